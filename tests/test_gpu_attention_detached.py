"""The attention calls serve inference: with inputs that require gradients they
give the same bits, and a result that carries none, as their documentation says."""
import numpy as np
import pytest
import torch

from attention_parity import SM, bf16

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def test_results_are_detached_as_documented():
    rng = np.random.default_rng(1)
    pos = torch.tensor([9, 30, -1], dtype=torch.int32, device="cuda")
    q, C = bf16(rng, 3, 16, 576).cuda(), bf16(rng, 40, 576).cuda()
    qe, kv = bf16(rng, 3, 4, 192).cuda(), bf16(rng, 40, 4, 256).cuda()
    lat = lambda: S.latent_attention(q, C, SM, pos=pos, with_lse=True)  # noqa: E731
    exp = lambda: S.expanded_attention(qe, kv, C.detach()[:, 512:], pos, SM, with_lse=True)  # noqa: E731
    want = [*lat(), *exp()]
    for t in (q, C, qe, kv):
        t.requires_grad_()
    got = [*lat(), *exp()]
    assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, want))
    assert "carries no gradient" in S.latent_attention.__doc__ and "carries no gradient" in S.expanded_attention.__doc__
