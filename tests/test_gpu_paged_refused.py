"""Refused calls of the paged caches, the rotation, the norm and the attention of drafted
tokens leave their outputs as they were."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_amd as S
from attention_parity import SM, bf16
from paged_parity import ints, rotation

pytestmark = pytest.mark.gpu


def _unchanged(refused, outputs):
    """Each of the calls is refused, and none writes to any of the outputs."""
    before = [t.clone() for t in outputs]
    for call in refused:
        with pytest.raises((S.MisaError, ValueError)):
            call()
    torch.cuda.synchronize()
    for t, b in zip(outputs, before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
def test_refused_appends_write_nothing(fp8):
    rng = np.random.default_rng(1)
    x, i, t, rot, w = bf16(rng, 2, 576).cuda(), ints([0, 1]), ints([[0], [1]]), rotation(8).cuda(), bf16(rng, 512).cuda()
    if fp8:
        cache = dict(C=torch.zeros(32, 512, dtype=torch.uint8, device="cuda"), c_scale=torch.ones(32, device="cuda"),
                     rope=bf16(rng, 32, 64).cuda())
    else:
        cache = dict(C=bf16(rng, 32, 576).cuda())
    ok = dict(x=x, seq=i, pos=i, table=t, page=16, **cache)
    bad = [dict(x=x[:, :512]), dict(seq=i.long()), dict(pos=i[:1]), dict(table=t[0]), dict(weight=w[:64]), dict(rot=rot[:, :32]),
           dict(rot_at=0), dict(pairs=True), dict(rot=rot.double()), dict(x=x.t().contiguous().t()), dict(page=12), dict(rot=rot, rot_at=0),
           dict(turn=i), dict(weight=w, eps=-1.0), dict(page=(1 << 32) + 16)]
    _unchanged([lambda kw=kw: S.paged_append(**(ok | kw)) for kw in bad], list(cache.values()))
    before = cache["C"].clone()
    S.paged_append(**ok)                                       # and the call itself does write
    assert not torch.equal(cache["C"].view(torch.uint8), before.view(torch.uint8))


def test_refused_rotations_norms_and_attention_write_nothing():
    rng = np.random.default_rng(2)
    q, to, rot, pos = bf16(rng, 2, 3, 64).cuda(), bf16(rng, 2, 3, 64).cuda(), rotation(8).cuda(), ints([1, 2])
    _unchanged([lambda: S.rotate(q[:, :, :32].contiguous(), pos, rot, out=to), lambda: S.rotate(q, pos.long(), rot, out=to),
                lambda: S.rotate(q[:1].expand(2, 3, 64), pos, rot, out=to), lambda: S.rotate(q, pos[:1], rot, out=to)], [to])
    x, w, y, s = bf16(rng, 3, 64).cuda(), bf16(rng, 64).cuda(), bf16(rng, 3, 64).cuda(), bf16(rng, 3, 64).cuda()
    _unchanged([lambda: S.rms_norm(x, w, -1.0, out=y), lambda: S.rms_norm(x, w, group=128, out=y), lambda: S.rms_norm(x, w[:32], out=y),
                lambda: S.rms_norm(x, w, residual=x[:2], out=y, out_sum=s), lambda: S.rms_norm(x, w, out=y, out_sum=s)], [y, s])
    qa, C, out = bf16(rng, 2, 70, 4, 576).cuda(), bf16(rng, 256, 576).cuda(), bf16(rng, 2, 70, 4, 512).cuda()
    ok = dict(q=qa, prefix=ints([5, 6]), table=ints([[0, 1], [2, 3]]), page=64, C=C, sm_scale=SM, out=out)
    one = torch.ones(2, 70, dtype=torch.int64, device="cuda")
    bad = [dict(mask=one), dict(mask=one[:, :, None].int()), dict(page=24), dict(longest=-1), dict(sm_scale=float("inf")),
           dict(ws=torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[16:]), dict(prefix=ints([5]))]
    _unchanged([lambda kw=kw: S.tree_attention(**(ok | kw)) for kw in bad], [out])
