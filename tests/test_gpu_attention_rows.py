"""A row of attention depends on its own query and its own keys, to the bit: a
score that is out of all proportion (or infinite) for the queries that see its
key, or for one head, changes no bit of the rows that share a wave or a workgroup
with them. Every width, keys in one share of several tiles and split."""
import numpy as np
import pytest
import torch

from attention_cut import EXPANDED, LATENT, cut_of
from attention_parity import SM, bf16, gpu, latent_cache

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _equal(got, want, rows):
    assert bool(rows.any()) and not bool(rows.all())
    assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][rows], want[1][rows])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,rows,cut", [
    (2, 3, 130, (16, False)), (20, 3, 1000, (16, True)), (260, 3, 130, (32, False)), (128, 3, 400, (32, True)),
    (260, 20, 130, (64, False)), (130, 20, 700, (64, True)), (520, 3, 130, (128, False)), (260, 3, 700, (128, True))])
def test_prefix_a_key_that_others_see(T, H, rows, cut, fp8):
    rng = np.random.default_rng(T + H + rows)
    cache = gpu(latent_cache(rng, rows, fp8)[0])
    q = bf16(rng, T, H, 576).cuda()
    key = 100                                                  # in the second tile; the queries that do not see it
    sees = np.arange(T) % 2 == 0                               # see others of that tile
    pos = np.where(sees, rng.integers(key, rows, T), rng.integers(70, key, T))
    call = lambda: S.latent_attention(q, sm_scale=SM, pos=_ints(pos), with_lse=True, **cache)  # noqa: E731
    ran, want = cut_of(call, LATENT)
    assert ran == cut
    part, col = (cache["rope"], 5) if fp8 else (cache["C"], 517)
    others = torch.from_numpy(~sees).cuda()
    for x in (2.0 ** 20, -2.0 ** 20, float("inf")):
        part[key, col] = x
        _equal(call(), want, others)


@pytest.mark.parametrize("T,H,L,cut", [(300, 16, 300, (128, False)), (300, 2, 5000, (128, True)),
                                       (500, 256, 512, (256, False)), (500, 64, 3000, (256, True))])
def test_expanded_a_key_that_others_see(T, H, L, cut):
    rng = np.random.default_rng(T + H + L)
    q, kv, rope = bf16(rng, T, H, 192).cuda(), bf16(rng, L, H, 256).cuda(), bf16(rng, L, 64).cuda()
    key = L - 38                                               # not the first of its tile
    sees = np.arange(T) % 2 == 0
    pos = np.where(sees, rng.integers(key, L, T), rng.integers(key // 64 * 64, key, T))
    call = lambda: S.expanded_attention(q, kv, rope, _ints(pos), SM, with_lse=True)  # noqa: E731
    ran, want = cut_of(call, EXPANDED)
    assert ran == cut
    others = torch.from_numpy(~sees).cuda()
    for x in (2.0 ** 20, -2.0 ** 20, float("inf")):
        rope[key, 5] = x
        _equal(call(), want, others)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,k,cut", [
    (2, 3, 130, (16, False)), (20, 3, 1000, (16, True)), (130, 20, 130, (32, False)), (20, 20, 2000, (32, True)),
    (130, 33, 130, (64, False)), (64, 33, 1000, (64, True)), (130, 70, 130, (128, False)), (70, 70, 2000, (128, True))])
def test_list_another_head(T, H, k, cut, fp8):
    rng = np.random.default_rng(T + H + k)
    cache = gpu(latent_cache(rng, k + 50, fp8)[0])
    q = bf16(rng, T, H, 576).cuda()
    idx = _ints(rng.integers(0, k + 50, (T, k)))
    call = lambda: S.latent_attention(q, sm_scale=SM, idx=idx, with_lse=True, **cache)  # noqa: E731
    ran, want = cut_of(call, LATENT)
    assert ran == cut
    others = torch.ones(T, H, dtype=torch.bool, device="cuda")
    others[:, 1] = False
    was = q[:, 1].clone()
    for x in (was * 256, torch.full_like(was, float("nan")), torch.full_like(was, float("inf"))):
        q[:, 1] = x
        _equal(call(), want, others)


@pytest.mark.parametrize("T,H,L,cut", [(300, 16, 300, (128, False)), (300, 2, 5000, (128, True)),
                                       (500, 256, 512, (256, False)), (500, 64, 3000, (256, True))])
def test_expanded_another_query(T, H, L, cut):
    rng = np.random.default_rng(T + H + L + 1)
    q, kv, rope = bf16(rng, T, H, 192).cuda(), bf16(rng, L, H, 256).cuda(), bf16(rng, L, 64).cuda()
    call = lambda: S.expanded_attention(q, kv, rope, _ints(np.arange(L - T, L)), SM, with_lse=True)  # noqa: E731
    ran, want = cut_of(call, EXPANDED)
    assert ran == cut
    others = torch.arange(T, device="cuda") % 32 != 9
    was = q[~others].clone()
    for x in (was * 256, torch.full_like(was, float("nan")), torch.full_like(was, float("inf"))):
        q[~others] = x
        _equal(call(), want, others)
