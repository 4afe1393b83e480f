"""Queries, caches, keys and values given as int16 bit patterns are bfloat16
numbers to every call, and what comes back is bfloat16."""
import numpy as np
import pytest
import torch

from attention_parity import SM, bf16, gpu, latent_cache

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _bits(t):
    return t.view(torch.int16) if t is not None and t.dtype == torch.bfloat16 else t


def _same(got, want):
    assert got[0].dtype == torch.bfloat16 and got[1].dtype == torch.float32
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("k", [0, 100])
def test_latent_from_bits(k, fp8):
    rng = np.random.default_rng(k + fp8)
    T, H, rows = 3, 20, 150
    cache = gpu(latent_cache(rng, rows, fp8)[0])
    q = bf16(rng, T, H, 576).cuda()
    kw = dict(idx=_ints(rng.integers(-1, rows, (T, k)))) if k else dict(pos=_ints([149, 70, -1]))
    want = S.latent_attention(q, sm_scale=SM, with_lse=True, **cache, **kw)
    _same(S.latent_attention(_bits(q), sm_scale=SM, with_lse=True, **{n: _bits(v) for n, v in cache.items()}, **kw), want)
    assert S.latent_attention(_bits(q), sm_scale=SM, **cache, **kw).dtype == torch.bfloat16
    mine = torch.zeros_like(want[0])
    got = S.latent_attention(_bits(q), sm_scale=SM, **cache, **kw, out=mine)
    assert got is mine and torch.equal(mine, want[0])


def test_expanded_from_bits():
    rng = np.random.default_rng(3)
    T, H, L = 40, 2, 90
    q, kv, rope = bf16(rng, T, H, 192).cuda(), bf16(rng, L, H, 256).cuda(), bf16(rng, L, 64).cuda()
    pos = _ints(np.arange(L - T, L))
    want = S.expanded_attention(q, kv, rope, pos, SM, with_lse=True)
    _same(S.expanded_attention(_bits(q), _bits(kv), _bits(rope), pos, SM, with_lse=True), want)
    assert S.expanded_attention(_bits(q), kv, rope, pos, SM).dtype == torch.bfloat16


def test_empty_batch_from_bits():
    C = torch.zeros(4, 576, dtype=torch.int16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = S.latent_attention(torch.empty(0, 16, 576, dtype=torch.int16, device="cuda"), C, SM, pos=none)
    assert out.dtype == torch.bfloat16 and tuple(out.shape) == (0, 16, 512)


@pytest.mark.parametrize("fp8", [False, True])
def test_caches_from_bits(fp8):
    rng = np.random.default_rng(4)
    x, slots = bf16(rng, 9, 576).cuda(), _ints([3, 0, -1, 8, 1, 12, 5, 2, 40])
    cache = gpu(latent_cache(rng, 13, fp8)[0])
    other = {n: (None if v is None else v.clone()) for n, v in cache.items()}
    S.cache_write(x, slots, **cache)
    S.cache_write(_bits(x), slots, **{n: _bits(v) for n, v in other.items()})
    for n, v in cache.items():
        assert v is None or torch.equal(v.view(torch.uint8), other[n].view(torch.uint8))
    got = S.cache_read(slots, **{n: _bits(v) for n, v in other.items()})
    assert got.dtype == torch.bfloat16 and torch.equal(got, S.cache_read(slots, **cache))
