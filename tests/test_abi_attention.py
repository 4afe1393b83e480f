"""Argument checks of the cache and attention entry points that need no GPU:
bad calls are refused before anything is enqueued, empty ones are no-ops, and
workspace sizes are planned on the host. The oracle's coding of a row is pinned
against torch's cast here too."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
import sparse_attention_indexer_block_amd as S
from oracle.attention import attend, code_row, latent_keys

FAKE = 1 << 20  # an aligned, never-dereferenced address: validation must fail first


def _cache(**kw):
    a = dict(rows=1000, d=512, dr=64, dtype=1, c=FAKE, scale=FAKE, rope=FAKE)
    a.update(kw)
    return S.Cache(*a.values())


BAD_CACHE = [
    (dict(dtype=2), -1), (dict(rows=0), -1), (dict(rows=-5), -1), (dict(rows=(1 << 30) + 1), -2), (dict(d=0), -1),
    (dict(dr=-1), -1), (dict(d=256), -2), (dict(dr=32), -2), (dict(c=None), -1), (dict(c=FAKE + 8), -1),
    (dict(scale=None), -1), (dict(scale=FAKE + 2), -1), (dict(rope=None), -1), (dict(rope=FAKE + 8), -1),
    (dict(dr=0), -1), (dict(dtype=0), -1), (dict(dtype=0, scale=None), -1),
]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_cache_checks(kw, status):
    L, c = S.lib(), _cache(**kw)
    assert L.misa_cache_write(ctypes.byref(c), FAKE, 3, FAKE, None) == status
    assert L.misa_cache_read(ctypes.byref(c), FAKE, 3, FAKE, None) == status
    p = _latent(cache=c)
    assert L.misa_latent_attention(ctypes.byref(p), FAKE, FAKE, FAKE, 1 << 40, None) == status
    assert L.misa_latent_workspace_bytes(ctypes.byref(p)) == 0
    assert L.misa_last_error() != b""


def test_cache_call_checks():
    L, c = S.lib(), _cache()
    w = lambda x=FAKE, n=3, s=FAKE: L.misa_cache_write(ctypes.byref(c), x, n, s, None)  # noqa: E731
    r = lambda o=FAKE, n=3, s=FAKE: L.misa_cache_read(ctypes.byref(c), s, n, o, None)  # noqa: E731
    assert w(n=-1) == w(x=None) == w(x=FAKE + 8) == w(s=None) == w(s=FAKE + 1) == -1
    assert r(n=-1) == r(o=None) == r(o=FAKE + 8) == r(s=None) == r(s=FAKE + 1) == -1
    assert w(x=None, n=0, s=None) == r(o=None, n=0, s=None) == 0
    assert L.misa_cache_write(None, FAKE, 1, FAKE, None) == -1


def _latent(**kw):
    a = dict(T=4, H=16, k=64, sm_scale=0.1, q=FAKE, idx=FAKE, pos=None, base=None, cache=_cache())
    a.update(kw)
    return S.LatentProblem(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(T=1 << 20, H=1 << 11), -2), (dict(sm_scale=math.nan), -1),
    (dict(sm_scale=math.inf), -1), (dict(k=0), -1), (dict(k=-1), -1), (dict(k=(1 << 30) + 1), -2), (dict(idx=None), -1),
    (dict(idx=FAKE + 2), -1), (dict(pos=FAKE), -1), (dict(idx=None, k=0), -1), (dict(idx=None, k=0, pos=FAKE + 1), -1),
    (dict(q=None), -1), (dict(q=FAKE + 8), -1), (dict(base=FAKE + 2), -1), (dict(cache=_cache(d=128)), -2),
    (dict(cache=_cache(dr=0, rope=None)), -2),
])
def test_latent_checks(kw, status):
    p = _latent(**kw)
    assert S.lib().misa_latent_attention(ctypes.byref(p), FAKE, FAKE, FAKE, 1 << 40, None) == status
    assert S.lib().misa_last_error() != b""


def test_latent_call_checks():
    L, p = S.lib(), _latent()
    f = lambda out=FAKE, lse=FAKE, ws=FAKE, n=1 << 40: L.misa_latent_attention(ctypes.byref(p), out, lse, ws, n, None)  # noqa: E731
    assert f(out=None) == f(out=FAKE + 8) == f(lse=FAKE + 2) == -1
    need = L.misa_latent_workspace_bytes(ctypes.byref(p))
    assert need >= 256
    assert f(n=need - 1) == f(ws=None) == f(ws=FAKE + 16) == -3
    assert L.misa_latent_attention(None, FAKE, FAKE, FAKE, 1 << 40, None) == -1
    e = _latent(T=0, q=None, idx=None)
    assert L.misa_latent_attention(ctypes.byref(e), None, None, None, 0, None) == 0
    assert L.misa_latent_workspace_bytes(ctypes.byref(e)) >= 256


def _expanded(**kw):
    a = dict(T=4, H=16, L=100, sm_scale=0.1, q=FAKE, kv=FAKE, rope=FAKE, rope_ld=64, pos=FAKE, base=None)
    a.update(kw)
    return S.ExpandedProblem(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(T=1 << 20, H=1 << 11), -2), (dict(L=0), -1), (dict(L=(1 << 30) + 1), -2),
    (dict(sm_scale=math.nan), -1), (dict(rope_ld=63), -1), (dict(rope_ld=68), -1), (dict(rope_ld=-64), -1),
    (dict(q=None), -1), (dict(kv=FAKE + 8), -1), (dict(rope=None), -1), (dict(rope=FAKE + 2), -1), (dict(pos=None), -1),
    (dict(base=FAKE + 1), -1),
])
def test_expanded_checks(kw, status):
    p = _expanded(**kw)
    assert S.lib().misa_expanded_attention(ctypes.byref(p), FAKE, FAKE, FAKE, 1 << 40, None) == status
    assert S.lib().misa_last_error() != b""


def test_expanded_call_checks():
    L, p = S.lib(), _expanded()
    f = lambda out=FAKE, lse=FAKE, ws=FAKE, n=1 << 40: L.misa_expanded_attention(ctypes.byref(p), out, lse, ws, n, None)  # noqa: E731
    assert f(out=None) == f(out=FAKE + 8) == f(lse=FAKE + 2) == -1
    need = L.misa_expanded_workspace_bytes(ctypes.byref(p))
    assert f(n=need - 1) == f(ws=None) == f(ws=FAKE + 16) == -3
    e = _expanded(T=0, q=None, kv=None, rope=None, pos=None)
    assert L.misa_expanded_attention(ctypes.byref(e), None, None, None, 0, None) == 0


@pytest.mark.parametrize("T,H,rows,k", [(1, 1, 1, 1), (1, 16, 131072, 2048), (32, 128, 1 << 20, 2048), (16384, 128, 16384, 2048),
                                        (1, 128, 1 << 30, 1 << 30), (8, 20, 100, 1 << 30)])
def test_workspace_sizes(T, H, rows, k):
    L = S.lib()
    cap = 1 << 32  # partial sums of few rows; large calls need none
    for p in (_latent(T=T, H=H, k=k, cache=_cache(rows=rows)), _latent(T=T, H=H, k=0, idx=None, pos=FAKE, cache=_cache(rows=rows)),
              _latent(T=T, H=H, k=0, idx=None, pos=FAKE, base=FAKE, cache=_cache(rows=rows))):
        n = L.misa_latent_workspace_bytes(ctypes.byref(p))
        assert 256 <= n <= cap
    e = _expanded(T=T, H=H, L=rows)
    assert 256 <= L.misa_expanded_workspace_bytes(ctypes.byref(e)) <= cap


def test_binding_refuses_host_tensors_and_wrong_kinds():
    x = torch.zeros(2, 576, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        S.cache_write(x, i, torch.zeros(4, 576, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU tensor"):
        S.cache_read(i, torch.zeros(4, 512, dtype=torch.uint8), torch.ones(4), torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU tensor"):
        S.latent_attention(torch.zeros(2, 16, 576, dtype=torch.bfloat16), torch.zeros(4, 576, dtype=torch.bfloat16), 1.0, pos=i)
    with pytest.raises(ValueError, match="GPU tensor"):
        S.expanded_attention(torch.zeros(2, 4, 192, dtype=torch.bfloat16), torch.zeros(4, 4, 256, dtype=torch.bfloat16),
                             torch.zeros(4, 64, dtype=torch.bfloat16), i, 1.0)
    with pytest.raises(ValueError, match="missing"):
        S.cache_read(None, None)


# ------------------------------------------------------------- oracle pins

def test_oracle_codes_equal_torchs_cast():
    rng = np.random.default_rng(1)
    for scale in (1.0, 1e-3, 1e20, 2.0 ** -120):
        x = torch.from_numpy((rng.standard_normal((50, 64)) * scale).astype(np.float32)).bfloat16()
        for r in x:
            codes, s = code_row(r.to(torch.float64).numpy())
            assert math.frexp(s)[0] == 0.5
            a = float(r.abs().max())
            assert a <= 448 * s and (a > 448 * s / 2 or s == 2.0 ** -126)
            assert np.array_equal(codes, (r.float() / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(2)
    K, V = rng.standard_normal((7, 5)), rng.standard_normal((7, 3))
    out, z, _, _ = attend(np.zeros(5), K, V, 0.3)                       # equal scores: the mean
    assert np.allclose(out, V.mean(0)) and math.isclose(z, math.log(7))
    out, z, A, G = attend(np.ones(5), K[:1], V[:1], 0.3)                # one key: its value
    assert np.allclose(out, V[0]) and math.isclose(z, 0.3 * K[0].sum()) and math.isclose(G, 0.3 * np.abs(K[0]).sum())
    q = rng.standard_normal(5)
    e = [math.exp(0.3 * float(sum(a * b for a, b in zip(q, k)))) for k in K]
    out, z, _, _ = attend(q, K, V, 0.3)
    assert np.allclose(out, sum(w * v for w, v in zip(e, V)) / sum(e)) and math.isclose(z, math.log(sum(e)))
    twice, _, _, _ = attend(q, np.vstack([K, K[:1]]), np.vstack([V, V[:1]]), 0.3)  # a repeated key counts twice
    e[0] *= 2
    assert np.allclose(twice, sum(w * v for w, v in zip(e, V)) / sum(e))
    assert attend(q, K[:0], V[:0], 0.3)[1] == -math.inf


def test_oracle_keys_of_a_query():
    assert list(latent_keys(10, idx=[3, -1, 9, 3], base=2)) == [5, 5]
    assert list(latent_keys(10, pos=3, base=8)) == [8, 9]
    assert list(latent_keys(4, pos=2 ** 31 - 1)) == [0, 1, 2, 3]
    assert not len(latent_keys(10, pos=-1)) and not len(latent_keys(10, pos=3, base=-1)) and not len(latent_keys(10, idx=[1], base=-1))
