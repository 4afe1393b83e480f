"""Argument checks of the norm's, the paged caches' and the drafted tokens' entry
points that need no GPU: bad calls are refused before anything is enqueued, empty ones
are no-ops, and workspace sizes are planned on the host. The oracle is pinned here too."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_amd as S
from oracle.attention import attend
from oracle.paged import norm_row, page_row, rotate_row, tree_rows
from test_abi_attention import BAD_CACHE, FAKE, _cache

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def _pages(**kw):
    a = dict(table=FAKE, seqs=3, per=10, page=64)
    a.update(kw)
    return S.Pages(*a.values())


def _rot(**kw):
    a = dict(rot=FAKE, positions=100, pairs=0)
    a.update(kw)
    return S.Rotation(*a.values())


def _append(**kw):
    a = dict(n=5, x=FAKE, x_ld=576, seq=FAKE, pos=FAKE, turn=None, weight=FAKE, w_dtype=0, rot_at=512, eps=1e-6,
             rotation=_rot(), pages=_pages(), cache=_cache())
    a.update(kw)
    return S.AppendProblem(*a.values())


BAD_PAGES = [(dict(seqs=-1), INVALID), (dict(per=0), INVALID), (dict(page=0), INVALID), (dict(page=-64), INVALID),
             (dict(page=48), INVALID), (dict(seqs=(1 << 22) + 1), UNSUPPORTED), (dict(per=1 << 23, page=64), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(n=(1 << 25) + 1), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(x_ld=575), INVALID), (dict(x_ld=568), INVALID), (dict(x_ld=580), INVALID), (dict(x_ld=1 << 41), UNSUPPORTED),
    (dict(seq=None), INVALID), (dict(seq=FAKE + 2), INVALID), (dict(pos=None), INVALID), (dict(pos=FAKE + 1), INVALID),
    (dict(turn=FAKE + 2), INVALID), (dict(turn=FAKE, rotation=_rot(rot=None)), INVALID), (dict(weight=FAKE + 8), INVALID),
    (dict(w_dtype=2), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(rot_at=0), INVALID), (dict(rot_at=448), INVALID), (dict(rotation=_rot(rot=FAKE + 4)), INVALID),
    (dict(rotation=_rot(positions=0)), INVALID), (dict(rotation=_rot(pairs=2)), INVALID),
    (dict(pages=_pages(table=None)), INVALID), (dict(pages=_pages(table=FAKE + 2)), INVALID),
    (dict(cache=_cache(d=128, dr=0, rope=None), x_ld=128, rot_at=32), INVALID),
    (dict(cache=_cache(d=128, dr=0, rope=None), x_ld=128, rot_at=128), INVALID),
    (dict(cache=_cache(d=128, dr=0, rope=None), x_ld=128, rot_at=-64), INVALID),
])
def test_append_checks(kw, status):
    p = _append(**kw)
    assert S.lib().misa_paged_append(ctypes.byref(p), None) == status
    assert S.lib().misa_last_error() != b""


def test_append_of_nothing():
    for kw in (dict(n=0, x=None, seq=None, pos=None), dict(pages=_pages(seqs=0, table=None), x=None)):
        p = _append(**kw)
        assert S.lib().misa_paged_append(ctypes.byref(p), None) == 0
    assert S.lib().misa_paged_append(None, None) == INVALID


@pytest.mark.parametrize("kw,status", BAD_PAGES)
def test_pages_checks(kw, status):
    p, t = _append(pages=_pages(**kw)), _tree(pages=_pages(**kw))
    assert S.lib().misa_paged_append(ctypes.byref(p), None) == status
    assert S.lib().misa_tree_attention(ctypes.byref(t), FAKE, FAKE, FAKE, 1 << 40, None) == status
    assert S.lib().misa_tree_workspace_bytes(ctypes.byref(t)) == 0


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_paged_cache_checks(kw, status):
    p, t = _append(cache=_cache(**kw)), _tree(cache=_cache(**kw))
    assert S.lib().misa_paged_append(ctypes.byref(p), None) == status
    assert S.lib().misa_tree_attention(ctypes.byref(t), FAKE, FAKE, FAKE, 1 << 40, None) == status


def _rotate(**kw):
    a = dict(T=4, H=16, x=FAKE, x_t=16 * 64, x_h=64, pos=FAKE, rotation=_rot())
    a.update(kw)
    return S.RotateProblem(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(T=1 << 20, H=1 << 11), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(x_t=63), INVALID), (dict(x_t=-64), INVALID), (dict(x_h=68), INVALID),
    (dict(x_h=56), INVALID), (dict(pos=None), INVALID), (dict(rotation=_rot(rot=None)), INVALID),
    (dict(rotation=_rot(positions=-1)), INVALID), (dict(rotation=_rot(pairs=-1)), INVALID),
])
def test_rotate_checks(kw, status):
    p = _rotate(**kw)
    assert S.lib().misa_rotate(ctypes.byref(p), FAKE, 1024, 64, None) == status
    assert S.lib().misa_last_error() != b""


def test_rotate_call_checks():
    p = _rotate()
    f = lambda out=FAKE, t=1024, h=64: S.lib().misa_rotate(ctypes.byref(p), out, t, h, None)  # noqa: E731
    assert f(out=None) == f(out=FAKE + 8) == f(t=60) == f(h=0) == f(h=66) == S.lib().misa_rotate(None, FAKE, 64, 64, None) == INVALID
    e = _rotate(T=0, x=None, pos=None)
    assert S.lib().misa_rotate(ctypes.byref(e), None, 64, 64, None) == 0


def _norm(**kw):
    a = dict(n=5, width=512, x=FAKE, x_ld=512, residual=FAKE, weight=FAKE, w_dtype=0, dtype=1, group=0, eps=1e-6)
    a.update(kw)
    return S.NormProblem(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(n=(1 << 25) + 1), UNSUPPORTED), (dict(width=0), INVALID), (dict(width=12), INVALID),
    (dict(width=16392, x_ld=16392), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(group=64), INVALID),
    (dict(group=128, dtype=0), INVALID), (dict(x_ld=504), INVALID), (dict(x_ld=514), INVALID), (dict(x=None), INVALID),
    (dict(x=FAKE + 2), INVALID), (dict(residual=FAKE + 8), INVALID), (dict(weight=None), INVALID),
    (dict(weight=FAKE + 8), INVALID), (dict(w_dtype=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(dtype=0), INVALID), (dict(residual=None), INVALID),
])
def test_norm_checks(kw, status):
    p = _norm(**kw)  # (the last two: a scale for a bf16 result, a sum without residual)
    assert S.lib().misa_rms_norm(ctypes.byref(p), FAKE, FAKE, FAKE, None) == status
    assert S.lib().misa_last_error() != b""


def test_calls_past_a_launch_are_refused():
    # a launch has fewer than 2^32 threads
    p = _rotate(T=1 << 22, H=65)
    assert S.lib().misa_rotate(ctypes.byref(p), FAKE, 65 * 64, 64, None) == UNSUPPORTED
    assert b"2^28" in S.lib().misa_last_error()
    for n, width in ((1 << 25, 264), ((1 << 19) + 1, 16384), ((1 << 24) + 1, 512)):
        p = _norm(n=n, width=width, x_ld=width)
        assert S.lib().misa_rms_norm(ctypes.byref(p), FAKE, FAKE, FAKE, None) == UNSUPPORTED
        assert b"2^33" in S.lib().misa_last_error()


def test_norm_call_checks():
    p = _norm()
    f = lambda y=FAKE, s=FAKE, t=FAKE: S.lib().misa_rms_norm(ctypes.byref(p), y, s, t, None)  # noqa: E731
    assert f(y=None) == f(y=FAKE + 8) == f(s=None) == f(s=FAKE + 2) == f(t=FAKE + 8) == INVALID
    assert S.lib().misa_rms_norm(None, FAKE, FAKE, FAKE, None) == INVALID
    e = _norm(n=0, x=None, residual=None)
    assert S.lib().misa_rms_norm(ctypes.byref(e), None, None, None, None) == 0


def _tree(**kw):
    a = dict(N=4, H=16, k=0, words=1, sm_scale=0.1, longest=0, q=FAKE, prefix=FAKE, mask=FAKE, idx=None, pages=_pages(),
             cache=_cache())
    a.update(kw)
    return S.TreeProblem(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), INVALID), (dict(N=(1 << 16) + 1), UNSUPPORTED), (dict(H=0), INVALID), (dict(N=1 << 16, H=1 << 14), UNSUPPORTED),
    (dict(N=1 << 12, pages=_pages(seqs=1 << 11)), UNSUPPORTED), (dict(sm_scale=math.nan), INVALID),
    (dict(sm_scale=2.4e38), INVALID), (dict(words=0), INVALID), (dict(words=-1), INVALID), (dict(words=1025), UNSUPPORTED),
    (dict(mask=None), INVALID), (dict(mask=FAKE + 4), INVALID), (dict(k=5), INVALID), (dict(k=0, idx=FAKE), INVALID),
    (dict(k=-1, idx=FAKE), INVALID), (dict(k=(1 << 24) + 1, idx=FAKE), UNSUPPORTED), (dict(k=8, idx=FAKE + 2), INVALID),
    (dict(k=1 << 24, idx=FAKE, N=64), UNSUPPORTED), (dict(longest=-1), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(prefix=None), INVALID), (dict(prefix=FAKE + 2), INVALID), (dict(pages=_pages(table=None)), INVALID),
    (dict(cache=_cache(d=128)), UNSUPPORTED), (dict(cache=_cache(dr=0, rope=None)), UNSUPPORTED),
])
def test_tree_checks(kw, status):
    p = _tree(**kw)
    assert S.lib().misa_tree_attention(ctypes.byref(p), FAKE, FAKE, FAKE, 1 << 40, None) == status
    assert S.lib().misa_last_error() != b""


def test_tree_call_checks():
    L = S.lib()
    for p in (_tree(), _tree(k=100, idx=FAKE), _tree(mask=None, words=0)):
        f = lambda out=FAKE, lse=FAKE, ws=FAKE, n=1 << 40: L.misa_tree_attention(ctypes.byref(p), out, lse, ws, n, None)  # noqa: E731
        assert f(out=None) == f(out=FAKE + 8) == f(lse=FAKE + 2) == INVALID
        need = L.misa_tree_workspace_bytes(ctypes.byref(p))
        assert need >= 256
        assert f(n=need - 1) == f(ws=None) == f(ws=FAKE + 16) == WORKSPACE
    assert L.misa_tree_attention(None, FAKE, FAKE, FAKE, 1 << 40, None) == INVALID
    e = _tree(pages=_pages(seqs=0, table=None), q=None, prefix=None, mask=FAKE)
    assert L.misa_tree_attention(ctypes.byref(e), None, None, None, 0, None) == 0
    assert L.misa_tree_workspace_bytes(ctypes.byref(e)) >= 256


@pytest.mark.parametrize("seqs,N,H", [(1, 1, 1), (1, 64, 128), (2, 64, 128), (32, 4, 128), (256, 1, 16), (256, 8, 128), (257, 8, 128),
                                      (4096, 1, 128), (64, 1024, 16), (1 << 22, 1, 1)])
@pytest.mark.parametrize("per,page,longest", [(1, 1, 0), (2048, 64, 0), (2048, 64, 100), (1 << 22, 64, 0)])
def test_tree_workspace_sizes(seqs, N, H, per, page, longest):
    p = _tree(N=N, H=H, mask=None, words=0, longest=longest, pages=_pages(seqs=seqs, per=per, page=page))
    assert 256 <= S.lib().misa_tree_workspace_bytes(ctypes.byref(p)) <= 1 << 30  # partial sums of few rows; large calls need none


def test_binding_refuses_host_tensors_and_wrong_kinds():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        S.rms_norm(b(2, 64), b(64))
    with pytest.raises(ValueError, match="rows"):
        S.rms_norm(None, b(64))
    with pytest.raises(ValueError, match="GPU tensor"):
        S.paged_append(b(2, 576), i, i, i[None], 64, b(4, 576))
    with pytest.raises(ValueError, match="GPU tensor"):
        S.rotate(b(2, 4, 64), i, torch.zeros(5, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        S.tree_attention(b(1, 2, 4, 576), i[:1], i[None], 64, b(4, 576), 1.0)


# ------------------------------------------------------------- oracle pins

def test_oracle_norm_closed_forms():
    w = np.array([1.0, 2.0, -1.0, 0.5])
    assert np.allclose(norm_row(np.array([3.0, 3.0, -3.0, 3.0]), w, 0.0), [1, 2, 1, 0.5])      # equal magnitudes: the weights
    assert np.allclose(norm_row(np.array([1.0, 0, 0, 0]), w, 0.75), [1, 0, 0, 0])               # 1 / sqrt(1/4 + 3/4)
    x = np.random.default_rng(0).standard_normal(64)
    assert np.allclose(norm_row(5 * x, np.ones(64), 0.0), norm_row(x, np.ones(64), 0.0))        # a scale cancels


def test_oracle_rotation_closed_forms():
    x = np.random.default_rng(1).standard_normal(64)
    turn = lambda a: np.concatenate([np.cos(a), np.sin(a)])  # noqa: E731
    a, b = np.linspace(0, 3, 32), np.linspace(1, -2, 32)
    for pairs in (False, True):
        assert np.allclose(rotate_row(x, turn(0 * a), pairs), x)
        assert np.allclose(rotate_row(rotate_row(x, turn(a), pairs), turn(b), pairs), rotate_row(x, turn(a + b), pairs))
        # products of two turned rows depend on the difference of their angles alone
        y = np.random.default_rng(2).standard_normal(64)
        assert np.isclose(rotate_row(x, turn(a + 1), pairs) @ rotate_row(y, turn(b + 1), pairs),
                          rotate_row(x, turn(a), pairs) @ rotate_row(y, turn(b), pairs))
    e = np.zeros(64)
    e[0] = 1.0
    q = turn(np.full(32, np.pi / 2))
    assert np.allclose(rotate_row(e, q, False)[32], 1) and np.allclose(rotate_row(e, q, True)[1], 1)


def test_oracle_pages_and_trees():
    table = np.array([[2, 0], [-1, 3]], dtype=np.int32)
    at = [page_row(table, 4, 15, 0, j) for j in range(9)]
    assert at == [8, 9, 10, 11, 0, 1, 2, 3, -1] and page_row(table, 4, 15, 1, 2) == -1
    assert page_row(table, 4, 15, 1, 6) == 14 and page_row(table, 4, 15, 1, 7) == -1 and page_row(table, 4, 15, 2, 0) == -1
    assert list(tree_rows(table, 4, 16, 0, 3, 1)) == [8, 9, 10, 11, 0]                  # three committed, nodes 0 and 1
    assert list(tree_rows(table, 4, 16, 0, 3, 2, mask=[0b101])) == [8, 9, 10, 11, 1]
    assert list(tree_rows(table, 4, 16, 0, 3, 0, mask=[0b1], idx=[2, -1, 0, 2, 3])) == [10, 8, 10, 11]
    assert not len(tree_rows(table, 4, 16, 0, 3, 0, mask=[0])) and not len(tree_rows(table, 4, 16, 0, -1, 0))
    assert list(tree_rows(table, 4, 16, 0, 100, 0)) == [8, 9, 10, 11, 0, 1, 2, 3]
    assert attend(np.ones(3), np.ones((0, 3)), np.ones((0, 2)), 1.0)[1] == -math.inf
