"""Inputs and comparisons of the tests of the norm, of paged caches and of the
attention of drafted tokens.

Tolerances, from the arithmetic (u = 2^-24: half a step of fp32): h = x + r is off by
u |h|; the reciprocal root, formed in 64 bits, by u once it is fp32; the products h * r
and (h r) * w by u each: a normed value by 4 u |y|. A rotated value is two products
(u each of them) and their sum (u of it): 2 u (|a| + |b|) for cosines and sines of at
most 1. Then one rounding: to bf16 half a step, 2^-8 of the value or 2^-134 below the
normal range, to a code half a step, 2^-4 of it or half of the smallest code's 2^-9
times the scale. A row's scale is the oracle's unless its largest value is as near to a
power's border as its own error."""
from __future__ import annotations

import numpy as np
import torch

import oracle as O
from attention_parity import HALF, U, check_rows, f64
from oracle.paged import tree_rows

TINY = 2.0 ** -134


def ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def words(a):
    """Masks (Python integers below 2^64, any nesting) as an int64 GPU tensor."""
    return torch.from_numpy(np.asarray(a, dtype=np.uint64).view(np.int64)).cuda()


def rotation(positions):
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def tables(rng, seqs, per, spare=2):
    """Pages of the sequences in random order out of a pool: table [seqs, per], pages of the pool."""
    pool = seqs * per + spare
    return rng.permutation(pool)[:seqs * per].reshape(seqs, per).astype(np.int32), pool


def check_bf16(where, got, want, err):
    """bf16 values against float64 ones whose fp32 forms are off by err."""
    off = np.abs(f64(got) - want)
    tol = np.maximum(HALF * np.abs(want), TINY) + 1.01 * err
    assert (off <= tol).all(), f"{where}: off by {off.max():.3e}, {np.max(off / tol):.2f} of the tolerance"


def check_codes(where, codes, scale, want, err):
    """A row's E4M3FN codes and scale against float64 values whose fp32 forms are off by err."""
    scale = float(scale)
    top = float(np.abs(want).max())
    if top == 0.0:
        assert scale == 1.0 and (codes & 0x7f == 0).all(), where
        return
    slack = 1.01 * float(err.max())
    assert scale >= 2.0 ** -126 and np.log2(scale) == round(np.log2(scale)), where
    assert top - slack <= 448 * scale and (top + slack > 224 * scale or scale == 2.0 ** -126), f"{where}: {top} at scale {scale}"
    off = np.abs(O.decode_e4m3fn(codes) * scale - want)
    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * scale) + 1.1 * err
    assert (off <= tol).all(), f"{where}: off by {off.max():.3e}, {np.max(off / tol):.2f} of the tolerance"


def check_tree(label, out, lse, q, K, table, page, prefix, mask=None, idx=None, only=None):
    """out [S, N, H, 512], lse [S, N, H] (GPU) against the oracle; K [rows, 576] float64, mask [S][N][words]."""
    S, N, H = q.shape[:3]
    flat = lambda t: t.reshape(S * N, *t.shape[2:])  # noqa: E731

    def rows_of(t, h):
        s, i = divmod(t, N)
        r = tree_rows(table, page, K.shape[0], s, int(prefix[s]), i, None if mask is None else mask[s][i],
                      None if idx is None else idx[s, i])
        return K[r], K[r][:, :512]
    check_rows(label, flat(out), flat(lse), flat(q), rows_of, 512, only=only)


def random_trees(rng, S, N, pad=0, words_a_mask=None):
    """Masks [S][N][words] of random trees; the last `pad` nodes are padding."""
    W = words_a_mask or -(-N // 64)
    got = []
    for _ in range(S):
        mine = []
        for j in range(N - pad):
            up = int(rng.integers(-1, j)) if j else -1
            mine.append((mine[up] if up >= 0 else 0) | 1 << j)
        got.append([[m >> (64 * w) & (2 ** 64 - 1) for w in range(W)] for m in mine + [0] * pad])
    return got
