"""Plain float64 oracle of the norm, of paged caches and of the attention of
drafted tokens (test infrastructure only; it shares no code with the HIP library)."""
from __future__ import annotations

import numpy as np


def norm_row(h: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    """One row h of float64 values, normed."""
    return h / np.sqrt(np.dot(h, h) / len(h) + eps) * weight


def rotate_row(x: np.ndarray, rot: np.ndarray, pairs: bool) -> np.ndarray:
    """64 values x rotated by the angles whose 32 cosines and 32 sines are rot."""
    out = np.empty(64)
    for i in range(32):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + 32)
        out[a] = x[a] * rot[i] - x[b] * rot[32 + i]
        out[b] = x[b] * rot[i] + x[a] * rot[32 + i]
    return out


def page_row(table: np.ndarray, page: int, rows: int, s: int, j: int) -> int:
    """The cache row of position j of sequence s, or -1."""
    seqs, per = table.shape
    if not 0 <= s < seqs or j < 0 or j // page >= per or table[s, j // page] < 0:
        return -1
    row = int(table[s, j // page]) * page + j % page
    return row if row < rows else -1


def tree_rows(table, page, rows, s, prefix, node, mask=None, idx=None) -> np.ndarray:
    """The cache rows that are keys of one node: mask is its list of words (None: a chain), idx its list of positions."""
    seqs, per = table.shape
    if prefix < 0:
        return np.zeros(0, dtype=np.int64)
    n = min(int(prefix), per * page)
    if mask is None:
        bits = list(range(node + 1))
    else:
        bits = [64 * w + b for w, word in enumerate(mask) for b in range(64) if (int(word) >> b) & 1]
        if not bits:
            return np.zeros(0, dtype=np.int64)
    at = list(range(n)) if idx is None else [int(j) for j in idx if 0 <= j < n]
    found = [page_row(table, page, rows, s, j) for j in at + [n + b for b in bits]]
    return np.array([r for r in found if r >= 0], dtype=np.int64)
