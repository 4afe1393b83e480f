"""Plain float64 oracle of the caches and of latent attention (test
infrastructure only; it shares no code with the HIP library).

Rows are decoded to float64 from their bits; every function takes and returns
numpy arrays. `magnitude` terms serve the tests' tolerances.
"""
from __future__ import annotations

import math

import numpy as np

from .indexer import decode_e4m3fn

E4M3_VALUES = decode_e4m3fn(np.arange(256, dtype=np.uint8))


def code_row(x: np.ndarray):
    """E4M3FN codes (uint8) and the scale of one row x of float64 values: the
    scale is the smallest power of two from 2^-126 with max|x| <= 448 scale (1
    for a zero row); ties go to the even code."""
    if not np.isfinite(x).all():
        return None, math.nan
    a = float(np.abs(x).max()) if x.size else 0.0
    e = -126
    while a > 448.0 * 2.0 ** e:
        e += 1
    scale = 1.0 if a == 0.0 else 2.0 ** e
    mags = E4M3_VALUES[:127]  # codes 0 .. 126: 0 to 448 in ascending order
    y = np.abs(x) / scale
    hi = np.clip(np.searchsorted(mags, y, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - mags[lo], mags[hi] - y
    pick = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    pick = np.where(y >= mags[hi], hi, pick)
    return (pick + 128 * np.signbit(x)).astype(np.uint8), scale


def attend(q: np.ndarray, K: np.ndarray, V: np.ndarray, sm: float):
    """One query row over its keys: (out, log-sum, sum p|V|, max sum |q||K|).
    q [d], K [n, d], V [n, dv]; no keys: zeros and -inf."""
    if K.shape[0] == 0:
        return np.zeros(V.shape[1]), -math.inf, np.zeros(V.shape[1]), 0.0
    s = (K @ q) * sm
    top = s.max()
    e = np.exp(s - top)
    p = e / e.sum()
    return p @ V, top + math.log(e.sum()), p @ np.abs(V), float((np.abs(K) @ np.abs(q)).max()) * abs(sm)


def latent_keys(rows: int, pos=None, idx=None, base: int = 0) -> np.ndarray:
    """The cache rows that are keys of one query."""
    if base < 0:
        return np.zeros(0, dtype=np.int64)
    if idx is not None:
        r = np.asarray(idx, dtype=np.int64)
        r = r[r >= 0] + base
        return r[r < rows]
    return np.arange(base, min(rows, base + max(0, int(pos) + 1)), dtype=np.int64)
