"""Inputs of the cache and attention tests, and the comparison with the oracle.

Tolerances, from the arithmetic (u = 2^-24: half a step of fp32, b = 2^-8: of
bf16). A score is a sum of n_d exact products (bf16 times bf16 or a code) in
fp32, scaled: it is off by at most (n_d + 8) u G with G = sm * max_s sum |q||k|.
A weight exp(S - reference) carries that and the exponential's own error
(2^-21), once in the sum and once in the total: eps = 2 (n_d + 8) u G + 2^-20.
It is rounded to bf16 (b) and summed in fp32 over n keys ((n + 16) u), and the
result is rounded to bf16 (b). So
    |out - oracle| <= (b + eps + (n + 16) u) sum p|v| + b |oracle|
(a 1% margin covers products of these terms), and
    |lse - oracle| <= (n_d + 8) u G + (n + 16) u + 2^-20 + 8 u |oracle|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle as O
from oracle.attention import attend, latent_keys

U, HALF = 2.0 ** -24, 2.0 ** -8
SM = 192 ** -0.5


def bf16(rng, *shape, scale=1.0):
    """Random bf16 values as a CPU tensor."""
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).bfloat16()


def f64(t):
    return t.cpu().to(torch.float64).numpy()


def latent_cache(rng, rows, fp8):
    """A latent cache on the CPU and its rows in float64: ({C, c_scale, rope}, [rows, 576])."""
    if not fp8:
        C = bf16(rng, rows, 576)
        return dict(C=C, c_scale=None, rope=None), f64(C)
    x = rng.standard_normal((rows, 512)) * np.exp(0.5 * rng.standard_normal((rows, 1)))
    scale = (np.abs(x).max(1) / 448.0 * (0.9 + 0.2 * rng.random(rows))).astype(np.float32)  # any scale is read
    codes = torch.from_numpy(np.clip(x / scale[:, None], -448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
    rope = bf16(rng, rows, 64)
    K = np.concatenate([O.decode_e4m3fn(codes.view(torch.uint8).numpy()) * scale.astype(np.float64)[:, None],
                        f64(rope)], 1)
    return dict(C=codes, c_scale=torch.from_numpy(scale), rope=rope), K


def gpu(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def check_rows(label, got, lse, q, rows_of, dv, sm=SM, only=None):
    """got [T, H, dv] and lse [T, H] (GPU) against the oracle; rows_of(t, h) gives K, V of the query's keys."""
    got, lse = f64(got), f64(lse)
    T, H = lse.shape
    for t in (range(T) if only is None else only):
        for h in range(H):
            K, V = rows_of(t, h)
            n, nd = K.shape
            want, z, A, G = attend(f64(q[t, h]), K, V, sm)
            where = f"{label} t={t} h={h} n={n}"
            if n == 0:
                assert (got[t, h] == 0).all() and lse[t, h] == -math.inf, where
                continue
            eps = 2 * (nd + 8) * U * G + 2.0 ** -20
            tol = 1.01 * ((HALF + eps + (n + 16) * U) * A + HALF * np.abs(want))
            off = np.abs(got[t, h] - want)
            assert (off <= tol).all(), f"{where}: off by {off.max():.3e}, {np.max(off / tol):.2f} of the tolerance"
            ztol = 1.01 * ((nd + 8) * U * G + (n + 16) * U + 2.0 ** -20 + 8 * U * abs(z))
            assert abs(lse[t, h] - z) <= ztol, f"{where}: lse off by {abs(lse[t, h] - z):.3e} (tolerance {ztol:.3e})"


def check_latent(label, got, lse, q, K, pos=None, idx=None, base=None, only=None):
    def rows_of(t, h):
        r = latent_keys(K.shape[0], None if pos is None else pos[t], None if idx is None else idx[t],
                        0 if base is None else int(base[t]))
        return K[r], K[r][:, :512]
    check_rows(label, got, lse, q, rows_of, 512, only=only)


def check_expanded(label, got, lse, q, kv, rope, pos, base=None, only=None):
    kv, rope = f64(kv), f64(rope)
    L = kv.shape[0]

    def rows_of(t, h):
        r = latent_keys(L, pos[t], None, 0 if base is None else int(base[t]))
        return np.concatenate([kv[r, h, :128], rope[r]], 1), kv[r, h, 128:]
    check_rows(label, got, lse, q, rows_of, 128, only=only)
