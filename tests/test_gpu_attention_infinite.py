"""Scores of minus infinity and values that are infinite, in keys that a query
sees: what the formula gives (a weight of zero times an infinite value is NaN), on
every width, whatever tile the key lies in."""
import numpy as np
import pytest
import torch

from attention_cut import LATENT, cut_of
from attention_parity import SM, U, bf16, f64, gpu, latent_cache
from oracle.attention import attend, latent_keys

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")

SHARED = [(2, 3, 130, (16, False)), (20, 3, 1000, (16, True)), (260, 3, 130, (32, False)), (128, 3, 400, (32, True)),
          (260, 20, 130, (64, False)), (130, 20, 700, (64, True)), (520, 3, 130, (128, False)), (260, 3, 700, (128, True))]
LISTS = [(2, 3, 130, (16, False)), (20, 3, 1000, (16, True)), (130, 20, 130, (32, False)), (20, 20, 2000, (32, True)),
         (130, 33, 130, (64, False)), (64, 33, 1000, (64, True)), (130, 70, 130, (128, False)), (70, 70, 2000, (128, True))]


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _infinite_scale(rng, T, H, rows, key):
    """A coded cache and queries whose every score with row `key` is -inf, by its infinite scale alone."""
    cache, K = latent_cache(rng, rows, True)
    q = bf16(rng, T, H, 576)
    q[:, :, :512] = q[:, :, :512].abs().clamp(min=0.01)
    cache["C"].view(torch.uint8)[key] = 0xb8                   # -1 in every place
    K[key, :512] = -1.0
    cache["c_scale"][key] = 1.0
    return q, cache, K


def _check(got, clean, q, K, keys_of, key, only):
    sees = np.array([key in keys_of(t) for t in range(q.shape[0])])
    assert sees.any()
    out, lse = got
    assert bool(out.cpu()[torch.from_numpy(sees)].isnan().all())
    assert torch.equal(out.cpu()[torch.from_numpy(~sees)], clean[0].cpu()[torch.from_numpy(~sees)])
    assert torch.equal(lse.cpu()[torch.from_numpy(~sees)], clean[1].cpu()[torch.from_numpy(~sees)])

    for t in only:                                             # the key weighs nothing in the log-sum
        r = keys_of(t)
        r = r[r != key]
        for h in range(q.shape[1]):
            _, z, _, G = attend(f64(q[t, h]), K[r], K[r][:, :512], SM)
            tol = 1.01 * ((584 * U) * G + (len(r) + 16) * U + 2.0 ** -20 + 8 * U * abs(z))
            assert sees[t] and abs(float(lse[t, h]) - z) <= tol, (t, h)


@pytest.mark.parametrize("T,H,rows,cut", SHARED)
def test_prefix_with_an_infinite_scale(T, H, rows, cut):
    rng = np.random.default_rng(T + H + rows)
    key = 100
    q, cache, K = _infinite_scale(rng, T, H, rows, key)
    sees = np.arange(T) % 2 == 0
    pos = np.where(sees, rng.integers(key, rows, T), rng.integers(70, key, T))
    pos[0] = key                                               # the key in the query's last tile, and (below) in a full one
    pos[T // 2 * 2 - 2] = rows - 1
    call = lambda: S.latent_attention(q.cuda(), sm_scale=SM, pos=_ints(pos), with_lse=True, **gpu(cache))  # noqa: E731
    ran, clean = cut_of(call, LATENT)
    assert ran == cut
    cache["c_scale"][key] = float("inf")
    _check(call(), clean, q, K, lambda t: latent_keys(rows, int(pos[t])), key, [0, T // 2 * 2 - 2])


@pytest.mark.parametrize("T,H,k,cut", LISTS)
def test_list_with_an_infinite_scale(T, H, k, cut):
    rng = np.random.default_rng(T + H + k)
    rows, key = k + 50, 17
    q, cache, K = _infinite_scale(rng, T, H, rows, key)
    idx = rng.integers(key + 1, rows, (T, k))
    idx[::2, 90] = key
    call = lambda: S.latent_attention(q.cuda(), sm_scale=SM, idx=_ints(idx), with_lse=True, **gpu(cache))  # noqa: E731
    ran, clean = cut_of(call, LATENT)
    assert ran == cut
    cache["c_scale"][key] = float("inf")
    _check(call(), clean, q, K, lambda t: latent_keys(rows, None, idx[t]), key, [0])
