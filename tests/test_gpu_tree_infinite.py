"""Scores of minus infinity and near the lowest number, infinite scales and values at their
limit, in keys that drafted tokens see: what the formula gives, on every width of the
attention over pages, whole and split, in committed keys and in drafted ones."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_amd as S
from attention_parity import SM, U, bf16, check_rows, f64, gpu, latent_cache
from oracle.attention import attend
from oracle.paged import tree_rows
from paged_parity import ints, random_trees, words
from test_gpu_attention_infinite import LN2
from test_gpu_tree_attention import cut_of

pytestmark = pytest.mark.gpu

PAGE = 64
CASES = [  # sequences, nodes, heads, longest prefix, the cut
    (260, 1, 3, 130, (16, False)), (2, 1, 3, 600, (16, True)), (300, 2, 16, 130, (32, False)), (9, 17, 3, 700, (32, True)),
    (70, 3, 33, 130, (64, False)), (40, 6, 20, 1000, (64, True)), (100, 3, 33, 130, (128, False)), (3, 50, 100, 900, (128, True)),
    (40, 16, 3, 1000, (128, True))]


def _scene(rng, seqs, N, longest, fp8):
    """Lengths, pages of each sequence's own, a cache and its rows, and trees."""
    per = -(-(longest + N) // PAGE)
    prefix = rng.integers(70, longest + 1, seqs)
    prefix[0] = longest
    table = rng.permutation(seqs * per).reshape(seqs, per).astype(np.int32)
    cache, K = latent_cache(rng, seqs * per * PAGE, fp8)
    return prefix, table, cache, K, random_trees(rng, seqs, N)


def _row(table, s, j):
    return int(table[s, j // PAGE]) * PAGE + j % PAGE


def _keys(table, K, prefix, mask, N):
    def rows(t):
        s, i = divmod(t, N)
        return tree_rows(table, PAGE, K.shape[0], s, int(prefix[s]), i, mask[s][i])
    return rows


def _call(q, prefix, table, cache, mask, longest, cut, sm=SM):
    ran, (out, lse) = cut_of(lambda: S.tree_attention(q.cuda(), ints(prefix), ints(table), PAGE, sm_scale=sm, mask=words(mask),
                                                      longest=longest, with_lse=True, **gpu(cache)))
    assert ran == cut
    return out.flatten(0, 1), lse.flatten(0, 1)


@pytest.mark.parametrize("seqs,N,H,longest,cut", CASES)
def test_an_infinite_scale(seqs, N, H, longest, cut):
    # every score with one committed key of the first sequence and with one drafted key of the last is -inf, by the key's scale
    rng = np.random.default_rng(seqs * N + H)
    prefix, table, cache, K, mask = _scene(rng, seqs, N, longest, True)
    q = bf16(rng, seqs, N, H, 576)
    q[..., :512] = q[..., :512].abs().clamp(min=0.01)
    bad = [_row(table, 0, 66), _row(table, seqs - 1, int(prefix[-1]) + N // 2)]
    for r in bad:
        cache["C"].view(torch.uint8)[r] = 0xb8                 # -1 in every place
        cache["c_scale"][r], K[r, :512] = 1.0, -1.0
    clean = _call(q, prefix, table, cache, mask, longest, cut)
    cache["c_scale"][bad] = float("inf")
    out, lse = _call(q, prefix, table, cache, mask, longest, cut)
    keys = _keys(table, K, prefix, mask, N)
    sees = torch.tensor([bool(np.isin(bad, keys(t)).any()) if t < N or t >= (seqs - 1) * N else False for t in range(seqs * N)])
    assert sees[:N].all() and sees[-N:].any()
    out, lse, clean = out.cpu(), lse.cpu(), [x.cpu() for x in clean]
    assert bool(out[sees].isnan().all()) and torch.equal(out[~sees], clean[0][~sees]) and torch.equal(lse[~sees], clean[1][~sees])
    flat = q.flatten(0, 1)
    for t in [0, (seqs - 1) * N + N // 2]:                     # the key weighs nothing in the log-sum
        r = np.setdiff1d(keys(t), bad)
        for h in range(min(H, 8)):
            _, z, _, G = attend(f64(flat[t, h]), K[r], K[r][:, :512], SM)
            tol = 1.01 * ((584 * U) * G + (len(r) + 16) * U + 2.0 ** -20 + 8 * U * abs(z))
            assert sees[t] and abs(float(lse[t, h]) - z) <= tol, (t, h)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", CASES)
def test_keys_that_score_minus_infinity(seqs, N, H, longest, cut, fp8):
    # all keys of the first sequence, all committed ones of the second, the first 66 and node 0 of the last
    rng = np.random.default_rng(seqs + N * H)
    prefix, table, cache, K, mask = _scene(rng, seqs, N, longest, fp8)
    q = bf16(rng, seqs, N, H, 576)
    q[..., 520] = 0.5
    low = {_row(table, 0, j) for j in range(prefix[0] + N)} | {_row(table, 1, j) for j in range(prefix[1])}
    if seqs > 2:
        low |= {_row(table, seqs - 1, j) for j in [*range(66), int(prefix[-1])]}
    low = np.array(sorted(low))
    (cache["rope"] if fp8 else cache["C"])[low, 8 if fp8 else 520] = float("-inf")
    out, lse = _call(q, prefix, table, cache, mask, longest, cut)
    assert bool(out[:N].isnan().all()) and bool((lse[:N] == -np.inf).all()) and bool(out[N:].isfinite().all())
    keys = _keys(table, K, prefix, mask, N)
    held = {}

    def finite(t, h):
        if t not in held:
            held.clear()
            r = np.setdiff1d(keys(t), low)
            held[t] = K[r], K[r][:, :512]
        return held[t]
    check_rows("the other keys", out, lse, q.flatten(0, 1), finite, 512, only=sorted({N, 2 * N - 1, (seqs - 1) * N, seqs * N - 1}))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", CASES)
def test_keys_after_scores_of_the_lowest_number(seqs, N, H, longest, cut, fp8):
    # a tile of keys whose scores are the lowest finite number, -(2 - 2^-23) 2^127, in three exact parts; then
    # keys of score 0, beside which they weigh nothing. With `all` every key scores it, and they weigh alike.
    rng = np.random.default_rng(seqs + H)
    per = -(-(longest + N) // PAGE)
    prefix = rng.integers(70, longest + 1, seqs)
    prefix[0] = longest
    cache, _ = latent_cache(rng, 2 * PAGE, fp8)
    cache["C"][:PAGE], cache["C"][PAGE:] = cache["C"][0].clone(), cache["C"][PAGE].clone()
    rope = cache["rope"] if fp8 else cache["C"][:, 512:]
    rope[:, 8:11] = 0.0
    rope[:PAGE, 8:11] = -torch.tensor([2 - 2.0 ** -7, 2.0 ** -7 - 2.0 ** -15, 2.0 ** -15 - 2.0 ** -23]).bfloat16() * 2.0 ** 63
    if fp8:
        cache["c_scale"][:] = 1.0
    q = torch.zeros(seqs, N, H, 576, dtype=torch.bfloat16)
    q[..., 520:523] = 2.0 ** 64
    mask, value = random_trees(rng, seqs, N), cache["C"][:, :512].float().bfloat16()
    seen = np.repeat(prefix, N) + np.array([bin(m[0]).count("1") for s in range(seqs) for m in mask[s]])
    for low, first in (("first", 1), ("all", per)):
        table = np.ones((seqs, per), dtype=np.int32)
        table[:, :first] = 0
        out, lse = _call(q, prefix, table, cache, mask, longest, cut, sm=LN2)
        assert torch.equal(out.cpu(), value[0 if low == "all" else PAGE].expand_as(out))
        n, z = (seen, -(2 - 2.0 ** -23) * 2.0 ** 127 * LN2) if low == "all" else (seen - 64, 0.0)
        want = torch.from_numpy(z + np.log(n))[:, None]
        tol = 2.0 ** -21 * 2.4e38 if low == "all" else (longest + N + 16) * U + 2.0 ** -20 + 8 * U * want.abs()
        assert bool(((lse.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", CASES)
def test_values_at_their_limit(seqs, N, H, longest, cut, fp8):
    # weights reach 2^31 before a reference is raised: keys times values stay below 2^96
    rng = np.random.default_rng(seqs * N * H)
    prefix, table, cache, K, mask = _scene(rng, seqs, N, longest, fp8)
    q = torch.zeros(seqs, N, H, 576, dtype=torch.bfloat16)
    q[..., 520] = 1.0
    large = 2.0 ** (95 - int(np.ceil(np.log2(longest + N))) - 3)   # (the cache's values are below 2^3 without it)
    rope = cache["rope"] if fp8 else cache["C"][:, 512:]
    rope[:, 8] = 31.0                                          # (scores rise after the first tile)
    rope[torch.tensor([_row(table, s, j) for s in range(seqs) for j in range(64)]), 8] = 0.0
    if fp8:
        cache["c_scale"] *= large / 448
        K[:, :512] *= large / 448
    else:
        cache["C"][:, :512] = cache["C"][:, :512].clamp(-8, 8) * large
        K[:, :512] = f64(cache["C"][:, :512])
    K[:, 512:] = f64(rope)
    out, lse = _call(q, prefix, table, cache, mask, longest, cut, sm=LN2)
    keys, held = _keys(table, K, prefix, mask, N), {}

    def rows(t, h):
        if t not in held:
            held.clear()
            held[t] = K[keys(t)], K[keys(t)][:, :512]
        return held[t]
    check_rows("large values", out, lse, q.flatten(0, 1), rows, 512, sm=LN2, only=[0, N - 1, seqs * N - 1])
