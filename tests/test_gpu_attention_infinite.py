"""Scores of minus infinity and near the lowest number, and values that are infinite, in keys that a query
sees: what the formula gives (a weight of zero times an infinite value is NaN), on
every width, whatever tile the key lies in."""
import numpy as np
import pytest
import torch

from attention_cut import EXPANDED, LATENT, cut_of
from attention_parity import SM, U, bf16, check_rows, f64, gpu, latent_cache
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


# ------------------------------------------------ scores near the lowest number

LN2 = 0.6931471824645996                                       # times log2(e) in fp32: 1


def _far_below(rng, T, H, rows, width, rotary, fp8=False):
    """Queries and a cache whose every score in powers of two is -1.9375 * 2^127 (-3.297e38), by one rotary value."""
    q = torch.zeros(T, H, width, dtype=torch.bfloat16)
    q[:, :, width - rotary + 8] = 2.0 ** 64
    cache, K = latent_cache(rng, rows, fp8)
    (cache["rope"] if fp8 else cache["C"])[:, 8 if fp8 else 520] = -1.9375 * 2.0 ** 63
    return q, cache, K


def _own_row(out, lse, want, n):
    """Every key of the query is the same row: its values, and its score plus log n."""
    assert torch.equal(out.cpu(), want.expand_as(out).to(torch.bfloat16))
    z = lse.cpu().double()
    assert bool((z - (-1.9375 * 2.0 ** 127 * LN2 + np.log(n))).abs().max() <= 2.0 ** -21 * 2.3e38)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,k,cut", LISTS)
def test_list_of_scores_far_below_zero(T, H, k, cut, fp8):
    q, cache, K = _far_below(np.random.default_rng(k), T, H, 40, 576, 64)
    if fp8:                                                    # (scales of 1: the values are exact in bf16)
        q, cache, K = _far_below(np.random.default_rng(k), T, H, 40, 576, 64, True)
        cache["c_scale"][:] = 1.0
    vals = cache["C"][:, :512].float()
    idx = torch.arange(T)[:, None].expand(T, k) % 40
    ran, (out, lse) = cut_of(lambda: S.latent_attention(q.cuda(), sm_scale=LN2, idx=_ints(idx), with_lse=True, **gpu(cache)), LATENT)
    assert ran == cut
    _own_row(out, lse, vals[torch.arange(T) % 40][:, None], k)


@pytest.mark.parametrize("T,H,rows,cut", SHARED)
def test_prefix_of_scores_far_below_zero(T, H, rows, cut):
    q, cache, K = _far_below(np.random.default_rng(rows), T, H, rows, 576, 64)
    cache["C"][:] = cache["C"][:1].clone()
    pos = np.full(T, rows - 1)
    pos[::2] = rows - 60
    ran, (out, lse) = cut_of(lambda: S.latent_attention(q.cuda(), sm_scale=LN2, pos=_ints(pos), with_lse=True, **gpu(cache)), LATENT)
    assert ran == cut
    _own_row(out, lse, cache["C"][0, :512], rows)


@pytest.mark.parametrize("T,H,L,cut", [(300, 16, 300, (128, False)), (300, 2, 5000, (128, True)),
                                       (500, 256, 512, (256, False)), (500, 64, 3000, (256, True))])
def test_expanded_scores_far_below_zero(T, H, L, cut):
    q, _, _ = _far_below(np.random.default_rng(L), T, H, 1, 192, 64)
    kv = bf16(np.random.default_rng(L), 1, H, 256)
    rope = torch.zeros(L, 64, dtype=torch.bfloat16)
    rope[:, 8] = -1.9375 * 2.0 ** 63
    call = lambda: S.expanded_attention(q.cuda(), kv.cuda().expand(L, H, 256).contiguous(), rope.cuda(),  # noqa: E731
                                        _ints(np.arange(L - T, L)), LN2, with_lse=True)
    ran, (out, lse) = cut_of(call, EXPANDED)
    assert ran == cut
    _own_row(out, lse, kv[0, :, 128:], L)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,k,cut", LISTS)
def test_keys_after_scores_of_the_lowest_number(T, H, k, cut, fp8):
    # a tile of keys whose scores are the lowest finite number, -(2 - 2^-23) 2^127, in three exact parts; then
    # keys of score 0, beside which they weigh nothing
    cache, K = latent_cache(np.random.default_rng(k), 40, fp8)
    q = torch.zeros(T, H, 576, dtype=torch.bfloat16)
    q[:, :, 520:523] = 2.0 ** 64
    rope = cache["rope"] if fp8 else cache["C"][:, 512:]
    rope[:, 8:11] = 0.0
    rope[0, 8:11] = -torch.tensor([2 - 2.0 ** -7, 2.0 ** -7 - 2.0 ** -15, 2.0 ** -15 - 2.0 ** -23]).bfloat16() * 2.0 ** 63
    if fp8:
        cache["c_scale"][:] = 1.0
    idx = torch.zeros(T, k, dtype=torch.int64)
    idx[:, 64:] = 7
    ran, (out, lse) = cut_of(lambda: S.latent_attention(q.cuda(), sm_scale=LN2, idx=_ints(idx), with_lse=True, **gpu(cache)), LATENT)
    assert ran == cut
    assert torch.equal(out.cpu(), cache["C"][7, :512].float().bfloat16().expand(T, H, 512))
    assert bool((lse.cpu().double() - np.log(k - 64)).abs().max() <= (k + 16) * U + 2.0 ** -20 + 8 * U * np.log(k))


# ---------------------------------------------- queries whose keys all score -inf

def _minus_inf_rows(rng, T, H, rows, fp8, upto):
    """Rows 0 .. upto - 1 score -inf with every query, by one rotary value; their values are finite."""
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    q[:, :, 520] = 0.5
    (cache["rope"] if fp8 else cache["C"])[:upto, 8 if fp8 else 520] = float("-inf")
    return q, cache, K


def _check_minus_inf(got, q, K, keys_of, upto, only):
    """keys_of(t): the query's keys; those below `upto` score -inf."""
    out, lse = (x.cpu() for x in got)
    kinds = set()
    for t in only:
        r = keys_of(t)
        real = r[r >= upto]
        kind = "none" if not len(r) else "all -inf" if not len(real) else "some"
        kinds.add(kind)
        if kind == "none":
            assert not out[t].any() and bool((lse[t] == -np.inf).all()), t
        elif kind == "all -inf":
            assert bool(out[t].isnan().all()) and bool((lse[t] == -np.inf).all()), t
    check_rows("the other keys", got[0], got[1], q, lambda t, h: (K[keys_of(t)[keys_of(t) >= upto]], K[keys_of(t)[keys_of(t) >= upto]][:, :512]), 512,
               only=[t for t in only if (keys_of(t) >= upto).any()])
    assert "all -inf" in kinds
    return kinds


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,k,cut", LISTS)
def test_list_of_keys_that_score_minus_infinity(T, H, k, cut, fp8):
    rng = np.random.default_rng(T + H + k)
    rows, upto = k + 50, 9
    q, cache, K = _minus_inf_rows(rng, T, H, rows, fp8, upto)
    idx = rng.integers(0, rows, (T, k))
    idx[0] = rng.integers(0, upto, k)                          # all of them -inf
    if T > 2:
        idx[1] = -1                                            # no key
        idx[2] = -1                                            # one, -inf, the rest padding
        idx[2, k - 2] = 3
        idx[3, :k - 1] = rng.integers(0, upto, k - 1)          # one that is not, in the last place
        idx[3, k - 1] = upto
    call = lambda: S.latent_attention(q.cuda(), sm_scale=SM, idx=_ints(idx), with_lse=True, **gpu(cache))  # noqa: E731
    ran, got = cut_of(call, LATENT)
    assert ran == cut
    _check_minus_inf(got, q, K, lambda t: latent_keys(rows, None, idx[t]), upto, sorted({0, 1, 2, 3, T - 1} & set(range(T))))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("based", [False, True])
@pytest.mark.parametrize("T,H,rows", [(2, 3, 130), (20, 3, 1000), (260, 3, 130), (128, 3, 400), (260, 20, 130), (130, 20, 700), (520, 3, 130),
                                      (260, 3, 700), (130, 33, 130), (64, 33, 1000), (130, 70, 130), (70, 70, 2000)])
def test_prefix_of_keys_that_score_minus_infinity(T, H, rows, based, fp8):
    rng = np.random.default_rng(T + H + rows)
    upto = 75                                                  # the first tile and a part of the second
    q, cache, K = _minus_inf_rows(rng, T, H, rows, fp8, upto)
    pos = rng.integers(-1, rows, T)
    pos[0], pos[1], pos[T - 1] = 5, 80, upto - 1
    if T > 2:
        pos[2], pos[3], pos[4] = -1, upto, rows - 1
    base = rng.integers(0, 9, T) if based else np.zeros(T, dtype=np.int64)
    base[:2] = 0
    if T == 2:
        pos[1] = upto - 1
    args = dict(sm_scale=SM, pos=_ints(pos), base=_ints(base) if based else None, with_lse=True)
    got = S.latent_attention(q.cuda(), **gpu(cache), **args)
    _check_minus_inf(got, q, K, lambda t: latent_keys(rows, int(pos[t]), None, int(base[t])), upto,
                     sorted({0, 1, 2, 3, 4, T - 1} & set(range(T))))


@pytest.mark.parametrize("T,H,L,cut", [(300, 16, 300, (128, False)), (300, 2, 5000, (128, True)),
                                       (500, 256, 512, (256, False)), (500, 64, 3000, (256, True))])
def test_expanded_keys_that_score_minus_infinity(T, H, L, cut):
    rng = np.random.default_rng(T + H + L)
    q, kv, rope = bf16(rng, T, H, 192), bf16(rng, L, H, 256), bf16(rng, L, 64)
    q[:, :, 136] = 0.5
    upto = L - 90
    rope[:upto, 8] = float("-inf")
    pos = rng.integers(-1, L, T)
    pos[:6] = [5, upto - 1, -1, upto, L - 1, 0]
    call = lambda: S.expanded_attention(q.cuda(), kv.cuda(), rope.cuda(), _ints(pos), SM, with_lse=True)  # noqa: E731
    ran, (out, lse) = cut_of(call, EXPANDED)
    assert ran == cut
    n = torch.from_numpy(pos + 1).cuda()
    assert bool(out[(n > 0) & (n <= upto)].isnan().all()) and not bool(out[n == 0].any())
    assert bool((lse[n <= upto] == float("-inf")).all()) and bool(lse[n > upto].isfinite().all())
    kd, rd = f64(kv[:, :2]), f64(rope)
    check_rows("the other keys", out[:, :2], lse[:, :2], q[:, :2],
               lambda t, h: (np.concatenate([kd[upto:pos[t] + 1, h, :128], rd[upto:pos[t] + 1]], 1), kd[upto:pos[t] + 1, h, 128:]),
               128, only=[3, 4])


# ------------------------------------------------------------- values at their limit

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,k,cut", LISTS)
def test_values_at_their_limit(T, H, k, cut, fp8):
    # weights reach 2^31 before a reference is raised: keys times values stay below 2^96
    rng = np.random.default_rng(T + H + k)
    rows = 60
    cache, K = latent_cache(rng, rows, fp8)
    q = torch.zeros(T, H, 576, dtype=torch.bfloat16)
    q[:, :, 520] = 1.0
    large = 2.0 ** (95 - int(np.ceil(np.log2(k))) - 3)         # (the cache's values are below 2^3 without it)
    rope = cache["rope"] if fp8 else cache["C"][:, 512:]
    rope[:30, 8], rope[30:, 8] = 0.0, 31.0
    if fp8:
        cache["c_scale"] *= large / 448
        K[:, :512] *= large / 448
    else:
        cache["C"][:, :512] = cache["C"][:, :512].clamp(-8, 8) * large
        K[:, :512] = f64(cache["C"][:, :512])
    K[:, 512:] = f64(rope)
    idx = rng.integers(0, 30, (T, k))
    idx[:, 64:] = rng.integers(30, rows, (T, k - 64))          # (scores rise after the first tile)
    ran, (out, lse) = cut_of(lambda: S.latent_attention(q.cuda(), sm_scale=LN2, idx=_ints(idx), with_lse=True, **gpu(cache)), LATENT)
    assert ran == cut
    check_rows("large values", out, lse, q, lambda t, h: (K[idx[t]], K[idx[t]][:, :512]), 512, sm=LN2, only=[0, T - 1])
