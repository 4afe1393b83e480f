"""Every way that a call of the attention is cut, with the cut asserted: a size
that the cost model moves to another kernel fails here by name. Prefixes of
queries that share their keys and of queries with a base of their own, lists, and
the expanded form with keys and values that are not finite on both of its widths."""
import numpy as np
import pytest
import torch

from attention_cut import EXPANDED, LATENT, cut_of
from attention_parity import SM, bf16, check_expanded, check_latent, check_rows, f64, gpu, latent_cache
from oracle.attention import latent_keys

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _bad_row(cache, row, fp8, bad):
    d = {n: (None if v is None else v.clone()) for n, v in cache.items()}
    if fp8:
        d["C"].view(torch.uint8)[row] = 0x7f
        d["c_scale"][row] = bad
        d["rope"][row] = bad
    else:
        d["C"][row] = bad
    return d


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,rows,cut", [
    (2, 3, 64, (16, False)), (2, 3, 200, (16, True)), (260, 3, 64, (32, False)), (70, 3, 400, (32, True)),
    (260, 20, 64, (64, False)), (70, 20, 1000, (64, True)), (520, 3, 64, (128, False)), (260, 3, 700, (128, True))])
def test_prefix_of_shared_keys(T, H, rows, cut, fp8):
    rng = np.random.default_rng(T + H + rows)
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    pos = np.linspace(rows - 1, 0, T).astype(np.int32)
    ran, (out, lse) = cut_of(lambda: S.latent_attention(q.cuda(), sm_scale=SM, pos=_ints(pos), with_lse=True, **gpu(cache)), LATENT)
    assert ran == cut
    check_latent("shared", out, lse, q, K, pos=pos, only=sorted({0, 1, T // 2, T - 1}))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,rows,cut", [
    (2, 3, 64, (16, False)), (2, 3, 200, (16, True)), (130, 20, 64, (32, False)), (20, 20, 2000, (32, True)),
    (130, 40, 64, (64, False)), (20, 100, 1000, (64, True)), (130, 70, 64, (128, False)), (70, 70, 2000, (128, True))])
def test_prefix_of_each_sequence(T, H, rows, cut, fp8):
    # several sequences in one cache: the rows before a base and after the end are other sequences' keys
    rng = np.random.default_rng(T + H + rows)
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    base = rng.integers(0, rows, T).astype(np.int32)
    base[0] = 0
    pos = rng.integers(0, rows, T).astype(np.int32)
    pos[0], pos[1] = rows - 1, -1
    if T > 8:
        pos[2], base[3], base[4], pos[5], base[5] = 2 ** 31 - 1, -1, rows, 0, rows - 1
        pos[6], base[6] = -2 ** 31, 2 ** 31 - 1
    args = dict(sm_scale=SM, pos=_ints(pos), base=_ints(base), with_lse=True)
    ran, (out, lse) = cut_of(lambda: S.latent_attention(q.cuda(), **gpu(cache), **args), LATENT)
    assert ran == cut
    check_latent("base", out, lse, q, K, pos=pos, base=base, only=sorted({0, 1, 2, 3, 4, 5, 6, T // 2, T - 1} & set(range(T))))
    row = rows // 2 + 5
    sees = torch.tensor([row in latent_keys(rows, int(p), None, int(b)) for p, b in zip(pos, base)])
    for bad in (float("nan"), float("inf")):
        o2, z2 = S.latent_attention(q.cuda(), **gpu(_bad_row(cache, row, fp8, bad)), **args)
        assert torch.equal(o2.cpu()[~sees], out.cpu()[~sees]) and torch.equal(z2.cpu()[~sees], lse.cpu()[~sees])
        assert bool(o2.cpu()[sees].isnan().all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,k,cut", [
    (2, 3, 64, (16, False)), (2, 3, 200, (16, True)), (130, 20, 64, (32, False)), (20, 20, 2000, (32, True)),
    (130, 40, 64, (64, False)), (20, 100, 1000, (64, True)), (130, 70, 64, (128, False)), (70, 70, 2000, (128, True))])
def test_lists(T, H, k, cut, fp8):
    rng = np.random.default_rng(T + H + k)
    rows = k + 100
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    idx = rng.integers(-40, rows, (T, k)).astype(np.int32)
    idx[idx < 0] = -1
    idx[1, 1:] = -1
    ran, (out, lse) = cut_of(lambda: S.latent_attention(q.cuda(), sm_scale=SM, idx=_ints(idx), with_lse=True, **gpu(cache)), LATENT)
    assert ran == cut
    check_latent("list", out, lse, q, K, idx=idx, only=sorted({0, 1, T // 2, T - 1}))


@pytest.mark.parametrize("T,H,L,cut", [(300, 64, 300, (128, False)), (300, 2, 5000, (128, True)),
                                       (500, 256, 512, (256, False)), (500, 64, 3000, (256, True))])
def test_expanded_with_bad_keys_and_values(T, H, L, cut):
    # two sequences and keys of nobody between them; what is not finite reaches the queries that see it
    rng = np.random.default_rng(T + H + L)
    q, kv, rope = bf16(rng, T, H, 192), bf16(rng, L, H, 256), bf16(rng, L, 64)
    n0, first1 = L // 2 - 20, L // 2 + 20
    half = T // 2
    base = np.where(np.arange(T) < half, 0, first1).astype(np.int32)
    pos = np.concatenate([np.linspace(0, n0 - 1, half), np.linspace(-9, L - first1 - 1, T - half)]).astype(np.int32)
    qg, kg, rg = q.cuda(), kv.cuda(), rope.cuda()
    args = (_ints(pos), SM)
    ran, (out, lse) = cut_of(lambda: S.expanded_attention(qg, kg, rg, *args, base=_ints(base), with_lse=True), EXPANDED)
    assert ran == cut
    some = [0, 1, half - 1, half, T - 1]
    kd, rd = f64(kv[:, :2]), f64(rope)

    def rows_of(t, h):
        r = latent_keys(L, int(pos[t]), None, int(base[t]))
        return np.concatenate([kd[r, h, :128], rd[r]], 1), kd[r, h, 128:]
    check_rows("expanded", out[:, :2], lse[:, :2], q[:, :2], rows_of, 128, only=some)

    kg[n0:first1] = float("nan")                              # keys of nobody
    rg[n0:first1] = float("inf")
    o2, z2 = S.expanded_attention(qg, kg, rg, *args, base=_ints(base), with_lse=True)
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    v, w, u = n0 * 3 // 4, first1 + (L - first1) // 2, L - 1
    kg[v, 1, 130], kg[w, 0, 200], rg[u] = float("nan"), float("-inf"), float("nan")
    o2, z2 = S.expanded_attention(qg, kg, rg, *args, base=_ints(base), with_lse=True)
    sees = lambda r: torch.tensor([r in latent_keys(L, int(p), None, int(b)) for p, b in zip(pos, base)]).cuda()  # noqa: E731
    hit = torch.zeros(T, H, 128, dtype=torch.bool, device="cuda")
    hit[sees(v), 1, 2] = True
    hit[sees(w), 0, 72] = True
    hit[sees(u)] = True
    assert bool(sees(v).any()) and bool(sees(w).any()) and bool(sees(u).any()) and not bool(hit.all())
    assert torch.equal(o2[~hit], out[~hit]) and bool(o2[sees(u)].isnan().all()) and bool(o2[sees(v), 1, 2].isnan().all())
    assert bool((o2[sees(w) & ~sees(u), 0, 72] == float("-inf")).all())
    assert torch.equal(z2[~sees(u)], lse[~sees(u)]) and bool(z2[sees(u)].isnan().all())
