"""Attention of drafted tokens over paged caches against the oracle in 64 bits: every
cut of a call (asserted by the launches' names), chains, trees and padding, sequences of
different lengths, selections, pages of 1 to 1024 rows and pages that are missing, and
what a query does not see."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_amd as S
from attention_parity import SM, bf16, gpu, latent_cache
from paged_parity import check_tree, ints, random_trees, tables, words

pytestmark = pytest.mark.gpu

NAMES = {16: "k_tree_16", 32: "k_tree_32", 64: "k_tree_64", 128: "k_tree_128"}


def cut_of(call):
    """(rows of a workgroup, whether parts were joined) of the one call that call() makes, and its result."""
    torch.cuda.synchronize()
    S.profile_reset()
    S.profile_enable(True)
    try:
        got = call()
        torch.cuda.synchronize()
    finally:
        S.profile_enable(False)
    ran = [rows for rows, name in NAMES.items() if S.profile_read(name)[1]]
    joined, total = S.profile_read("k_tree_join")[1], S.profile_read("")[1]
    S.profile_reset()
    assert len(ran) == 1 and total == 1 + joined, (ran, joined, total)
    return (ran[0], joined == 1), got


def _some(S_, N, count=8):
    T = S_ * N
    return sorted({0, 1 % T, N - 1, T // 2, T - 1, *np.linspace(0, T - 1, count).astype(int).tolist()})


CUTS = [  # sequences, nodes, heads, longest prefix, the cut
    (2, 1, 3, 50, (16, False)), (2, 1, 3, 600, (16, True)), (3, 5, 16, 50, (16, False)), (300, 2, 16, 100, (32, False)),
    (9, 17, 3, 700, (32, True)), (70, 3, 33, 30, (64, False)), (40, 6, 20, 1000, (64, True)), (300, 2, 128, 100, (128, False)),
    (20, 16, 3, 700, (32, False)), (4, 7, 128, 500, (16, False)), (3, 40, 40, 300, (32, False)),
    (24, 4, 128, 2000, (64, True)), (40, 16, 3, 1000, (128, True))]  # (the last: rows of four nodes share a workgroup)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", CUTS)
def test_every_cut(seqs, N, H, longest, cut, fp8):
    rng = np.random.default_rng(seqs * N + H + longest)
    page = 64
    per = -(-(longest + N) // page)
    table, pool = tables(rng, seqs, per)
    cache, K = latent_cache(rng, pool * page, fp8)
    q = bf16(rng, seqs, N, H, 576)
    prefix = rng.integers(0, longest + 1, seqs)
    prefix[0], prefix[-1] = longest, 0
    if seqs > 4:
        prefix[2] = -1
    mask = random_trees(rng, seqs, N, pad=1 if N > 2 else 0)
    call = lambda m: S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=m, longest=longest, with_lse=True,  # noqa: E731
                                      **gpu(cache))
    only = _some(seqs, N)
    ran, (out, lse) = cut_of(lambda: call(words(mask)))
    assert ran == cut
    check_tree("trees", out, lse, q, K, table, page, prefix, mask=mask, only=only)
    ran, (out, lse) = cut_of(lambda: call(None))
    assert ran == cut
    check_tree("chains", out, lse, q, K, table, page, prefix, only=only)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 2, 16, 128, 1024])
@pytest.mark.parametrize("H", [1, 16, 40])
def test_pages(page, H, fp8):
    rng = np.random.default_rng(page + H)
    seqs, N = 3, 6
    per = -(-200 // page)
    table, pool = tables(rng, seqs, per)
    cache, K = latent_cache(rng, pool * page - (page // 2 if page > 1 else 0), fp8)   # the last page is cut short
    table[1, per // 2] = -1                                          # a page that is gone
    if page <= 16:
        table[2, :per - 1] = table[0, :per - 1]                      # a shared prompt
        table[2, 0] = 1 << 26                                        # no page of this cache
    q, prefix = bf16(rng, seqs, N, H, 576), [194, 130, 63]
    mask = random_trees(rng, seqs, N)
    out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=words(mask), with_lse=True, **gpu(cache))
    check_tree(f"page {page}", out, lse, q, K, table, page, prefix, mask=mask)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H", [(1, 1, 16), (2, 130, 2), (2, 70, 20), (1, 200, 40)])
def test_long_chains_and_masks_of_several_words(seqs, N, H, fp8):
    rng = np.random.default_rng(N)
    page, longest = 32, 150
    table, pool = tables(rng, seqs, -(-(longest + N) // page))
    cache, K = latent_cache(rng, pool * page, fp8)
    q, prefix = bf16(rng, seqs, N, H, 576), rng.integers(0, longest + 1, seqs)
    only = _some(seqs, N, 10)
    out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, with_lse=True, **gpu(cache))
    check_tree("chain", out, lse, q, K, table, page, prefix, only=only)
    mask = random_trees(rng, seqs, N, words_a_mask=-(-N // 64) + 1)
    out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=words(mask), with_lse=True, **gpu(cache))
    check_tree("tree", out, lse, q, K, table, page, prefix, mask=mask, only=only)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,k", [(1, 1, 16, 1), (2, 3, 5, 100), (3, 7, 64, 300), (1, 70, 20, 65), (40, 2, 128, 64), (2, 2, 16, 1100)])
def test_selections(seqs, N, H, k, fp8):
    rng = np.random.default_rng(seqs + N + k)
    page, longest = 16, 700
    table, pool = tables(rng, seqs, -(-(longest + N) // page))
    table[0, 2] = -1
    cache, K = latent_cache(rng, pool * page, fp8)
    q, prefix = bf16(rng, seqs, N, H, 576), rng.integers(0, longest + 1, seqs)
    prefix[0] = longest
    if seqs > 2:
        prefix[1] = -1
    idx = rng.integers(-1, longest + 20, (seqs, N, k)).astype(np.int32)       # some past the prefix, some twice
    idx[-1, -1] = -1                                                           # no selection at all
    idx[0, 0, 0] = 2 ** 31 - 1
    mask = random_trees(rng, seqs, N, pad=1 if N > 2 else 0)
    for m in (mask, None):
        out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=None if m is None else words(m),
                                    idx=ints(idx), with_lse=True, **gpu(cache))
        check_tree("selection", out, lse, q, K, table, page, prefix, mask=m, idx=idx, only=_some(seqs, N))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", CUTS)
def test_what_a_query_does_not_see_has_no_effect(seqs, N, H, longest, cut, fp8):
    # every row outside the committed keys and a mask's nodes holds NaN or an infinity, and so do padding's queries
    rng = np.random.default_rng(seqs + N + H)
    page, per = 16, -(-(longest + N + 20) // 16)
    table, pool = tables(rng, seqs, per)
    cache, _ = latent_cache(rng, pool * page, fp8)
    prefix = rng.integers(0, longest + 1, seqs)
    prefix[0] = longest
    if seqs > 4:
        prefix[1] = -5
    mask = random_trees(rng, seqs, N, pad=1 if N > 2 else 0)
    if N > 4:                                                                  # the last node sees itself alone, and no other sees it
        for s in range(seqs):
            mask[s][N - 2] = [1 << (N - 2)]
    seen = torch.zeros(pool * page, dtype=torch.bool)
    for s in range(seqs):
        at = list(range(prefix[s])) + [prefix[s] + b for b in range(N) if any(m[0] >> b & 1 for m in mask[s])] if prefix[s] >= 0 else []
        seen[[int(table[s, j // page]) * page + j % page for j in at]] = True
    q = bf16(rng, seqs, N, H, 576)
    call = lambda q, c: S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=words(mask), longest=longest,  # noqa: E731
                                         with_lse=True, **gpu(c))
    want = call(q, cache)
    bad, qbad = {n: None if t is None else t.clone() for n, t in cache.items()}, q.clone()
    junk = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(pool * page) % 3]
    if fp8:
        bad["c_scale"][~seen] = junk[~seen]
        bad["C"].view(torch.uint8)[~seen] = 0x7f
        bad["rope"][~seen] = junk[~seen, None].bfloat16()
    else:
        bad["C"][~seen] = junk[~seen, None].bfloat16()
    dead = torch.tensor([[prefix[s] < 0 or not any(mask[s][i]) for i in range(N)] for s in range(seqs)])
    qbad[dead] = float("nan")
    got = call(qbad, bad)
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
    assert bool((got[0].cpu()[dead] == 0).all()) and bool((got[1].cpu()[dead] == -float("inf")).all())
    assert bool(got[0].isfinite().all())
    if N > 4:
        # a node that holds NaN: those that see it, and no other
        row = int(table[0, (prefix[0] + N - 2) // page]) * page + (prefix[0] + N - 2) % page
        if fp8:
            bad["c_scale"][row] = float("nan")
        else:
            bad["C"][row] = float("nan")
        out, lse = call(qbad, bad)
        assert bool(out[0, N - 2].isnan().all()) and bool(lse[0, N - 2].isnan().all())
        out[0, N - 2], lse[0, N - 2] = got[0][0, N - 2], got[1][0, N - 2]
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_longest_decides_the_cut_alone(fp8):
    rng = np.random.default_rng(11)
    seqs, N, H, page = 6, 3, 24, 64
    table, pool = tables(rng, seqs, 32)
    cache, K = latent_cache(rng, pool * page, fp8)
    q, prefix = bf16(rng, seqs, N, H, 576), [2045, 3, 700, 0, 64, 1999]
    for longest in (0, 1, 100, 2000, 1 << 30):
        out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, longest=longest, with_lse=True, **gpu(cache))
        check_tree(f"longest {longest}", out, lse, q, K, table, page, prefix, only=[0, 2, 4, 9, 13, 17])


def test_one_token_equals_latent_attention():
    # pages in order: the same keys as a prefix or a list gives, to within the roundings of another cut
    rng = np.random.default_rng(12)
    rows, T, H = 1000, 3, 16
    cache, K = latent_cache(rng, rows, True)
    q, pos = bf16(rng, T, H, 576), np.array([999, 400, 0])
    table = np.tile(np.arange(rows // 8, dtype=np.int32), (T, 1))
    out, lse = S.tree_attention(q[:, None].contiguous().cuda(), ints(pos), ints(table), 8, sm_scale=SM, with_lse=True, **gpu(cache))
    check_tree("one token", out, lse, q[:, None], K, table, 8, pos)
    idx = np.where(np.arange(rows) <= pos[:, None], np.arange(rows), -1)
    lists = S.latent_attention(q.cuda(), sm_scale=SM, idx=ints(idx), with_lse=True, **gpu(cache))
    assert bool(((lists[1] - lse[:, 0]).abs() <= 1e-5 * lse[:, 0].abs()).all())
    assert bool(((lists[0] - out[:, 0]).float().abs() <= 2.0 ** -5).all())      # two results of a few tenths, each off by 2^-7 of sum p|v|


def test_bits_streams_graphs_and_workspaces():
    rng = np.random.default_rng(13)
    seqs, N, H, page, longest = 5, 8, 32, 16, 900
    table, pool = tables(rng, seqs, -(-(longest + N) // page))
    cache, _ = latent_cache(rng, pool * page, True)
    q, prefix, mask = bf16(rng, seqs, N, H, 576).cuda(), ints([900, 10, 500, 0, -1]), words(random_trees(rng, seqs, N))
    idx = ints(rng.integers(-1, longest, (seqs, N, 200)))
    c, t = gpu(cache), ints(table)
    side = torch.cuda.Stream()
    for kw in (dict(), dict(idx=idx)):
        p = S.make_tree_problem(q, prefix, t, page, sm_scale=SM, mask=mask, longest=longest, **c, **kw)
        n = S.lib().misa_tree_workspace_bytes(p)
        assert n > 256
        ws, out = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda"), torch.empty(seqs, N, H, 512, dtype=torch.bfloat16, device="cuda")
        call = lambda **k: S.tree_attention(q, prefix, t, page, sm_scale=SM, mask=mask, longest=longest, with_lse=True, **c, **kw, **k)  # noqa: E731
        want = call()
        got = call(ws=ws, out=out)
        assert got[0] is out and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert bool((ws[n:] == 255).all())                                     # nothing behind the workspace
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = call()
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        g, ws = torch.cuda.CUDAGraph(), torch.empty(n, dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(g):
            got = call(ws=ws)
        for i in range(4):
            ws.fill_(i * 85)
            got[0].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(call()[0], want[0])                             # eager work between the replays
        # another batch through the same graph: what lies in the inputs is read anew
        prefix.copy_(ints([1, 2, 900, -1, 33]))
        fresh = call()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], fresh[0]) and torch.equal(got[1], fresh[1])
        prefix.copy_(ints([900, 10, 500, 0, -1]))


def test_a_rows_bits_are_its_own():
    # the same sequence alone and among others, under the same cut of its keys: a batch of equal sequences
    rng = np.random.default_rng(14)
    N, H, page = 4, 48, 64
    table, pool = tables(rng, 1, 5)
    cache, _ = latent_cache(rng, pool * page, False)
    q = bf16(rng, 1, N, H, 576)
    for seqs in (300, 600):                                                    # (never split)
        many = q.expand(seqs, N, H, 576).contiguous()
        noise = many.clone()
        noise[1:] = bf16(rng, seqs - 1, N, H, 576)
        call = lambda x: S.tree_attention(x.cuda(), ints([300] * seqs), ints(np.tile(table, (seqs, 1))), page, sm_scale=SM, **gpu(cache))  # noqa: E731
        a, b = call(many), call(noise)
        assert bool((a == a[0]).all()) and torch.equal(a[0], b[0])


def test_rows_far_into_a_long_cache():
    rng = np.random.default_rng(15)
    rows, page = 4_200_000, 64                                                 # byte offsets pass 2^32
    C = torch.full((rows, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    far = rows // page - 1
    table = np.array([[far, 0, far - 1]], dtype=np.int32)
    at = np.concatenate([np.arange(64) + v * page for v in table[0]])
    K = bf16(rng, 192, 576)
    C[torch.from_numpy(at).cuda()] = K.cuda()
    q = bf16(rng, 1, 2, 16, 576)
    out, lse = S.tree_attention(q.cuda(), ints([150]), ints(table), page, C, SM, with_lse=True)
    check_tree("far", out, lse, q, K.double().numpy(), np.array([[0, 1, 2]]), page, [150])
    idx = ints(np.arange(150)[None, None].repeat(2, 1))
    out, lse = S.tree_attention(q.cuda(), ints([150]), ints(table), page, C, SM, idx=idx, with_lse=True)
    check_tree("far, a list", out, lse, q, K.double().numpy(), np.array([[0, 1, 2]]), page, [150])


def test_empty_calls_and_refusals():
    rng = np.random.default_rng(16)
    C, q = bf16(rng, 64, 576).cuda(), bf16(rng, 2, 3, 4, 576).cuda()
    t, n = ints([[0, 1], [2, 3]]), ints([5, 6])
    out, lse = S.tree_attention(q[:0], n[:0], t[:0], 16, C, SM, with_lse=True)
    assert out.shape == (0, 3, 4, 512) and lse.shape == (0, 3, 4)
    i64 = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    assert S.tree_attention(q[:0], n[:0], t[:0], 16, C, SM, mask=i64[:0], idx=i64.int()[:0, :, None]).shape == (0, 3, 4, 512)
    ok = dict(q=q, prefix=n, table=t, page=16, C=C, sm_scale=SM)
    for bad, text in [(dict(q=q[0]), "4 dimensions"), (dict(q=q[..., :512].contiguous()), "q has shape"), (dict(prefix=n.long()), "prefix must be"),
                      (dict(prefix=n[:1]), "prefix has shape"), (dict(table=t[:1]), "sequences"), (dict(table=t[0]), "2 dimensions"),
                      (dict(mask=i64.int()), "mask must be"), (dict(mask=i64[:, :2]), "mask has shape"), (dict(mask=i64[0]), "mask"),
                      (dict(idx=i64.int()), "3 dimensions"), (dict(idx=i64.int()[:, :2, None]), "idx has shape"),
                      (dict(out=torch.empty(2, 3, 4, 512, device="cuda")), "out must be")]:
        with pytest.raises(ValueError, match=text):
            S.tree_attention(**(ok | bad))
    for bad, text in [(dict(page=24), "power of two"), (dict(longest=-1), "longest"), (dict(sm_scale=float("nan")), "sm_scale"),
                      (dict(C=C[:, :128].contiguous()), "d = 512"), (dict(mask=i64[..., None][..., :0]), "one word"),
                      (dict(idx=i64.int()[..., None][..., :0]), "one column")]:
        with pytest.raises((S.MisaError, ValueError), match=text):
            S.tree_attention(**(ok | bad))
    q.requires_grad_()
    assert not S.tree_attention(**ok).requires_grad
