"""Attention of drafted tokens where the cut and the masks are large, against the oracle in
64 bits: batches of 65 to 256 sequences whose keys are split (a lane of the cut then holds
several sequences), 256 sequences beside 257, and masks and chains of several words on every
width, whole and split, with words of one mask in different splits."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_amd as S
from attention_parity import SM, bf16, check_rows, gpu, latent_cache
from oracle.paged import tree_rows
from paged_parity import ints, random_trees, words
from test_gpu_tree_attention import cut_of

pytestmark = pytest.mark.gpu


def _check(label, out, lse, q, K, table, page, prefix, mask, only):
    """As check_tree, with the keys of a node gathered once for all of its heads."""
    N, held = q.shape[1], {}

    def rows_of(t, h):
        if t not in held:
            held.clear()
            s, i = divmod(t, N)
            r = tree_rows(table, page, K.shape[0], s, int(prefix[s]), i, None if mask is None else mask[s][i])
            held[t] = K[r], K[r][:, :512]
        return held[t]
    flat = lambda t: t.reshape(-1, *t.shape[2:])  # noqa: E731
    check_rows(label, flat(out), flat(lse), flat(q), rows_of, 512, only=only)


def _splits(ws, seqs):
    """(first slot, splits) of each sequence, as the call left them in front of its workspace."""
    return ws[:seqs * 8].view(torch.int32).cpu().numpy().reshape(seqs, 2)


def _call(q, prefix, table, page, cache, mask, longest):
    """The call with a workspace of its own: the cut, the splits of each sequence (None: whole), out, lse."""
    kw = dict(sm_scale=SM, mask=None if mask is None else words(mask), longest=longest, **gpu(cache))
    a = (q.cuda(), ints(prefix), ints(table), page)
    n = S.lib().misa_tree_workspace_bytes(S.make_tree_problem(*a, **kw))
    ws = torch.full((n + 1024,), 255, dtype=torch.uint8, device="cuda")
    ran, (out, lse) = cut_of(lambda: S.tree_attention(*a, with_lse=True, ws=ws, **kw))
    assert bool((ws[n:] == 255).all())
    return ran, _splits(ws, q.shape[0]) if ran[1] else None, out, lse


BATCHES = [  # sequences, nodes, heads, longest prefix, rows of a workgroup
    (65, 1, 16, 8000, 16), (100, 1, 16, 8000, 16), (128, 1, 16, 4000, 16), (129, 1, 16, 3000, 16), (255, 1, 20, 4000, 32),
    (200, 2, 16, 3000, 32), (128, 2, 40, 3000, 64), (200, 1, 64, 4000, 64), (256, 1, 128, 3000, 128), (66, 2, 128, 3000, 128),
    (129, 3, 20, 4000, 128), (256, 1, 16, 3000, 16)]


def _batch(rng, seqs, N, longest, page=64):
    """Lengths of very different sequences, the longest in the last 64, on pages that they share, and whose pages: all."""
    per, pool = -(-(longest + N) // page), 100
    prefix = rng.integers(0, 200, seqs)
    prefix[[0, 63, seqs - 3]], prefix[[1, 64, seqs - 2]] = 0, -1
    prefix[seqs - 1] = longest
    prefix[rng.integers(2, 62, 5)] = rng.integers(longest // 2, longest, 5)
    prefix[62], prefix[min(127, seqs - 4)], prefix[min(128, seqs - 5)] = longest - 7, longest // 2, longest // 3
    return prefix, rng.integers(0, pool, (seqs, per)).astype(np.int32), pool * page


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,rows", BATCHES)
def test_batches_of_many_sequences_are_split(seqs, N, H, longest, rows, fp8):
    rng = np.random.default_rng(seqs * N + H + longest)
    prefix, table, pool = _batch(rng, seqs, N, longest)
    cache, K = latent_cache(rng, pool, fp8)
    q, mask = bf16(rng, seqs, N, H, 576), random_trees(rng, seqs, N, pad=1 if N > 2 else 0)
    ran, cut, out, lse = _call(q, prefix, table, 64, cache, mask, longest)
    assert ran == (rows, True)
    first, splits = cut[:, 0], cut[:, 1]
    assert (splits >= 1).all() and (first == np.concatenate([[0], np.cumsum(splits)[:-1]])).all()
    assert splits[seqs - 1] > 1 and splits[62] > 1 and (splits[prefix < 0] == 1).all()
    at = {0, 1, 2, 62, 63, 64, 65, 126, 127, 128, 129, 191, 192, seqs - 5, seqs - 4, seqs - 3, seqs - 2, seqs - 1}
    only = sorted({s * N + i for s in at if s < seqs for i in {0, N - 1}})
    _check("batch", out, lse, q, K, table, 64, prefix, mask, only)
    dead = torch.from_numpy(prefix < 0)
    assert bool((out.cpu()[dead] == 0).all()) and bool((lse.cpu()[dead] == -float("inf")).all())
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("fp8", [False, True])
def test_256_sequences_beside_257(fp8):
    # the larger batch keeps sequences whole; what the sequences give is the same to within the cuts' roundings
    rng = np.random.default_rng(257)
    prefix, table, pool = _batch(rng, 257, 1, 3000)
    prefix[255] = 3000
    cache, K = latent_cache(rng, pool, fp8)
    q = bf16(rng, 257, 1, 16, 576)
    only = [0, 1, 62, 63, 64, 65, 127, 128, 252, 253, 254, 255]
    ran, cut, out, lse = _call(q[:256], prefix[:256], table[:256], 64, cache, None, 3000)
    assert ran == (16, True) and cut[255, 1] > 1
    _check("256", out, lse, q[:256], K, table, 64, prefix, None, only)
    ran, cut, out, lse = _call(q, prefix, table, 64, cache, None, 3000)
    assert ran == (16, False)
    _check("257", out, lse, q, K, table, 64, prefix, None, [*only, 256])


WORDS = [  # sequences, nodes, heads, longest prefix, the cut
    (2, 128, 128, 3000, (128, True)), (4, 70, 128, 2000, (128, True)), (1, 65, 128, 4000, (128, True)), (2, 130, 128, 1500, (128, True)),
    (3, 70, 128, 300, (128, False)), (2, 200, 128, 500, (128, False)), (1, 130, 40, 6000, (128, True)), (6, 70, 16, 9000, (128, True)),
    (2, 130, 20, 500, (64, False)), (2, 65, 20, 2000, (64, True)), (1, 130, 20, 2000, (64, True)), (1, 70, 3, 40000, (32, True))]


def _nodes(seqs, N):
    """Nodes on both sides of the words' borders, shared out to the first and the last sequence."""
    return sorted({s * N + i for s, some in ((0, (0, 1, 64, N - 2)), (seqs - 1, (63, 65, 127, 128, N - 1))) for i in some if i < N})


def _alone(node, W):
    """A mask of W words that names its node and no other."""
    return [1 << node % 64 if w == node // 64 else 0 for w in range(W)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", WORDS)
def test_masks_of_several_words_on_every_width(seqs, N, H, longest, cut, fp8):
    rng = np.random.default_rng(seqs * N + H + longest)
    page, pool = 32, 200
    table = rng.integers(0, pool, (seqs, -(-(longest + N) // page))).astype(np.int32)
    cache, K = latent_cache(rng, pool * page, fp8)
    q, prefix = bf16(rng, seqs, N, H, 576), rng.integers(longest // 2, longest + 1, seqs)
    prefix[0] = longest
    mask = random_trees(rng, seqs, N, pad=1)
    for i in (1, N - 2):                                                        # nothing of the last word, nothing of the first
        mask[0][i] = _alone(i, -(-N // 64))
    for m in (mask, None):
        ran, _, out, lse = _call(q, prefix, table, page, cache, m, longest)
        assert ran == cut
        _check("words" if m else "chain", out, lse, q, K, table, page, prefix, m, _nodes(seqs, N))
        assert bool(out.isfinite().all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,H,per,n,cut", [(512, 16, 200, 100, (128, True)), (400, 1, 40, 100, (128, True)), (130, 20, 5, 100, (64, True)),
                                           (100, 16, 5, 60, (32, True)), (100, 1, 5, 60, (32, True))])
def test_words_of_a_mask_in_different_splits(N, H, per, n, cut, fp8):
    # planned for a long prefix, run on a short one: the words' tiles are most of the keys
    rng = np.random.default_rng(N + H)
    page, pool, prefix, held = 1024, 3, [n], -(-n // 64)
    table = rng.integers(0, pool, (1, per)).astype(np.int32)
    cache, K = latent_cache(rng, pool * page, fp8)
    q, mask = bf16(rng, 1, N, H, 576), random_trees(rng, 1, N, pad=1)
    for m in (mask, None):
        ran, parts, out, lse = _call(q, prefix, table, page, cache, m, 0)
        tiles = held + -(-N // 64)
        share = -(-tiles // parts[0, 1])
        assert ran == cut and any(b > held for b in range(share, tiles, share))     # a border between words
        _check("words", out, lse, q, K, table, page, prefix, m, sorted({*_nodes(1, N), N // 2, 200 % N, 448 % N, 449 % N}))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", WORDS[:7] + WORDS[8:10])
def test_what_a_query_does_not_see_has_no_effect_past_one_word(seqs, N, H, longest, cut, fp8):
    rng = np.random.default_rng(seqs + N + H)
    page, W = 16, -(-N // 64)
    per = -(-(longest + N + 20) // page)
    table = rng.permutation(seqs * per).reshape(seqs, per).astype(np.int32)
    cache, _ = latent_cache(rng, seqs * per * page, fp8)
    prefix = rng.integers(longest // 2, longest + 1, seqs)
    prefix[0] = longest
    mask, lone = random_trees(rng, seqs, N, pad=1), N - 2
    for s in range(seqs):
        mask[s][lone] = _alone(lone, W)                                         # sees itself, and no other sees it
    assert not any(mask[s][i][lone // 64] >> lone % 64 & 1 for s in range(seqs) for i in range(N) if i != lone)
    row = lambda s, j: int(table[s, j // page]) * page + j % page  # noqa: E731
    seen = torch.zeros(seqs * per * page, dtype=torch.bool)
    for s in range(seqs):
        named = [b for b in range(64 * W) if any(m[b // 64] >> b % 64 & 1 for m in mask[s])]
        seen[[row(s, j) for j in [*range(prefix[s]), *(prefix[s] + b for b in named)]]] = True
    q = bf16(rng, seqs, N, H, 576)
    ran, _, *want = _call(q, prefix, table, page, cache, mask, longest)
    assert ran == cut
    junk = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(len(seen)) % 3]
    bad, qbad = {n: None if t is None else t.clone() for n, t in cache.items()}, q.clone()
    if fp8:
        bad["c_scale"][~seen], bad["rope"][~seen] = junk[~seen], junk[~seen, None].bfloat16()
        bad["C"].view(torch.uint8)[~seen] = 0x7f
    else:
        bad["C"][~seen] = junk[~seen, None].bfloat16()
    qbad[:, N - 1] = float("nan")                                               # padding
    _, _, *got = _call(qbad, prefix, table, page, bad, mask, longest)
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
    assert bool((got[0][:, N - 1] == 0).all()) and bool((got[1][:, N - 1] == -float("inf")).all())
    (bad["c_scale"] if fp8 else bad["C"])[row(0, prefix[0] + lone)] = float("nan")  # the lone node: itself and no other
    _, _, out, lse = _call(qbad, prefix, table, page, bad, mask, longest)
    assert bool(out[0, lone].isnan().all()) and bool(lse[0, lone].isnan().all())
    out[0, lone], lse[0, lone] = got[0][0, lone], got[1][0, lone]
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
