"""Attention of drafted tokens where the running maximum of the softmax has to be lifted
again and again, by some rows of a workgroup and not by others; negative and zero scales;
and the same bits from calls that run at once."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_amd as S
from attention_parity import SM, bf16, gpu, latent_cache
from paged_parity import check_tree, ints, random_trees, tables, words
from test_gpu_tree_attention import cut_of

pytestmark = pytest.mark.gpu

WIDTHS = [  # sequences, nodes, heads, longest prefix, the cut
    (1, 1, 16, 700, (16, True)), (9, 17, 3, 700, (32, True)), (40, 6, 20, 1000, (64, True)), (3, 50, 100, 500, (128, False)),
    (3, 50, 100, 900, (128, True))]


def _inputs(rng, seqs, N, H, longest, fp8):
    page = 32
    table, pool = tables(rng, seqs, -(-(longest + N) // page))
    cache, K = latent_cache(rng, pool * page, fp8)
    prefix = np.full(seqs, longest)
    prefix[1:] = rng.integers(longest // 2, longest, seqs - 1)
    return page, table, cache, K, bf16(rng, seqs, N, H, 576), prefix, random_trees(rng, seqs, N)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", WIDTHS)
def test_scores_that_climb(seqs, N, H, longest, cut, fp8):
    # the first rotary value climbs by 52 every 40 positions, so that a score moves by 30 (43 powers
    # of two) a step: up, down, or not at all, by 32 heads together and in the last kind by every other row
    rng = np.random.default_rng(seqs + N + H + longest)
    page, table, cache, K, q, prefix, mask = _inputs(rng, seqs, N, H, longest, fp8)
    j = np.arange(table.shape[1] * page)
    for s in range(seqs):
        at = table[s, j // page] * page + j % page
        level = torch.from_numpy(52.0 * (j // 40)).bfloat16()
        (cache["rope"][:, 0] if fp8 else cache["C"][:, 512])[torch.from_numpy(at)] = level
        K[at, 512] = level.double().numpy()
    kind = np.arange(N * H).reshape(N, H) // 32 % 4
    q[..., 512] = torch.from_numpy(np.where(kind == 0, 8.0, np.where(kind == 1, 0.0, np.where(kind == 2, -8.0, 8.0 * (np.arange(H) % 2))))).bfloat16()
    call = lambda: S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=words(mask), longest=longest,  # noqa: E731
                                    with_lse=True, **gpu(cache))
    ran, (out, lse) = cut_of(call)
    assert ran == cut
    T = seqs * N
    check_tree("climbing", out, lse, q, K, table, page, prefix, mask=mask, only=sorted({0, 1 % T, N - 1, T // 2, T - 1}))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", WIDTHS)
def test_negative_and_zero_scales(seqs, N, H, longest, cut, fp8):
    rng = np.random.default_rng(seqs * N + H + longest)
    page, table, cache, K, q, prefix, mask = _inputs(rng, seqs, N, H, longest, fp8)
    T = seqs * N
    for sm, sign in ((-SM, -1.0), (0.0, 0.0)):                                  # sm q.k = SM (sign q).k, exactly
        out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=sm, mask=words(mask), longest=longest,
                                    with_lse=True, **gpu(cache))
        check_tree(f"scale {sm}", out, lse, sign * q, K, table, page, prefix, mask=mask, only=sorted({0, T // 2, T - 1}))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest,cut", WIDTHS[2:])
def test_calls_at_once(seqs, N, H, longest, cut, fp8):
    rng = np.random.default_rng(longest)
    page, table, cache, _, q, prefix, mask = _inputs(rng, seqs, N, H, longest, fp8)
    c, t, n, m = gpu(cache), ints(table), ints(prefix), words(mask)
    qs = [q.cuda(), (0.5 * q).cuda()]
    call = lambda x, ws=None: S.tree_attention(x, n, t, page, sm_scale=SM, mask=m, longest=longest, with_lse=True, ws=ws, **c)  # noqa: E731
    want = [call(x) for x in qs]
    size = S.lib().misa_tree_workspace_bytes(S.make_tree_problem(qs[0], n, t, page, sm_scale=SM, mask=m, longest=longest, **c))
    streams, ws = [torch.cuda.Stream() for _ in qs], [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(qs[i], ws[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
