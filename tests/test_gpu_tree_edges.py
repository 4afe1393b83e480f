"""Attention of drafted tokens at the ends of its tables and sizes, against the oracle in 64
bits: prefixes that reach and pass the table's end, so that drafted positions lie in no page;
more heads than a workgroup has rows; masks that name positions behind the nodes; and lists
whose positions and nodes meet those ends."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_amd as S
from attention_parity import SM, bf16, gpu, latent_cache
from paged_parity import check_tree, ints, random_trees, tables, words
from test_gpu_tree_attention import NAMES

pytestmark = pytest.mark.gpu


def _widths(call):
    """Rows of the workgroups that call() ran with (the last launch of the attention itself), and its result."""
    torch.cuda.synchronize()
    S.profile_reset()
    S.profile_enable(True)
    try:
        got = call()
        torch.cuda.synchronize()
    finally:
        S.profile_enable(False)
    ran = {rows for rows, name in NAMES.items() if S.profile_read(name)[1]}
    S.profile_reset()
    return ran, got


ENDS = [(2, 6, 3, 70, 16), (5, 17, 3, 700, 16), (9, 17, 3, 700, 32), (70, 3, 33, 128, 64), (3, 50, 100, 250, 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("seqs,N,H,cap,rows", ENDS)
def test_prefixes_at_the_tables_end(seqs, N, H, cap, rows, page, fp8):
    rng = np.random.default_rng(seqs + N + page)
    per = -(-cap // page)
    table, pool = tables(rng, seqs, per, spare=0)
    cache, K = latent_cache(rng, pool * page, fp8)
    full = per * page
    prefix = np.array([full - 2, full, full + 1000, 2 ** 31 - 1, full - N, full - 1])[np.arange(seqs) % 6]
    q, mask = bf16(rng, seqs, N, H, 576), random_trees(rng, seqs, N)
    only = sorted({s * N + i for s in range(min(seqs, 6)) for i in {0, 1, N - 1}})
    for m in (mask, None):
        for idx in (None, np.stack([rng.integers(-1, full + 5, (N, 40)) for _ in range(seqs)]).astype(np.int32)):
            call = lambda: S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=None if m is None else words(m),  # noqa: E731
                                            idx=None if idx is None else ints(idx), with_lse=True, **gpu(cache))
            ran, (out, lse) = _widths(call)
            assert ran == (set() if idx is not None else {rows})
            check_tree("end", out, lse, q, K, table, page, prefix, mask=m, idx=idx, only=only)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest", [(1, 1, 300, 500), (1, 1, 129, 90), (3, 2, 257, 200), (70, 1, 161, 100), (300, 1, 136, 60), (2, 5, 1000, 64)])
def test_more_heads_than_rows_of_a_workgroup(seqs, N, H, longest, fp8):
    rng = np.random.default_rng(seqs + H)
    page = 32
    table, pool = tables(rng, seqs, -(-(longest + N) // page))
    cache, K = latent_cache(rng, pool * page, fp8)
    q, prefix = bf16(rng, seqs, N, H, 576), rng.integers(0, longest + 1, seqs)
    prefix[0] = longest
    out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, longest=longest, with_lse=True, **gpu(cache))
    check_tree("heads", out, lse, q, K, table, page, prefix, only=sorted({0, seqs * N // 2, seqs * N - 1}))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,N,H,longest", [(2, 3, 3, 100), (5, 17, 3, 700), (40, 6, 20, 200), (3, 50, 100, 200)])
def test_masks_that_name_positions_behind_the_nodes(seqs, N, H, longest, fp8):
    # bit b is position prefix + b, whether or not a node of this call is there
    rng = np.random.default_rng(N + H)
    page = 16
    table, pool = tables(rng, seqs, -(-(longest + 100) // page))
    table[0, -1] = -1
    cache, K = latent_cache(rng, pool * page, fp8)
    q, prefix = bf16(rng, seqs, N, H, 576), rng.integers(longest // 2, longest + 1, seqs)
    prefix[0] = longest
    mask = [[[int(rng.integers(0, 2 ** 63)) | 1 << 63, int(rng.integers(0, 2 ** 63)) << 1 | 1] for _ in range(N)] for _ in range(seqs)]
    out, lse = S.tree_attention(q.cuda(), ints(prefix), ints(table), page, sm_scale=SM, mask=words(mask), longest=longest, with_lse=True,
                                **gpu(cache))
    check_tree("behind", out, lse, q, K, table, page, prefix, mask=mask, only=sorted({0, 1, N - 1, seqs * N // 2, seqs * N - 1}))


@pytest.mark.parametrize("fp8", [False, True])
def test_one_token_with_and_without_a_mask(fp8):
    rng = np.random.default_rng(5)
    table, pool = tables(rng, 9, 20)
    cache, _ = latent_cache(rng, pool * 16, fp8)
    q, prefix = bf16(rng, 9, 1, 16, 576), rng.integers(0, 300, 9)
    call = lambda m: S.tree_attention(q.cuda(), ints(prefix), ints(table), 16, sm_scale=SM, mask=m, with_lse=True, **gpu(cache))  # noqa: E731
    (a, b), (c, d) = call(None), call(torch.ones(9, 1, dtype=torch.int64, device="cuda"))
    assert torch.equal(a, c) and torch.equal(b, d)
