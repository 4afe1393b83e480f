"""Sizes of the norm, the paged caches and the drafted tokens that are refused where an
answer would be a wrong one (no GPU needed)."""
import ctypes

import pytest

import sparse_attention_indexer_block_amd as S
from test_abi_attention import FAKE
from test_abi_paged import INVALID, _pages, _tree


@pytest.mark.parametrize("N,words", [(65, 1), (128, 1), (129, 2), (1 << 16, 1023)])
def test_a_mask_has_a_bit_for_every_node(N, words):
    # a node past the mask's last word could not name itself
    L = S.lib()
    for kw in (dict(), dict(k=8, idx=FAKE)):
        p = _tree(N=N, words=words, **kw)
        assert L.misa_tree_attention(ctypes.byref(p), FAKE, FAKE, FAKE, 1 << 40, None) == INVALID
        assert b"words" in L.misa_last_error()
        assert L.misa_tree_workspace_bytes(ctypes.byref(p)) == 0
        for enough in (words + 1, min(words + 5, 1024)):
            p = _tree(N=N, words=enough, **kw)
            if kw and 3 * N * (8 + 64 * enough) > 1 << 31:                 # three sequences' lists of rows have a limit of their own
                assert L.misa_tree_workspace_bytes(ctypes.byref(p)) == 0 and b"2^31" in L.misa_last_error()
            else:
                assert L.misa_tree_workspace_bytes(ctypes.byref(p)) >= 256
    p = _tree(N=N, words=words, pages=_pages(seqs=0, table=None))          # an empty batch has no masks
    assert L.misa_tree_attention(ctypes.byref(p), None, None, None, 0, None) == 0
