"""Sizes of the norm, the paged caches and the drafted tokens that are refused where an
answer would be a wrong one (no GPU needed)."""
import ctypes
import math

import pytest
import torch

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


class _Far:
    """What the binding asks of a GPU tensor, without one, so that its shape may be any."""
    is_cuda, requires_grad = True, False

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


WIDE = 1 << 32
b16, i32, i64, f32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


@pytest.mark.parametrize("kw,name", [
    (dict(page=WIDE + 64), "page"), (dict(longest=WIDE + 5), "longest"), (dict(longest=-WIDE), "longest"),
    (dict(table=_Far((1, WIDE + 2), i32)), "pages"), (dict(mask=_Far((1, 4, WIDE + 1), i64)), "words"),
    (dict(idx=_Far((1, 4, WIDE + 3), i32)), "idx")])
def test_the_binding_passes_on_no_size_past_32_bits_for_trees(kw, name):
    # (the C structures would take such a number modulo 2^32)
    a = dict(q=_Far((1, 4, 16, 576), b16), prefix=_Far((1,), i32), table=_Far((1, 8), i32), page=64, C=_Far((512, 576), b16), sm_scale=0.1)
    assert S.make_tree_problem(**a).pages.page == 64
    with pytest.raises(ValueError, match=f"{name}.*32 bits"):
        S.make_tree_problem(**(a | kw))


@pytest.mark.parametrize("n,width,name", [(WIDE + 5, 8, "rows"), (1, WIDE + 8, "width")])
def test_the_binding_passes_on_no_size_past_32_bits_for_the_norm(n, width, name, monkeypatch):
    monkeypatch.setattr(S, "_on", lambda *a: pytest.fail(f"called with {a[2].n} rows of {a[2].width}"))
    out = _Far((n, width), b16)
    with pytest.raises(ValueError, match=f"{name}.*32 bits"):
        S.rms_norm(_Far((n, width), b16), _Far((width,), f32), out=out)


@pytest.mark.parametrize("kw,name", [(dict(page=WIDE + 64), "page"), (dict(table=_Far((1, WIDE + 2), i32)), "pages"),
                                     (dict(rot=_Far((8, 64), f32), rot_at=WIDE + 512), "rot_at")])
def test_the_binding_passes_on_no_size_past_32_bits_for_appends(kw, name, monkeypatch):
    monkeypatch.setattr(S, "_on", lambda *a: pytest.fail("called"))
    a = dict(x=_Far((2, 576), b16), seq=_Far((2,), i32), pos=_Far((2,), i32), table=_Far((1, 8), i32), page=64, C=_Far((512, 576), b16))
    with pytest.raises(ValueError, match=f"{name}.*32 bits"):
        S.paged_append(**(a | kw))


def test_the_binding_passes_on_no_size_past_32_bits_for_lists():
    with pytest.raises(ValueError, match="idx.*32 bits"):
        S.make_latent_problem(_Far((1, 16, 576), b16), _Far((512, 576), b16), 0.1, idx=_Far((1, WIDE + 2), i32))
