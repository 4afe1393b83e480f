"""Limits of the attention entry points' arguments that need no GPU: softmax
scales whose product with log2(e) is no fp32 number are refused, those below are not."""
import ctypes

import pytest

import sparse_attention_indexer_block_amd as S

FAKE = 1 << 20  # an aligned, never-dereferenced address: validation must fail first


def _problems(sm):
    cache = S.Cache(1000, 512, 64, S.KDT_FP8, FAKE, FAKE, FAKE)
    L = S.lib()
    return [(S.LatentProblem(4, 16, 100, sm, FAKE, FAKE, None, None, cache), L.misa_latent_attention, L.misa_latent_workspace_bytes),
            (S.ExpandedProblem(4, 16, 100, sm, FAKE, FAKE, FAKE, 64, FAKE, None), L.misa_expanded_attention,
             L.misa_expanded_workspace_bytes)]


@pytest.mark.parametrize("sm", [2.36e38, -2.36e38, 3.4e38, -3.4e38])
def test_softmax_scales_past_the_range_are_refused(sm):
    for p, call, need in _problems(sm):
        assert need(ctypes.byref(p)) == 0
        assert call(ctypes.byref(p), FAKE, FAKE, FAKE, 1 << 40, None) == -1
        assert b"sm_scale" in S.lib().misa_last_error()


@pytest.mark.parametrize("sm", [2.35e38, -2.35e38, 0.0, -0.0, 1e-45])
def test_softmax_scales_inside_the_range_are_taken(sm):
    for p, call, need in _problems(sm):
        assert need(ctypes.byref(p)) >= 256
        assert call(ctypes.byref(p), None, FAKE, FAKE, 1 << 40, None) == -1  # (for the missing result)
        assert b"out" in S.lib().misa_last_error()
