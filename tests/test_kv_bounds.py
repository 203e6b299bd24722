"""Sizes at the edge of what the paged cache's calls take (host only: fake
device addresses are never dereferenced, every call fails before a launch)."""

import ctypes

import pytest

import weight_only_int4_quantize_amd as awq

from test_kv_checks import SHAPE, attend, cache, read, seqs, write

LONGEST = 2 ** 31 - 1024    # whole splits of 1024 positions in 32 bits


@pytest.fixture(scope="module")
def L():
    return awq.load()


@pytest.mark.parametrize("max_len", [LONGEST + 1, 2 ** 31 - 300, 2 ** 31 - 257])
def test_lengths_past_whole_splits(L, max_len):
    """One split has to hold every position, or a call without a workspace
    would have parts and nowhere to put them."""
    s = seqs(n_seqs=1, max_pages=1 << 25, table_stride=1 << 25, max_len=max_len)
    for call in (attend, read, write):
        assert call(L, cache(), s) == SHAPE
    for max_tokens in (1, 5, 500):
        s.max_tokens = max_tokens
        assert L.awq_kv_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(s), 4) == 0


def test_longest_length_is_taken(L):
    s = seqs(n_seqs=1, max_pages=1 << 25, table_stride=1 << 25, max_len=LONGEST)
    need = L.awq_kv_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(s), 4)
    assert need > 0
    assert attend(L, cache(), s, ws=0x10000, nbytes=need - 1) == 5      # past the shape checks


def test_output_rows_that_interleave(L):
    """Strides of head_dim and more whose tokens and heads still meet: token 1
    of head 0 would be head 1 of token 0, written by two blocks."""
    c, s = cache(), seqs()
    for strides in ((128, 128), (256, 256), (256, 128), (384, 128), (128, 256), (128, 15 * 128 - 8), (504, 128)):
        assert attend(L, c, s, os=strides) == SHAPE, strides
    # taken (what fails is the workspace, checked behind the strides)
    for strides in ((512, 128), (1024, 128), (128, 15 * 128), (136, 16 * 136), (1024, 256)):
        assert attend(L, c, s, os=strides, ws=0x10000, nbytes=0) == 5, strides
    assert attend(L, c, s, os=(128, 128), n=1, ws=0x10000, nbytes=0) == 5      # one token: no two meet
    one = cache(n_kv_heads=1)
    assert attend(L, one, s, os=(128, 0), heads=1, ws=0x10000, nbytes=0) == 5
