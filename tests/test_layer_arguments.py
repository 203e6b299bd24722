"""Arguments of the operators between a decoder layer's linear layers at the ends
of their ranges (host only): integers that size what a call fills, of other kinds
than Python's own and past what a C int holds; the norm's offset; strides."""

import ctypes

import numpy as np
import pytest

import weight_only_int4_quantize_amd as awq


@pytest.fixture
def entry(monkeypatch):
    """awq_rope_frequencies behind a check that what it is given to fill holds
    rotary_dim / 2 numbers."""
    lib = awq.load()
    given = []

    class Guarded:
        def __getattr__(self, name):
            return getattr(lib, name)

        def awq_rope_frequencies(self, r, *a):
            given.append(len(a[-2]))
            assert ctypes.c_int(r).value // 2 <= len(a[-2]) or not 2 <= ctypes.c_int(r).value <= 4096
            return lib.awq_rope_frequencies(r, *a)

    monkeypatch.setattr(awq, "_lib", Guarded())
    return given


@pytest.mark.parametrize("kind", [int, np.int32, np.int64, np.uint16])
def test_rotary_dim_of_any_integer_kind(entry, kind):
    want, m = awq.rope_frequencies(64, 50000.0, "yarn", 4.0, 4096)
    got, n = awq.rope_frequencies(kind(64), 50000.0, "yarn", 4.0, 4096)
    assert entry == [32, 32] and got == want and n == m


def test_rotary_dim_past_a_c_int(entry):
    for bad in (2 ** 32 + 64, -2 ** 32 + 64, 2 ** 31):
        with pytest.raises(ValueError, match="rotary_dim"):
            awq.rope_frequencies(bad)
    for bad in (64.0, "64", None, np.float32(64)):
        with pytest.raises(TypeError, match="rotary_dim"):
            awq.rope_frequencies(bad)
    for bad in (0, 1, 7, -64, 4098, True):
        with pytest.raises(awq.AwqError):
            awq.rope_frequencies(bad)


def test_norm_offsets():
    L = awq.load()
    for bad in (1e36, 65505.0, -65536.0, float("nan"), float("inf")):
        assert L.awq_rmsnorm(0x10000, 64, None, 0, None, 0, None, bad, 1e-5, 4, 64, 0, 0, 0x20000, 64, None, None) == 4
    for good in (65504.0, -65504.0, 1.0):       # (no rows: nothing to do)
        assert L.awq_rmsnorm(0x10000, 64, None, 0, None, 0, None, good, 1e-5, 0, 64, 0, 0, 0x20000, 64, None, None) == 0


@pytest.mark.parametrize("stride", [2 ** 39, 2 ** 40 - 1])
def test_interleaved_rows_of_the_largest_strides(stride):
    """Rows of the rotation's output that share memory, their tokens' reach past
    64 bits."""
    L = awq.load()
    table = awq._RopeTableStruct(0x10000, 128, 0, 1.0)
    q = awq._RopeHeadsStruct(0x10000, 0x20000, 256, 128, stride, 2 ** 39, 65535)
    for n in (2 ** 24 - 1, 2 ** 23 + 1, 2 ** 23 + 5, 1000):
        assert L.awq_rope(ctypes.byref(table), 0x10000, None, ctypes.byref(q), None, 128, n, None) == 2
