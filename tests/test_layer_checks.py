"""Argument checks of the norm, the rotary positions and the 4-bit cache (host
only: fake device addresses are never dereferenced, every call fails before a
launch or has nothing to do), the frequencies, and pins of the CPU oracle."""

import ctypes
import math

import numpy as np
import pytest

import weight_only_int4_quantize_amd as awq
from oracle import layer_oracle as lo
from test_kv_checks import attend, cache, read, seqs, write

OK, NULL, SHAPE, ALIGN, CONFIG, WORKSPACE = 0, 1, 2, 3, 4, 5
FAKE = 0x10000
INT4 = awq.KV_FORMATS["int4"]


@pytest.fixture(scope="module")
def L():
    return awq.load()


# ---------------------------------------------------------------- the 4-bit cache

@pytest.mark.parametrize("call", [write, read, attend])
def test_cache_checks(L, call):
    for kw, expect in [(dict(k_scales=FAKE + 8), ALIGN), (dict(v_scales=FAKE + 4), ALIGN), (dict(k_codes=FAKE + 8), ALIGN),
                       (dict(head_dim=80), CONFIG), (dict(head_dim=32), CONFIG), (dict(page_size=16), CONFIG),
                       (dict(v_scales=None), NULL), (dict(n_pages=0), SHAPE), (dict(format=2), CONFIG),
                       (dict(format=3), CONFIG), (dict(format=5), CONFIG)]:
        assert call(L, cache(**{"format": INT4, **kw}), seqs()) == expect, kw
    for empty in (dict(n_seqs=0), dict(max_tokens=0)):
        assert call(L, cache(format=INT4), seqs(**empty)) == OK
    assert call(L, cache(format=INT4), seqs(), n=0) == OK


def test_more_blocks_than_a_launch_takes(L):
    pages = seqs(max_tokens=2 ** 31 - 1, max_len=1 << 30, max_pages=1 << 25, table_stride=1 << 25, n_seqs=1)
    assert write(L, cache(page_size=32, format=INT4), pages, n=2 ** 31 - 1) == SHAPE
    many = cache(n_kv_heads=40000, format=INT4)
    assert attend(L, many, seqs(max_tokens=20), heads=40000) == SHAPE


def test_workspace_query(L):
    q = L.awq_kv_attention_workspace_bytes
    for fmt in (0, INT4):
        assert q(ctypes.byref(cache(format=fmt)), ctypes.byref(seqs(n_seqs=1, max_tokens=1, max_len=1 << 20)), 4) > 0
    assert q(ctypes.byref(cache(format=3)), ctypes.byref(seqs()), 4) == 0


def test_cache_class_refuses():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.KVCache(torch.zeros(1, 1, 4, 64, 16, dtype=torch.uint8), torch.zeros(1, 1, 2, 128, 16, dtype=torch.uint8),
                    torch.zeros(1, 1, 4, 64, 2).half(), torch.zeros(1, 1, 2, 64).half(), "int4")
    with pytest.raises(ValueError, match="fmt"):
        awq.KVCache.empty(1, 1, 128, 64, "int2", "cpu")


# ---------------------------------------------------------------- the norm

def norm(L, x=FAKE, xs=64, r=None, rs=0, ro=None, ros=0, w=FAKE, offset=0.0, eps=1e-5, rows=4, width=64, fmt=0, group=0,
         out=FAKE + 0x10000, os=64, scales=FAKE):
    return L.awq_rmsnorm(x, xs, r, rs, ro, ros, w, offset, eps, rows, width, fmt, group, out, os, scales, None)


def test_norm_checks(L):
    for bad in (3, -1):
        assert norm(L, fmt=bad) == CONFIG
    assert norm(L, group=32) == CONFIG                          # fp16 has no scales
    for g in (16, 48, 1024, -32):
        assert norm(L, fmt=1, group=g) == CONFIG
    assert norm(L, fmt=1, group=128) == SHAPE                   # width 64
    for bad in (-1e-9, float("nan"), float("inf")):
        assert norm(L, eps=bad) == CONFIG
    assert norm(L, offset=float("nan")) == CONFIG
    assert norm(L, rows=-1) == SHAPE and norm(L, rows=2 ** 31) == SHAPE
    assert norm(L, width=0) == SHAPE and norm(L, width=2 ** 24 + 1) == SHAPE
    assert norm(L, xs=-1) == SHAPE and norm(L, os=63) == SHAPE and norm(L, os=2 ** 40) == SHAPE
    assert norm(L, r=FAKE, rs=-1) == SHAPE and norm(L, ro=FAKE * 3, ros=63) == SHAPE
    assert norm(L, rows=0) == OK and norm(L, rows=0, x=None, out=None) == OK
    assert norm(L, x=None) == NULL and norm(L, out=None) == NULL and norm(L, fmt=2, scales=None) == NULL
    assert norm(L, x=FAKE + 1) == ALIGN and norm(L, w=FAKE + 1) == ALIGN and norm(L, fmt=1, scales=FAKE + 2) == ALIGN
    assert norm(L, out=FAKE + 0x10001) == ALIGN
    # aliases: the strides must be the same ones, 8 bits over 16 never
    assert norm(L, out=FAKE, xs=80) == SHAPE and norm(L, r=FAKE * 2, rs=64, ro=FAKE * 2, ros=65) == SHAPE
    assert norm(L, fmt=1, out=FAKE) == SHAPE and norm(L, fmt=2, r=FAKE * 2, rs=64, out=FAKE * 2) == SHAPE
    assert norm(L, ro=FAKE * 5, ros=64, out=FAKE * 5) == SHAPE
    assert norm(L, rows=2 ** 31 - 1, width=64) == SHAPE         # more blocks than a launch takes
    assert norm(L, rows=2 ** 24, width=2 ** 20, xs=2 ** 20, os=2 ** 20) == SHAPE


# ---------------------------------------------------------------- rotary positions

def heads(**kw):
    return awq._RopeHeadsStruct(*{**dict(x=FAKE, y=FAKE * 2, its=256, ihs=128, ots=256, ohs=128, heads=2), **kw}.values())


def rope(L, freqs=FAKE, r=128, layout=0, m=1.0, positions=FAKE, s=None, q=None, k=None, dim=128, n=3):
    t = awq._RopeTableStruct(freqs, r, layout, m)
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    return L.awq_rope(ctypes.byref(t), positions, ref(s), ref(heads() if q is None else q), ref(k), dim, n, None)


def test_rope_checks(L):
    assert L.awq_rope(None, FAKE, None, None, None, 128, 3, None) == NULL
    assert rope(L, layout=2) == CONFIG and rope(L, layout=-1) == CONFIG and rope(L, m=float("inf")) == CONFIG
    for kw in (dict(r=0), dict(r=63), dict(r=130), dict(dim=0), dict(dim=4098), dict(n=-1), dict(n=2 ** 24)):
        assert rope(L, **kw) == SHAPE, kw
    assert rope(L, positions=None) == NULL and rope(L, s=seqs()) == NULL        # neither, both
    for kw in (dict(n_seqs=-1), dict(n_seqs=32768), dict(max_tokens=-1), dict(max_len=2 ** 31 - 1)):
        assert rope(L, positions=None, s=seqs(**kw)) == SHAPE, kw
    for kw, expect in [(dict(heads=-1), SHAPE), (dict(heads=65536), SHAPE), (dict(its=-1), SHAPE), (dict(ihs=-1), SHAPE),
                       (dict(ots=127), SHAPE), (dict(ohs=64), SHAPE), (dict(ots=200), SHAPE), (dict(ots=2 ** 40), SHAPE),
                       (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=FAKE + 1), ALIGN), (dict(y=FAKE + 1), ALIGN),
                       (dict(y=FAKE, its=512), SHAPE)]:
        assert rope(L, q=heads(**kw)) == expect, kw
        assert rope(L, k=heads(**kw)) == expect, kw
    assert rope(L, freqs=None) == NULL and rope(L, freqs=FAKE + 4) == ALIGN and rope(L, positions=FAKE + 2) == ALIGN
    assert rope(L, positions=None, s=seqs(cu_tokens=None)) == NULL
    assert rope(L, positions=None, s=seqs(kv_len=FAKE + 1)) == ALIGN
    # nothing to do
    assert rope(L, n=0) == OK and rope(L, n=0, positions=None) == OK
    assert rope(L, q=heads(heads=0)) == OK
    assert rope(L, positions=None, s=seqs(n_seqs=0)) == OK and rope(L, positions=None, s=seqs(max_tokens=0)) == OK


@pytest.mark.parametrize("scaling", sorted(awq.ROPE_SCALINGS))
@pytest.mark.parametrize("r,base,factor,length", [(128, 10000.0, 4.0, 4096.0), (64, 500000.0, 8.0, 8192.0),
                                                  (10, 10000.0, 1.0, 100.0), (256, 1e6, 40.0, 32768.0), (4, 100.0, 2.0, 7.0)])
def test_frequencies(scaling, r, base, factor, length):
    got, m = awq.rope_frequencies(r, base, scaling, factor, length)
    want, wm = lo.rope_frequencies(r, base, scaling, factor, length)
    np.testing.assert_allclose(got, want, rtol=1e-14)
    assert math.isclose(m, wm, rel_tol=1e-15)
    plain, _ = awq.rope_frequencies(r, base)
    # the fastest pair stays (but for plain interpolation), none turns faster, none slower than factor times
    assert (np.array(got) <= np.array(plain) * (1 + 1e-15)).all()
    assert (np.array(got) >= np.array(plain) / factor * (1 - 1e-12)).all()


def test_frequency_checks():
    for kw in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=4098), dict(base=1.0), dict(base=float("nan")),
               dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=float("inf")),
               dict(scaling="ntk", rotary_dim=2, factor=2.0), dict(scaling="yarn", factor=2.0),
               dict(scaling="yarn", factor=2.0, trained_len=100, low=2.0, high=1.0),
               dict(scaling="wavelength", factor=2.0, trained_len=-1.0),
               dict(scaling="wavelength", factor=2.0, trained_len=10, low=0.0)):
        with pytest.raises(awq.AwqError):
            awq.rope_frequencies(**{"rotary_dim": 64, **kw})
    with pytest.raises(ValueError, match="scaling"):
        awq.rope_frequencies(64, scaling="other")
    L = awq.load()
    assert L.awq_rope_frequencies(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None, None) == NULL
    assert L.awq_rope_frequencies(64, 1e4, 5, 1.0, 0.0, 0.0, 0.0, FAKE, FAKE) == CONFIG


# ---------------------------------------------------------------- the oracle

def test_oracle_groups_by_hand():
    x = np.array([[3.0, 18.0, 3.5, 4.5, 5.5, 10.0] + [7.0] * 26], np.float16)
    c, s = lo.groups4(x)
    assert list(s[0]) == [1.0, 3.0]
    assert list(c[0, :6]) == [0, 15, 0, 2, 2, 7]            # halves to even: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    np.testing.assert_array_equal(lo.numbers4(c, s)[0, :3], np.float16([3, 18, 3]))
    c, s = lo.groups4(np.full((1, 32), 1000.5, np.float16))
    assert (c == 0).all() and s[0, 0] == 0 and (lo.numbers4(c, s) == np.float16(1000.5)).all()
    # a step is never above a fifteenth of the range, and the top never passes the group's
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((5000, 32)) * np.exp2(rng.integers(-16, 13, (5000, 1)))).astype(np.float16)
    x[0], x[0, 0], x[0, 1] = 0, 65504, -65504
    c, s = lo.groups4(x)
    y = lo.numbers4(c, s).astype(np.float64)
    assert np.isfinite(y).all() and (y.max(-1) <= x.max(-1)).all() and (y.min(-1) == x.min(-1)).all()
    step = s[:, :1].astype(np.float64)
    cut = (x.max(-1) - x.min(-1).astype(np.float64))[:, None] - 15 * step
    assert (cut >= 0).all()
    assert (np.abs(y - x) <= step / 2 + cut + 2.0 ** -11 * np.abs(y) + 2.0 ** -25).all()


def test_oracle_layouts():
    rng = np.random.default_rng(2)
    c = rng.integers(0, 16, (3, 2, 64, 96)).astype(np.uint8)
    np.testing.assert_array_equal(lo.load_k(lo.store_k(c)), c)
    np.testing.assert_array_equal(lo.load_v(lo.store_v(c)), c)
    # header's order: of eight, number 2 j in bits 4 j, number 2 j + 1 in bits 16 + 4 j
    word = int.from_bytes(bytes(lo.store_k(c)[1, 0, 2, 5, 4:8]), "little")
    assert [word >> (4 * (i // 2) + 16 * (i % 2)) & 15 for i in range(8)] == list(c[1, 0, 5, 72:80])
    word = int.from_bytes(bytes(lo.store_v(c)[2, 1, 1, 50, 12:16]), "little")
    assert [word >> (4 * (i // 2) + 16 * (i % 2)) & 15 for i in range(8)] == list(c[2, 1, 56:64, 50])


def test_oracle_rope_by_hand():
    x = np.arange(1, 5, dtype=np.float16).reshape(1, 1, 4)
    f = np.array([math.pi / 2, math.pi])
    y, _ = lo.rope(x, [1], f, "half")
    np.testing.assert_allclose(y[0, 0], [-3, -2, 1, -4], atol=1e-12)        # (1, 3) by a quarter, (2, 4) by a half turn
    y, _ = lo.rope(x, [1], f, "interleaved", 2.0)
    np.testing.assert_allclose(y[0, 0], [-4, 2, -6, -8], atol=1e-12)


def test_oracle_norm_by_hand():
    x = np.array([[3.0, 4.0]], np.float16)
    h, y = lo.rmsnorm(x, np.float16([2, 1]), 0.0, np.float16([[0, 0]]))
    np.testing.assert_allclose(y, [[6 / math.sqrt(12.5), 4 / math.sqrt(12.5)]])
    np.testing.assert_allclose(lo.norm_scales(np.array([[1.0, -2.0, 0.0, 0.0]]), "int8", 2), [[2 / 127, 1e-5 / 127]])
