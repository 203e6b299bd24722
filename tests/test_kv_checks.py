"""The paged 8-bit cache's and the attention's argument checks (host only:
fake device addresses are never dereferenced, every call fails before a
launch or has nothing to do), the binding's own checks, and pins of the CPU
oracle they are compared with."""

import ctypes

import numpy as np
import pytest

import weight_only_int4_quantize_amd as awq
from oracle import kv_oracle

OK, NULL, SHAPE, ALIGN, CONFIG, WORKSPACE = 0, 1, 2, 3, 4, 5
FAKE = 0x10000
FAKE_ODD = 0x10008


@pytest.fixture(scope="module")
def L():
    return awq.load()


def cache(**kw):
    base = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, n_pages=8, n_kv_heads=2, page_size=64,
                head_dim=128, format=0)
    return awq._KVCacheStruct(**{**base, **kw})


def seqs(**kw):
    base = dict(block_table=FAKE, cu_tokens=FAKE, kv_len=FAKE, table_stride=4, max_pages=4, n_seqs=3, max_tokens=5,
                max_len=256)
    return awq._KVSeqsStruct(**{**base, **kw})


def write(L, c, s, k=FAKE, v=FAKE, strides=(256, 128, 256, 128), n=15):
    return L.awq_kv_write(ctypes.byref(c) if c else None, ctypes.byref(s) if s else None, k, strides[0], strides[1], v,
                          strides[2], strides[3], n, None)


def read(L, c, s, k=FAKE, v=FAKE, n=15):
    return L.awq_kv_read(ctypes.byref(c) if c else None, ctypes.byref(s) if s else None, k, v, n, None)


def attend(L, c, s, q=FAKE, out=FAKE, qs=(512, 128), os=(512, 128), n=15, heads=4, scale=0.1, causal=1, window=0,
           lse=None, ws=None, nbytes=0):
    return L.awq_kv_attention(ctypes.byref(c) if c else None, ctypes.byref(s) if s else None, q, qs[0], qs[1], n, heads,
                              scale, causal, window, out, os[0], os[1], lse, ws, nbytes, None)


BAD_CACHE = [
    (dict(format=2), CONFIG), (dict(format=-1), CONFIG),
    (dict(page_size=16), CONFIG), (dict(page_size=48), CONFIG), (dict(page_size=512), CONFIG), (dict(page_size=0), CONFIG),
    (dict(head_dim=80), CONFIG), (dict(head_dim=0), CONFIG), (dict(head_dim=512), CONFIG),
    (dict(n_pages=0), SHAPE), (dict(n_pages=2 ** 31), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(n_kv_heads=65536), SHAPE),
    (dict(k_codes=None), NULL), (dict(v_codes=None), NULL), (dict(k_scales=None), NULL), (dict(v_scales=None), NULL),
    (dict(k_codes=FAKE_ODD), ALIGN), (dict(v_codes=FAKE_ODD), ALIGN), (dict(k_scales=FAKE + 2), ALIGN),
    (dict(v_scales=FAKE + 1), ALIGN),
]
BAD_SEQS = [
    (dict(n_seqs=-1), SHAPE), (dict(n_seqs=32768), SHAPE), (dict(max_pages=-1), SHAPE), (dict(table_stride=3), SHAPE),
    (dict(max_tokens=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(max_len=2 ** 31 - 1), SHAPE),
    (dict(max_tokens=2 ** 31), SHAPE),
    (dict(block_table=None), NULL), (dict(cu_tokens=None), NULL), (dict(kv_len=None), NULL),
    (dict(block_table=FAKE + 2), ALIGN), (dict(cu_tokens=FAKE + 2), ALIGN), (dict(kv_len=FAKE + 1), ALIGN),
]


@pytest.mark.parametrize("call", [write, read, attend])
def test_cache_and_batch_checks(L, call):
    assert call(L, None, seqs()) == NULL and call(L, cache(), None) == NULL
    for kw, expect in BAD_CACHE:
        assert call(L, cache(**kw), seqs()) == expect, kw
    for kw, expect in BAD_SEQS:
        assert call(L, cache(), seqs(**kw)) == expect, kw
    assert call(L, cache(), seqs(), n=-1) == SHAPE
    # nothing to do
    assert call(L, cache(), seqs(n_seqs=0)) == OK
    assert call(L, cache(), seqs(max_tokens=0)) == OK
    assert call(L, cache(), seqs(), n=0) == OK


def test_write_and_read_checks(L):
    assert write(L, cache(), seqs(), k=None) == NULL and write(L, cache(), seqs(), v=None) == NULL
    assert write(L, cache(), seqs(), k=FAKE_ODD) == ALIGN and write(L, cache(), seqs(), v=FAKE_ODD) == ALIGN
    for i in range(4):
        for bad in (4, -8):
            st = [256, 128, 256, 128]
            st[i] = bad
            assert write(L, cache(), seqs(), strides=st) == SHAPE
    assert write(L, cache(), seqs(max_pages=0)) == OK
    assert read(L, cache(), seqs(), k=None, v=None) == OK
    assert read(L, cache(), seqs(), k=FAKE_ODD) == ALIGN and read(L, cache(), seqs(), v=FAKE_ODD) == ALIGN


def test_attention_checks(L):
    c, s = cache(), seqs()
    assert attend(L, c, s, heads=0) == SHAPE and attend(L, c, s, heads=3) == SHAPE
    assert attend(L, c, s, n=2 ** 30) == SHAPE          # rows x heads past 32 bits
    assert attend(L, c, seqs(max_tokens=2 ** 30)) == SHAPE
    assert L.awq_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(seqs(max_tokens=2 ** 30)), 4) == 0
    assert attend(L, c, s, qs=(4, 128)) == SHAPE and attend(L, c, s, qs=(512, -8)) == SHAPE
    assert attend(L, c, s, os=(4, 128)) == SHAPE and attend(L, c, s, os=(512, 12)) == SHAPE
    for bad in (float("nan"), float("inf")):
        assert attend(L, c, s, scale=bad) == CONFIG
    assert attend(L, c, s, causal=2) == CONFIG
    assert attend(L, c, s, window=-1) == CONFIG and attend(L, c, s, causal=0, window=4) == CONFIG
    assert attend(L, c, s, q=None) == NULL and attend(L, c, s, out=None) == NULL
    assert attend(L, c, s, q=FAKE_ODD) == ALIGN and attend(L, c, s, out=FAKE_ODD) == ALIGN
    assert attend(L, c, s, lse=FAKE + 2) == ALIGN
    assert attend(L, c, s, ws=FAKE + 128, nbytes=1 << 30) == ALIGN
    need = L.awq_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(s), 4)
    assert need > 0 and attend(L, c, s, ws=FAKE, nbytes=need - 1) == WORKSPACE


def test_outputs_that_share_memory(L):
    c, s = cache(), seqs()
    assert attend(L, c, s, os=(0, 128)) == SHAPE and attend(L, c, s, os=(512, 0)) == SHAPE
    assert attend(L, c, s, os=(64, 1920)) == SHAPE


def test_more_blocks_than_a_launch_takes(L):
    q = L.awq_kv_attention_workspace_bytes
    many = cache(n_kv_heads=40000)          # two row tiles of 40000 heads
    assert q(ctypes.byref(many), ctypes.byref(seqs(max_tokens=20)), 40000) == 0
    assert attend(L, many, seqs(max_tokens=20), heads=40000) == SHAPE
    loose = seqs(max_tokens=2 ** 30, n_seqs=1)
    assert q(ctypes.byref(cache(n_kv_heads=2)), ctypes.byref(loose), 2) == 0
    assert attend(L, cache(n_kv_heads=2), loose, heads=2) == SHAPE
    pages = seqs(max_tokens=2 ** 31 - 1, max_len=1 << 30, max_pages=1 << 25, table_stride=1 << 25, n_seqs=1)
    assert write(L, cache(page_size=32), pages, n=2 ** 31 - 1) == SHAPE


def test_workspace_query(L):
    q = L.awq_kv_attention_workspace_bytes
    c = cache()
    assert q(ctypes.byref(cache(head_dim=80)), ctypes.byref(seqs()), 4) == 0
    assert q(ctypes.byref(c), ctypes.byref(seqs()), 3) == 0 and q(None, ctypes.byref(seqs()), 4) == 0
    assert q(ctypes.byref(c), ctypes.byref(seqs(n_seqs=0)), 4) > 0
    # long sequences on few heads split, many sequences do not need to
    long = q(ctypes.byref(c), ctypes.byref(seqs(n_seqs=1, max_tokens=1, max_len=1 << 20)), 4)
    assert long > q(ctypes.byref(c), ctypes.byref(seqs(n_seqs=1, max_tokens=1, max_len=64)), 4)
    assert long < 1 << 28


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.KVCache(torch.zeros(1, 1, 8, 64, 16, dtype=torch.uint8), torch.zeros(1, 1, 4, 128, 16, dtype=torch.uint8),
                    torch.zeros(1, 1), torch.zeros(1, 1))
    with pytest.raises(ValueError, match="fmt"):
        awq.KVCache(None, None, None, None, "int3")
    t = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.KVSeqs(t, torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 1, 1)
    with pytest.raises(TypeError):
        awq.KVSeqs([[0]], None, None, 1, 1)


# ---------------------------------------------------------------- the oracle

def test_oracle_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(kv_oracle.e4m3_value(b), t)
    finite = b[~np.isnan(t)]
    np.testing.assert_array_equal(kv_oracle.e4m3_bits(kv_oracle.e4m3_value(finite)), finite)
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.01,
                        (t[:126:1] + t[1:127]) / 2]).astype(np.float32)     # midpoints: ties to even
    np.testing.assert_array_equal(kv_oracle.e4m3_round(x),
                                  torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_oracle_write_by_hand():
    """Two tokens of maximum 1.27, then one of 2.54: the scale doubles and the
    old codes halve (ties to even)."""
    codes, scales = np.zeros((1, 1, 32, 64)), np.zeros((1, 1), np.float32)
    x = np.zeros((2, 1, 64), np.float16)
    x[0, 0, :3] = [1.27, -0.03, 0.05]
    x[1, 0, 0] = -1.0
    table = [[0]]
    kv_oracle.write(codes, scales, x, table, [0, 2], [2], "int8")
    assert abs(scales[0, 0] - 0.01) < 1e-5
    assert list(codes[0, 0, 0, :3]) == [127, -3, 5] and codes[0, 0, 1, 0] == -100
    y = np.zeros((1, 1, 64), np.float16)
    y[0, 0, 0] = np.float16(1.27) * 2
    kv_oracle.write(codes, scales, y, table, [0, 1], [3], "int8")
    assert list(codes[0, 0, 0, :3]) == [64, -2, 2] and codes[0, 0, 1, 0] == -50 and codes[0, 0, 2, 0] == 127
    # a smaller token leaves the scale and the old codes alone
    before, s = codes.copy(), scales.copy()
    kv_oracle.write(codes, scales, y * 0 + np.float16(0.5), table, [0, 1], [4], "int8")
    np.testing.assert_array_equal(codes[0, 0, :3], before[0, 0, :3])
    np.testing.assert_array_equal(scales, s)


def test_oracle_attention_is_softmax():
    rng = np.random.default_rng(3)
    kc, vc = rng.integers(-127, 128, (2, 1, 32, 64)).astype(float), rng.integers(-127, 128, (2, 1, 32, 64)).astype(float)
    ks, vs = np.full((2, 1), 0.01, np.float32), np.full((2, 1), 0.02, np.float32)
    q = rng.standard_normal((1, 1, 64))
    out, lse, _, _ = kv_oracle.attention(q, kc, ks, vc, vs, [[1, 0]], [0, 1], [40], 0.125)
    k = np.concatenate([kc[1, 0], kc[0, 0]])[:40] * np.float64(np.float32(0.01))
    v = np.concatenate([vc[1, 0], vc[0, 0]])[:40] * np.float64(np.float32(0.02))
    t = 0.125 * k @ q[0, 0]
    w = np.exp(t)
    np.testing.assert_allclose(out[0, 0], (w / w.sum()) @ v, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse[0, 0], np.log(w.sum()), rtol=1e-12)
    # causal rows before the first token see nothing
    out, lse, _, _ = kv_oracle.attention(np.ones((3, 1, 64)), kc, ks, vc, vs, [[1, 0]], [0, 3], [1], 0.125)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2]).all()
