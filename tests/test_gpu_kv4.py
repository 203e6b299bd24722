"""The paged 4-bit cache (awq_kv_write, awq_kv_read with "int4") and the
attention over it (awq_kv_attention) against the CPU oracle.

Write: codes, steps and smallest numbers as the oracle's float32 steps give
them, exactly. Read: exactly. Attention: per element, with A = sum_j w_j |v_j|
over the exact weights w (sum 1), N the visible keys, D the channels,
u = 2^-24, S the largest scale * sum |q_d k_d| of a row, V the largest |v|:
  * a logit is D products summed in fp32, each step off by at most u of a
    partial sum no larger than S; the multiplication with the scale and the
    subtraction of the maximum (both below 1.45 S and 12 in the binary
    logarithm) round at most 4 u S + 16 u more: (D + 8) u S + 16 u, relative
    on a weight;
  * 2^x of the hardware is within 2^-22, the sums of N weights and their
    rescaling round 2 N u: together e = 2 ((D + 8) u S + 16 u + 2^-21 + 2 N u),
    once in the numerator, once in the denominator;
  * a weight enters the second product as two fp16 numbers, within 2^-20 of
    itself, or, where the second is subnormal, 2^-24 in units of which the
    row's largest weight is at least 2^12: N 2^-36 V;
  * the output is rounded to fp16: 2^-11 |o|, or 2^-25 for a subnormal.
so |err| <= (e + 2^-20) A + N 2^-36 V + 2^-11 |o| + 2^-25, and
|err lse| <= e + 2^-22 |lse| + 16 u.
"""

import numpy as np
import pytest

from oracle import kv_oracle, layer_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host, say  # noqa: E402


class Model:
    """A cache on the GPU, filled with garbage (codes 15, NaN scales), and the
    oracle's beside it, with a shuffled table."""

    def __init__(self, seed, n_seqs, heads, dim, page, max_len, spare=2):
        self.rng = np.random.default_rng(seed)
        self.page, self.heads, self.dim = page, heads, dim
        per = -(-max_len // page)
        self.pages = n_seqs * per + spare
        order = self.rng.permutation(self.pages).astype(np.int32)
        self.table = order[: n_seqs * per].reshape(n_seqs, per).copy()
        self.len = np.zeros(n_seqs, np.int32)
        self.cache = awq.KVCache.empty(self.pages, heads, dim, page, "int4", "cuda")
        self.cache.k_codes.fill_(0xFF)
        self.cache.v_codes.fill_(0xFF)
        self.cache.k_scales.fill_(float("nan"))
        self.cache.v_scales.fill_(float("nan"))
        shape = (self.pages, heads, page, dim)
        self.kc, self.vc = np.full(shape, 15, np.uint8), np.full(shape, 15, np.uint8)
        self.ks = np.full((self.pages, heads, page, dim // 32, 2), np.nan, np.float16)
        self.vs = np.full((self.pages, heads, page, 2), np.nan, np.float16)

    def seqs(self, new, lens=None, table=None, max_tokens=None, max_len=None):
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        lens = self.len if lens is None else np.asarray(lens, np.int32)
        table = self.table if table is None else table
        s = awq.KVSeqs(dev(np.ascontiguousarray(table)), dev(cu), dev(lens.copy()),
                       int(max(new, default=0)) if max_tokens is None else max_tokens,
                       int(lens.max(initial=0)) if max_len is None else max_len)
        return s, cu, lens, table

    def values(self, n, spread=1.0):
        x = self.rng.standard_normal((n, self.heads, self.dim)) * spread
        x[..., :2] *= 6.0
        return (x * np.exp(self.rng.standard_normal((n, 1, 1)) * 0.5)).astype(np.float16)

    def append(self, new, k=None, v=None, table=None, call=None):
        """Writes new[b] tokens behind every sequence, on both sides."""
        new = np.asarray(new)
        self.len = (self.len + new).astype(np.int32)
        s, cu, lens, table = self.seqs(new, table=table)
        k = self.values(int(new.sum())) if k is None else k
        v = self.values(int(new.sum()), 0.3) if v is None else v
        kd, vd = (dev(k), dev(v)) if call is None else call(k, v)
        awq.awq_kv_write(self.cache, s, kd, vd)
        lo.write(self.kc, self.ks, k, table, cu, lens, "k")
        lo.write(self.vc, self.vs, v, table, cu, lens, "v")

    def check(self, table=None):
        """Every written token's codes and scales; pages never written as they were."""
        torch.cuda.synchronize()
        table = self.table if table is None else table
        kb, vb = host(self.cache.k_codes), host(self.cache.v_codes)
        kc, vc = lo.load_k(kb), lo.load_v(vb)
        ks, vs = lo.load_k_scales(host(self.cache.k_scales)), lo.load_v_scales(host(self.cache.v_scales))
        used = np.zeros(self.pages, int)
        for b, n in enumerate(self.len):
            for p in range(-(-int(n) // self.page)):
                if 0 <= table[b, p] < self.pages:
                    used[table[b, p]] = min(self.page, n - p * self.page)
        for pid in range(self.pages):
            n = used[pid]
            if n == 0:
                assert (kb[pid] == 0xFF).all() and (vb[pid] == 0xFF).all()
                assert np.isnan(ks[pid]).all() and np.isnan(vs[pid]).all()
                continue
            np.testing.assert_array_equal(ks[pid, :, :n], self.ks[pid, :, :n])
            np.testing.assert_array_equal(vs[pid, :, :n], self.vs[pid, :, :n])
            np.testing.assert_array_equal(kc[pid, :, :n], self.kc[pid, :, :n])
            np.testing.assert_array_equal(vc[pid, :, :n], self.vc[pid, :, :n])
            # keys and scales of slots not written yet stay
            assert (kc[pid, :, n:] == 15).all() and np.isnan(ks[pid, :, n:]).all() and np.isnan(vs[pid, :, n:]).all()

    def check_read(self, new, table=None):
        s, cu, lens, table = self.seqs(new, table=table)
        k, v = awq.awq_kv_read(self.cache, s)
        torch.cuda.synchronize()
        for got, codes, scales, side in ((k, self.kc, self.ks, "k"), (v, self.vc, self.vs, "v")):
            want = np.zeros(got.shape, np.float16)
            lo.read(codes, scales, want, table, cu, lens, side)
            np.testing.assert_array_equal(host(got), want)

    def attend(self, q, new, lens=None, table=None, scale=None, causal=True, window=0, split=True, max_tokens=None,
               max_len=None, out=None):
        s, cu, lens, table = self.seqs(new, lens, table, max_tokens, max_len)
        scale = self.dim ** -0.5 if scale is None else scale
        ws = awq.kv_attention_workspace(self.cache, s, q.shape[1]) if split else None
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        qd = dev(q) if isinstance(q, np.ndarray) else q
        out = awq.awq_kv_attention(qd, self.cache, s, scale, causal, window, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        if ws is not None:
            assert not host(ws[:4096 * 4]).any()        # the counters are back at zero
        return host(out), host(lse), self.want(host(qd), table, cu, lens, scale, causal, window)

    def want(self, q, table, cu, lens, scale, causal=True, window=0):
        ks, vs = np.nan_to_num(self.ks), np.nan_to_num(self.vs)
        return lo.attention(q, self.kc, ks, self.vc, vs, table, cu, lens, scale, causal, window)

    def assert_attention(self, got, n_keys):
        o, lse, (eo, elog, spread, mass) = got
        u = 2.0 ** -24
        e = 2 * ((self.dim + 8) * u * mass + 16 * u + 2.0 ** -21 + 2 * n_keys * u)
        top = float(np.abs(lo.v_numbers(self.vc, np.nan_to_num(self.vs)).astype(np.float64)).max())
        tol = (e[..., None] + 2.0 ** -20) * spread + n_keys * 2.0 ** -36 * top + 2.0 ** -11 * np.abs(eo) + 2.0 ** -25
        err = np.abs(o.astype(np.float64) - eo)
        assert np.isfinite(o).all()
        assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"
        empty = np.isneginf(elog)
        assert np.isneginf(lse[empty]).all() and (o[empty] == 0).all()
        ok = ~empty
        lerr, ltol = np.abs(lse[ok] - elog[ok]), e[ok] + 2.0 ** -22 * np.abs(elog[ok]) + 16 * u
        assert (lerr <= ltol).all(), f"lse worst {np.max(lerr / ltol):.3f} of the bound"
        return float(np.max(err / tol)) if err.size else 0.0


# ---------------------------------------------------------------- write and read

@pytest.mark.parametrize("dim,page,heads", [(64, 32, 3), (96, 64, 1), (128, 64, 2), (192, 128, 2), (256, 256, 1)])
def test_write_and_read(dim, page, heads):
    """A ragged prompt, single tokens, a few at once over page borders, a
    sequence that gets none; then everything back, and the newest tokens only."""
    say("kv4 write", dim, page)
    m = Model([1, dim, page], 4, heads, dim, page, 3 * page + 40)
    m.append([page + 7, 1, 2 * page, 0])
    m.check()
    for step in range(4):
        m.append([1, 1, 0 if step == 2 else 1, 1], k=m.values(4 if step != 2 else 3, 4.0 ** step))
        m.check()
    m.append([page, 17, 3, 33])
    m.check()
    m.check_read(m.len)
    m.check_read(np.minimum(m.len, 5))


def test_write_strided_inputs():
    """k and v as slices of one packed projection, and head-major tensors."""
    m = Model([2], 2, 2, 128, 64, 200)

    def packed(k, v):
        t = torch.zeros(k.shape[0], 6, 128, dtype=torch.float16, device="cuda")
        t[:, 2:4], t[:, 4:6] = dev(k), dev(v)
        return t[:, 2:4], t[:, 4:6]

    def head_major(k, v):
        return tuple(dev(np.ascontiguousarray(t.transpose(1, 0, 2))).transpose(0, 1) for t in (k, v))

    m.append([70, 130], call=packed)
    m.append([1, 1], call=head_major)
    m.append([60, 5], call=head_major)
    m.check()


def test_write_extreme_values():
    """Zeros, constant groups far from zero, subnormals, the largest fp16
    numbers, infinities and NaN, groups whose quotients are halfway."""
    m = Model([3], 3, 2, 64, 32, 96)
    k = m.values(3 * 33)
    k[:20] = 0
    k[20:33] = np.float16(1000.5)
    k[33:50, 0] = np.float16(6e-8) * np.arange(17 * 64).reshape(17, 64) % 9
    k[66:, 0, :5] = [np.inf, -np.inf, np.nan, 65504, -65504]
    v = m.values(3 * 33)
    v[5, 1, 3], v[40, 0, 7], v[70, 1] = np.nan, -np.inf, np.nan
    v[50:60] = (m.rng.integers(0, 31, (10, 2, 64)) * 0.5 + 3).astype(np.float16)      # steps of 1, halves between
    v[50:60, :, 0], v[50:60, :, 1] = 3, 18
    m.append([33, 33, 33], k=k, v=v)
    m.check()
    k = m.values(3)
    k[0, 0, 0] = np.inf
    m.append([1, 1, 1], k=k)
    m.check()
    m.check_read(m.len)


@pytest.mark.parametrize("dim,page", [(64, 32), (128, 64)])
def test_write_among_later_tokens(dim, page):
    """Tokens written again, at every place of a word of eight, leave the later
    tokens of their pages."""
    m = Model(24, 2, 2, dim, page, 100)
    m.append([100, 70])
    for first, n in ((35, 1), (64, 3), (8, 8), (30, 7), (95, 4)):
        say("kv4 write among", dim, first, n)
        s, cu, lens, table = m.seqs([n, 0], lens=[first + n, 70])
        k, v = m.values(n), m.values(n, 0.3)
        awq.awq_kv_write(m.cache, s, dev(k), dev(v))
        lo.write(m.kc, m.ks, k, table, cu, lens, "k")
        lo.write(m.vc, m.vs, v, table, cu, lens, "v")
        m.check()
    m.check_read([100, 70])


def test_write_many_random_groups():
    """Half a million groups over 30 binary orders of magnitude."""
    m = Model([4], 1, 16, 256, 256, 4096)
    k, v = (m.values(4096, 1.0) for _ in range(2))
    scale = np.exp2(m.rng.integers(-16, 14, (4096, 16, 1))).astype(np.float32)
    k, v = (np.clip(t.astype(np.float32) * scale, -65504, 65504).astype(np.float16) for t in (k, v))
    m.append([4096], k=k, v=v)
    m.check()


def test_write_beyond_the_cache():
    """Pages the cache does not hold, more new tokens than the length, rows
    past n_tokens, lengths past the table: nothing else changes."""
    m = Model([5], 3, 2, 64, 32, 96)
    bad = m.table.copy()
    bad[0, 1], bad[1, 0], bad[2, 2] = -1, m.pages, 2 ** 31 - 1
    m.append([70, 40, 96], table=bad)
    m.check(table=bad)
    m.check_read(m.len, table=bad)
    # 5 new tokens of a sequence of length 2: only the last two are its
    m = Model([6], 1, 1, 64, 32, 32)
    m.len[:] = -3
    m.append([5])
    m.check()
    m.check_read([5])
    # a length past the table's pages counts as their tokens
    s = awq.KVSeqs(dev(m.table), dev(np.array([0, 1], np.int32)), dev(np.array([10 ** 6], np.int32)), 1, 10 ** 6)
    before = lo.load_k(host(m.cache.k_codes))
    awq.awq_kv_write(m.cache, s, dev(m.values(1)), dev(m.values(1)))
    torch.cuda.synchronize()
    now = lo.load_k(host(m.cache.k_codes))
    assert (now[m.table[0, 0], 0, :31] == before[m.table[0, 0], 0, :31]).all()
    # cu_tokens past the tensor's rows: clamped
    s = awq.KVSeqs(dev(m.table), dev(np.array([0, 500], np.int32)), dev(np.array([4], np.int32)), 500, 32)
    awq.awq_kv_write(m.cache, s, dev(m.values(3)), dev(m.values(3)))
    torch.cuda.synchronize()


def test_read_leaves_other_rows():
    m = Model([7], 2, 1, 64, 32, 64)
    m.append([40, 20])
    s, cu, lens, table = m.seqs([10, 5])
    k = torch.full((20, 1, 64), 3.0, dtype=torch.float16, device="cuda")
    v = k.clone()
    awq.awq_kv_read(m.cache, s, out=(k, v))
    torch.cuda.synchronize()
    for got, codes, scales, side in ((k, m.kc, m.ks, "k"), (v, m.vc, m.vs, "v")):
        want = np.full((20, 1, 64), 3.0, np.float16)
        lo.read(codes, scales, want, table, cu, lens, side)
        np.testing.assert_array_equal(host(got), want)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("dim,page,heads,ratio,lens,new", [
    (128, 64, 2, 4, [1, 63, 64, 65, 1000], [1, 1, 1, 1, 1]),        # decode, ragged
    (128, 64, 1, 1, [700], [1]),
    (64, 32, 3, 2, [33, 500, 31], [1, 1, 1]),                       # two pages a tile
    (96, 128, 1, 3, [300, 129], [5, 1]),                            # 15 rows of odd heads
    (128, 32, 2, 2, [77, 129], [1, 6]),
    (192, 32, 1, 8, [100, 257], [2, 4]),                            # two row tiles
    (256, 256, 1, 1, [513], [3]),
    (128, 64, 2, 4, [300, 64, 10], [100, 64, 1]),                   # prefill, ragged
    (64, 32, 1, 1, [130, 1], [130, 1]),
    (96, 64, 1, 5, [200], [77]),
    (128, 32, 1, 2, [190, 33], [60, 33]),
    (192, 128, 1, 1, [260], [200]),
    (256, 32, 1, 2, [150, 90], [90, 90]),
])
def test_attention(split, dim, page, heads, ratio, lens, new):
    say("kv4 attention", dim, page, lens, new, "split" if split else "whole")
    m = Model([10, dim, page, len(lens)], len(lens), heads, dim, page, max(lens))
    m.append(lens)
    q = (m.rng.standard_normal((sum(new), heads * ratio, dim)) * 2).astype(np.float16)
    worst = m.assert_attention(m.attend(q, new, split=split), max(lens))
    say("  worst", round(worst, 3), "of the bound")


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 50), (True, 64), (True, 1000)])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_attention_masks(causal, window, new):
    m = Model([11, window, new], 3, 2, 64, 64, 700)
    m.append([700, 130, 90])
    say("kv4 attention mask", causal, window, new)
    q = (m.rng.standard_normal((3 * new, 4, 64)) * 2).astype(np.float16)
    m.assert_attention(m.attend(q, [new] * 3, causal=causal, window=window), 700)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-40, 0.7])
def test_attention_scale(scale, new):
    m = Model([12, new], 2, 1, 128, 64, 200)
    m.append([200, 70])
    q = m.rng.standard_normal((2 * new, 2, 128)).astype(np.float16)
    m.assert_attention(m.attend(q, [new, new], scale=scale, window=0), 200)
    m.assert_attention(m.attend(q, [new, new], scale=scale, window=20), 200)


@pytest.mark.parametrize("ratio,new", [(2, 3), (2, 40)])
def test_attention_empty_rows(ratio, new):
    """Sequences of length zero, sequences without queries, more queries than
    tokens (the first see nothing), rows of no sequence."""
    m = Model([13, new], 4, 1, 64, 32, 100)
    m.append([100, 0, 2, 5])
    n = [new, new, new, 0]
    q = m.rng.standard_normal((3 * new + 4, ratio, 64)).astype(np.float16)
    q[-4:] = np.nan
    out = torch.full((3 * new + 4, ratio, 64), 5.0, dtype=torch.float16, device="cuda")
    s, cu, lens, table = m.seqs(n)
    ws = awq.kv_attention_workspace(m.cache, s, ratio)
    for causal in (True, False):
        out.fill_(5.0)
        lse = torch.full((3 * new + 4, ratio), 7.0, device="cuda")
        awq.awq_kv_attention(dev(q), m.cache, s, causal=causal, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert (host(out)[3 * new:] == 5).all() and (host(lse)[3 * new:] == 7).all()
        want = m.want(q[:3 * new], table, cu, lens, 0.125, causal)
        m.assert_attention((host(out)[:3 * new], host(lse)[:3 * new], want), 100)


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("new", [1, 50])
def test_attention_missing_pages(new, page):
    """Pages the cache does not hold are not seen, whatever is in page 0."""
    m = Model([14], 2, 2, 128, page, 300)
    m.append([300, 200])
    m.cache.k_scales[0].fill_(float("inf")), m.cache.v_scales[0].fill_(float("nan"))
    bad = m.table.copy()
    bad[m.table == 0] = -1          # page 0 is nobody's
    bad[0, 0], bad[0, 4], bad[1, 3], bad[1, :2] = -1, m.pages + 5, -7, -1
    q = m.rng.standard_normal((2 * new, 4, 128)).astype(np.float16)
    m.assert_attention(m.attend(q, [new, new], table=bad), 300)
    bad[1, :] = -1
    got = m.attend(q, [new, new], table=bad)
    m.assert_attention(got, 300)
    assert (got[0][new:] == 0).all()


@pytest.mark.parametrize("page", [32, 64, 256])
@pytest.mark.parametrize("new", [1, 9, 90])
def test_attention_nothing_before_the_window(new, page):
    """Positions before every query's window and behind the end hold NaN scales."""
    m = Model(25, 2, 2, 64, page, 420)
    m.append([400, 243])
    q = m.rng.standard_normal((2 * new, 4, 64)).astype(np.float16)
    plain = m.attend(q, [new, new], causal=True, window=21)
    m.assert_attention(plain, 21)
    for b in range(2):
        first = int(m.len[b]) - new - 20        # the first query's window
        for p in range(first // page + 1):
            pid, n = int(m.table[b, p]), min(page, first - p * page)
            m.cache.k_scales[pid, :, :, :n] = float("nan")
            m.cache.v_scales[pid, :, :, :n] = float("nan")
    got = m.attend(q, [new, new], causal=True, window=21)
    np.testing.assert_array_equal(got[0], plain[0])
    np.testing.assert_array_equal(got[1], plain[1])


@pytest.mark.parametrize("new", [2, 70])
def test_attention_values_far_apart(new):
    """Values whose sizes differ by 2^26 from token to token."""
    m = Model([15, new], 1, 1, 64, 32, 320)
    v = m.values(320, 1.0) * np.exp2(m.rng.integers(-13, 13, (320, 1, 1)))
    m.append([320], v=np.clip(v, -6e4, 6e4).astype(np.float16))
    q = m.rng.standard_normal((new, 2, 64)).astype(np.float16)
    m.assert_attention(m.attend(q, [new]), 320)
    m.assert_attention(m.attend(q, [new], window=16), 320)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_steep(new):
    """Logits of several hundred, rising and falling along the keys: the
    maximum moves in every tile, or never again."""
    for order in (1, -1):
        m = Model([16, new], 1, 1, 64, 64, 640)
        k = m.values(640, 0.1)
        k[:, 0, 3] = (np.arange(640)[::order] * 0.4).astype(np.float16)
        m.append([640], k=k)
        q = m.rng.standard_normal((new, 1, 64)).astype(np.float16)
        q[:, :, 3] = 8.0
        m.assert_attention(m.attend(q, [new], causal=False), 640)


@pytest.mark.parametrize("new", [1, 60])
def test_attention_nan_queries(new):
    """A NaN reaches its own row and no other."""
    m = Model([17, new], 2, 2, 64, 64, 300)
    m.append([300, 100])
    q = m.rng.standard_normal((2 * new, 4, 64)).astype(np.float16)
    clean = m.attend(q, [new, new])
    bad = q.copy()
    bad[0, 1, 5] = np.nan
    bad[-1, 2, 0] = np.inf
    o, lse, _ = m.attend(bad, [new, new])
    touched = np.zeros(o.shape[:2], bool)
    touched[0, 1] = touched[-1, 2] = True
    assert np.isnan(o[0, 1]).all() and np.isnan(lse[0, 1])
    np.testing.assert_array_equal(o[~touched], clean[0][~touched])
    np.testing.assert_array_equal(lse[~touched], clean[1][~touched])


def test_attention_strides_and_streams():
    """Head-major queries and outputs, another stream than the inputs'."""
    m = Model([18], 2, 2, 128, 64, 300)
    m.append([300, 100])
    q = m.rng.standard_normal((4, 8, 128)).astype(np.float16)
    qt = dev(np.ascontiguousarray(q.transpose(1, 0, 2))).transpose(0, 1)
    out = torch.zeros(8, 4, 128, dtype=torch.float16, device="cuda").transpose(0, 1)
    plain = m.attend(q, [2, 2])
    got = m.attend(qt, [2, 2], out=out)
    np.testing.assert_array_equal(got[0], plain[0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = m.attend(q, [2, 2])
    np.testing.assert_array_equal(got[0], plain[0])


def test_results_do_not_vary():
    m = Model([19], 2, 2, 128, 64, 5000)
    m.append([5000, 3000])
    for new in (1, 40):
        q = m.rng.standard_normal((2 * new, 8, 128)).astype(np.float16)
        s, *_ = m.seqs([new, new])
        ws = awq.kv_attention_workspace(m.cache, s, 8)
        first = awq.awq_kv_attention(dev(q), m.cache, s, workspace=ws)
        for _ in range(5):
            assert torch.equal(awq.awq_kv_attention(dev(q), m.cache, s, workspace=ws), first)


def test_graph_replay():
    """A captured decode step (write, attention, read) replayed with new
    tokens and lengths, with eager work between."""
    m = Model([20], 2, 2, 128, 64, 400)
    m.append([130, 62])
    table, lens = dev(m.table), dev(m.len + 1)
    s = awq.KVSeqs(table, dev(np.array([0, 1, 2], np.int32)), lens, 1, 400)
    k, v, q = (torch.zeros(2, h, 128, dtype=torch.float16, device="cuda") for h in (2, 2, 8))
    ws = awq.kv_attention_workspace(m.cache, s, 8)
    out, back = torch.zeros_like(q), (torch.zeros_like(k), torch.zeros_like(v))

    def step():
        awq.awq_kv_write(m.cache, s, k, v)
        awq.awq_kv_attention(q, m.cache, s, out=out, workspace=ws)
        awq.awq_kv_read(m.cache, s, out=back)

    lens.zero_()                    # the warm-up and the capture change nothing
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        kn, vn, qn = m.values(2), m.values(2, 0.3), m.rng.standard_normal((2, 8, 128)).astype(np.float16)
        k.copy_(dev(kn)), v.copy_(dev(vn)), q.copy_(dev(qn)), lens.copy_(dev(m.len + 1))
        graph.replay()
        torch.cuda.synchronize()
        m.len = (m.len + 1).astype(np.int32)
        cu = np.array([0, 1, 2], np.int32)
        lo.write(m.kc, m.ks, kn, m.table, cu, m.len, "k")
        lo.write(m.vc, m.vs, vn, m.table, cu, m.len, "v")
        m.check()
        lse = np.zeros((2, 8), np.float32)
        want = m.want(qn, m.table, cu, m.len, 128 ** -0.5)
        m.assert_attention((host(out), want[1].astype(np.float32), want), 400)
        m.check_read([1, 1])
        np.testing.assert_array_equal(host(awq.awq_kv_attention(q, m.cache, s, workspace=ws)), host(out))


def test_far_pages():
    """Pages past 2^31 bytes of codes."""
    heads, dim, page = 8, 256, 256
    pages = 2 ** 31 // (heads * dim * page // 2) + 40
    cache = awq.KVCache.empty(pages, heads, dim, page, "int4")
    table = dev(np.array([[pages - 1, 0, pages - 2]], np.int32))
    small = awq.KVCache.empty(3, heads, dim, page, "int4")
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(600, heads, dim, generator=g, device="cuda").half() for _ in range(2))
    outs = []
    for c, t in ((cache, table), (small, dev(np.array([[2, 0, 1]], np.int32)))):
        s = awq.KVSeqs(t, dev(np.array([0, 600], np.int32)), dev(np.array([600], np.int32)), 600, 600)
        awq.awq_kv_write(c, s, k, v)
        one = awq.KVSeqs(t, dev(np.array([0, 1], np.int32)), dev(np.array([600], np.int32)), 1, 600)
        outs.append((*awq.awq_kv_read(c, s), awq.awq_kv_attention(k, c, s), awq.awq_kv_attention(k[:1], c, one)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
