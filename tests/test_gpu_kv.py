"""The paged 8-bit cache (awq_kv_write, awq_kv_read) and the attention over
it (awq_kv_attention) against the CPU oracle.

Write: codes and scales bit for bit (the oracle takes the same float32
steps). Read: bit for bit. Attention: per element, with A = sum_j w_j |v_j|
over the exact weights w (sum 1), N the visible keys, D the channels,
u = 2^-24, S the largest scale * sum |q_d k_d| of a row:
  * a logit is D products summed in fp32 and two multiplications, each step
    off by at most u of a partial sum no larger than S (its log2 e multiple
    is rounded once more): (D + 4) u S absolute, so relative on a weight;
  * 2^x of the hardware and the reciprocal are within 2^-22 each, the sums of
    N weights and the rescaling per 64 keys round N + N / 16 times: together
    e = 2 ((D + 4) u S + 2^-21 + 2 N u), once in the numerator, once in the
    denominator;
  * a weight is rounded to fp16, half a step 2^-11 of it; in its unit (2^-14
    of the largest scale in decode, 2^-10 of up to twice it in prefill) the
    subnormal half step is 2^-34 of the largest page scale V at most, on N
    values of up to `top` steps: N 2^-34 top V;
  * the output is rounded to fp16: 2^-11 |o|, or 2^-25 for a subnormal.
so |err| <= (e + 2^-11) A + N 2^-34 top V + 2^-11 |o| + 2^-25, and |err lse| <= e + 2^-22 |lse|.
"""

import ctypes

import numpy as np
import pytest

from oracle import kv_oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host, say  # noqa: E402


class Model:
    """A cache on the GPU and the oracle's beside it, with a shuffled table."""

    def __init__(self, seed, n_seqs, heads, dim, page, fmt, max_len, garbage=0xFF, spare=2):
        self.rng = np.random.default_rng(seed)
        self.fmt, self.page, self.heads, self.dim = fmt, page, heads, dim
        per = -(-max_len // page)
        self.pages = n_seqs * per + spare
        order = self.rng.permutation(self.pages).astype(np.int32)
        self.table = order[: n_seqs * per].reshape(n_seqs, per).copy()
        self.len = np.zeros(n_seqs, np.int32)
        self.cache = awq.KVCache.empty(self.pages, heads, dim, page, fmt, "cuda")
        self.cache.k_codes.fill_(garbage)       # fp8 NaN, or code 127: nothing unwritten may matter
        self.cache.v_codes.fill_(garbage)
        self.cache.k_scales.fill_(float("nan"))
        self.cache.v_scales.fill_(float("nan"))
        shape = (self.pages, heads, page, dim)
        self.kc, self.vc = np.zeros(shape), np.zeros(shape)
        self.ks, self.vs = np.zeros(shape[:2], np.float32), np.zeros(shape[:2], np.float32)

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
        kv_oracle.write(self.kc, self.ks, k, table, cu, lens, self.fmt)
        kv_oracle.write(self.vc, self.vs, v, table, cu, lens, self.fmt)
        return s

    def check(self, table=None):
        """Every written token's codes, and its page's scales, bit for bit."""
        torch.cuda.synchronize()
        table = self.table if table is None else table
        got_k, got_v = kv_oracle.load_k(host(self.cache.k_codes)), kv_oracle.load_v(host(self.cache.v_codes))
        ks, vs = host(self.cache.k_scales), host(self.cache.v_scales)
        used = np.zeros(self.pages, int)
        for b, n in enumerate(self.len):
            for p in range(-(-int(n) // self.page)):
                if 0 <= table[b, p] < self.pages:
                    used[table[b, p]] = min(self.page, n - p * self.page)
        for pid in range(self.pages):
            n = used[pid]
            if n == 0:      # never written: as it was
                assert (got_k[pid] == 0xFF).all() and (got_v[pid] == 0xFF).all() and np.isnan(ks[pid]).all()
                continue
            np.testing.assert_array_equal(ks[pid], self.ks[pid])
            np.testing.assert_array_equal(vs[pid], self.vs[pid])
            np.testing.assert_array_equal(got_k[pid, :, :n], kv_oracle.to_bytes(self.kc[pid, :, :n], self.fmt))
            np.testing.assert_array_equal(got_v[pid, :, :n], kv_oracle.to_bytes(self.vc[pid, :, :n], self.fmt))

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
        want = kv_oracle.attention(host(qd), self.kc, self.ks, self.vc, self.vs, table, cu, lens, scale, causal, window)
        return host(out), host(lse), want

    def assert_attention(self, got, n_keys):
        o, lse, (eo, elog, spread, mass) = got
        u = 2.0 ** -24
        e = 2 * ((self.dim + 4) * u * mass + 2.0 ** -21 + 2 * n_keys * u)
        tol = (e[..., None] + 2.0 ** -11) * spread + 2.0 ** -11 * np.abs(eo) + 2.0 ** -25 + \
            n_keys * 2.0 ** -34 * float(kv_oracle.TOP[self.fmt]) * float(self.vs.max(initial=0))
        err = np.abs(o.astype(np.float64) - eo)
        assert np.isfinite(o).all()
        assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"
        empty = np.isneginf(elog)
        assert np.isneginf(lse[empty]).all() and (o[empty] == 0).all()
        ok = ~empty
        lerr, ltol = np.abs(lse[ok] - elog[ok]), e[ok] + 2.0 ** -22 * np.abs(elog[ok])
        assert (lerr <= ltol).all(), f"lse worst {np.max(lerr / ltol):.3f} of the bound"
        return float(np.max(err / tol)) if err.size else 0.0


# ---------------------------------------------------------------- write and read

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,page,heads", [(64, 32, 3), (96, 64, 1), (128, 64, 2), (192, 128, 2), (256, 256, 1)])
def test_write_steps_bit_exact(fmt, dim, page, heads):
    """A ragged prompt, single tokens (scales that grow and do not), a few at
    once over page borders, a sequence that gets none."""
    say("kv write", fmt, dim, page)
    m = Model([1, dim, page], 4, heads, dim, page, fmt, 3 * page + 40)
    m.append([page + 7, 1, 2 * page, 0])
    m.check()
    for step in range(4):
        m.append([1, 1, 0 if step == 2 else 1, 1], k=m.values(4 if step != 2 else 3, 4.0 ** step))
        m.check()
    m.append([page, 17, 3, 33])
    m.check()
    # read everything back, and the newest tokens only
    for new in (m.len, np.minimum(m.len, 5)):
        s, cu, lens, table = m.seqs(new)
        k, v = awq.awq_kv_read(m.cache, s)
        torch.cuda.synchronize()
        for got, codes, scales in ((k, m.kc, m.ks), (v, m.vc, m.vs)):
            want = np.zeros(got.shape, np.float16)
            kv_oracle.read(codes, scales, want, table, cu, lens)
            np.testing.assert_array_equal(host(got).view(np.uint16) & 0x7FFF, want.view(np.uint16) & 0x7FFF)
            np.testing.assert_array_equal(host(got), want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_strided_inputs(fmt):
    """k and v as slices of one packed projection, and head-major tensors."""
    m = Model([2], 2, 2, 128, 64, fmt, 200)

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


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_extreme_values(fmt):
    """Zeros, subnormals, the largest fp16 numbers, infinities and NaN."""
    m = Model([3], 3, 2, 64, 32, fmt, 96)
    k = m.values(3 * 33)
    k[:33] = 0
    k[33:66, 0] = np.float16(6e-8)
    k[66:, 0, :5] = [np.inf, -np.inf, np.nan, 65504, -65504]
    v = m.values(3 * 33)
    v[5, 1, 3], v[40, 0, 7], v[70, 1] = np.nan, -np.inf, np.nan
    m.append([33, 33, 33], k=k, v=v)
    m.check()
    k = m.values(3)
    k[0, 0, 0] = np.inf
    m.append([1, 1, 1], k=k)
    m.check()


def test_write_beyond_the_cache():
    """Pages the cache does not hold, more new tokens than the length, rows
    past n_tokens, lengths past the table: nothing else changes."""
    m = Model([4], 3, 2, 64, 32, "int8", 96)
    bad = m.table.copy()
    bad[0, 1], bad[1, 0], bad[2, 2] = -1, m.pages, 2 ** 31 - 1
    m.append([70, 40, 96], table=bad)
    m.check(table=bad)
    s, cu, lens, table = m.seqs(m.len, table=bad)
    k, v = awq.awq_kv_read(m.cache, s, out=(torch.full((206, 2, 64), 9.0, dtype=torch.float16, device="cuda"), None))
    assert v is None
    want = np.zeros((206, 2, 64), np.float16)
    kv_oracle.read(m.kc, m.ks, want, bad, cu, lens)
    np.testing.assert_array_equal(host(k), want)
    # 5 new tokens of a sequence of length 2: only the last two are its
    m = Model([5], 1, 1, 64, 32, "int8", 32)
    m.len[:] = -3
    m.append([5])
    m.check()
    s, *_ = m.seqs([5])
    k, _ = awq.awq_kv_read(m.cache, s)
    assert (host(k)[:3] == 0).all() and (host(k)[3:] != 0).any()
    # a length past the table's pages counts as their tokens
    before = host(m.cache.k_codes).copy()
    s = awq.KVSeqs(dev(m.table), dev(np.array([0, 1], np.int32)), dev(np.array([10 ** 6], np.int32)), 1, 10 ** 6)
    awq.awq_kv_write(m.cache, s, dev(m.values(1)), dev(m.values(1)))
    torch.cuda.synchronize()
    now = kv_oracle.load_k(host(m.cache.k_codes))
    assert (now[m.table[0, 0], 0, :31] == kv_oracle.load_k(before)[m.table[0, 0], 0, :31]).all()
    # cu_tokens past the tensor's rows: clamped
    s = awq.KVSeqs(dev(m.table), dev(np.array([0, 500], np.int32)), dev(np.array([4], np.int32)), 500, 32)
    awq.awq_kv_write(m.cache, s, dev(m.values(3)), dev(m.values(3)))
    torch.cuda.synchronize()


def test_read_leaves_other_rows():
    m = Model([6], 2, 1, 64, 32, "e4m3", 64)
    m.append([40, 20])
    s, cu, lens, table = m.seqs([10, 5])
    k = torch.full((20, 1, 64), 3.0, dtype=torch.float16, device="cuda")
    v = k.clone()
    awq.awq_kv_read(m.cache, s, out=(k, v))
    torch.cuda.synchronize()
    want = np.full((20, 1, 64), 3.0, np.float16)
    kv_oracle.read(m.vc, m.vs, want, table, cu, lens)
    np.testing.assert_array_equal(host(v), want)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("dim,page,heads,ratio,lens,new", [
    (128, 64, 2, 4, [1, 63, 64, 65, 1000], [1, 1, 1, 1, 1]),        # decode, ragged
    (128, 64, 1, 1, [700], [1]),
    (64, 32, 3, 2, [33, 500, 31], [1, 1, 1]),                       # two pages a tile
    (96, 128, 1, 3, [300, 129], [5, 1]),                            # 15 rows of odd heads
    (192, 32, 1, 8, [100, 257], [2, 4]),                            # two row tiles
    (256, 256, 1, 1, [513], [3]),
    (128, 64, 2, 4, [300, 64, 10], [100, 64, 1]),                   # prefill, ragged
    (64, 32, 1, 1, [130, 1], [130, 1]),
    (96, 64, 1, 5, [200], [77]),
    (192, 128, 1, 1, [260], [200]),
    (256, 32, 1, 2, [150, 90], [90, 90]),
])
def test_attention(fmt, split, dim, page, heads, ratio, lens, new):
    say("kv attention", fmt, dim, page, lens, new, "split" if split else "whole")
    m = Model([10, dim, page, len(lens)], len(lens), heads, dim, page, fmt, max(lens))
    m.append(lens)
    q = (m.rng.standard_normal((sum(new), heads * ratio, dim)) * 2).astype(np.float16)
    worst = m.assert_attention(m.attend(q, new, split=split), max(lens))
    say("  worst", round(worst, 3), "of the bound")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 50), (True, 64), (True, 1000)])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_attention_masks(fmt, causal, window, new):
    m = Model([11, window, new], 3, 2, 64, 64, fmt, 700)
    m.append([700, 130, 90])
    say("kv attention mask", fmt, causal, window, new)
    q = (m.rng.standard_normal((3 * new, 4, 64)) * 2).astype(np.float16)
    m.assert_attention(m.attend(q, [new] * 3, causal=causal, window=window), 700)


@pytest.mark.parametrize("ratio,new", [(2, 3), (2, 40)])
def test_attention_empty_rows(ratio, new):
    """Sequences of length zero, sequences without queries, more queries than
    tokens (the first see nothing), rows of no sequence."""
    m = Model([12, new], 4, 1, 64, 32, "e4m3", 100)
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
        want = kv_oracle.attention(q[:3 * new], m.kc, m.ks, m.vc, m.vs, table, cu, lens, 0.125, causal)
        m.assert_attention((host(out)[:3 * new], host(lse)[:3 * new], want), 100)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_missing_pages(new):
    """Pages the cache does not hold are not seen, whatever is in page 0."""
    m = Model([13], 2, 2, 128, 32, "e4m3", 300)
    m.append([300, 200])
    bad = m.table.copy()
    bad[0, 0], bad[0, 5], bad[1, 3], bad[1, :2] = -1, m.pages + 5, -7, -1
    q = m.rng.standard_normal((2 * new, 4, 128)).astype(np.float16)
    m.assert_attention(m.attend(q, [new, new], table=bad), 300)
    bad[1, :] = -1
    got = m.attend(q, [new, new], table=bad)
    m.assert_attention(got, 300)
    assert (got[0][new:] == 0).all()


@pytest.mark.parametrize("new", [2, 70])
def test_attention_scales_far_apart(new):
    """Pages whose value scales differ by 2^20, either way round, and the
    attention on the small ones."""
    for order in (1, -1):
        m = Model([14, new], 1, 1, 64, 32, "int8", 320)
        spreads = [2.0 ** -13, 2.0 ** 7, 1.0][::order]
        for i in range(9):
            m.append([32], v=(m.values(32).astype(np.float64) * spreads[i % 3]).astype(np.float16))
        q = m.rng.standard_normal((new, 2, 64)).astype(np.float16)
        m.assert_attention(m.attend(q, [new]), 320)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_large_logits(new):
    """Logits of thousands: one key takes the whole weight, and no overflow."""
    m = Model([15, new], 1, 1, 128, 64, "int8", 400)
    m.append([400], k=(m.values(400).astype(np.float64) * 100).astype(np.float16))
    q = (m.rng.standard_normal((new, 1, 128)) * 300).astype(np.float16)
    m.assert_attention(m.attend(q, [new]), 400)


def test_attention_strides_and_stream():
    """q and out as slices of packed tensors, on a stream of their own."""
    m = Model([16], 2, 2, 128, 64, "int8", 500)
    m.append([500, 77])
    for new in ([1, 1], [90, 40]):
        T = sum(new)
        big = torch.zeros(T, 8, 128, dtype=torch.float16, device="cuda")
        q = m.rng.standard_normal((T, 4, 128)).astype(np.float16)
        big[:, 2:6] = dev(q)
        out = torch.zeros(4, T, 128, dtype=torch.float16, device="cuda").transpose(0, 1)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            got = m.attend(big[:, 2:6], new, out=out)
        m.assert_attention(got, 500)


def test_attention_same_every_run_and_workspace_shared():
    """One workspace for calls of several shapes; equal bits on every run."""
    m = Model([17], 2, 2, 64, 64, "int8", 3000)
    m.append([3000, 1100])
    shapes = [([1, 1], 2), ([3, 2], 4), ([40, 80], 2), ([1, 1], 8)]
    handles = [(m.seqs(n)[0], r, dev(m.rng.standard_normal((sum(n), r, 64)).astype(np.float16))) for n, r in shapes]
    need = max(awq.kv_attention_workspace_bytes(m.cache, s, r) for s, r, _ in handles)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = [host(awq.awq_kv_attention(q, m.cache, s, workspace=ws)) for s, _, q in handles]
    for _ in range(3):
        for (s, _, q), want in zip(handles, first):
            np.testing.assert_array_equal(host(awq.awq_kv_attention(q, m.cache, s, workspace=ws)), want)


def test_bounds_may_be_loose():
    """max_tokens and max_len far above the batch's own, as a captured graph has them."""
    m = Model([18], 3, 1, 64, 64, "e4m3", 300)
    m.append([300, 5, 64])
    q = m.rng.standard_normal((3, 2, 64)).astype(np.float16)
    for mt, ml in ((1, 5000), (8, 300), (200, 100000)):
        m.assert_attention(m.attend(q, [1, 1, 1], max_tokens=mt, max_len=ml), 300)


def test_steps_in_a_graph():
    """Decode steps (write, attention) captured once and replayed with new
    tokens and lengths, eager work between the replays."""
    m = Model([19], 2, 2, 128, 32, "int8", 200)
    m.append([90, 31])
    k, v, q = (torch.zeros(2, h, 128, dtype=torch.float16, device="cuda") for h in (2, 2, 4))
    out = torch.zeros_like(q)
    lens = dev(m.len.copy())
    s = awq.KVSeqs(dev(m.table), dev(np.array([0, 1, 2], np.int32)), lens, 1, 200)
    ws = awq.kv_attention_workspace(m.cache, s, 4)

    def step():
        awq.awq_kv_write(m.cache, s, k, v)
        awq.awq_kv_attention(q, m.cache, s, out=out, workspace=ws)

    saved = [t.clone() for t in (m.cache.k_codes, m.cache.v_codes, m.cache.k_scales, m.cache.v_scales)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, o in zip((m.cache.k_codes, m.cache.v_codes, m.cache.k_scales, m.cache.v_scales), saved):
        t.copy_(o)
    for _ in range(5):
        nk, nv = m.values(2), m.values(2)
        nq = m.rng.standard_normal((2, 4, 128)).astype(np.float16)
        k.copy_(dev(nk)), v.copy_(dev(nv)), q.copy_(dev(nq))
        m.len += 1
        lens.copy_(dev(m.len))
        kv_oracle.write(m.kc, m.ks, nk, m.table, [0, 1, 2], m.len, "int8")
        kv_oracle.write(m.vc, m.vs, nv, m.table, [0, 1, 2], m.len, "int8")
        graph.replay()
        torch.cuda.synchronize()
        m.check()
        got = host(out).copy()
        want = kv_oracle.attention(nq, m.kc, m.ks, m.vc, m.vs, m.table, [0, 1, 2], m.len, 128 ** -0.5)
        u = 2.0 ** -24
        e = 2 * ((128 + 4) * u * want[3] + 2.0 ** -21 + 2 * 200 * u)
        tol = (e[..., None] + 2.0 ** -11) * want[2] + 2.0 ** -11 * np.abs(want[0]) + 2.0 ** -25
        assert (np.abs(got - want[0]) <= tol).all()
        out2 = awq.awq_kv_attention(q, m.cache, s)      # eager, without a workspace
        assert (np.abs(host(out2) - want[0]) <= tol).all()


@pytest.mark.parametrize("new", [2, 60])
def test_attention_scale_of_any_sign(new):
    m = Model([20, new], 2, 2, 64, 64, "int8", 200)
    m.append([200, 90])
    q = m.rng.standard_normal((2 * new, 4, 64)).astype(np.float16)
    for scale in (-0.2, 0.0, 1e-6, 3.0):
        m.assert_attention(m.attend(q, [new, new], scale=scale), 200)


@pytest.mark.parametrize("new", [1, 40])
def test_workspace_counts_the_loose_bound(new):
    """A workspace sized for a bound on the new tokens serves calls of fewer
    rows than the bound, on either side of the kernels' border."""
    m = Model([21, new], 1, 1, 64, 64, "int8", 2000)
    m.append([2000])
    q = m.rng.standard_normal((new, 2, 64)).astype(np.float16)
    for bound in (new, 16, 17, 500, 4000):
        if bound >= new:
            m.assert_attention(m.attend(q, [new], max_tokens=bound), 2000)


def test_far_pages():
    """Pages past 4 GiB of codes: writes, reads and attention address them."""
    heads, dim, page = 8, 128, 64
    per = heads * dim * page                    # bytes of a page's keys
    pages = (5 << 30) // per
    cache = awq.KVCache.empty(pages, heads, dim, page, "int8")
    rng = np.random.default_rng(22)
    ids = np.array([[pages - 1, 3, pages - 2], [0, pages // 2, pages - 7]], np.int32)
    lens = np.array([150, 170], np.int32)
    cu = np.array([0, 150, 320], np.int32)
    k, v = (rng.standard_normal((320, heads, dim)).astype(np.float16) for _ in range(2))
    s = awq.KVSeqs(dev(ids), dev(cu), dev(lens), 170, 170)
    awq.awq_kv_write(cache, s, dev(k), dev(v))
    gk, gv = awq.awq_kv_read(cache, s)
    # the oracle's cache holds the six pages alone
    small = np.arange(6, dtype=np.int32).reshape(2, 3)
    kc, vc = np.zeros((6, heads, page, dim)), np.zeros((6, heads, page, dim))
    ks, vs = np.zeros((6, heads), np.float32), np.zeros((6, heads), np.float32)
    kv_oracle.write(kc, ks, k, small, cu, lens, "int8")
    kv_oracle.write(vc, vs, v, small, cu, lens, "int8")
    for got, codes, scales in ((gk, kc, ks), (gv, vc, vs)):
        want = np.zeros(got.shape, np.float16)
        kv_oracle.read(codes, scales, want, small, cu, lens)
        np.testing.assert_array_equal(host(got), want)
    for n in (1, 50):
        cu2 = np.array([0, n, 2 * n], np.int32)
        q = rng.standard_normal((2 * n, 16, dim)).astype(np.float16)
        s2 = awq.KVSeqs(dev(ids), dev(cu2), dev(lens), n, 170)
        o = host(awq.awq_kv_attention(dev(q), cache, s2, workspace=awq.kv_attention_workspace(cache, s2, 16)))
        eo, _, spread, mass = kv_oracle.attention(q, kc, ks, vc, vs, small, cu2, lens, dim ** -0.5)
        tol = (2 * ((dim + 4) * 2.0 ** -24 * mass + 2.0 ** -20)[..., None] + 2.0 ** -11) * spread + \
            2.0 ** -11 * np.abs(eo) + 2.0 ** -24
        assert (np.abs(o - eo) <= tol).all()


def test_two_streams_at_once():
    """Two batches over one cache, on two streams with a workspace each."""
    m = Model([23], 2, 2, 128, 64, "e4m3", 3000)
    m.append([3000, 2500])
    sets = []
    for new in (1, 48):
        q = dev(m.rng.standard_normal((2 * new, 4, 128)).astype(np.float16))
        s = m.seqs([new, new])[0]
        ws = awq.kv_attention_workspace(m.cache, s, 4)
        sets.append((q, s, ws, host(awq.awq_kv_attention(q, m.cache, s, workspace=ws)), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, (q, s, ws, _, stream) in enumerate(sets):
            with torch.cuda.stream(stream):
                outs[i].append(awq.awq_kv_attention(q, m.cache, s, workspace=ws))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            np.testing.assert_array_equal(host(o), sets[i][3])


def test_wrong_tensors_are_refused():
    m = Model([24], 1, 2, 64, 32, "int8", 32)
    m.append([5])
    s, *_ = m.seqs([1])
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    kv = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    attend, write, read = awq.awq_kv_attention, awq.awq_kv_write, awq.awq_kv_read
    for bad, err in ((q.float(), TypeError), (q.cpu(), ValueError), (q[..., :32], ValueError), (q[0], ValueError),
                     (q.transpose(1, 2), ValueError), ([1], TypeError)):
        with pytest.raises(err):
            attend(bad, m.cache, s)
    with pytest.raises(awq.AwqError):
        attend(torch.zeros(1, 3, 64, dtype=torch.float16, device="cuda"), m.cache, s, out=torch.zeros(
            1, 3, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        attend(q, m.cache, s, out=q[:, :2])
    with pytest.raises(ValueError):
        attend(q, m.cache, s, lse=torch.zeros(1, 2, device="cuda"))
    with pytest.raises(TypeError):
        attend(q, m.cache, s, workspace=torch.zeros(99, device="cuda"))
    with pytest.raises(awq.AwqError):
        attend(q, m.cache, s, causal=False, window=3, out=torch.zeros_like(q))
    for bad in (kv.double(), kv[:, :1], kv.cpu()):
        with pytest.raises((TypeError, ValueError)):
            write(m.cache, s, bad, kv)
        with pytest.raises((TypeError, ValueError)):
            read(m.cache, s, out=(kv, bad))
    with pytest.raises(ValueError):
        write(m.cache, s, kv, torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        read(m.cache, s, n_tokens=3, out=(kv, kv.clone()))
    odd = torch.zeros(1 * 2 * 68 + 4, dtype=torch.float16, device="cuda").as_strided((1, 2, 64), (136, 68, 1))
    with pytest.raises(awq.AwqError):       # a head stride that is not a multiple of 8
        write(m.cache, s, odd, kv)
    m.check()                               # nothing was written


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("new", [2, 70])
def test_attention_query_not_finite(new, bad, split):
    """A query with a NaN gets NaN, in the output and in lse; neither it nor an
    infinity reaches another row, the ones of its block included."""
    m = Model([31, new], 2, 2, 128, 64, "int8", 1500)
    m.append([1500, 900])
    q = m.rng.standard_normal((2 * new, 4, 128)).astype(np.float16)
    clean = q.copy()
    q[1, 2, 77] = bad
    s, cu, lens, table = m.seqs([new, new])
    ws = awq.kv_attention_workspace(m.cache, s, 4) if split else None
    lse = torch.zeros(q.shape[:2], device="cuda")
    o = host(awq.awq_kv_attention(dev(q), m.cache, s, lse=lse, workspace=ws))
    lse = host(lse)
    if np.isnan(bad):
        assert np.isnan(o[1, 2]).all() and np.isnan(lse[1, 2])
    eo, el, spread, mass = kv_oracle.attention(clean, m.kc, m.ks, m.vc, m.vs, table, cu, lens, 128 ** -0.5)
    e = 2 * (132 * 2.0 ** -24 * mass + 2.0 ** -21 + 3000 * 2.0 ** -24)
    tol = (e[..., None] + 2.0 ** -11) * spread + 2.0 ** -11 * np.abs(eo) + 2.0 ** -25 + \
        1500 * 2.0 ** -34 * 127 * float(m.vs.max())
    others = np.ones(q.shape[:2], bool)
    others[1, 2] = False
    assert (np.abs(o - eo) <= tol)[others].all()
    assert (np.abs(lse - el) <= e + 2.0 ** -22 * np.abs(el))[others].all()
