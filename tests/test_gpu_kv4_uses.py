"""The 4-bit cache and its attention in uses of their own: the most sequences a
call takes, two graphs that take turns on one workspace, calls on two streams at
once, queries and outputs that broadcast or interleave.

Attention's bounds are test_gpu_kv4's.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_kv4 import Model  # noqa: E402
from test_gpu_parity import dev, host, say  # noqa: E402

U = 2.0 ** -24


@pytest.mark.parametrize("new", [1, 17])
def test_the_most_sequences(new):
    """32767 sequences of 17 tokens, their last `new` as queries: one row tile of
    16 and two; and the positions of the batch against the same ones given."""
    B, N, D = 32767, 17, 64
    say("kv4 sequences", B, new)
    g = torch.Generator(device="cuda").manual_seed(new)
    half = lambda *s: torch.randn(s, device="cuda", dtype=torch.float16, generator=g)  # noqa: E731
    cache = awq.KVCache.empty(B, 1, D, 32, "int4", "cuda")
    table = torch.randperm(B, device="cuda", generator=g).to(torch.int32).reshape(B, 1)
    lens = torch.full((B,), N, device="cuda", dtype=torch.int32)
    cu = lambda n: (torch.arange(B + 1, device="cuda") * n).to(torch.int32)  # noqa: E731
    whole = awq.KVSeqs(table, cu(N), lens, N, N)
    k, v = half(B * N, 1, D), half(B * N, 1, D)
    awq.awq_kv_write(cache, whole, k, v)
    kn, vn = (t.double().reshape(B, N, D) for t in awq.awq_kv_read(cache, whole))
    # fp16 s and lo: a number is within half a step and what s was cut by of its own
    for got, t in ((kn, k), (vn, v)):
        groups = t.double().reshape(B, N, -1, 32 if got is kn else D)
        s = (groups.amax(-1) - groups.amin(-1)) / 15
        err = (got.reshape(groups.shape) - groups).abs().amax(-1)
        top = groups.abs().amax(-1)
        assert (err <= 0.5 * s + 15 * 2.0 ** -10 * s + 15 * 2.0 ** -24 + 2.0 ** -11 * top).all()
    newest = awq.KVSeqs(table, cu(new), lens, new, N)
    q = half(B * new, 1, D)
    out = awq.awq_kv_attention(q, cache, newest)
    q64 = q.double().reshape(B, new, D)
    t = torch.matmul(q64, kn.transpose(1, 2).contiguous()) * D ** -0.5
    at = torch.arange(N, device="cuda")
    t = t.masked_fill(at[None, :] > at[N - new:, None], float("-inf"))
    w = torch.softmax(t, -1)
    want = torch.matmul(w, vn)
    spread = torch.matmul(w, vn.abs())
    mass = float((torch.matmul(q64.abs(), kn.abs().transpose(1, 2).contiguous()) * D ** -0.5).max())
    e = 2 * ((D + 8) * U * mass + 16 * U + 2.0 ** -21 + 2 * N * U)
    tol = (e + 2.0 ** -20) * spread + N * 2.0 ** -36 * float(vn.abs().max()) + 2.0 ** -11 * want.abs() + 2.0 ** -25
    assert ((out.double().reshape(B, new, D) - want).abs() <= tol).all()

    rope = awq.Rope(D)
    by_batch, _ = awq.awq_rope(q, None, rope, seqs=newest)
    positions = at[N - new:].to(torch.int32).repeat(B)
    given, _ = awq.awq_rope(q, None, rope, positions=positions)
    assert torch.equal(by_batch, given)


@pytest.mark.parametrize("dim,page,heads,ratio,new,causal,window", [
    (64, 32, 4, 8, 4, True, 0),
    (64, 64, 4, 1, 17, True, 30),
    (96, 64, 4, 3, 9, True, 0),
    (96, 32, 4, 1, 32, False, 0),
    (128, 64, 4, 8, 3, True, 0),
    (128, 32, 4, 5, 6, True, 33),
    (128, 256, 4, 2, 16, False, 0),
])
@pytest.mark.parametrize("split", [True, False])
def test_thirty_two_rows(dim, page, heads, ratio, new, causal, window, split):
    """17 to 32 rows a kv head in a batch of bounds long enough for blocks of 32
    rows: ragged lengths, missing pages, empty and short sequences, NaN queries,
    rows before a sequence's start."""
    say("kv4 rows", dim, page, ratio, new, window)
    lens = [700, 0, 1, new, 2300, 64, 333, new - 1]
    m = Model([45, dim, page, new], 8, heads, dim, page, max(lens))
    m.append(lens)
    news = [new, new, 1, new, new, 0, new, new]
    q = m.rng.standard_normal((sum(news), heads * ratio, dim)).astype(np.float16)
    table = m.table.copy()
    table[4, 3] = -1
    bound = 2 ** 16                 # 32 kv heads and more of 2^16 positions
    got = m.attend(q, news, table=table, causal=causal, window=window, split=split, max_len=bound)
    m.assert_attention(got, max(lens))
    # as two blocks of 16 rows
    two = m.attend(q, news, table=table, causal=causal, window=window, split=split)
    m.assert_attention(two, max(lens))
    q[news[0], 0] = np.nan          # a query of sequence 1, which is empty, and one of sequence 3
    q[2 * new + 2, 1 % (heads * ratio)] = np.nan
    o, lse, _ = m.attend(q, news, table=table, causal=causal, window=window, split=split, max_len=bound)
    hit = np.isnan(q).any(-1) & np.isfinite(got[1])
    assert np.isnan(o[hit]).all() and np.isnan(lse[hit]).all()
    np.testing.assert_array_equal(o[~hit], got[0][~hit])


def test_two_graphs_take_turns_on_a_workspace():
    m = Model(41, 3, 2, 128, 64, 1400)
    m.append([1300, 1, 700])
    cases = []
    for new, heads in (([1, 1, 1], 8), ([5, 0, 40], 4)):
        s, *_ = m.seqs(new)
        q = m.rng.standard_normal((sum(new), heads, 128)).astype(np.float16)
        cases.append((s, dev(q)))
    ws = max((awq.kv_attention_workspace(m.cache, s, q.shape[1]) for s, q in cases), key=lambda t: t.numel())
    want = [awq.awq_kv_attention(q, m.cache, s, workspace=ws).clone() for s, q in cases]
    graphs, outs = [], []
    for s, q in cases:
        out = torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            awq.awq_kv_attention(q, m.cache, s, out=out, workspace=ws)
        graphs.append(graph)
        outs.append(out)
    for turn in range(3):
        say("kv4 graphs in turn", turn)
        for graph, out, (s, q), w in zip(graphs, outs, cases, want):
            out.fill_(7.0)
            graph.replay()
            eager = awq.awq_kv_attention(q, m.cache, s, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(out, w) and torch.equal(eager, w)


def test_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    m = Model(42, 2, 2, 128, 64, 2100)
    m.append([2000, 900])
    s, *_ = m.seqs([1, 1])
    qs = [dev(m.rng.standard_normal((2, 8, 128)).astype(np.float16)) for _ in range(2)]
    ws = [awq.kv_attention_workspace(m.cache, s, 8) for _ in range(2)]
    want = [awq.awq_kv_attention(q, m.cache, s, workspace=w).clone() for q, w in zip(qs, ws)]
    outs = [[torch.zeros_like(q) for _ in range(20)] for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                awq.awq_kv_attention(qs[j], m.cache, s, out=outs[j][i], workspace=ws[j])
    torch.cuda.synchronize()
    for j in range(2):
        for out in outs[j]:
            assert torch.equal(out, want[j])


@pytest.mark.parametrize("new", [2, 40])
def test_broadcast_queries_and_interleaved_outputs(new):
    """One query for every head and token (strides 0), heads outermost in the output."""
    m = Model(43, 1, 2, 64, 32, 200)
    m.append([150])
    q = dev(m.rng.standard_normal(64).astype(np.float16)).expand(new, 6, 64)
    out = torch.full((6, new, 64), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    got = m.attend(q, [new], out=out)
    m.assert_attention(got, 150)
    same, *_ = m.attend(q.contiguous(), [new])
    np.testing.assert_array_equal(got[0], same)


def test_write_from_one_projection():
    """Keys and values as slices of one fused projection's rows, queries too."""
    m = Model(44, 2, 2, 96, 32, 90)
    rows = torch.zeros((70 + 33, 6 + 2 + 2, 96), dtype=torch.float16, device="cuda")

    def call(k, v):
        rows[:, 6:8] = dev(k)
        rows[:, 8:] = dev(v)
        return rows[:, 6:8], rows[:, 8:]

    m.append([70, 33], call=call)
    m.check()
    rows[:, :6] = dev(m.rng.standard_normal((103, 6, 96)).astype(np.float16))
    got = m.attend(rows[:, :6], [70, 33])
    m.assert_attention(got, 70)
