"""Uses of the paged cache's calls that its documentation allows and that are
off the usual path: pages shared by sequences, more query heads than a
decode tile's rows on one kv head, broadcast inputs, a bound below the
batch's tokens, and prompt chunks, reads and split linear layers in graphs."""

import numpy as np
import pytest

from oracle import kv_oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_kv import Model  # noqa: E402
from test_gpu_parity import dev, host, say  # noqa: E402


def near(m, o, want, n_keys, what=""):
    """The bound of test_gpu_attention_weights.py for weights in two parts."""
    eo, _, spread, mass = want
    e = 2 * ((m.dim + 4) * 2.0 ** -24 * mass + 2.0 ** -21 + 2 * n_keys * 2.0 ** -24)
    tol = (e + 2.0 ** -18)[..., None] * spread + 2.0 ** -11 * np.abs(eo) + 2.0 ** -25 + \
        n_keys * 2.0 ** -34 * float(kv_oracle.TOP[m.fmt]) * float(m.vs.max(initial=0))
    err = np.abs(o.astype(np.float64) - eo)
    assert np.isfinite(o).all() and (err <= tol).all(), f"{what} worst {np.max(err / tol):.3f} of the bound"


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
def test_shared_prefix(fmt, new):
    """Three sequences over the same first pages, each with a tail of its own;
    one of them names a page twice."""
    say("kv uses, shared prefix", fmt, new)
    m = Model([91, new], 3, 2, 64, 32, fmt, 32 * 6)
    m.table[1, :3] = m.table[2, :3] = m.table[0, :3]
    first = m.table.copy()
    m.len[:] = 0
    k, v = m.values(96), m.values(96)
    only = awq.KVSeqs(dev(first[:1]), dev(np.array([0, 96], np.int32)), dev(np.array([96], np.int32)), 96, 96)
    awq.awq_kv_write(m.cache, only, dev(k), dev(v))
    kv_oracle.write(m.kc, m.ks, k, first[:1], [0, 96], [96], fmt)
    kv_oracle.write(m.vc, m.vs, v, first[:1], [0, 96], [96], fmt)
    m.len[:] = 96
    m.append([50, 96, 64])
    twice = m.table.copy()
    twice[2, 4] = twice[2, 3]
    q = (m.rng.standard_normal((3 * new, 4, 64)) * 2).astype(np.float16)
    for table in (m.table, twice):
        o, _, want = m.attend(q, [new] * 3, table=table)
        near(m, o, want, 192)


@pytest.mark.parametrize("ratio,new", [(33, 1), (64, 1), (40, 3), (128, 1), (7, 5)])
@pytest.mark.parametrize("split", [True, False])
def test_many_query_heads(ratio, new, split):
    say("kv uses, query heads", ratio, new)
    m = Model([92, ratio], 2, 1, 64, 64, "int8", 2100)
    m.append([2100, 70])
    q = m.rng.standard_normal((2 * new, ratio, 64)).astype(np.float16)
    o, _, want = m.attend(q, [new, new], split=split)
    near(m, o, want, 2100)


def test_broadcast_inputs():
    """One token's keys and values for every head, one query for every row:
    strides of 0."""
    m = Model([94], 2, 4, 64, 32, "int8", 64)
    k1 = m.values(40)[:, :1]
    m.append([30, 10], k=np.broadcast_to(k1, (40, 4, 64)), v=np.broadcast_to(k1[:1], (40, 4, 64)),
             call=lambda k, v: (dev(k1).expand(40, 4, 64), dev(k1[:1]).expand(40, 4, 64)))
    m.check()
    q1 = m.rng.standard_normal((1, 1, 64)).astype(np.float16)
    for new in (1, 20):
        T = 2 * new
        o, _, want = m.attend(dev(q1).expand(T, 8, 64), [new, new])
        near(m, o, want, 30)


@pytest.mark.parametrize("new,bound", [(60, 32), (100, 64), (10, 1)])
def test_bound_below_the_tokens(new, bound):
    """Tokens past max_tokens, rounded up to whole pages or row tiles, are not
    processed; the ones before are, and nothing else changes."""
    m = Model([95, new], 1, 1, 64, 32, "int8", 128)
    s = awq.KVSeqs(dev(m.table), dev(np.array([0, new], np.int32)), dev(np.array([new], np.int32)), bound, new)
    k, v = m.values(new), m.values(new)
    awq.awq_kv_write(m.cache, s, dev(k), dev(v))
    done = min(new, -(-bound // 32) * 32)
    m.len[:] = done
    cu = [0, done]
    kv_oracle.write(m.kc, m.ks, k[:done], m.table, cu, m.len, "int8")
    kv_oracle.write(m.vc, m.vs, v[:done], m.table, cu, m.len, "int8")
    written = host(m.cache.k_scales).copy()
    more = ~np.isnan(written[m.table[0], 0])
    assert more[: -(-done // 32)].all()
    for p in range(-(-done // 32)):
        n = min(32, done - 32 * p)
        got = kv_oracle.load_k(host(m.cache.k_codes))[m.table[0, p], 0, :n]
        np.testing.assert_array_equal(got, kv_oracle.to_bytes(m.kc[m.table[0, p], 0, :n], "int8"))
    q = m.rng.standard_normal((new, 2, 64)).astype(np.float16)
    m.len[:] = done
    full, cu, lens, table = m.seqs([min(new, done)])
    low = awq.KVSeqs(full.block_table, full.cu_tokens, full.kv_len, min(bound, done), done)
    out = torch.full((done, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    awq.awq_kv_attention(dev(q[:done]), m.cache, low, out=out, workspace=awq.kv_attention_workspace(m.cache, low, 2))
    want = kv_oracle.attention(q[:done], m.kc, m.ks, m.vc, m.vs, m.table, cu, lens, 0.125)
    at = min(bound, done)
    near(m, host(out)[:at], tuple(w[:at] for w in want), done)


def replay(graph, eager, change, times=4):
    """Replays a graph with new inputs, eager work in between; `eager` computes
    what the graph's outputs have to be, bit for bit."""
    for i in range(times):
        change(i)
        graph.replay()
        torch.cuda.synchronize()
        junk = torch.randn(1 << 20, device="cuda").sum()       # other work on the device
        got, want = eager()
        for a, b in zip(got, want):
            np.testing.assert_array_equal(host(a), host(b))
        del junk


def captured(step):
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prompt_chunk_and_read_in_a_graph(fmt):
    """Two graphs of their own workspaces over one cache, replayed in turn."""
    m = Model([96], 2, 2, 64, 64, fmt, 1500)
    m.append([1500, 900])
    sets = []
    for new, ratio in ((70, 2), (1, 8)):
        lens = dev(m.len.copy())
        s = awq.KVSeqs(dev(m.table), dev(np.array([0, new, 2 * new], np.int32)), lens, new, 1500)
        q = dev(m.rng.standard_normal((2 * new, 2 * ratio, 64)).astype(np.float16))
        ws = awq.kv_attention_workspace(m.cache, s, 2 * ratio)
        out, k, v = torch.zeros_like(q), *(torch.zeros(2 * new, 2, 64, device="cuda").half() for _ in range(2))

        def step(q=q, s=s, ws=ws, out=out, k=k, v=v):
            awq.awq_kv_attention(q, m.cache, s, out=out, workspace=ws)
            awq.awq_kv_read(m.cache, s, out=(k, v))

        sets.append((captured(step), q, s, ws, out, k, v, lens))
    for i in range(3):
        for graph, q, s, ws, out, k, v, lens in sets:
            lens.copy_(dev(np.array([1500 - 100 * i, 900 - 71 * i], np.int32)))
            q.copy_(torch.randn_like(q))
            graph.replay()
            torch.cuda.synchronize()
            junk = torch.randn(1 << 20, device="cuda").sum()
            want = awq.awq_kv_attention(q, m.cache, s, workspace=torch.zeros_like(ws))
            wk, wv = awq.awq_kv_read(m.cache, s)
            for a, b in ((out, want), (k, wk), (v, wv)):
                np.testing.assert_array_equal(host(a), host(b))
            del junk


@pytest.mark.parametrize("M,N,K,G,bits,path", [(203, 1000, 4096, 64, 8, 0), (20, 520, 4096, 128, 4, 3),
                                               (129, 264, 1024, 32, 4, 0), (16, 4096, 1024, 128, 4, 0)])
def test_split_linear_layer_in_a_graph(M, N, K, G, bits, path):
    g = torch.Generator(device="cuda").manual_seed(97)
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).half()
    q = (awq.awq_quantize if bits == 4 else awq.awq_quantize_w8)(w, G)
    x, res = (torch.randn(M, n, generator=g, device="cuda").half() for n in (K, N))
    out, ws, ws2 = torch.zeros_like(res), awq.gemm_workspace(M, N, K), awq.gemm_workspace(M, N, K)
    call = lambda ws, out=None: awq.awq_gemm_fused(x, *q, G, activation="gelu", residual=res, path=path, workspace=ws,  # noqa: E731
                                                   out=out)
    graph = captured(lambda: call(ws, out))
    replay(graph, lambda: ([out], [call(ws2)]), lambda i: x.copy_(torch.randn_like(x)))
