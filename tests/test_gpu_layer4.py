"""A decoder layer's operators in a row over the 4-bit cache, as a serving
program calls them: norm with the residual's sum, q / k / v, rotary positions,
the cache's write, attention, the output projection with the residual, the
second norm, the gated feed-forward part. Every stage is compared with the CPU
oracle on that stage's own inputs (the norm, the rotation and the attention
within the bounds of their own tests, the linear layers within 1e-2 (|y| + 1)
and 1e-3 in the 2-norm, as in theirs), and the row, captured into a graph and
replayed with other tokens, gives what the eager calls give."""

import numpy as np
import pytest

import oracle
from oracle import layer_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_kv4 import Model  # noqa: E402
from test_gpu_norm import check_f16  # noqa: E402
from test_gpu_parity import dev, host, say  # noqa: E402
from test_gpu_rope import check as check_rope  # noqa: E402

K, HQ, HK, D, FF, G = 512, 8, 2, 64, 1408, 64


class Layer:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.w = {n: (rng.standard_normal((rows, cols)) * cols ** -0.5).astype(np.float16)
                  for n, rows, cols in (("q", HQ * D, K), ("k", HK * D, K), ("v", HK * D, K), ("o", K, HQ * D),
                                        ("gate", FF, K), ("up", FF, K), ("down", K, FF))}
        self.g = {n: (1 + 0.2 * rng.standard_normal(K)).astype(np.float16) for n in ("in", "post")}
        self.q = {n: awq.awq_quantize(dev(w), G) for n, w in self.w.items()}
        self.gd = {n: dev(g) for n, g in self.g.items()}
        self.rope = awq.Rope(D, scaling="yarn", factor=4.0, trained_len=64.0)

    def linear(self, name, x, **kw):
        return awq.awq_gemm_fused(x, *self.q[name], G, **kw)

    def run(self, x, h, cache, seqs, ws):
        """One pass: x the last layer's output, h the residual stream; every
        stage's tensors by name."""
        s = {"x": x.clone(), "h0": h.clone()}
        s["n1"] = awq.awq_rmsnorm(x, self.gd["in"], 1e-5, residual=h, residual_out=h)
        s["h1"] = h.clone()
        T = x.shape[0]
        s["q"], s["k"], s["v"] = (self.linear(n, s["n1"]).view(T, -1, D) for n in "qkv")
        s["q0"], s["k0"] = s["q"].clone(), s["k"].clone()
        awq.awq_rope(s["q"], s["k"], self.rope, seqs=seqs, out=(s["q"], s["k"]))
        awq.awq_kv_write(cache, seqs, s["k"], s["v"])
        s["a"] = awq.awq_kv_attention(s["q"], cache, seqs, workspace=ws)
        s["o"] = self.linear("o", s["a"].view(T, HQ * D))
        s["n2"] = awq.awq_rmsnorm(s["o"], self.gd["post"], 1e-5, residual=h, residual_out=h)
        s["h2"] = h.clone()
        s["up"] = self.linear("up", s["n2"])
        s["gate"] = self.linear("gate", s["n2"], activation="silu", mul=s["up"])
        s["y"] = self.linear("down", s["gate"])
        return s

    def exact(self, name, x):
        qw, sc, zr = (host(t) for t in self.q[name])
        return np.asarray(x, np.float64) @ oracle.dequantize(qw.view(np.uint32), sc, zr, G, self.w[name].shape[1]).T


def close(y, want, what):
    y = y.astype(np.float64)
    assert np.linalg.norm(y - want) <= 1e-3 * np.linalg.norm(want), what
    assert (np.abs(y - want) <= 1e-2 * (np.abs(want) + 1)).all(), what


def step(layer, m, new, graph=None):
    """New tokens behind every sequence of the model m, and the stages' checks."""
    T = int(np.sum(new))
    x, h = (m.rng.standard_normal((T, K)).astype(np.float16) for _ in range(2))
    m.len = (m.len + new).astype(np.int32)
    s, cu, lens, table = m.seqs(new)
    ws = awq.kv_attention_workspace(m.cache, s, HQ)
    out = layer.run(dev(x), dev(h), m.cache, s, ws)
    torch.cuda.synchronize()
    got = {n: host(t) for n, t in out.items()}
    check(layer, m, got, cu, lens, table)
    return x, h


def check(layer, m, got, cu, lens, table):
    T = got["x"].shape[0]
    _, y = lo.rmsnorm(got["x"], layer.g["in"], 1e-5, got["h0"])
    check_f16(got["n1"], y, K)
    np.testing.assert_array_equal(got["h1"], (got["x"].astype(np.float32) + got["h0"].astype(np.float32)).astype(np.float16))
    for n in "qkv":
        raw = got[n + "0"] if n != "v" else got["v"]
        close(raw.reshape(T, -1), layer.exact(n, got["n1"]), n)
    f, amp = lo.rope_frequencies(D, scaling="yarn", factor=4.0, length=64.0)
    pos = np.concatenate([np.arange(L - (b - a), L) for a, b, L in zip(cu[:-1], cu[1:], lens)])
    check_rope(got["q"], got["q0"], pos, f, "half", amp)
    check_rope(got["k"], got["k0"], pos, f, "half", amp)
    lo.write(m.kc, m.ks, got["k"], table, cu, lens, "k")
    lo.write(m.vc, m.vs, got["v"], table, cu, lens, "v")
    m.check()
    want = m.want(got["q"], table, cu, lens, D ** -0.5)
    m.assert_attention((got["a"], want[1].astype(np.float32), want), int(lens.max()))
    close(got["o"], layer.exact("o", got["a"].reshape(T, -1)), "o")
    _, y = lo.rmsnorm(got["o"], layer.g["post"], 1e-5, got["h1"])
    check_f16(got["n2"], y, K)
    gate = layer.exact("gate", got["n2"])
    close(got["gate"], gate / (1 + np.exp(-gate)) * got["up"].astype(np.float64), "gate")
    close(got["y"], layer.exact("down", got["gate"]), "down")


def test_layer():
    """A ragged prompt, then single tokens, then a few at once."""
    layer = Layer(1)
    m = Model([21], 3, HK, D, 32, 200)
    for new in ([70, 5, 33], [1, 1, 1], [1, 1, 1], [2, 9, 40]):
        say("layer", new)
        step(layer, m, np.array(new))


def test_layer_in_a_graph():
    layer = Layer(2)
    m = Model([22], 2, HK, D, 64, 300)
    step(layer, m, np.array([100, 30]))
    table, lens = dev(m.table), dev(m.len.copy())
    cu = np.array([0, 1, 2], np.int32)
    seqs = awq.KVSeqs(table, dev(cu), lens, 1, 300)
    ws = awq.kv_attention_workspace(m.cache, seqs, HQ)
    x, h = (torch.zeros(2, K, dtype=torch.float16, device="cuda") for _ in range(2))
    lens.zero_()                    # the warm-up and the capture write nothing
    layer.run(x, h, m.cache, seqs, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.run(x, h, m.cache, seqs, ws)
    for _ in range(3):
        m.len = (m.len + 1).astype(np.int32)
        x.copy_(dev(m.rng.standard_normal((2, K)).astype(np.float16)))
        h.copy_(dev(m.rng.standard_normal((2, K)).astype(np.float16)))
        lens.copy_(dev(m.len))
        h_in = h.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: host(t).copy() for n, t in out.items()}
        check(layer, m, got, cu, m.len, m.table)
        again = layer.run(x, h_in, m.cache, seqs, ws)      # the same tokens once more, eagerly
        torch.cuda.synchronize()
        for n, t in again.items():
            np.testing.assert_array_equal(host(t), got[n], err_msg=n)


def test_eight_bit_norm_feeds_a_product():
    """The norm's codes and scales stand for the fp16 norm within their steps,
    in a product that takes them apart: y = s (c . W^T)."""
    layer = Layer(3)
    rng = np.random.default_rng(23)
    x, h = (rng.standard_normal((9, K)).astype(np.float16) for _ in range(2))
    _, y = lo.rmsnorm(x, layer.g["in"], 1e-5, h)
    w = layer.w["gate"].astype(np.float64)
    for fmt, step_of in (("int8", lambda y, s: s / 2), ("e4m3", lambda y, s: np.maximum(2.0 ** -4 * np.abs(y), s * 2.0 ** -10))):
        codes, scales = awq.awq_rmsnorm(dev(x), layer.gd["in"], 1e-5, residual=dev(h), fmt=fmt)
        z = host(codes.float()).astype(np.float64) @ w.T * host(scales).astype(np.float64)
        # each element off by its step and the norm's own 1e-5, so a product by their sum times |w|
        tol = (step_of(y, host(scales).astype(np.float64)) + 1e-5 * np.abs(y)) @ np.abs(w).T
        assert (np.abs(z - y @ w.T) <= tol).all()
