"""awq_gemm_fused on the kernels that only large calls reach (the 256-row
tiles, whole, split and with a split last round) and on the skinny kernel's
splits, against float64.

The fp32 sum v of an output adds K / 16 products of 16, is rescaled K / G
times, scaled once and joined from up to 8 parts, each step off by u = 2^-24
of a partial sum below S = sum |x w|: |v - v64| <= (K / 16 + 2 K / G + 8) u S.
Behind it (see test_gpu_epilogue.py)
  |err| <= |mul| (1.13 |v - v64| + 2^-18 |act| + 2^-22)
           + 2^-22 (|act mul| + |residual|) + 2^-11 |y| + 2^-25.
"""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import say  # noqa: E402

COUNTERS = 4096         # bytes of the linear layer's workspace before the parked parts, on 256 CUs


@pytest.fixture(scope="module", autouse=True)
def cu256():
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are a 256-CU device's")


def act64(v, name):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


class Layer:
    def __init__(self, M, N, K, G, bits):
        self.M, self.N, self.K, self.G, self.bits = M, N, K, G, bits
        g = torch.Generator(device="cuda").manual_seed(M * 7 + N * 3 + K + bits)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x = randn(M, K).half()
        self.q = (awq.awq_quantize if bits == 4 else awq.awq_quantize_w8)((randn(N, K) * 0.02).half(), G)
        self.bias, self.mul, self.res = (randn(N) * 0.5).half(), randn(M, N).half(), (randn(M, N) * 2).half()
        words, s, z = self.q
        per = 32 // bits
        c = torch.stack([(words >> (bits * i)) & (2 ** bits - 1) for i in range(per)], -1).flatten(1).double()
        w = (c - z.double().repeat_interleave(G, 1)) * s.double().repeat_interleave(G, 1)
        self.v64 = self.x.double() @ w.t().contiguous()
        self.off = (K / 16 + 2 * K / G + 8) * 2.0 ** -24 * (self.x.double().abs() @ w.abs().t().contiguous())

    def run(self, act, b, m, r, path, ws, out=None):
        return awq.awq_gemm_fused(self.x, *self.q, self.G, bias=self.bias if b else None, activation=act,
                                  mul=self.mul if m else None, residual=self.res if r else None, path=path,
                                  workspace=ws, out=out)

    def check(self, y, act, b, m, r):
        assert y.isfinite().all()
        a = act64(self.v64 + (self.bias.double() if b else 0), act)
        mul = self.mul.double() if m else torch.ones((), dtype=torch.float64, device="cuda")
        res = self.res.double() if r else torch.zeros((), dtype=torch.float64, device="cuda")
        want = a * mul + res
        tol = mul.abs() * (1.13 * self.off + 2.0 ** -18 * a.abs() + 2.0 ** -22) + \
            2.0 ** -22 * ((a * mul).abs() + res.abs()) + 2.0 ** -11 * want.abs() + 2.0 ** -25
        err = (y.double() - want).abs()
        worst = float((err / tol).max())
        assert bool((err <= tol).all()), f"{act}: worst {worst:.3f} of the bound"


def hold(M, N, K, G, bits, path, with_ws, kernel, split):
    say("fused", M, N, K, G, bits, path, kernel, "split" if split else "whole")
    assert awq.gemm_fused_kernel(M, N, K, G, bits, path, with_ws) == kernel
    lay = Layer(M, N, K, G, bits)
    ws = awq.gemm_workspace(M, N, K) if with_ws else None
    for act, b, m, r in (("silu", 1, 1, 1), ("none", 0, 0, 1), ("gelu", 1, 0, 0), ("gelu_tanh", 0, 1, 0),
                         ("relu", 1, 1, 0)):
        if ws is not None:
            ws.zero_()
        y = lay.run(act, b, m, r, path, ws)
        lay.check(y, act, b, m, r)
        if ws is not None:      # the counters are back at zero; parts were parked where it splits
            assert not ws[:COUNTERS].any()
            assert bool(ws[COUNTERS:].any()) == split
        assert torch.equal(lay.run(act, b, m, r, path, ws), y)
    # the operands overwritten in place
    want = lay.run("silu", 1, 1, 1, path, ws)
    for name in ("res", "mul"):
        keep = getattr(lay, name)
        setattr(lay, name, keep.clone())
        got = lay.run("silu", 1, 1, 1, path, ws, out=getattr(lay, name))
        assert torch.equal(got, want), name
        setattr(lay, name, keep)


@pytest.mark.parametrize("bits,G", [(4, 128), (4, 64), (8, 64), (8, 256)])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("M,N,K,with_ws,split", [
    (1024, 8192, 4096, True, True),         # 256 x 256 tiles, 128 of them: stream-K
    (2048, 4864, 256, False, False),        # 152 of them, whole
    (1536, 11008, 2048, True, True),        # 516 tiles of 256 x 128: a round and a split tail
    (1100, 4104, 256, False, False),        # 165 of them, whole
])
def test_large_tiles(M, N, K, with_ws, split, odd, bits, G):
    if odd:             # rows that make no 16-byte pieces, ragged tiles
        M, N = M - 3, N - 5
    hold(M, N, K, G, bits, awq.PATH_AUTO, with_ws, "gemm", split)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("N", [104, 101])
def test_tall_narrow_layer(N, bits):
    """171 tiles of 256 x 128 in one column: the narrow tile's stream-K."""
    hold(43700, N, 5888, 128, bits, awq.PATH_AUTO, True, "gemm", True)


@pytest.mark.parametrize("with_ws,split", [(True, True), (False, False)])
@pytest.mark.parametrize("M,N,K", [(129, 264, 1024), (300, 520, 2048), (129, 261, 1024)])
def test_groups_of_32(M, N, K, with_ws, split):
    """The older form, with 16-byte accesses and without."""
    hold(M, N, K, 32, 4, awq.PATH_AUTO, with_ws, "gemm", split)


@pytest.mark.parametrize("with_ws", [True, False])
@pytest.mark.parametrize("M,N,K,G,path", [
    (12, 520, 4096, 128, 3), (20, 520, 4096, 128, 3), (32, 1000, 4096, 64, 3), (33, 520, 4096, 256, 3),
    (64, 1003, 4096, 128, 3), (41, 520, 4096, 32, 3),
    (40, 700, 4096, 32, 0), (64, 520, 2048, 32, 0),
])
def test_skinny(M, N, K, G, path, with_ws):
    """One, two and four row blocks; with a workspace K is split over blocks."""
    if path == 0 and awq.gemm_fused_kernel(M, N, K, G, 4, path, with_ws) != "skinny":
        pytest.skip("another kernel without a workspace")
    hold(M, N, K, G, 4, path, with_ws, "skinny", with_ws)


def test_skinny_large_layer():
    """What a decode batch of a large layer takes by itself."""
    hold(20, 8192, 28672, 128, 4, awq.PATH_AUTO, True, "skinny", True)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,N", [(65, 1000), (203, 1003), (500, 1000)])
def test_small_tiles_split(M, N, bits):
    hold(M, N, 4096, 64, bits, awq.PATH_AUTO, True, "gemm_small", True)
