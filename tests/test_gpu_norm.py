"""The root-mean-square norm (awq_rmsnorm) against the CPU oracle.

Per element, with u = 2^-24 and K the width: h is one fp32 sum (u), the squares
are summed by 64 threads or more with at most K / 64 + 32 steps each before and
in the exchange, the quotient, the square root and the reciprocal round four
times more: e = ((K / 64 + 36) / 2 + 4 + 4) u on y with its two products. fp16
adds half a step, 2^-11 |y| or 2^-25. A stored code stands for code * s, s off
by e + 3 u: int8 within s / 2 of y, e4m3 within 2^-4 |y| or s 2^-10, plus
(e + 8 u) |y| for y and 1 / s.
"""

import numpy as np
import pytest

from oracle import layer_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host, say  # noqa: E402

U = 2.0 ** -24


def bound(K):
    return ((K / 64 + 36) / 2 + 8) * U


def inputs(seed, T, K, residual=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K)) * np.exp(rng.standard_normal((T, 1)))
    x[:, : max(1, K // 50)] *= 10
    r = rng.standard_normal((T, K)) * 2 if residual else None
    w = 1 + 0.3 * rng.standard_normal(K)
    return x.astype(np.float16), None if r is None else r.astype(np.float16), w.astype(np.float16)


def check_f16(y, want, K):
    tol = (bound(K) + 2.0 ** -11) * np.abs(want) + 2.0 ** -25
    err = np.abs(y.astype(np.float64) - want)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"


def check_8bit(codes, scales, want, fmt, group):
    T, K = want.shape
    s = lo.norm_scales(want, fmt, group)
    got = scales.astype(np.float64)
    assert got.shape == s.shape
    e = bound(K)
    assert (np.abs(got - s) <= (e + 3 * U) * s).all()
    step = np.repeat(got, K // got.shape[1], 1)
    err = np.abs(codes.astype(np.float64) * step - want)
    if fmt == "int8":
        tol = step * 0.5 + (e + 8 * U) * np.abs(want)
    else:
        tol = np.maximum(2.0 ** -4 * np.abs(want), step * 2.0 ** -10) + (e + 8 * U) * np.abs(want)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"


def values(codes):
    return host(codes.float() if codes.dtype == torch.float8_e4m3fn else codes)


WIDTHS = [1, 7, 8, 63, 64, 513, 1000, 1024, 2047, 2048, 2056, 4096, 5001, 8192, 8200, 11008, 16384, 20000, 32768, 40003]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("T", [1, 5])
def test_widths(K, T):
    say("rmsnorm", T, K)
    x, r, w = inputs([1, K], T, K)
    h, y = lo.rmsnorm(x, w, 1e-5, r)
    out = torch.full((T, K), 7.0, dtype=torch.float16, device="cuda")
    got = awq.awq_rmsnorm(dev(x), dev(w), 1e-5, residual=dev(r), residual_out=out)
    np.testing.assert_array_equal(host(out), (x.astype(np.float32) + r.astype(np.float32)).astype(np.float16))
    check_f16(host(got), y, K)
    for fmt in ("int8", "e4m3"):
        codes, scales = awq.awq_rmsnorm(dev(x), dev(w), 1e-5, residual=dev(r), fmt=fmt)
        check_8bit(values(codes), host(scales), y, fmt, 0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 512])
@pytest.mark.parametrize("K", [512, 1536, 8192, 33280])
def test_groups(fmt, group, K):
    x, r, w = inputs([2, K, group], 3, K)
    _, y = lo.rmsnorm(x, w, 1e-6, r)
    codes, scales = awq.awq_rmsnorm(dev(x), dev(w), 1e-6, residual=dev(r), fmt=fmt, group_size=group)
    check_8bit(values(codes), host(scales), y, fmt, group)


@pytest.mark.parametrize("weight,offset,residual", [(True, 0.0, False), (True, 1.0, True), (False, 0.0, True),
                                                    (False, 1.0, False), (True, -0.5, False)])
def test_weights_and_offsets(weight, offset, residual):
    x, r, w = inputs([3], 4, 1000, residual)
    w = (w - offset).astype(np.float16) if weight else None
    _, y = lo.rmsnorm(x, w, 1e-3, r, offset)
    got = awq.awq_rmsnorm(dev(x), None if w is None else dev(w), 1e-3, residual=None if r is None else dev(r),
                          weight_offset=offset)
    check_f16(host(got), y, 1000)


@pytest.mark.parametrize("K", [999, 4096, 40000])
def test_in_place_and_strides(K):
    """The sum over the residual, over x; y over x; rows of a wider tensor, at
    addresses that are not multiples of 16; a broadcast residual."""
    x, r, w = inputs([4, K], 6, K)
    h, y = lo.rmsnorm(x, w, 1e-5, r)
    h16 = (x.astype(np.float32) + r.astype(np.float32)).astype(np.float16)
    xd, rd = dev(x), dev(r)
    got = awq.awq_rmsnorm(xd, dev(w), residual=rd, residual_out=rd)
    np.testing.assert_array_equal(host(rd), h16)
    np.testing.assert_array_equal(host(xd), x)
    check_f16(host(got), y, K)
    rd = dev(r)
    got = awq.awq_rmsnorm(xd, dev(w), residual=rd, residual_out=rd, out=xd)
    assert got is xd
    np.testing.assert_array_equal(host(rd), h16)
    check_f16(host(xd), y, K)
    xd, rd = dev(x), dev(r)
    awq.awq_rmsnorm(xd, dev(w), residual=rd, residual_out=xd, out=rd)
    np.testing.assert_array_equal(host(xd), h16)
    check_f16(host(rd), y, K)
    wide = [torch.full((6, K + 11), 5.0, dtype=torch.float16, device="cuda") for _ in range(4)]
    views = [t[:, 3: 3 + K] for t in wide]
    views[0].copy_(dev(x)), views[1].copy_(dev(r))
    wv = torch.zeros(K + 1, dtype=torch.float16, device="cuda")[1:]
    wv.copy_(dev(w))
    awq.awq_rmsnorm(views[0], wv, residual=views[1], residual_out=views[2], out=views[3])
    np.testing.assert_array_equal(host(views[2]), h16)
    check_f16(host(views[3]), y, K)
    for t in wide:
        assert (host(t)[:, :3] == 5).all() and (host(t)[:, 3 + K:] == 5).all()
    codes = torch.full((6, K + 5), 9, dtype=torch.int8, device="cuda")
    _, s = awq.awq_rmsnorm(views[0], wv, residual=views[1], fmt="int8", out=codes[:, 1: K + 1])
    check_8bit(host(codes)[:, 1: K + 1], host(s), y, "int8", 0)
    assert (host(codes)[:, 0] == 9).all() and (host(codes)[:, K + 1:] == 9).all()
    one = r[:1]
    _, y = lo.rmsnorm(x, w, 1e-5, np.repeat(one, 6, 0))
    check_f16(host(awq.awq_rmsnorm(dev(x), dev(w), residual=dev(one).expand(6, K))), y, K)


@pytest.mark.parametrize("K", [64, 5000, 40000])
def test_extreme_rows(K):
    """Zeros, subnormals, the largest numbers, infinities and NaN: each row by
    itself."""
    x, _, w = inputs([5, K], 7, K, False)
    x[0] = 0
    x[1] = np.float16(6e-8)
    x[2] = 65504
    x[3, 5], x[4, 7], x[4, 8] = np.nan, np.inf, -np.inf
    x[5] = 0
    x[5, 3] = 65504
    with np.errstate(invalid="ignore"):
        _, y = lo.rmsnorm(x, w, 1e-5)
    got = host(awq.awq_rmsnorm(dev(x), dev(w)))
    good = [0, 1, 2, 5, 6]
    with np.errstate(over="ignore"):
        fits = np.abs(y[good]).max(1) < 65504
    check_f16(got[good][fits], y[good][fits], K)
    assert np.isnan(got[3]).all()
    assert np.isnan(got[4, 7:9]).all() and (got[4, :7] == 0).all() and (got[4, 9:] == 0).all()
    for fmt in ("int8", "e4m3"):
        codes, scales = awq.awq_rmsnorm(dev(x), dev(w), fmt=fmt)
        codes, scales = values(codes), host(scales)
        check_8bit(codes[good], scales[good], y[good], fmt, 0)
        assert np.isnan(scales[3:5]).all() and (codes[3:5] == 0).all()
        if K % 32 == 0:
            codes, scales = awq.awq_rmsnorm(dev(x), dev(w), fmt=fmt, group_size=32)
            codes, scales = values(codes), host(scales)
            check_8bit(codes[good], scales[good], y[good], fmt, 32)
            assert np.isnan(scales[3]).all() and np.isnan(scales[4, 0]) and (codes[4] == 0).all()
            assert (scales[4, 1:] > 0).all()


def test_a_nan_weight_stays_in_its_group():
    x, r, w = inputs([6], 2, 256)
    w[70] = np.nan
    y = host(awq.awq_rmsnorm(dev(x), dev(w), residual=dev(r)))
    assert np.isnan(y[:, 70]).all() and np.isfinite(np.delete(y, 70, 1)).all()
    codes, scales = awq.awq_rmsnorm(dev(x), dev(w), residual=dev(r), fmt="int8", group_size=64)
    assert np.isnan(host(scales)[:, 1]).all() and np.isfinite(np.delete(host(scales), 1, 1)).all()
    assert (host(codes)[:, 64:128] == 0).all()


def test_many_rows_and_none():
    for T in (0, 1, 3, 4, 1000):
        x, r, w = inputs([7], T, 96) if T else (np.zeros((0, 96), np.float16),) * 2 + (np.ones(96, np.float16),)
        got = awq.awq_rmsnorm(dev(x), dev(w), residual=dev(r))
        if T:
            check_f16(host(got), lo.rmsnorm(x, w, 1e-5, r)[1], 96)


def test_graph_replay_and_streams():
    x, r, w = inputs([8], 17, 4096)
    xd, rd, wd = dev(x), dev(r), dev(w)
    y, total = torch.zeros_like(xd), torch.zeros_like(xd)
    codes, scales = torch.zeros(17, 4096, dtype=torch.int8, device="cuda"), torch.zeros(17, 32, device="cuda")

    def step():
        awq.awq_rmsnorm(xd, wd, residual=rd, residual_out=total, out=y)
        awq.awq_rmsnorm(total, wd, fmt="int8", group_size=128, out=codes, scales=scales)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x, r, _ = inputs([9, i], 17, 4096)
        xd.copy_(dev(x)), rd.copy_(dev(r))
        graph.replay()
        torch.cuda.synchronize()
        got = [host(t).copy() for t in (y, total, codes, scales)]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()
        torch.cuda.synchronize()
        for a, t in zip(got, (y, total, codes, scales)):
            np.testing.assert_array_equal(a, host(t))
        check_f16(got[0], lo.rmsnorm(x, w, 1e-5, r)[1], 4096)


def test_python_path_gives_the_same(monkeypatch):
    x, r, w = inputs([10], 3, 999)

    def run():
        outs = [awq.awq_rmsnorm(dev(x), dev(w), 1e-4, residual=dev(r), weight_offset=1)]
        outs += awq.awq_rmsnorm(dev(x), fmt="e4m3")
        outs += awq.awq_rmsnorm(dev(x[:, :960].copy()), fmt="int8", group_size=32)
        return [values(t) for t in outs]

    want = run()
    monkeypatch.setattr(awq, "_fast", (None, *(awq._fast or awq._fast_calls())[1:]))
    for a, b in zip(run(), want):
        np.testing.assert_array_equal(a, b)


def test_binding_refusals():
    x, r, w = (dev(t) for t in inputs([11], 2, 64))
    with pytest.raises(ValueError, match="fmt"):
        awq.awq_rmsnorm(x, w, fmt="int4")
    with pytest.raises(TypeError):
        awq.awq_rmsnorm(x.float(), w)
    with pytest.raises(ValueError, match="2-D"):
        awq.awq_rmsnorm(x[0], w)
    with pytest.raises(ValueError, match="weight"):
        awq.awq_rmsnorm(x, w[:60])
    with pytest.raises(ValueError, match="residual"):
        awq.awq_rmsnorm(x, w, residual=r[:1])
    with pytest.raises(ValueError, match="contiguous"):
        awq.awq_rmsnorm(x.t().contiguous().t(), w)
    with pytest.raises(TypeError, match="out"):
        awq.awq_rmsnorm(x, w, fmt="int8", out=torch.zeros_like(x))
    with pytest.raises(ValueError, match="scales"):
        awq.awq_rmsnorm(x, w, fmt="int8", scales=torch.zeros(2, 2, device="cuda"))
    for kw in (dict(group_size=32), dict(fmt="int8", group_size=48), dict(eps=-1.0), dict(eps=float("nan")),
               dict(weight_offset=float("inf"))):
        with pytest.raises(awq.AwqError):
            awq.awq_rmsnorm(x, w, **kw)
    with pytest.raises(awq.AwqError):       # outputs whose rows share memory
        awq.awq_rmsnorm(x, w, out=torch.zeros(64, dtype=torch.float16, device="cuda").expand(2, 64))
