"""awq_gemm_fused on sums that are not finite: a NaN stays a NaN behind every
activation, an infinity gives what the formula gives, and the other rows and
columns keep their bits. On every kernel of the linear layer."""

import numpy as np
import pytest

import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host, say  # noqa: E402

NAN, INF = float("nan"), float("inf")
# act(v) of v = NaN, inf, -inf. SiLU and the GELUs of -inf are limits of the
# form -inf * 0, which an implementation may answer by the limit or by NaN.
EXPECT = {"none": (NAN, INF, -INF), "relu": (NAN, INF, 0.0), "silu": (NAN, INF, None), "gelu": (NAN, INF, None),
          "gelu_tanh": (NAN, INF, None)}

# M, N, K, G, bits, path, workspace
CALLS = [
    (1, 520, 1024, 128, 4, 0, False),       # GEMV, one-shot
    (2, 520, 11008, 128, 4, 0, False),      # streaming
    (4, 136, 16384, 128, 4, 1, False),      # few rows
    (16, 520, 1024, 128, 4, 0, True),       # column tiles
    (20, 520, 4096, 128, 4, 3, True),       # skinny, split
    (20, 520, 4096, 128, 4, 3, False),
    (70, 520, 1024, 128, 4, 0, True),       # small tiles, vector accesses
    (70, 517, 1024, 128, 4, 0, True),       # element by element
    (70, 520, 512, 32, 4, 2, False),        # the older form
    (70, 517, 512, 32, 4, 2, True),
    (1, 520, 1024, 128, 8, 0, False),       # W8
    (70, 520, 1024, 128, 8, 0, True),
]


@pytest.mark.parametrize("act", list(awq.ACTIVATIONS))
@pytest.mark.parametrize("M,N,K,G,bits,path,with_ws", CALLS)
def test_nonfinite_sums(M, N, K, G, bits, path, with_ws, act):
    say("fused, not finite", M, N, K, G, bits, path, with_ws, act)
    lay = synth.make_layer(N, K, M, seed=[61, M, N, K], w_std=0.02)
    q = oracle.quantize(lay["w"], G) if bits == 4 else oracle.quantize_w8(lay["w"], G)
    t = (dev(lay["x"]), dev(q[0].view(np.int32)), dev(q[1]), dev(q[2]))
    ws = awq.gemm_workspace(M, N, K) if with_ws else None
    rng = np.random.default_rng([62, M])
    bias = rng.standard_normal(N).astype(np.float16)
    mul = rng.uniform(0.5, 2.0, (M, N)).astype(np.float16)
    res = rng.standard_normal((M, N)).astype(np.float16)

    def run(b, x=None):
        t_ = t if x is None else (x,) + t[1:]
        return host(awq.awq_gemm_fused(*t_, G, bias=dev(b), activation=act, mul=dev(mul), residual=dev(res), path=path,
                                       workspace=ws))

    clean = run(bias)
    assert np.isfinite(clean).all()
    # the bias makes three columns' sums not finite: the same for all rows
    bad = bias.copy()
    cols = [0, N // 2 + 1, N - 1]
    bad[cols] = [NAN, INF, -INF]
    got = run(bad)
    for c, want in zip(cols, EXPECT[act]):
        if want is None:
            assert (np.isnan(got[:, c]) | (got[:, c] == res[:, c])).all(), (act, c)
        elif np.isnan(want):
            assert np.isnan(got[:, c]).all(), (act, "NaN became", got[:, c])
        elif np.isinf(want):
            np.testing.assert_array_equal(got[:, c], np.full(M, want, np.float16))
        else:
            np.testing.assert_array_equal(got[:, c], res[:, c])
    others = np.ones(N, bool)
    others[cols] = False
    np.testing.assert_array_equal(got[:, others], clean[:, others])
    # a NaN in one row of x: that row alone, all of it
    x = lay["x"].copy()
    x[M - 1, K // 3] = np.nan
    got = run(bias, dev(x))
    assert np.isnan(got[M - 1]).all()
    np.testing.assert_array_equal(got[: M - 1], clean[: M - 1])
