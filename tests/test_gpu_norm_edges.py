"""The norm (awq_rmsnorm) at the edges of its arguments.

The bounds are test_gpu_norm's.
"""

import numpy as np
import pytest

from oracle import layer_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_norm import check_8bit, check_f16, inputs, values  # noqa: E402
from test_gpu_parity import dev, host, say  # noqa: E402


def test_group_sizes_of_any_integer_kind():
    """Numpy's integers as Python's own; past a C int, where ctypes would cut
    them to an ordinary group and the call fill more scales than there are, no
    call."""
    x, _, w = inputs([21], 2, 64, False)
    xd, wd = dev(x), dev(w)
    _, y = lo.rmsnorm(x, w)
    for kind in (int, np.int32, np.int64):
        codes, scales = awq.awq_rmsnorm(xd, wd, fmt="int8", group_size=kind(32))
        check_8bit(host(codes), host(scales), y, "int8", 32)
    for bad in (-2 ** 32 + 32, 2 ** 32 + 32, 2 ** 31):
        say("rmsnorm group", bad)
        with pytest.raises(ValueError, match="group_size"):
            awq.awq_rmsnorm(xd, wd, fmt="int8", group_size=bad)
    for bad in (32.0, "32", None):
        with pytest.raises(TypeError, match="group_size"):
            awq.awq_rmsnorm(xd, wd, fmt="int8", group_size=bad)


@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.1e-38, 1.2e-38, 1e-30])
def test_the_smallest_eps(eps, fmt):
    """Rows of zeros are zeros with any eps > 0, subnormal numbers among them; the
    smallest fp16 numbers are not the eps' business."""
    x, _, w = inputs([22], 4, 96, False)
    x[0] = 0
    x[1] = np.float16(6e-8)
    x[2] = 0
    x[2, 5] = np.float16(6e-8)
    _, y = lo.rmsnorm(x, w, eps)
    assert np.isfinite(y).all() and not y[0].any()
    got = awq.awq_rmsnorm(dev(x), dev(w), eps, fmt=fmt)
    if fmt is None:
        check_f16(host(got), y, 96)
    else:
        check_8bit(values(got[0]), host(got[1]), y, fmt, 0)


@pytest.mark.parametrize("offset", [1e36, -65505.0, 65504.0, -65504.0])
def test_the_largest_offsets(offset):
    """An offset as large as the largest weight: the 8-bit scales hold y, as far
    from fp16 as it is. One past that is refused: the unscaled products pass
    fp32, and finite rows had infinite scales."""
    x, r, w = inputs([23], 3, 256)
    x[1] = 65504
    x[2] = np.float16(6e-8)
    r[2] = 0
    _, y = lo.rmsnorm(x, w, 1e-5, r, offset)
    for fmt in ("int8", "e4m3"):
        call = lambda: awq.awq_rmsnorm(dev(x), dev(w), residual=dev(r), weight_offset=offset, fmt=fmt, group_size=64)  # noqa: E731
        if abs(offset) > 65504:
            with pytest.raises(awq.AwqError):
                call()
        else:
            codes, scales = call()
            check_8bit(values(codes), host(scales), y, fmt, 64)
