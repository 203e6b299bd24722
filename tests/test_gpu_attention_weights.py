"""The weights of awq_kv_attention's second product: what their rounding to
fp16 may cost, whatever scales the pages have.

With the names of test_gpu_kv.py (A = sum_j w_j |v_j|, N the visible keys,
e the fp32 steps' share), a weight enters as one or two fp16 numbers: half a
step 2^-11 of it, and below fp16's normal range half a subnormal step 2^-25
in a unit in which the row's largest product C = max_j w_j s_j of a weight
and its page's scale is at least 2^9. A value is at most `top` steps of its
scale, so the subnormals cost N 2^-34 top C: a bound by what the row itself
weighs, not by the largest scale in the cache. Hence
  |err| <= (e + 2^-11) A + N 2^-34 top C + 2^-11 |o| + 2^-25.
"""

import numpy as np
import pytest

from oracle import kv_oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv import Model  # noqa: E402
from test_gpu_parity import say  # noqa: E402

U = 2.0 ** -24


def largest_product(m, q, length, new, scale, window):
    """max_j w_j s_j of every row of a one-sequence, one-kv-head model."""
    ids = m.table[0, : -(-length // m.page)]
    k = (m.kc[ids, 0] * m.ks[ids, 0].astype(np.float64)[:, None, None]).reshape(-1, m.dim)[:length]
    s = np.repeat(m.vs[ids, 0].astype(np.float64), m.page)[:length]
    c = np.zeros(q.shape[:2])
    for i in range(new):
        p = length - new + i
        see = slice(max(0, p - window + 1) if window else 0, p + 1)
        for h in range(q.shape[1]):
            t = scale * (k[see] @ q[i, h].astype(np.float64))
            w = np.exp(t - t.max())
            c[i, h] = (w / w.sum() * s[see]).max()
    return c


def hold(m, got, c, n_keys):
    o, _, (eo, _, spread, mass) = got
    e = 2 * ((m.dim + 4) * U * mass + 2.0 ** -21 + 2 * n_keys * U)
    tol = (e + 2.0 ** -11)[..., None] * spread + 2.0 ** -11 * np.abs(eo) + 2.0 ** -25 + \
        (n_keys * 2.0 ** -34 * float(kv_oracle.TOP[m.fmt]) * c)[..., None]
    err = np.abs(o.astype(np.float64) - eo)
    say("  worst", float(np.max(err / tol)), "of the bound")
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("small", [2e-5, 1e-3, 0.5])
@pytest.mark.parametrize("length,new", [(164, 2), (200, 70)])
def test_large_page_outside_the_window(fmt, page, small, length, new):
    """The first 64 tokens' values are near fp16's largest, the others small;
    some rows of a block see the former, the rest (behind the window) do not
    and must not lose their own values' bits to them."""
    say("weights, large page masked", fmt, page, small, length, new)
    m = Model([51, page, length], 1, 1, 64, page, fmt, length)
    v = (m.rng.uniform(0.5, 1.0, (length, 1, 64)) * small).astype(np.float16)
    v[:64] = (m.rng.uniform(-1, 1, (64, 1, 64)) * 6e4).astype(np.float16)
    m.append([length], k=m.values(length), v=v)
    q = m.rng.standard_normal((new, 2, 64)).astype(np.float16)
    got = m.attend(q, [new], window=100)
    hold(m, got, largest_product(m, q, length, new, 64 ** -0.5, 100), 100)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("small", [2e-5, 1e-3])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("new", [2, 70])
def test_small_page_takes_the_weight(fmt, page, small, order, new):
    """Keys of the pages with large values point away from the queries, whose
    weight (below e^-50) is on the pages with small ones; either comes first."""
    say("weights, small page attended", fmt, page, small, order, new)
    length = 256
    m = Model([52, page, new], 1, 1, 64, page, fmt, length)
    big = (np.arange(length) // 64 % 2 == 0) if order == 1 else (np.arange(length) // 64 % 2 == 1)
    sign = np.where(big, -1.0, 1.0)[:, None, None]
    k = (sign * m.rng.uniform(0.8, 1.0, (length, 1, 64))).astype(np.float16)
    v = (m.rng.uniform(0.5, 1.0, (length, 1, 64)) * np.where(big, 6e4, small)[:, None, None]).astype(np.float16)
    m.append([length], k=k, v=v)
    q = m.rng.uniform(3.5, 4.5, (new, 2, 64)).astype(np.float16)
    got = m.attend(q, [new])
    hold(m, got, largest_product(m, q, length, new, 64 ** -0.5, 0), length)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,page", [(64, 32), (96, 64), (128, 64), (192, 128), (256, 64)])
@pytest.mark.parametrize("new", [2, 16, 70])
def test_opposite_values_cancel(fmt, dim, page, new):
    """Two visible keys of nearly equal weight and opposite values: the output
    is a small difference, in which a weight rounded to one fp16 number
    (2^-11 of A) would show. As two, a weight is within 2^-20 of itself (both
    parts toward zero); its exponent, at most 16, is rounded twice and the
    scales' logarithm, exponential and reciprocal add 2^-22 each, together
    below 2^-18: |err| <= (e + 2^-18) A + N 2^-34 top C + 2^-11 |o| + 2^-25."""
    say("weights, opposite values", fmt, dim, page, new)
    length = 130
    m = Model([53, dim, new], 1, 1, dim, page, fmt, length)
    v = (m.rng.uniform(50, 100, (length, 1, 1)) * np.where(np.arange(length) % 2, 1.0, -1.0)[:, None, None] *
         np.ones((1, 1, dim))).astype(np.float16)
    v[:, :, ::3] = v[:, :, ::3] / 2
    v[1::2] = -v[0::2]
    m.append([length], k=m.values(length), v=v)
    q = (m.rng.standard_normal((new, 2, dim)) * 0.02).astype(np.float16)
    o, _, (eo, _, spread, mass) = m.attend(q, [new], window=2)
    c = largest_product(m, q, length, new, dim ** -0.5, 2)
    e = 2 * ((dim + 4) * U * mass + 2.0 ** -21 + 4 * U)
    tol = (e + 2.0 ** -18)[..., None] * spread + 2.0 ** -11 * np.abs(eo) + 2.0 ** -25 + \
        (2 * 2.0 ** -34 * float(kv_oracle.TOP[m.fmt]) * c)[..., None]
    err = np.abs(o.astype(np.float64) - eo)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n_seqs,longest,new", [(1500, 40, 2), (1500, 40, 1), (6, 300, 200)])
def test_every_weight_has_both_parts(fmt, n_seqs, longest, new):
    """Some 2^17 weights of short sequences, where a single one that is off by
    a step of fp16 shows in the outputs: the bound of the test above."""
    say("weights, both parts", fmt, n_seqs, new)
    m = Model([93], n_seqs, 1, 64, 32, fmt, longest)
    lens = m.rng.integers(0, longest + 1, n_seqs)
    m.append(lens)
    count = np.minimum(lens, m.rng.integers(0, new + 1, n_seqs))
    q = m.rng.standard_normal((int(count.sum()), 2, 64)).astype(np.float16)
    for split in (True, False):
        o, _, (eo, _, spread, mass) = m.attend(q, list(count), split=split)
        e = 2 * ((m.dim + 4) * U * mass + 2.0 ** -21 + 2 * longest * U)
        tol = (e + 2.0 ** -18)[..., None] * spread + 2.0 ** -11 * np.abs(eo) + 2.0 ** -25 + \
            longest * 2.0 ** -34 * float(kv_oracle.TOP[fmt]) * float(m.vs.max())
        err = np.abs(o.astype(np.float64) - eo)
        assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"
