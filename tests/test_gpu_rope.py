"""Rotary positions (awq_rope) against the CPU oracle.

Per element of a pair (a, b), with u = 2^-24 and m the amplitude: the reduced
angle is rounded to fp32 (2^-25 of a turn, pi 2^-24 = 3.2 u on sine and cosine;
the fp64 steps before it at most 2^-25 of a turn at 2^31 positions more), sine
and cosine are within 4 units of the last place (4 u), the amplitude, its
product, and the two products and the sum of the rotation round 5 times:
(2 * 3.2 + 4 + 5) u m (|a| + |b|), and fp16 adds 2^-11 |y| or 2^-25.
"""

import numpy as np
import pytest

from oracle import layer_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host, say  # noqa: E402


def check(y, x, positions, freqs, layout, m=1.0):
    want, size = lo.rope(x, positions, freqs, layout, m)
    tol = 16 * 2.0 ** -24 * abs(m) * size + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    r = 2 * len(freqs)
    err = np.abs(y.astype(np.float64) - want)
    assert (err[..., :r] <= tol[..., :r]).all(), f"worst {np.max(err[..., :r] / tol[..., :r]):.3f} of the bound"
    np.testing.assert_array_equal(y[..., r:], x[..., r:])


def heads(seed, T, hq, hk, D):
    rng = np.random.default_rng(seed)
    q, k = (rng.standard_normal((T, h, D)).astype(np.float16) * 3 for h in (hq, hk))
    return rng, q, k


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,r,hq,hk,T", [(128, 128, 32, 8, 5), (128, 64, 4, 4, 70), (64, 64, 3, 1, 1), (80, 20, 5, 5, 9),
                                         (96, 24, 2, 1, 3), (256, 256, 8, 1, 2), (2, 2, 7, 3, 4), (100, 34, 1, 1, 3),
                                         (50, 50, 3, 2, 2), (512, 128, 2, 2, 2), (4096, 4096, 1, 1, 1)])
def test_shapes(layout, D, r, hq, hk, T):
    say("rope", layout, D, r)
    rng, q, k = heads([1, D, r], T, hq, hk, D)
    pos = rng.integers(0, 5000, T).astype(np.int32)
    f, _ = lo.rope_frequencies(r)
    rope = awq.Rope(r, layout=layout)
    qo, ko = awq.awq_rope(dev(q), dev(k), rope, dev(pos))
    check(host(qo), q, pos, f, layout)
    check(host(ko), k, pos, f, layout)
    # in place, and one tensor alone
    qd, kd = dev(q), dev(k)
    got = awq.awq_rope(qd, kd, rope, dev(pos), out=(qd, kd))
    assert got[0] is qd and got[1] is kd
    assert torch.equal(qd, qo) and torch.equal(kd, ko)
    q2, none = awq.awq_rope(dev(q), None, rope, dev(pos))
    assert none is None and torch.equal(q2, qo)
    none, k2 = awq.awq_rope(None, dev(k), rope, dev(pos))
    assert none is None and torch.equal(k2, ko)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "wavelength"])
def test_scaled_far_positions(layout, scaling):
    rng, q, k = heads([2], 40, 2, 1, 128)
    pos = np.concatenate([rng.integers(0, 2 ** 21, 36), [0, 1, 2 ** 31 - 1, -(2 ** 31)]]).astype(np.int32)
    f, m = lo.rope_frequencies(96, 50000.0, scaling, 8.0, 8192.0)
    rope = awq.Rope(96, 50000.0, layout, scaling, 8.0, 8192.0)
    np.testing.assert_allclose(host(rope.freqs), f, rtol=1e-14)
    qo, ko = awq.awq_rope(dev(q), dev(k), rope, dev(pos))
    # (of far positions the fp64 product itself is the definition: the table's own frequencies)
    check(host(qo), q, pos, host(rope.freqs), layout, m)
    check(host(ko), k, pos, host(rope.freqs), layout, m)


def test_turning_back():
    """Positions p, then -p, is the input up to the roundings; frequencies of
    one's own."""
    rng, q, _ = heads([3], 20, 4, 1, 64)
    pos = rng.integers(0, 100000, 20).astype(np.int32)
    f = rng.uniform(0.0, 1.0, 32)
    rope = awq.Rope.of(dev(f), "half", 2.0)
    y, _ = awq.awq_rope(dev(q), None, rope, dev(pos))
    check(host(y), q, pos, f, "half", 2.0)
    back, _ = awq.awq_rope(y, None, awq.Rope.of(dev(f), "half", 0.5), dev(-pos))
    assert np.abs(host(back).astype(np.float64) - q).max() <= 4 * 2.0 ** -11 * np.abs(q).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_alignment(layout):
    """Slices of one packed projection at odd addresses, in place and out;
    head-major outputs; a broadcast input."""
    rng, q, k = heads([4], 6, 4, 2, 64)
    pos = rng.integers(0, 500, 6).astype(np.int32)
    f, _ = lo.rope_frequencies(32)
    rope = awq.Rope(32, layout=layout)
    packed = torch.full((6, 6 * 64 + 5), 9.0, dtype=torch.float16, device="cuda")
    qv, kv = packed[:, 1:257].unflatten(1, (4, 64)), packed[:, 257:385].unflatten(1, (2, 64))
    qv.copy_(dev(q)), kv.copy_(dev(k))
    qo, ko = awq.awq_rope(qv, kv, rope, dev(pos))
    check(host(qo), q, pos, f, layout)
    out = (torch.zeros(4, 6, 64, dtype=torch.float16, device="cuda").transpose(0, 1),
           torch.zeros(2, 6, 64, dtype=torch.float16, device="cuda").transpose(0, 1))
    awq.awq_rope(qv, kv, rope, dev(pos), out=out)
    assert torch.equal(out[0], qo) and torch.equal(out[1], ko)
    awq.awq_rope(qv, kv, rope, dev(pos), out=(qv, kv))
    assert torch.equal(qv, qo) and torch.equal(kv, ko)
    assert (host(packed)[:, 0] == 9).all() and (host(packed)[:, 385:] == 9).all()
    wide, _ = awq.awq_rope(dev(q[:1]).expand(6, 4, 64), None, rope, dev(pos))
    check(host(wide), np.repeat(q[:1], 6, 0), pos, f, layout)


def test_batch_positions():
    """The newest tokens of ragged sequences: none, more than the length,
    rows of no sequence, bounds below the counts."""
    rng, q, k = heads([5], 24, 2, 1, 64)
    new, lens = [3, 0, 7, 1, 9], [3, 5, 1000, 131072, 4]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(new, lens)])
    f, _ = lo.rope_frequencies(64)
    rope = awq.Rope(64)
    table = torch.zeros(5, 0, dtype=torch.int32, device="cuda")
    s = awq.KVSeqs(table, dev(cu), dev(np.array(lens, np.int32)), 9, 131072)
    qd, kd = dev(q), dev(k)
    awq.awq_rope(qd, kd, rope, seqs=s, out=(qd, kd))
    check(host(qd)[:20], q[:20], pos, f, "half")
    check(host(kd)[:20], k[:20], pos, f, "half")
    np.testing.assert_array_equal(host(qd)[20:], q[20:])
    fresh, _ = awq.awq_rope(dev(q), None, rope, seqs=s)
    assert torch.equal(fresh[:20], qd[:20]) and not fresh[20:].any()
    # the same positions as a tensor
    t, _ = awq.awq_rope(dev(q[:20]), None, rope, dev(pos.astype(np.int32)))
    assert torch.equal(t, qd[:20])
    # new tokens past max_tokens and rows past the tensor are left
    s = awq.KVSeqs(table, dev(cu), dev(np.array(lens, np.int32)), 4, 131072)
    part = dev(q[:15])
    awq.awq_rope(part, None, rope, seqs=s, out=(part, None))
    done = np.zeros(15, bool)
    for b, n in enumerate(new):
        done[cu[b]: cu[b] + min(n, 4)] = True
    check(host(part)[done], q[:15][done], pos[:15][done], f, "half")
    np.testing.assert_array_equal(host(part)[~done], q[:15][~done])
    # arrays that lie: nothing leaves the tensors
    wild = awq.KVSeqs(table, dev(np.array([-5, 3, 900, 2 ** 31 - 1, 1, 7], np.int32)),
                      dev(np.array([2 ** 31 - 1, -4, 0, 9, 1], np.int32)), 1000, 131072)
    awq.awq_rope(dev(q), dev(k), rope, seqs=wild)
    torch.cuda.synchronize()


def test_values_that_are_not_finite():
    """They reach their own pair alone."""
    rng, q, _ = heads([6], 3, 2, 1, 64)
    pos = np.array([5, 6, 7], np.int32)
    rope = awq.Rope(64)
    clean = host(awq.awq_rope(dev(q), None, rope, dev(pos))[0])
    bad = q.copy()
    bad[1, 0, 3], bad[2, 1, 40] = np.nan, np.inf
    got = host(awq.awq_rope(dev(bad), None, rope, dev(pos))[0])
    same = np.ones(q.shape, bool)
    same[1, 0, [3, 35]] = same[2, 1, [8, 40]] = False
    np.testing.assert_array_equal(got[same], clean[same])
    assert not np.isfinite(got[~same]).any()


def test_graph_replay_and_streams():
    rng, q, k = heads([7], 8, 8, 2, 128)
    rope = awq.Rope(128, scaling="yarn", factor=4.0, trained_len=4096)
    f, m = lo.rope_frequencies(128, scaling="yarn", factor=4.0, length=4096)
    qd, kd, pos = dev(q), dev(k), torch.zeros(8, dtype=torch.int32, device="cuda")
    out = (torch.zeros_like(qd), torch.zeros_like(kd))
    awq.awq_rope(qd, kd, rope, pos, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.awq_rope(qd, kd, rope, pos, out=out)
    for _ in range(3):
        p = rng.integers(0, 16384, 8).astype(np.int32)
        pos.copy_(dev(p))
        graph.replay()
        torch.cuda.synchronize()
        check(host(out[0]), q, p, f, "half", m)
        first = out[0].clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            again = awq.awq_rope(qd, kd, rope, pos)
        torch.cuda.synchronize()
        assert torch.equal(again[0], first)


def test_python_path_gives_the_same(monkeypatch):
    rng, q, k = heads([8], 5, 3, 2, 80)
    pos = dev(rng.integers(0, 500, 5).astype(np.int32))
    rope = awq.Rope(40, layout="interleaved")
    s = awq.KVSeqs(torch.zeros(2, 0, dtype=torch.int32, device="cuda"), dev(np.array([0, 2, 4], np.int32)),
                   dev(np.array([9, 2], np.int32)), 2, 9)
    run = lambda: [*awq.awq_rope(dev(q), dev(k), rope, pos), *awq.awq_rope(dev(q), dev(k), rope, seqs=s)]  # noqa: E731
    want = run()
    monkeypatch.setattr(awq, "_fast", (None, *(awq._fast or awq._fast_calls())[1:]))
    for a, b in zip(run(), want):
        assert torch.equal(a, b)


def test_binding_refusals():
    _, q, k = heads([9], 4, 2, 1, 64)
    q, k, rope = dev(q), dev(k), awq.Rope(64)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="either"):
        awq.awq_rope(q, k, rope)
    with pytest.raises(ValueError, match="positions"):
        awq.awq_rope(q, k, rope, pos[:3])
    with pytest.raises(TypeError, match="positions"):
        awq.awq_rope(q, k, rope, pos.long())
    with pytest.raises(ValueError, match="rotates"):
        awq.awq_rope(q[..., :32].contiguous(), None, rope, pos)
    with pytest.raises(ValueError, match="same tokens"):
        awq.awq_rope(q, k[:3], rope, pos)
    with pytest.raises(TypeError, match="float16"):
        awq.awq_rope(q.float(), None, rope, pos)
    with pytest.raises(ValueError, match="contiguous"):
        awq.awq_rope(q.transpose(1, 2).contiguous().transpose(1, 2), None, rope, pos)
    with pytest.raises(ValueError, match="out"):
        awq.awq_rope(q, None, rope, pos, out=(q[:2], None))
    with pytest.raises(ValueError, match="layout"):
        awq.Rope(64, layout="other")
    with pytest.raises(ValueError, match="scaling"):
        awq.Rope(64, scaling="other")
    with pytest.raises(awq.AwqError):
        awq.Rope(63)
    with pytest.raises(awq.AwqError):       # in place with other strides
        awq.awq_rope(q.new_zeros(8, 2, 64)[:4], None, rope, pos, out=(q.new_zeros(64).expand(4, 2, 64), None))
