"""Token tensors with fewer rows than cu_tokens names: the rows that are there
keep the positions that cu_tokens and kv_len give them, the others are
skipped."""

import numpy as np
import pytest

from oracle import kv_oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_kv import Model  # noqa: E402
from test_gpu_parity import dev, host, say  # noqa: E402

HELD, NEW = [50, 33, 0, 90], [40, 70, 45, 3]        # sequence rows 0.., 40.., 110.., 155..


def batch(m, new, lens):
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return awq.KVSeqs(dev(m.table), dev(cu), dev(np.asarray(lens, np.int32)), max(new), int(max(lens))), cu


def present(rows):
    """New tokens of each sequence that `rows` rows hold."""
    first = np.concatenate([[0], np.cumsum(NEW)])
    return np.clip(rows - first[:-1], 0, NEW)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("rows", [158, 157, 130, 111, 75, 41, 7])
def test_write_fewer_rows(fmt, rows):
    say("kv write, rows", rows)
    m = Model([71, rows], 4, 2, 64, 32, fmt, 160)
    m.append(HELD)
    lens = np.array(HELD) + NEW
    s, _ = batch(m, NEW, lens)
    k, v = m.values(rows), m.values(rows, 3.0)
    awq.awq_kv_write(m.cache, s, dev(k), dev(v))
    # the same rows as a batch of their own
    here = present(rows)
    m.len = (np.array(HELD) + here).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(here)]).astype(np.int32)
    kv_oracle.write(m.kc, m.ks, k, m.table, cu, m.len, fmt)
    kv_oracle.write(m.vc, m.vs, v, m.table, cu, m.len, fmt)
    m.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("rows", [158, 130, 75, 7])
def test_read_fewer_rows(fmt, rows):
    m = Model([72], 4, 2, 64, 32, fmt, 160)
    lens = np.array(HELD) + NEW
    m.append(lens)
    s, cu = batch(m, NEW, lens)
    all_k, all_v = (host(t) for t in awq.awq_kv_read(m.cache, s))
    k, v = awq.awq_kv_read(m.cache, s, n_tokens=rows)
    np.testing.assert_array_equal(host(k), all_k[:rows])
    np.testing.assert_array_equal(host(v), all_v[:rows])
    # more new tokens than the length: rows at positions below 0 are 0, the
    # rows behind the tensor's end untouched
    s, _ = batch(m, NEW, np.minimum(lens, 20))
    all_k, _ = (host(t) for t in awq.awq_kv_read(m.cache, s))
    big = torch.full((158 + 50, 2, 64), 9.0, dtype=torch.float16, device="cuda")
    awq.awq_kv_read(m.cache, s, out=(big[:rows], None))
    np.testing.assert_array_equal(host(big)[:rows], all_k[:rows])
    assert (host(big)[rows:] == 9).all()


@pytest.mark.parametrize("new,rows", [([1, 1, 1, 1], 3), ([5, 2, 4, 3], 9), (NEW, 130), (NEW, 75), (NEW, 7)])
def test_attention_fewer_rows(new, rows):
    m = Model([73], 4, 2, 64, 32, "int8", 160)
    lens = np.array(HELD) + NEW
    m.append(lens)
    s, cu = batch(m, new, lens)
    T = int(cu[-1])
    q = m.rng.standard_normal((T, 4, 64)).astype(np.float16)
    whole = host(awq.awq_kv_attention(dev(q), m.cache, s))
    for ws in (None, awq.kv_attention_workspace(m.cache, s, 4)):
        part = host(awq.awq_kv_attention(dev(q[:rows]), m.cache, s, workspace=ws))
        want = kv_oracle.attention(q, m.kc, m.ks, m.vc, m.vs, m.table, cu, lens, 64 ** -0.5)
        u = 2.0 ** -24
        e = 2 * (68 * u * want[3] + 2.0 ** -21 + 2 * 160 * u)
        tol = (e + 2.0 ** -18)[..., None] * want[2] + 2.0 ** -11 * np.abs(want[0]) + 2.0 ** -25 + \
            160 * 2.0 ** -34 * 127 * float(m.vs.max())
        assert (np.abs(part.astype(np.float64) - want[0][:rows]) <= tol[:rows]).all()
        assert (np.abs(whole.astype(np.float64) - want[0]) <= tol).all()
