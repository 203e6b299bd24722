"""A batch whose table has no pages: nothing is held, so nothing is written,
tokens read back as 0 and attention sees nothing."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host  # noqa: E402


def half(*shape, value=None):
    if value is not None:
        return torch.full(shape, value, dtype=torch.float16, device="cuda")
    return torch.randn(*shape, device="cuda").half()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,new", [([5, 0, 40], [3, 1, 40]), ([0, 0, 0], [1, 1, 1])])
def test_table_without_pages(fmt, lens, new):
    cache = awq.KVCache.empty(4, 2, 64, 32, fmt)
    cache.k_codes.fill_(0xFF), cache.v_codes.fill_(0xFF)
    cache.k_scales.fill_(float("nan")), cache.v_scales.fill_(float("nan"))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    s = awq.KVSeqs(torch.zeros(3, 0, dtype=torch.int32, device="cuda"), dev(cu), dev(np.array(lens, np.int32)),
                   max(new), max(lens))
    awq.awq_kv_write(cache, s, half(T, 2, 64), half(T, 2, 64))
    torch.cuda.synchronize()
    assert (host(cache.k_codes) == 0xFF).all() and (host(cache.v_codes) == 0xFF).all()
    assert np.isnan(host(cache.k_scales)).all() and np.isnan(host(cache.v_scales)).all()
    k, v = half(T + 3, 2, 64, value=9.0), half(T + 3, 2, 64, value=9.0)
    awq.awq_kv_read(cache, s, out=(k, v))
    for t in (k, v):
        assert (host(t)[:T] == 0).all() and (host(t)[T:] == 9).all()
    k, v = awq.awq_kv_read(cache, s)
    assert k.shape == (T, 2, 64) and not host(k).any() and not host(v).any()
    for workspace in (None, awq.kv_attention_workspace(cache, s, 4)):
        out, lse = half(T + 3, 4, 64, value=9.0), torch.full((T + 3, 4), 7.0, device="cuda")
        awq.awq_kv_attention(half(T + 3, 4, 64), cache, s, out=out, lse=lse, workspace=workspace)
        assert (host(out)[:T] == 0).all() and (host(out)[T:] == 9).all()
        assert np.isneginf(host(lse)[:T]).all() and (host(lse)[T:] == 7).all()
