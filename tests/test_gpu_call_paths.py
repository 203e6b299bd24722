"""The serving calls' two marshalling paths, the call extension and Python:
the same results, and neither keeps other Python threads from running."""

import ctypes
import threading
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host  # noqa: E402


def extension():
    ext = (awq._fast or awq._fast_calls())[0]
    if ext is None:
        pytest.skip("the call extension is not built")
    return ext


def batch(new, lens, page=32):
    rng = np.random.default_rng(81)
    per = -(-max(lens) // page)
    table = rng.permutation(len(lens) * per).astype(np.int32).reshape(len(lens), per)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return awq.KVSeqs(dev(table), dev(cu), dev(np.array(lens, np.int32)), max(new), max(lens)), len(lens) * per


def run_all():
    """Every serving call, with and without each of its optional tensors."""
    g = torch.Generator(device="cuda").manual_seed(82)
    half = lambda *s: torch.randn(*s, generator=g, device="cuda").half()  # noqa: E731
    outs = []
    for quantize, G in ((awq.awq_quantize, 128), (awq.awq_quantize_w8, 64)):
        w = quantize(half(264, 512) * 0.05, G)
        for M in (1, 12, 70):
            x, mul, res, bias = half(M, 512), half(M, 264), half(M, 270)[:, 3:267], half(264)
            ws = awq.gemm_workspace(M, 264, 512)
            outs.append(awq.awq_gemm_fused(x, *w, G))
            outs.append(awq.awq_gemm_fused(x, *w, G, bias=bias, activation="silu", mul=mul, residual=res, workspace=ws))
            y = mul.clone()
            assert awq.awq_gemm_fused(x, *w, G, residual=y, out=y, path=awq.PATH_AUTO) is y
            outs.append(y)
    for fmt in awq.KV_FORMATS:
        new, lens = [30, 1, 0, 17], [100, 1, 0, 40]
        s, pages = batch(new, lens)
        cache = awq.KVCache.empty(pages, 2, 64, 32, fmt)
        cache.k_codes.zero_(), cache.v_codes.zero_()
        full, _ = batch(lens, lens)
        kv = half(sum(lens), 6, 64)
        assert awq.awq_kv_write(cache, full, kv[:, 2:4], kv[:, 4:]) is None
        awq.awq_kv_write(cache, s, half(48, 2, 64) * 9, half(48, 2, 64) * 9)
        outs += [cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales]
        outs += [*awq.awq_kv_read(cache, s), *awq.awq_kv_read(cache, s, n_tokens=48)]
        out = (torch.full((50, 2, 64), 5.0, device="cuda").half(), None)
        assert awq.awq_kv_read(cache, s, out=out)[1] is None
        outs.append(out[0])
        q = half(48, 6, 64)
        ws = awq.kv_attention_workspace(cache, s, 6)
        for kw in (dict(), dict(scale=0.5, causal=False), dict(window=9, workspace=ws)):
            outs.append(awq.awq_kv_attention(q, cache, s, **kw))
            out, lse = torch.zeros(6, 48, 64, device="cuda").half().transpose(0, 1), torch.zeros(48, 6, device="cuda")
            assert awq.awq_kv_attention(q, cache, s, out=out, lse=lse, **kw) is out
            outs += [out, lse]
    torch.cuda.synchronize()
    return [host(o).copy() for o in outs]


def test_python_path_gives_the_same(monkeypatch):
    extension()
    want = run_all()
    entries = awq._fast[1:]
    monkeypatch.setattr(awq, "_fast", (None, *entries))
    got = run_all()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("call", ["kv_write", "kv_read", "kv_attention"])
def test_other_threads_run(call):
    """A call that takes long (a full queue makes a launch wait) leaves the
    interpreter to other threads: the C library's usleep stands for the entry
    point, its argument for the cache's address."""
    ext = extension()
    entry = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    t = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    dev_index, pause = t.get_device(), 400_000
    args = {"kv_write": (pause, 0, 4, 64, t, t), "kv_read": (pause, 0, 4, 64, t, t),
            "kv_attention": (pause, 0, 64, t, 1.0, True, 0, t, None, None)}[call]
    times = []

    def long_call():
        times.append(time.perf_counter())
        getattr(ext, call)(entry, 0, dev_index, *args)
        times.append(time.perf_counter())

    thread = threading.Thread(target=long_call)
    ticks = []
    thread.start()
    while thread.is_alive():
        time.sleep(0.005)
        ticks.append(time.perf_counter())
    thread.join()
    start, end = times
    assert end - start >= 0.39
    # some 80 ticks fall into the call; none does while it keeps the interpreter
    during = sum(start + 0.02 < t < end - 0.02 for t in ticks)
    assert during >= 5, f"the other thread ran {during} times in {end - start:.3f} s"
