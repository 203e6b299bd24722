"""Attention over the 4-bit cache where a sequence's keys are many blocks' parts:
more than eight of them (the join takes eight at a time), blocks of 32 rows,
parts that some rows see nothing of, maxima that rise and fall from part to part;
and two row tiles of the most sequences that a call takes.

Attention's bounds are test_gpu_kv4's.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_kv4 import Model  # noqa: E402
from test_gpu_parity import say  # noqa: E402

U = 2.0 ** -24


def steep(m, k, order):
    """Keys whose channel 3 grows, falls, or goes up and down along the positions."""
    n = len(k)
    t = np.arange(n)
    k[:, :, 3] = {"up": t, "down": n - 1 - t, "waves": n / 4 * (1 + np.sin(t / 700.0))}[order][:, None] * (160.0 / n)
    return k


def parts(m, new, ratio, rows, max_len=None):
    """Parts that the call's bounds make of a sequence's keys, in blocks of `rows`
    rows: from the size of the workspace, 4096 counters and what a part leaves."""
    s, *_ = m.seqs(new, max_len=max_len)
    tiles = -(-max(new) * ratio // rows) * len(new) * m.heads
    room = awq.kv_attention_workspace_bytes(m.cache, s, m.heads * ratio) - 4096 * 4
    assert room % (tiles * rows * (m.dim + 2) * 4) == 0
    return room // (tiles * rows * (m.dim + 2) * 4)


@pytest.mark.parametrize("order", ["flat", "up", "down", "waves"])
@pytest.mark.parametrize("dim,page,heads,ratio,len_,new", [
    (128, 64, 2, 1, 5000, 1),           # 20 parts of 256 positions
    (64, 32, 1, 8, 4800, 1),            # 19
    (256, 64, 1, 4, 2500, 3),           # 10, 12 rows
    (192, 128, 1, 8, 5000, 3),          # two blocks of 16 rows
    (96, 64, 2, 3, 4096 + 7, 5),        # 17, the last of 7 positions
])
def test_many_parts(dim, page, heads, ratio, len_, new, order):
    say("kv4 parts", dim, page, len_, new, order)
    m = Model([51, dim, new], 1, heads, dim, page, len_)
    k = m.values(len_, 0.5)
    if order != "flat":
        steep(m, k, order)
    m.append([len_], k=k)
    assert parts(m, [new], ratio, 16) > 8
    q = m.rng.standard_normal((new, heads * ratio, dim)).astype(np.float16)
    if order != "flat":
        q[:, :, 3] = 8.0 if dim < 100 else 12.0
    for window in (0, len_ - 300, 2000):
        worst = m.assert_attention(m.attend(q, [new], window=window), len_)
        say("  worst", round(worst, 3), "of the bound")
    m.assert_attention(m.attend(q, [new], causal=False), len_)


@pytest.mark.parametrize("len_", [32768, 32768 - 5, 20000])
def test_the_most_parts(len_):
    """One kv head: 128 parts."""
    say("kv4 parts", len_)
    m = Model([52, len_], 1, 1, 64, 256, len_)
    m.append([len_], k=steep(m, m.values(len_, 0.5), "waves"))
    assert parts(m, [1], 3, 16) > 64 or len_ < 32768
    q = m.rng.standard_normal((1, 3, 64)).astype(np.float16)
    q[:, :, 3] = 6.0
    m.assert_attention(m.attend(q, [1]), len_)
    q[0, 1, 7] = np.nan
    o, lse, want = m.attend(q, [1])
    assert np.isnan(o[0, 1]).all() and np.isnan(lse[0, 1])
    rest = [0, 2]
    m.assert_attention((o[:, rest], lse[:, rest], tuple(w[:, rest] for w in want)), len_)


@pytest.mark.parametrize("dim,page,ratio,news", [(128, 64, 8, 4), (64, 32, 4, 6), (96, 64, 2, 16), (128, 32, 1, 32)])
@pytest.mark.parametrize("order", ["flat", "waves"])
def test_parts_of_thirty_two_rows(dim, page, ratio, news, order):
    """17 to 32 rows a kv head, up to three parts of 4096 positions: 32 kv heads,
    the bound 2^16. Windows that leave rows without a position of a part."""
    say("kv4 parts, 32 rows", dim, page, ratio, news, order)
    lens = [9000, 5000, 4096 + news // 2, 8192, 4097, 100, 0, news]
    m = Model([53, dim, news], 8, 4, dim, page, max(lens))
    k = m.values(sum(lens), 0.5)
    if order == "waves":
        at = np.cumsum([0] + lens)
        for b, n in enumerate(lens):
            if n:
                steep(m, k[at[b]: at[b + 1]], "waves")
    m.append(lens, k=k)
    new = [news] * 6 + [0, news]
    assert parts(m, new, ratio, 32, 2 ** 16) == 16
    q = m.rng.standard_normal((sum(new), 4 * ratio, dim)).astype(np.float16)
    if order == "waves":
        q[:, :, 3] = 6.0
    for causal, window in ((True, 0), (True, news // 2), (True, 4100), (False, 0)):
        got = m.attend(q, new, causal=causal, window=window, max_len=2 ** 16)
        m.assert_attention(got, max(lens))


def test_ten_parts_of_thirty_two_rows():
    """One sequence of 16 kv heads, the bound 2^16: parts of 2048 positions."""
    say("kv4 ten parts, 32 rows")
    m = Model([54], 1, 16, 64, 64, 18500)
    m.append([18500], k=steep(m, m.values(18500, 0.5), "waves"))
    assert parts(m, [3], 8, 32, 2 ** 16) == 32
    q = m.rng.standard_normal((3, 128, 64)).astype(np.float16)
    q[:, :, 3] = 6.0
    for window in (0, 9000):
        m.assert_attention(m.attend(q, [3], window=window, max_len=2 ** 16), 18500)


def test_two_row_tiles_of_the_most_sequences():
    """32767 sequences of 17 tokens, all of them queries, 192 channels: two blocks
    of 16 rows a sequence, as far as a launch's second dimension goes."""
    B, N, D = 32767, 17, 192
    say("kv4 sequences", B, D)
    g = torch.Generator(device="cuda").manual_seed(55)
    half = lambda *s: torch.randn(s, device="cuda", dtype=torch.float16, generator=g)  # noqa: E731
    cache = awq.KVCache.empty(B, 1, D, 32, "int4", "cuda")
    table = torch.randperm(B, device="cuda", generator=g).to(torch.int32).reshape(B, 1)
    lens = torch.full((B,), N, device="cuda", dtype=torch.int32)
    cu = (torch.arange(B + 1, device="cuda") * N).to(torch.int32)
    s = awq.KVSeqs(table, cu, lens, N, N)
    awq.awq_kv_write(cache, s, half(B * N, 1, D), half(B * N, 1, D))
    kn, vn = (t.double().reshape(B, N, D) for t in awq.awq_kv_read(cache, s))
    q = half(B * N, 1, D)
    out = awq.awq_kv_attention(q, cache, s)
    q64 = q.double().reshape(B, N, D)
    kt = kn.transpose(1, 2).contiguous()
    at = torch.arange(N, device="cuda")
    t = torch.matmul(q64, kt) * D ** -0.5
    w = torch.softmax(t.masked_fill(at[None, :] > at[:, None], float("-inf")), -1)
    want, spread = torch.matmul(w, vn), torch.matmul(w, vn.abs())
    mass = float((torch.matmul(q64.abs(), kt.abs()) * D ** -0.5).max())
    e = 2 * ((D + 8) * U * mass + 16 * U + 2.0 ** -21 + 2 * N * U)
    tol = (e + 2.0 ** -20) * spread + N * 2.0 ** -36 * float(vn.abs().max()) + 2.0 ** -11 * want.abs() + 2.0 ** -25
    assert ((out.double().reshape(B, N, D) - want).abs() <= tol).all()
    # a few sequences of it as a batch of their own
    few = [0, 1, 16383, 16384, 32766]
    t5 = table[few].contiguous()
    rows = torch.cat([torch.arange(b * N, b * N + N, device="cuda") for b in few])
    s5 = awq.KVSeqs(t5, cu[: len(few) + 1].contiguous(), lens[: len(few)].contiguous(), N, N)
    assert torch.equal(awq.awq_kv_attention(q[rows].contiguous(), cache, s5), out[rows])
