"""Attention over positions that no query of the call sees and that nobody has
written: behind the rows that a token tensor holds where cu_tokens names more,
behind those that max_tokens leaves over, and before every query's window. What
such a place holds (NaN codes, steps and scales that are NaN or infinite) changes
no row.

Attention's bounds are test_gpu_kv's and test_gpu_kv4's.
"""

import numpy as np
import pytest

from oracle import kv_oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

import test_gpu_kv as kv8  # noqa: E402
import test_gpu_kv4 as kv4  # noqa: E402
from test_gpu_parity import dev, host, say  # noqa: E402

FORMATS = ["int4", "e4m3", "int8"]
GARBAGE = [float("nan"), float("inf")]


def model(fmt, seed, n_seqs, heads, dim, page, max_len, garbage):
    if fmt == "int4":
        m = kv4.Model(seed, n_seqs, heads, dim, page, max_len)
    else:
        m = kv8.Model(seed, n_seqs, heads, dim, page, fmt, max_len)
    m.cache.k_scales.fill_(garbage)
    m.cache.v_scales.fill_(garbage)
    return m


def want_of(m, fmt, q, cu, lens, window):
    if fmt == "int4":
        return m.want(q, m.table, cu, lens, m.dim ** -0.5, True, window)
    return kv_oracle.attention(q, m.kc, m.ks, m.vc, m.vs, m.table, cu, lens, m.dim ** -0.5, True, window)


def check(m, fmt, new, here, bound, rows, ratio, window=0, max_len=None, split=True):
    """A batch of `new` tokens a sequence of which `here` are written (the model
    holds them as its newest), bounded by `bound`, the tensors holding `rows`
    rows: the rows of the tokens in `here` as the oracle's, the others as they
    were."""
    new, here = np.asarray(new), np.asarray(here)
    lens = m.len + new - here
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s = awq.KVSeqs(dev(m.table), dev(cu), dev(lens.astype(np.int32)), int(bound),
                   int(lens.max()) if max_len is None else max_len)
    q = m.rng.standard_normal((rows, m.heads * ratio, m.dim)).astype(np.float16)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = awq.kv_attention_workspace(m.cache, s, m.heads * ratio) if split else None
    awq.awq_kv_attention(dev(q), m.cache, s, window=window, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    mine = np.concatenate([cu[b] + np.arange(n) for b, n in enumerate(here)]).astype(int)
    want = want_of(m, fmt, q[mine], np.concatenate([[0], np.cumsum(here)]), m.len, window)
    m.assert_attention((host(out)[mine], host(lse)[mine], want), int(m.len.max()))
    others = np.setdiff1d(np.arange(rows), mine)
    assert (host(out)[others] == 7).all() and (host(lse)[others] == 7).all()


SHAPES = [      # dim, page, heads, ratio, tokens held before, new ones
    (64, 32, 2, 2, [50, 31, 90], [3, 8, 4]),            # a block of 16 rows
    (128, 64, 1, 1, [1000, 33, 64], [1, 12, 1]),        # parts to join
    (128, 64, 2, 8, [7, 60, 0], [4, 4, 4]),             # two blocks of 16 rows
    (256, 32, 1, 4, [40, 64, 0], [2, 7, 1]),
    (96, 32, 2, 3, [70, 129, 5], [40, 100, 9]),         # 128 rows a block
    (192, 128, 1, 1, [10, 120, 300], [70, 200, 3]),
    (64, 64, 1, 2, [3, 64, 700], [1, 90, 64]),
]


@pytest.mark.parametrize("garbage", GARBAGE)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,page,heads,ratio,held,new", SHAPES)
def test_rows_that_are_not_there(dim, page, heads, ratio, held, new, fmt, garbage):
    """Tensors with fewer rows than cu_tokens names: the tokens behind them were
    never written."""
    for have in (1, new[1] // 2, new[1] - 1):
        rows = new[0] + have
        say("unseen rows", fmt, garbage, dim, page, new, rows)
        m = model(fmt, [81, dim, have], 3, heads, dim, page, max(h + n for h, n in zip(held, new)), garbage)
        here = [new[0], have, 0]
        m.append(np.array(held) + here)
        check(m, fmt, new, here, max(new), rows, ratio)
        check(m, fmt, new, here, max(new), rows, ratio, window=20, split=False)


@pytest.mark.parametrize("garbage", GARBAGE)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,page,heads,ratio,held,new", SHAPES)
def test_a_bound_below_the_tokens(dim, page, heads, ratio, held, new, fmt, garbage):
    """New tokens past max_tokens: not written, not processed, in the way of nobody."""
    for bound in {1, max(1, max(new) // 3), max(1, max(new) - 1)}:
        say("unseen tokens", fmt, garbage, dim, page, new, bound)
        m = model(fmt, [82, dim, bound], 3, heads, dim, page, max(h + n for h, n in zip(held, new)), garbage)
        here = np.minimum(new, bound)
        m.append(np.array(held) + here)
        check(m, fmt, new, here, bound, sum(new), ratio)
        check(m, fmt, new, here, bound, sum(new), ratio, window=9, split=False)


@pytest.mark.parametrize("garbage", GARBAGE)
@pytest.mark.parametrize("page", [32, 64])
def test_blocks_of_thirty_two_rows(page, garbage):
    """The same over the 4-bit cache where 17 to 32 rows are one block's."""
    say("unseen, 32 rows", page, garbage)
    bound = 2 ** 16             # 32 kv heads of 2^16 positions
    held, new = [700, 0, 1, 64, 333, 30, 31, 96], [6, 6, 1, 6, 6, 6, 0, 6]
    lens = [h + n for h, n in zip(held, new)]
    m = model("int4", [83, page], 8, 4, 128, page, max(lens), garbage)
    here = np.minimum(new, [6, 6, 1, 6, 2, 0, 0, 0])
    m.append(np.array(held) + here)
    check(m, "int4", new, here, 6, int(here.sum()), 4, max_len=bound)
    m = model("int4", [84, page], 8, 4, 128, page, max(lens), garbage)
    here = np.minimum(new, 5)
    m.append(np.array(held) + here)
    check(m, "int4", new, here, 5, sum(new), 4, max_len=bound)


@pytest.mark.parametrize("garbage", GARBAGE)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [32, 64, 256])
@pytest.mark.parametrize("new", [1, 9, 90])
def test_nothing_before_the_window(new, page, fmt, garbage):
    """A sequence whose first tokens were never written, its first written one
    the first that any window reaches."""
    W = 21
    say("unseen before the window", fmt, garbage, page, new)
    for first in (0, 32, 45, 63):
        n = W + new - 1
        m = model(fmt, [85, page, new], 1, 2, 64, page, first + n, garbage)
        if fmt != "int4":
            # a page written from its middle keeps what its scale was
            m.cache.k_scales.fill_(0.0)
            m.cache.v_scales.fill_(0.0)
            for p in range(first // page):
                m.cache.k_scales[m.table[0, p]] = garbage
                m.cache.v_scales[m.table[0, p]] = garbage
        m.len[:] = first
        m.append([n])
        q = m.rng.standard_normal((new, 4, 64)).astype(np.float16)
        for split in (True, False):
            m.assert_attention(m.attend(q, [new], window=W, split=split), n)
