"""CPU oracle of the paged 8-bit key / value cache and the attention over it
(NumPy; imports nothing of the library).

The write is done in IEEE float32 step by step as include/awq.h states it, so
codes and scales compare bit for bit; the attention is float64 from the exact
stored numbers. A cache here is [pages, heads, page, D] int/float numbers (the
stored codes without scale) plus fp32 scales; `store_k` / `store_v` give the
byte layouts of the library's tensors.
"""

from __future__ import annotations

import numpy as np

TOP = {"int8": np.float32(127.0), "e4m3": np.float32(448.0)}
FLOOR = np.float32(1e-5)


def e4m3_round(v):
    """float32/64 -> nearest e4m3 value (ties to even), |v| <= 464."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(divide="ignore"):
        exp = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = 2.0 ** (exp - 3)
    return np.rint(v / step) * step


def e4m3_bits(v):
    """Exact e4m3 values -> their bytes."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    exp = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    normal = a >= 2.0 ** -6
    mant = np.where(normal, a / 2.0 ** exp * 8 - 8, a / 2.0 ** -9)
    code = np.where(normal, (exp + 7) * 8 + mant, mant).astype(np.int64)
    return (code | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def e4m3_value(b):
    """Bytes -> e4m3 values (the NaN codes 0x7f, 0xff as nan)."""
    b = np.asarray(b, dtype=np.int64)
    exp, mant = (b >> 3) & 15, b & 7
    v = np.where(exp == 0, mant * 2.0 ** -9, (8 + mant) * 2.0 ** (exp - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def to_code(v, fmt):
    """float32 scaled values -> the format's numbers (int8 codes or e4m3 values)."""
    v = np.clip(np.asarray(v, dtype=np.float32), -TOP[fmt], TOP[fmt])
    return np.rint(v).astype(np.float64) if fmt == "int8" else e4m3_round(v)


def to_bytes(codes, fmt):
    return (codes + 128).astype(np.uint8) if fmt == "int8" else e4m3_bits(codes)


def from_bytes(b, fmt):
    return b.astype(np.float64) - 128 if fmt == "int8" else e4m3_value(b)


def store_k(t):
    p, h, n, d = t.shape
    return np.ascontiguousarray(t.reshape(p, h, n, d // 16, 16).transpose(0, 1, 3, 2, 4))


def load_k(t):
    p, h, dc, n, _ = t.shape
    return np.ascontiguousarray(t.transpose(0, 1, 3, 2, 4)).reshape(p, h, n, dc * 16)


def store_v(t):
    p, h, n, d = t.shape
    return np.ascontiguousarray(t.reshape(p, h, n // 16, 16, d).transpose(0, 1, 2, 4, 3))


def load_v(t):
    p, h, nc, d, _ = t.shape
    return np.ascontiguousarray(t.transpose(0, 1, 2, 4, 3)).reshape(p, h, nc * 16, d)


def positions(table, cu, kv_len, page, n_pages):
    """Per row of the token tensors: (row, sequence, position, page id or -1)."""
    out = []
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            pos = kv_len[b] - n + i
            pid = -1
            if pos >= 0:
                pid = int(table[b][pos // page])
                if not 0 <= pid < n_pages:
                    pid = -1
            out.append((cu[b] + i, b, pos, pid))
    return out


def write(codes, scales, x, table, cu, kv_len, fmt):
    """New rows x [T, H, D] (fp16) into codes [pages, H, page, D] (numbers) and
    scales [pages, H], in place."""
    page = codes.shape[2]
    x = np.asarray(x, dtype=np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-65504), np.float32(65504)))
    todo = {}
    for row, b, pos, pid in positions(table, cu, kv_len, page, codes.shape[0]):
        if pos >= 0 and pid >= 0:
            todo.setdefault((b, pos // page, pid), []).append((pos % page, row))
    for (_, _, pid), rows in todo.items():
        slots = np.array([s for s, _ in rows])
        new = x[[r for _, r in rows]]                               # [n, H, D]
        t0 = int(slots.min())
        put = np.maximum(np.abs(new).max(axis=(0, 2)), FLOOR) / TOP[fmt]
        old = scales[pid].copy()
        s = np.maximum(old, put) if t0 > 0 else put
        inv = np.float32(1) / s
        for h in range(codes.shape[1]):
            if t0 > 0 and s[h] > old[h]:
                shrink = old[h] * inv[h]
                codes[pid, h, :t0] = to_code(codes[pid, h, :t0].astype(np.float32) * shrink, fmt)
            codes[pid, h, slots] = to_code(new[:, h] * inv[h], fmt)
        scales[pid] = s


def read(codes, scales, out, table, cu, kv_len):
    """fp16(code * scale) of the newest tokens into out [T, H, D]."""
    page = codes.shape[2]
    for row, b, pos, pid in positions(table, cu, kv_len, page, codes.shape[0]):
        out[row] = 0 if pid < 0 else (codes[pid, :, pos % page].astype(np.float32) *
                                      scales[pid][:, None]).astype(np.float16)


def attention(q, k_codes, k_scales, v_codes, v_scales, table, cu, kv_len, scale, causal=True, window=0):
    """float64 (out, lse, spread, logit_mass): the outputs [T, Hq, D], the
    log-sum-exp [T, Hq], sum_j w_j |v_j| (what a relative error of the weights
    is multiplied by) and max_j scale * sum_d |q_d k_jd| (what one of the
    logits' is)."""
    T, hq, d = q.shape
    pages, heads, page, _ = k_codes.shape
    r = hq // heads
    out, spread = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, mass = np.full((T, hq), -np.inf), np.zeros((T, hq))
    q = np.asarray(q, dtype=np.float64)
    for b in range(len(kv_len)):
        L, n = int(kv_len[b]), int(cu[b + 1] - cu[b])
        ids = [int(table[b][p]) for p in range(-(-L // page))]
        ok = np.repeat([0 <= i < pages for i in ids], page)[:L].astype(bool) if L else np.zeros(0, bool)
        safe = [i if 0 <= i < pages else 0 for i in ids]
        for h in range(heads):
            if L:
                k = (k_codes[safe, h] * k_scales[safe, h].astype(np.float64)[:, None, None]).reshape(-1, d)[:L]
                v = (v_codes[safe, h] * v_scales[safe, h].astype(np.float64)[:, None, None]).reshape(-1, d)[:L]
            for i in range(n):
                pos = L - n + i
                j = np.arange(L)
                see = ok.copy()
                if causal:
                    see &= j <= pos
                if window:
                    see &= j > pos - window
                if not see.any():
                    continue
                kk, vv = k[see], v[see]
                for g in range(r):
                    row, head = cu[b] + i, h * r + g
                    t = scale * (kk @ q[row, head])
                    mx = t.max()
                    w = np.exp(t - mx)
                    lse[row, head] = mx + np.log(w.sum())
                    w /= w.sum()
                    out[row, head] = w @ vv
                    spread[row, head] = w @ np.abs(vv)
                    mass[row, head] = abs(scale) * (np.abs(kk) @ np.abs(q[row, head])).max()
    return out, lse, spread, mass
