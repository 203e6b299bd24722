"""CPU oracle of the operators between a decoder layer's linear layers: the
root-mean-square norm, rotary positions, and the 4-bit key / value cache (NumPy;
imports nothing of the library).

The cache's write is done in IEEE float32 step by step as include/awq.h states
it, so codes and scales compare bit for bit; everything else is float64. A 4-bit
cache here is codes [pages, heads, page, D] (0 .. 15) with steps and smallest
numbers, fp16: keys [pages, heads, page, D / 32, 2], values [pages, heads, page,
2]; `store_*` and `load_*` give the byte layouts of the library's tensors.
"""

from __future__ import annotations

import math

import numpy as np

from . import kv_oracle

NIBBLES = (0, 2, 4, 6, 1, 3, 5, 7)      # the code of each nibble of a word


# ---------------------------------------------------------------- norm

def rmsnorm(x, weight=None, eps=1e-5, residual=None, offset=0.0):
    """float64 (h, y)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    if weight is not None:
        y = y * (np.float64(np.float32(offset)) + np.asarray(weight, np.float64))
    return h, y


def norm_scales(y, fmt, group=0):
    """float64 scales [T, K / group or 1] of y."""
    T, K = y.shape
    top = np.abs(y).reshape(T, -1, group or K).max(-1)
    return np.maximum(top, 1e-5) / (127.0 if fmt == "int8" else 448.0)


# ---------------------------------------------------------------- rotary positions

def rope_frequencies(r, base=10000.0, scaling="none", factor=1.0, length=0.0, low=1.0, high=None):
    """([r / 2] radians per position, amplitude) by the written formulas."""
    high = (32.0 if scaling == "yarn" else 4.0) if high is None else high
    i = np.arange(r // 2)
    f = np.power(base * factor ** (r / (r - 2.0)) if scaling == "ntk" else base, -2.0 * i / r)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        ends = [r * math.log(length / (2 * math.pi * t)) / (2 * math.log(base)) for t in (high, low)]
        a, b = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), r - 1)
        ramp = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "wavelength":
        keep = np.clip((length / (2 * math.pi / f) - low) / (high - low), 0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    return f, 1.0


def rope(x, positions, freqs, layout="half", amplitude=1.0):
    """float64 [T, heads, D] of x rotated; and |a| + |b| of every element's pair."""
    x = np.asarray(x, np.float64)
    r = 2 * len(freqs)
    z = np.exp(1j * np.asarray(positions, np.float64)[:, None] * freqs)[:, None] * amplitude
    a, b = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    y, size = x.copy(), np.zeros_like(x)
    w = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = w.real, w.imag
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


# ---------------------------------------------------------------- the 4-bit cache

def groups4(x):
    """Groups x [..., n] (finite fp16 numbers) -> codes [..., n], (s, lo) [..., 2]."""
    x = np.asarray(x, np.float32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    want = (hi - lo) / np.float32(15)
    s = want.astype(np.float16)
    s = np.where(s.astype(np.float32) > want, np.nextafter(s, np.float16(0)), s)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((x - lo) / s.astype(np.float32))
    codes = np.where(s > 0, np.clip(q, 0, 15), 0).astype(np.uint8)
    return codes, np.concatenate([s, lo.astype(np.float16)], -1)


def numbers4(codes, s_lo):
    """The cached numbers fp16(lo + s c) of groups: the sum is exact in float64."""
    s, lo = s_lo[..., :1].astype(np.float64), s_lo[..., 1:].astype(np.float64)
    return (lo + s * codes).astype(np.float16)


def k_numbers(codes, scales):
    g = codes.reshape(*codes.shape[:-1], -1, 32)
    return numbers4(g, scales).reshape(codes.shape)


def v_numbers(codes, scales):
    return numbers4(codes, scales)


def finite(x):
    x = np.asarray(x, np.float16).astype(np.float32)
    return np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-65504), np.float32(65504)))


def write(codes, scales, x, table, cu, kv_len, side):
    """New rows x [T, H, D] (fp16) into the cache of one side ("k" or "v"), in place."""
    page = codes.shape[2]
    x = finite(x)
    g = x.reshape(*x.shape[:-1], -1, 32) if side == "k" else x
    c, s = groups4(g)
    c = c.reshape(x.shape)
    for row, _, pos, pid in kv_oracle.positions(table, cu, kv_len, page, codes.shape[0]):
        if pos >= 0 and pid >= 0 and row < len(x):
            codes[pid, :, pos % page] = c[row]
            scales[pid, :, pos % page] = s[row]


def read(codes, scales, out, table, cu, kv_len, side):
    """The cached numbers of the newest tokens into out [T, H, D]."""
    page = codes.shape[2]
    for row, _, pos, pid in kv_oracle.positions(table, cu, kv_len, page, codes.shape[0]):
        if pid < 0:
            out[row] = 0
        else:
            f = k_numbers if side == "k" else v_numbers
            out[row] = f(codes[pid, :, pos % page], scales[pid, :, pos % page])


def attention(q, kc, ks, vc, vs, table, cu, kv_len, scale, causal=True, window=0):
    """As kv_oracle.attention, over the 4-bit cache's numbers."""
    one = np.ones(kc.shape[:2])
    return kv_oracle.attention(q, k_numbers(kc, ks).astype(np.float64), one, v_numbers(vc, vs).astype(np.float64), one,
                               table, cu, kv_len, scale, causal, window)


def to_nibbles(codes):
    """[..., 8 n] codes -> [..., 4 n] bytes."""
    c = codes.astype(np.uint8).reshape(*codes.shape[:-1], -1, 8)[..., list(NIBBLES)]
    c = c.reshape(*c.shape[:-1], 4, 2)
    return (c[..., 0] | (c[..., 1] << 4)).reshape(*codes.shape[:-1], -1)


def from_nibbles(b):
    c = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1, 8)
    out = np.empty_like(c)
    out[..., list(NIBBLES)] = c
    return out.reshape(*b.shape[:-1], -1)


def store_k(codes):
    p, h, n, d = codes.shape
    return np.ascontiguousarray(to_nibbles(codes.reshape(p, h, n, d // 32, 32)).transpose(0, 1, 3, 2, 4))


def load_k(b):
    c = from_nibbles(b).transpose(0, 1, 3, 2, 4)
    return np.ascontiguousarray(c).reshape(*c.shape[:3], -1)


def load_k_scales(s):
    return np.ascontiguousarray(s.transpose(0, 1, 3, 2, 4))


def store_v(codes):
    p, h, n, d = codes.shape
    return to_nibbles(np.ascontiguousarray(codes.reshape(p, h, n // 32, 32, d).transpose(0, 1, 2, 4, 3)))


def load_v(b):
    c = from_nibbles(b).transpose(0, 1, 2, 4, 3)
    return np.ascontiguousarray(c).reshape(c.shape[0], c.shape[1], -1, c.shape[4])


def load_v_scales(s):
    return np.ascontiguousarray(s.transpose(0, 1, 3, 2))
