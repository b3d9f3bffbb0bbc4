"""Decoder-layer operators in float64: the norm of the residual stream, groups
in 8 bits, the paged cache and causal attention over it.  Test infrastructure:
plain loops over the definitions, no shortcut shared with the kernels."""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
HOLD = 240.0 * 2.0 ** 120      # largest magnitude a group keeps


def bf16_values(bits: np.ndarray) -> np.ndarray:
    """float64 values of bf16 bit patterns."""
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_table() -> np.ndarray:
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 of mantissa;
    0x7F and 0xFF are NaN, there are no infinities."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if b & 127 == 127:
            mag = math.nan
        out[b] = -mag if b & 128 else mag
    return out


_TABLE = e4m3_table()
_POS = _TABLE[:127]            # 0 .. 448, rising


def e4m3_bits(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 of values up to 448 in magnitude, ties to the even pattern."""
    a = np.abs(x)
    i = np.clip(np.searchsorted(_POS, a, side="right") - 1, 0, 126)
    j = np.minimum(i + 1, 126)
    lo, hi = a - _POS[i], _POS[j] - a
    up = (hi < lo) | ((hi == lo) & (i % 2 == 1) & (j > i))
    b = np.where(up, j, i).astype(np.uint8)
    b = np.where(np.isnan(x), 127, b).astype(np.uint8)
    return (b | np.where(np.signbit(x), 128, 0).astype(np.uint8)).astype(np.uint8)


def scale_exponent(amax: np.ndarray) -> np.ndarray:
    """The smallest e with amax <= 448 * 2^e, within -120..120; -120 for 0."""
    e = np.full(amax.shape, -120, np.int64)
    for idx in np.ndindex(amax.shape):
        a = float(amax[idx])
        while e[idx] < 120 and a > E4M3_MAX * 2.0 ** int(e[idx]):
            e[idx] += 1
    return e


def quantise(x: np.ndarray):
    """(e4m3 bytes, scale bytes) of groups along the last dimension.  NaN has
    no part in a group's scale."""
    x = np.where(np.isnan(x), x, np.clip(x, -HOLD, HOLD))
    amax = np.max(np.where(np.isnan(x), 0.0, np.abs(x)), axis=-1)
    e = scale_exponent(amax)
    q = e4m3_bits(x / np.exp2(e.astype(np.float64))[..., None])
    return q, (e + 127).astype(np.uint8)


def dequantise(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return _TABLE[q] * np.exp2(scale.astype(np.float64) - 127.0)[..., None]


def rms_norm(x, weight, eps, residual=None):
    """(y, h) in float64."""
    h = x if residual is None else x + residual
    return h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * weight, h


def cache_row(slot: int, page: int):
    return slot // page, slot % page


def paged_attention(q, k, v, table, cu_q, kv_len, window=0, scale=None):
    """(out, sum of probability times |v|) in float64.  q [tokens, heads, dim];
    k, v [pages, kv_heads, page, dim]; the loops follow the definition."""
    tokens, heads, dim = q.shape
    _, kv_heads, page, _ = k.shape
    g = heads // kv_heads
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(kv_len)):
        n, m = int(cu_q[b + 1] - cu_q[b]), int(kv_len[b])
        for i in range(n):
            p = m - n + i
            lo = max(0, p - window + 1) if window else 0
            keys = np.arange(lo, p + 1)
            if not len(keys):
                continue
            pages, at = table[b][keys // page], keys % page
            for h in range(heads):
                kk, vv = k[pages, h // g, at], v[pages, h // g, at]
                z = kk @ q[cu_q[b] + i, h] * scale
                w = np.exp(z - z.max())
                w /= w.sum()
                out[cu_q[b] + i, h] = w @ vv
                mag[cu_q[b] + i, h] = w @ np.abs(vv)
    return out, mag
