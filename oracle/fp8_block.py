"""e4m3 KV cache with one scale per (block, kv head): append and decode (test infrastructure).

  * a row at offset 0 starts a block afresh;
  * scale = the smallest power of two >= 2^-126 with |x| <= 448 * scale over the finite values
    of the rows since then, never smaller than it was;
  * code = e4m3(x / scale), nearest even, saturated (infinities too; NaN gives a NaN code);
  * rows already there when the scale grows: code' = e4m3(value(code) * old / new).
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .fp8 import E4M3_MAX, e4m3_to_float
from .paged_attention import bf16_bits_to_f64, softmax_attention

LUT = np.array([e4m3_to_float(c) for c in range(256)], dtype=np.float64)


def needed_scale(values: np.ndarray) -> float:
    """Smallest power of two >= 2^-126 whose product with 448 is not below any finite |value|."""
    v = np.abs(np.asarray(values, np.float64))
    v = v[np.isfinite(v)]
    top = Fraction(float(v.max())) if v.size else Fraction(0)
    k = -126
    while Fraction(E4M3_MAX) * Fraction(2) ** k < top:
        k += 1
    return math.ldexp(1.0, k)



def encode(y: np.ndarray) -> np.ndarray:
    """e4m3 codes of float64 values: by nearest neighbour on the grid, ties to the even code."""
    y = np.asarray(y, np.float64)
    flat = y.reshape(-1)
    out = np.zeros(flat.shape, np.uint8)
    grid = LUT[:0x7F]                       # values of the codes 0x00 .. 0x7E, rising
    a = np.minimum(np.abs(np.where(np.isnan(flat), 0.0, flat)), E4M3_MAX)
    hi = np.clip(np.searchsorted(grid, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a     # exact: both have few bits
    pick = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(hi % 2 == 0, hi, lo)))
    out = pick.astype(np.uint8) | np.where(np.signbit(flat), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(flat), 0x7F, out).astype(np.uint8).reshape(y.shape)


def append(codes, scales, x, block_tables, cu, ctx):
    """Copies of (codes [nb, bs, Hkv, D], scales [nb, Hkv]) after the rows x (bf16 bits
    [T, Hkv, D]) were appended as the last positions of each sequence's context."""
    codes, scales = np.array(codes, copy=True), np.array(scales, np.float32, copy=True)
    xf = bf16_bits_to_f64(x)
    bs, hkv = codes.shape[1], codes.shape[2]
    for s in range(len(ctx)):
        t, end = int(cu[s]), int(cu[s + 1])
        p = int(ctx[s]) - (end - t)
        while t < end:
            b, r = int(block_tables[s, p // bs]), p % bs
            n = min(bs - r, end - t)
            for g in range(hkv):
                rows = xf[t:t + n, g]
                need = needed_scale(rows)
                old = float(scales[b, g]) if r else 0.0
                new = max(old, need)
                if r and new != old:
                    codes[b, :r, g] = encode(LUT[codes[b, :r, g]] * (old / new))
                codes[b, r:r + n, g] = encode(rows / new)
                scales[b, g] = new
            t, p = t + n, p + n
    return codes, scales


def dequantize(codes, scales):
    return LUT[np.asarray(codes, np.uint8)] * np.asarray(scales, np.float64)[:, None, :, None]


def decode(q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, scale):
    """Textbook float64 attention of the values the pools hold."""
    B, Hq, D = q.shape
    nb, bs, Hkv, _ = np.asarray(k_codes).shape
    G = Hq // Hkv
    qf = bf16_bits_to_f64(q)
    scale = float(np.float32(scale))
    out = np.zeros((B, Hq, D))
    for s in range(B):
        ctx = int(context_lens[s])
        if ctx <= 0:
            continue
        blocks = np.asarray(block_tables[s, : -(-ctx // bs)], np.int64)
        K = dequantize(k_codes[blocks], k_scales[blocks]).reshape(-1, Hkv, D)[:ctx]
        V = dequantize(v_codes[blocks], v_scales[blocks]).reshape(-1, Hkv, D)[:ctx]
        for h in range(Hq):
            out[s, h] = softmax_attention(qf[s, h], K[:, h // G], V[:, h // G], scale)
    return out
