"""Rotary positions in float64 (test infrastructure only).

The first 2 * len(inv_freq) dims of a head form pairs; pair i of a token at position p is
turned by p * inv_freq[i] (the fp32 table read as exact numbers) and scaled by `amplitude`.
Half layout: dims (i, i + half); interleaved: dims (2 i, 2 i + 1). Other dims are copied.
"""
from __future__ import annotations

import math

import numpy as np


def rotate(x: np.ndarray, positions, inv_freq, interleaved: bool, amplitude: float = 1.0):
    """x float64 [T, H, D] -> float64, unrounded."""
    y = np.array(x, dtype=np.float64, copy=True)
    f = np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    amp = float(np.float32(amplitude))
    h = len(f)
    for t, p in enumerate(np.asarray(positions)):
        for i in range(h):
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
            ang = math.fmod(int(p) * f[i], 2.0 * math.pi)
            c, s = amp * math.cos(ang), amp * math.sin(ang)
            a, b = x[t, :, ia].astype(np.float64), x[t, :, ib].astype(np.float64)
            y[t, :, ia], y[t, :, ib] = a * c - b * s, b * c + a * s
    return y


def inv_freq(rot_dim: int, base: float, scaling: str = "none", factor: float = 1.0,
             original_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(float64 table, amplitude): base^(-2 i / rot_dim), stretched for longer contexts."""
    half = rot_dim // 2
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = np.array([base ** (-2.0 * i / rot_dim) for i in range(half)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":
        # the pair that makes n turns within the original context: original / wavelength = n
        # with wavelength = 2 pi base^(2 i / rot_dim), solved for i
        def pair(n):
            return rot_dim / 2 * math.log(original_context / (2 * math.pi * n), base)
        lo, hi = pair(beta_fast), pair(beta_slow)
        ramp = np.clip((np.arange(half) - lo) / (hi - lo), 0.0, 1.0)
        return f * (1 - ramp) + f / factor * ramp, 1.0 + 0.1 * math.log(factor)
    return f, 1.0
