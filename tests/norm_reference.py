"""Norm and rotation of heads in 64 bits, with the terms of the error bounds, for the tests.

Written from the formulas of include/dflash.h; shares no code with the library."""
from __future__ import annotations

import numpy as np

import cache_reference as R


def norm_error(hd):
    """Relative error of x / sqrt(mean(x^2) + eps) in fp32: hd squares summed (half of their
    error under the root), a reciprocal root within two steps, one product."""
    return hd / 2 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -24


def forward(x, w, pos, eps, layout, rd, freqs, m, half):
    """-> y, bound of its error (x [T][heads][hd], 64 bits; half: half a step of the type)"""
    hd = x.shape[-1]
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y, size = R.rope(n * w, pos, layout, rd, freqs, m)
    # the norm's and the weight product's errors, then the turn's 4e-7 (test_gpu_cache.py)
    return y, size * (norm_error(hd) + 2.0 ** -24 + 4e-7) + half * np.abs(y) * 1.01 + 1e-38


def backward(x, w, dy, pos, eps, layout, rd, freqs, m, half, depth):
    """-> dx, its bound, dw, its bound (depth: most fp32 additions that a term of dw goes through)"""
    hd, e = x.shape[-1], norm_error(x.shape[-1])
    inv = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * inv
    g, size = R.rope(dy, pos, layout, rd, freqs, m, True)
    dn, dn_err = g * w, size * np.abs(w) * (4e-7 + 2.0 ** -24)
    dot = (dn * n).mean(-1, keepdims=True)
    dot_err = (dn_err * np.abs(n) + np.abs(dn * n) * (e + (hd + 2) * 2.0 ** -24)).mean(-1, keepdims=True)
    dx = inv * (dn - n * dot)
    err = inv * (dn_err + np.abs(n) * dot_err + np.abs(n * dot) * (e + 2.0 ** -23) + (np.abs(dn) + np.abs(n * dot)) * (e + 2.0 ** -23))
    dw = (g * n).sum((0, 1))
    dw_err = (size * np.abs(n) * (4e-7 + e) + np.abs(g * n) * (depth + 1) * 2.0 ** -24).sum((0, 1))
    return dx, err + half * np.abs(dx) * 1.01 + 1e-38, dw, dw_err
