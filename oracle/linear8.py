"""Rows rounded to 8 bits and the 8-bit product with its epilogue -- oracle side (test infrastructure only).

    quantize:  scale = max |row| / 127,  q = round(127 x / max |row|), ties to even
    linear:    y = act(xs ws (xq . wq^T) + b) + r, sums in whole numbers, the rest in float64
"""
from __future__ import annotations

import numpy as np

from .linear import ACT, SLOPE


def quantize(x):
    """(q int8, scale f32) of x [m, k], given as float64 with the values of f16 or bf16 numbers.

    127 x is exact in float64, and the quotient's distance from any n + 1/2 that it does not equal is over 2^-32 of it, so
    its rounding to float64 does not carry it across; nor does that of a / 127 across a border between f32 numbers.
    """
    a = np.abs(x).max(-1, initial=0.0)
    fine = np.isfinite(a)
    safe = np.where(fine & (a > 0), a, 1.0)[:, None]
    q = np.where((fine & (a > 0))[:, None], np.rint(127 * np.where(fine[:, None], x, 0.0) / safe), 0.0)
    return q.astype(np.int8), np.where(fine, a / 127, np.nan).astype(np.float32)


def linear(xq, xs, wq, ws, bias=None, act="none", residual=None):
    """(y, z, p): the result, the activation's argument and the scaled product."""
    total = xq.astype(np.int64) @ wq.astype(np.int64).T
    p = total.astype(np.float64) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    z = p if bias is None else p + bias
    y = ACT[act](z)
    return (y if residual is None else y + residual), z, p


def tolerance(y, z, p, act, half_step, low, bias=None, residual=None):
    """half_step of the result (2^-11 f16, 2^-8 bf16) and `low` below its normal numbers; through the activation's slope
    the f32 roundings of the sum, of its two scalings and of the sum with the bias; of the activation's value 2^-19, growing
    past arguments of 32 as their f32 step does (its exponential or erfc); one f32 rounding of the sum with the residual."""
    a = ACT[act](z)
    b = 0.0 if bias is None else np.abs(bias)
    r = 0.0 if residual is None else np.abs(residual)
    return (half_step * np.abs(y) + low + SLOPE * 2.0 ** -24 * (4 * np.abs(p) + b) +
            2.0 ** -19 * np.abs(a) * (1 + np.abs(z) / 32) + 2.0 ** -24 * (np.abs(a) + r))
