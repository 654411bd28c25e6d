"""W4A16 product with bias, activation and residual -- oracle side (test infrastructure only).

    y = act(x . w + b) + r,   w[k, n] = int4(W, k, n) * S[k // 128, n],   all in float64
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc, expit

from .qkv import dequantize

ACT = {
    "none": lambda z: z,
    "relu": lambda z: np.where(z < 0, 0.0, z),
    "gelu": lambda z: z * erfc(-z / np.sqrt(2.0)) / 2,
    "gelu_tanh": lambda z: z * expit(2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)),
    "silu": lambda z: z * expit(z),
}
SLOPE = 1.13      # the largest slope of any of them (gelu at sqrt 2: 1.129)


def linear(x, w, s, bias=None, act="none", residual=None):
    """(y, z, t): the result, the activation's argument and sum |x w| + |b|."""
    wd = dequantize(w, s)
    xd = x.astype(np.float64)
    z, t = xd @ wd, np.abs(xd) @ np.abs(wd)
    if bias is not None:
        z, t = z + bias.astype(np.float64), t + np.abs(bias.astype(np.float64))
    y = ACT[act](z)
    if residual is not None:
        y = y + residual.astype(np.float64)
    return y, z, t


def tolerance(y, z, t, act, residual=None):
    """Half a step of f16 (2^-11, below 2^-14 an absolute 2^-25); the f32 accumulation, 1e-5 of sum |x w| + |b|, through
    the activation's slope; 2^-19 of the activation's value for its exponential or erfc (an f32 argument of up to 32
    significant in units of 2^-24); one f32 rounding of the sum with the residual."""
    a = ACT[act](z)
    r = 0.0 if residual is None else np.abs(residual.astype(np.float64))
    return 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + SLOPE * 1e-5 * t + 2.0 ** -19 * np.abs(a) + 2.0 ** -24 * (np.abs(a) + r)
