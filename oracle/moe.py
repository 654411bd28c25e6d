"""Mixture-of-experts feed-forward on W4A16 weights -- oracle side (test infrastructure only), token by token in float64."""
from __future__ import annotations

import numpy as np

from .linear import ACT, SLOPE
from .qkv import dequantize


def choose(x, router, top_k, normalize):
    """Chosen experts [t][top_k], best first, and their shares.  Every score is summed in the same order, so that equal
    rows of the router have equal scores; a score that is NaN comes last."""
    chosen, shares = [], []
    for row in x.astype(np.float64):
        with np.errstate(all="ignore"):
            z = (row * router.astype(np.float64)).sum(-1)
            order = sorted(range(len(z)), key=lambda e: (np.isnan(z[e]), -z[e] if not np.isnan(z[e]) else 0.0, e))[:top_k]
            part = np.exp(z - z[order[0]])
            chosen.append(order)
            shares.append(part[order] / (part[order].sum() if normalize else part.sum()))
    return chosen, shares


def moe(x, router, w_gate, s_gate, w_up, s_up, w_down, s_down, top_k, normalize=True, act="silu", residual=None):
    """(y, tolerance).  The tolerance: gate, up and down products 1e-5 of their sums of magnitudes (f32 accumulation) each,
    the first through the activation's slope; h 2^-19 for the activation, 2^-22 for its product, 2^-22 of itself and 2^-23
    of the row's largest for what is kept of it (csrc/moe_w4a16.hip); shares 2^-18 (a step of f32 for exp,
    the f32 sum of up to 512 of them, the quotient);
    f32 sums over experts and parts (1e-5); half a step of f16 for y."""
    t, hidden = x.shape
    chosen, shares = choose(x, router, top_k, normalize)
    y = np.zeros((t, hidden)) if residual is None else residual.astype(np.float64)
    total = np.abs(y) * 2.0 ** -23
    for e in sorted({e for c in chosen for e in c}):
        rows = [i for i in range(t) if e in chosen[i]]
        p = np.array([shares[i][chosen[i].index(e)] for i in rows])[:, None]
        g, u, d = dequantize(w_gate[e], s_gate[e]), dequantize(w_up[e], s_up[e]), dequantize(w_down[e], s_down[e])
        xr = x[rows].astype(np.float64)
        gate, up = xr @ g, xr @ u
        a = ACT[act](gate)
        h = a * up
        dh = (SLOPE * 1e-5 * (np.abs(xr) @ np.abs(g)) * np.abs(up) + np.abs(a) * 1e-5 * (np.abs(xr) @ np.abs(u)) +
              (2.0 ** -19 + 2.0 ** -21) * np.abs(h) + 2.0 ** -23 * np.abs(h).max(-1, keepdims=True))
        out = h @ d
        size = np.abs(h) @ np.abs(d)
        y[rows] += p * out
        total[rows] += p * (dh @ np.abs(d) + 1e-5 * size + 2.0 ** -18 * np.abs(out) + 1e-5 * size)
    return y, total + 2.0 ** -11 * np.abs(y) + 2.0 ** -25
