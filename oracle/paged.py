"""Rotary positions, the paged cache and attention over it -- oracle side (test infrastructure only).

Written from the definitions in float64, token by token:

* a sequence s has the new tokens of rows q_start[s] .. q_start[s+1]-1 and lens[s] tokens in all, the new ones
  last; its token at position c is in slot c % page of page table[s][c // page]; a page id outside [0, pages) is
  not there;
* pair j of a head turns by positions[axis(j)][t] * inv_freq[j];
* a row at position p sees c <= p (c < lens, page there), with a window only c > p - window or c < sinks; its
  output is the softmax-weighted mean of the visible V, zero when it sees nothing.
"""
from __future__ import annotations

import math

import numpy as np


def rows_of(q_start, lens, tokens):
    """(sequence, position) of every row; (-1, -1) for rows of no sequence."""
    out = [(-1, -1)] * tokens
    for s in range(len(lens)):
        for t in range(max(0, int(q_start[s])), min(tokens, int(q_start[s + 1]))):
            out[t] = (s, int(lens[s]) - (int(q_start[s + 1]) - t))
    return out


def slot(table, page, pages, s, c):
    """Row of the cache [pages * page, ...] holding position c of sequence s, or -1."""
    if c < 0 or c // page >= table.shape[1]:
        return -1
    i = int(table[s, c // page])
    return i * page + c % page if 0 <= i < pages else -1


def rotate(x, positions, inv_freq, sections, interleaved):
    """x [T, heads, d] float64 -> turned."""
    T, _, d = x.shape
    half = len(inv_freq)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    y = x.copy()
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        for t in range(T):
            a = float(positions[axis[j]][t]) * float(inv_freq[j])
            c, s = math.cos(a), math.sin(a)
            y[t, :, i0] = x[t, :, i0] * c - x[t, :, i1] * s
            y[t, :, i1] = x[t, :, i0] * s + x[t, :, i1] * c
    return y


def append(cache, new, table, q_start, lens):
    """cache [pages, page, heads, d] with the rows of ``new`` [T, heads, d] written to their slots."""
    pages, page = cache.shape[:2]
    out = cache.copy()
    flat = out.reshape((pages * page,) + cache.shape[2:])
    for t, (s, pos) in enumerate(rows_of(q_start, lens, new.shape[0])):
        at = -1 if s < 0 else slot(table, page, pages, s, pos)
        if at >= 0:
            flat[at] = new[t]
    return out


def visible(table, page, pages, s, pos, length, window, sinks):
    """Positions a row at ``pos`` of sequence s sees, and their slots."""
    cs = [c for c in range(0, min(pos + 1, length)) if not window or c > pos - window or c < sinks]
    pairs = [(c, slot(table, page, pages, s, c)) for c in cs]
    return [c for c, i in pairs if i >= 0], [i for _, i in pairs if i >= 0]


def attention(q, k_cache, v_cache, table, q_start, lens, scale, window=0, sinks=0):
    """Returns (out [T, hq, d], bound terms): see ``attention_tolerance``."""
    T, hq, d = q.shape
    pages, page, hkv, _ = k_cache.shape
    kf, vf = k_cache.reshape(-1, hkv, d), v_cache.reshape(-1, hkv, d)
    out = np.zeros((T, hq, d))
    mean_abs, score, vmax = np.zeros((T, hq, d)), np.zeros((T, hq)), np.zeros((T, hq, d))
    count = np.zeros((T,))
    for t, (s, pos) in enumerate(rows_of(q_start, lens, T)):
        slots = visible(table, page, pages, s, pos, int(lens[s]), window, sinks)[1] if s >= 0 else []
        count[t] = len(slots)
        if not slots:
            continue
        for h in range(hq):
            kh = h // (hq // hkv)
            K, V = kf[slots, kh], vf[slots, kh]
            with np.errstate(all="ignore"):
                z = scale * (K @ q[t, h])
                top = z.max()
                p = np.exp(z - (0.0 if top == -np.inf else top))
                if p.sum() == 0:
                    continue
                w = p / p.sum()
                out[t, h] = w @ V
                mean_abs[t, h] = w @ np.abs(V)
                score[t, h] = abs(scale) * (np.abs(K) @ np.abs(q[t, h])).max()
                vmax[t, h] = np.abs(V).max(0)
    return out, (mean_abs, score, vmax, count)


def attention_tolerance(y, terms, eps, min_normal):
    """Bound of |out - y| for 16-bit inputs and outputs, f32 scores and sums, and weights rounded to 16 bits.

    Half a step eps / 2 for the output; half a step for each weight, against the weighted mean of |v|; a score off
    by delta moves every weight by exp(+-delta), and the mean by at most 2 delta of it, where delta counts d + 8
    roundings (2^-24) of the products, the scale and the exponent's argument, on sum |q k| * scale + 1; the two
    sums of n terms take 2 n roundings; below the smallest normal number steps are absolute.
    """
    mean_abs, score, vmax, count = terms
    d = y.shape[-1]
    u = 2.0 ** -24
    delta = (d + 8) * u * (score + 1.0)[..., None]
    n = count[:, None, None]
    sub = eps * min_normal / 2
    return eps / 2 * np.abs(y) + (eps / 2 + 2 * delta + 2 * (n + 8) * u) * mean_abs + sub * (1 + n * vmax)


def rotate_tolerance(x, y, sections, interleaved, eps, min_normal):
    """Bound of |turned - y|: half a step of the output type, and 2^-21 of the pair's length for a sine and cosine
    off by 4 steps of 2^-24 each, the two products and the sum."""
    half = sum(sections)
    hyp = np.zeros_like(y)
    j = np.arange(half)
    i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    hyp[..., i0] = hyp[..., i1] = np.hypot(x[..., i0], x[..., i1])
    return eps / 2 * np.abs(y) + 2.0 ** -21 * hyp + np.where(hyp > 0, eps * min_normal / 2, 0.0)
