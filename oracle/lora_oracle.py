"""CPU oracle (numpy, fp64) of the low-rank adapters beside the experts'
projections, row by row, with bounds of what fp32 sums may lose.

Pinned by tests/test_lora_cpu.py: hand-worked adapters of rank one, and the
merged weights W + s B A.

`pairs[d][e]` is adapter d's (A, B, scale) for expert e (shared experts behind
the routed ones) in fp64, or None.
"""
from __future__ import annotations

import numpy as np

EPS32 = 2.0 ** -24   # half a unit in the last place, relative


def rows_of(sorted_pair, ids, T, k, E, n_shared):
    """(token, expert) of every row; expert -1: no row."""
    flat = np.asarray(ids).ravel()
    out = [(p // k, int(flat[p])) if 0 <= p < T * k else (0, -1) for p in np.asarray(sorted_pair)]
    return out + [(t, E + s) for s in range(n_shared) for t in range(T)]


def product(A, B, scale, v_in):
    """(s B (A v), bound).  Exact products, K sums of A v and rank of B v, each
    at most that many roundings of partial sums (and one per 32 of a matrix
    step); B v runs on three parts of v, so three times its sums; one rounding
    each for the scale, the parts of K and the weight."""
    K, r = A.shape[1], A.shape[0]
    v = A @ v_in
    mag = np.abs(A) @ np.abs(v_in)
    y = scale * (B @ v)
    bound = abs(scale) * (np.abs(B) @ mag) * (K + K / 32 + 3 * r + 16) * EPS32
    return y, bound


def gateup(gu, x, rows, adapter, pairs, widths, ld, bf16):
    """(h, bound) [R][ld] in fp64 from gu [R][2 ld], x [T][H]; NaN where no row
    or no column is."""
    R = len(rows)
    h = np.full((R, ld), np.nan)
    bound = np.zeros((R, ld))
    for r, (t, e) in enumerate(rows):
        if e < 0:
            continue
        I = widths[e]
        g, u = gu[r, :I].copy(), gu[r, ld:ld + I].copy()
        dg, du = np.zeros(I), np.zeros(I)
        d = int(adapter[t])
        if 0 <= d < len(pairs) and pairs[d][e] is not None:
            A, B, s = pairs[d][e]
            rank = A.shape[0] // 2
            yg, dg = product(A[:rank], B[:I], s, x[t])
            yu, du = product(A[rank:], B[I:], s, x[t])
            g += yg
            u += yu
            dg = dg + EPS32 * np.abs(g)
            du = du + EPS32 * np.abs(u)
        with np.errstate(over="ignore"):
            sl = g / (1 + np.exp(-g))
        h[r, :I] = sl * u
        # |SiLU'| <= 1.1; exponential, division and products lose a few units,
        # the exponential's argument |g| of them
        loose = (1.1 * dg * (np.abs(u) + du) + np.abs(sl) * du
                 + (16 + 2 * np.abs(g)) * EPS32 * np.abs(h[r, :I]))
        half = 2.0 ** -8 * (np.abs(h[r, :I]) + loose) + 2.0 ** -133 if bf16 else 2.0 ** -149
        bound[r, :I] = loose + half
    return h, bound


def down(base, h, rows, adapter, pairs, widths, w, pair_pos, gates, T, k, bf16):
    """(out, bound) [T][H] in fp64 from base [T][H] and h [R][ld]."""
    out = base.copy()
    mag, off = np.abs(base), np.zeros_like(base)
    n_sh = gates.shape[1]
    terms = 0
    for t in range(T):
        d = int(adapter[t])
        if not 0 <= d < len(pairs):
            continue
        choices = [(int(pair_pos[t * k + j]), w[t, j]) for j in range(k)]
        choices += [(T * k + s * T + t, gates[t, s]) for s in range(n_sh)]
        for r, wt in choices:
            if r < 0 or rows[r][1] < 0 or pairs[d][rows[r][1]] is None:
                continue
            e = rows[r][1]
            A, B, s = pairs[d][e]
            y, b = product(A, B, s, h[r, :widths[e]])
            out[t] += wt * y
            off[t] += np.abs(wt) * b
            # the sum runs over all the rows' ranks as one
            mag[t] += np.abs(wt * s) * (np.abs(B) @ (np.abs(A) @ np.abs(h[r, :widths[e]])))
            terms = max(terms, A.shape[0])
    loose = off + (3 * (k + n_sh) * terms + 16) * EPS32 * mag
    half = 2.0 ** -8 * (np.abs(out) + loose) + 2.0 ** -133 if bf16 else EPS32 * np.abs(out)
    return out, loose + half
