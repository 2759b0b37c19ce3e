"""CPU oracle (numpy, fp64) of the MXFP4 operators: the format, the row
quantiser, and the layer's projections with bounds of what fp32 sums may lose.

Pinned by tests/test_mx_cpu.py: hand-worked codes, ties and scales; a search
over all 15 values for the nearest one; closed forms of one-weight layers.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def unpack(codes):
    """uint8 [..., C/2] to codes 0..15 [..., C], even index in the low nibble."""
    codes = np.asarray(codes, dtype=np.uint8)
    out = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=np.uint8)
    out[..., 0::2] = codes & 15
    out[..., 1::2] = codes >> 4
    return out


def pack(nib):
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).astype(np.uint8)


def values(codes, scales):
    """The values (fp64) of codes [..., C/2] and scales [..., C/32]."""
    nib = unpack(codes)
    v = np.where(nib & 8, -GRID[nib & 7], GRID[nib & 7])
    s = np.asarray(scales).astype(np.int64)
    unit = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(unit, BLOCK, axis=-1)


def quantise(rows):
    """fp64 (fp32- or bf16-valued) rows [..., C] to (codes, scales)."""
    rows = np.asarray(rows, dtype=np.float64)
    b = rows.reshape(rows.shape[:-1] + (rows.shape[-1] // BLOCK, BLOCK))
    bad = ~np.isfinite(b).all(axis=-1)
    fin = np.where(np.isfinite(b), b, 0.0)
    a = np.abs(fin).max(axis=-1)
    _, e = np.frexp(a)                       # a = m * 2^e, m in [0.5, 1)
    ex = np.where(a > 0, np.maximum(e - 3, -127), -127)
    m = np.abs(fin) / np.ldexp(1.0, ex)[..., None]
    # the nearest of the grid; of two equally near ones the even code (codes
    # alternate between even and odd mantissas)
    idx = np.searchsorted((GRID[1:] + GRID[:-1]) / 2, m, side="left")
    mid = np.concatenate([(GRID[1:] + GRID[:-1]) / 2, [np.inf]])
    tie = m == mid[np.minimum(idx, 7)]
    idx = np.where(tie & (idx % 2 == 1), idx + 1, idx)
    nib = (idx + 8 * np.signbit(fin)).astype(np.uint8)
    nib[bad] = 0
    scales = np.where(bad, 255, ex + 127).astype(np.uint8)
    return pack(nib.reshape(rows.shape)), scales


def activations(rows, act):
    """What the projection multiplies: the rows themselves, or their MXFP4 values."""
    rows = np.asarray(rows, dtype=np.float64)
    return rows if act == "a16" else values(*quantise(rows))


EPS32 = 2.0 ** -24   # half a unit in the last place, relative


def project(rows, w):
    """(rows @ w.T, the most that fp32 sums of its K products may be off).

    The products are exact in fp32 (4-bit times bf16 or 4-bit); K products
    summed in any order lose at most (K - 1) roundings of partial sums, each
    at most EPS32 times the sum of the magnitudes; one more per step of the
    matrix instruction (at most K / 32) covers its alignment of addends."""
    K = rows.shape[1]
    return rows @ w.T, (K + K / 32 + 4) * EPS32 * (np.abs(rows) @ np.abs(w).T)


def gateup(rows, w13, I):
    """(h unrounded, the bound of the kernel's bf16 h) for fp64 rows."""
    y, d = project(rows, w13)
    g, u, dg, du = y[:, :I], y[:, I:], d[:, :I], d[:, I:]
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    h = s * u
    # |SiLU'| <= 1.1; exp, divide and the products lose a few units of fp32;
    # then half a step of bf16, and its smallest step near zero
    loose = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 16 * EPS32 * np.abs(h)
    return h, loose + 2.0 ** -8 * (np.abs(h) + loose) + 2.0 ** -133


def combine(w, y, dy, pair_pos, T, k, gates):
    """(out, bound of the fp32 sum) of y rows [P + n_shared*T][H], weights w
    [T][k], pair_pos [T*k] (-1: absent), gates [T][n_shared]."""
    P, n_sh = T * k, gates.shape[1]
    out = np.zeros((T, y.shape[1]))
    mag, off = np.zeros_like(out), np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            p = pair_pos[t * k + j]
            if p >= 0:
                out[t] += w[t, j] * y[p]
                mag[t] += np.abs(w[t, j] * y[p])
                off[t] += abs(w[t, j]) * dy[p]
        for s in range(n_sh):
            r = P + s * T + t
            out[t] += gates[t, s] * y[r]
            mag[t] += np.abs(gates[t, s] * y[r])
            off[t] += gates[t, s] * dy[r]
    # k + n_shared roundings of the sum, and those of the gate (a few units)
    return out, off * (1 + 16 * EPS32) + (k + n_sh + 16) * EPS32 * (mag + off)
