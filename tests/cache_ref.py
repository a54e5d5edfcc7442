"""The decode cache's operators in 64 bits, straight from their definitions (numpy; tests only)."""
from __future__ import annotations

import math

import numpy as np


def decode_e4m3(codes):
    """The number that each E4M3 byte stands for (float64)."""
    c = np.asarray(codes, dtype=np.int64)
    sign, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(sign == 1, -v, v)


def e4m3_grid():
    """All finite E4M3 numbers, ascending."""
    v = decode_e4m3(np.arange(256))
    return np.unique(v[np.isfinite(v)])


def attend(q, rows_of, lengths, scale, window):
    """q [R][m][Hq][D] float64; rows_of(r, h, j) -> (keys [n][D], values [n][V]) of positions j.
    Returns out, lse, and per output the sum of p |v| and per row the sum over a key of |q| |k|
    (the largest key's), from which the tests derive how far a kernel may be off."""
    R, m, Hq, D = q.shape
    outs = None
    lse = np.full((R, m, Hq), -np.inf)
    logit = np.zeros((R, m, Hq))
    for r in range(R):
        for i in range(m):
            last = int(lengths[r]) - m + i
            first = max(0, last - window + 1) if window else 0
            j = np.arange(first, last + 1)
            for g in range(Hq):
                k, v = rows_of(r, g, j)
                if outs is None:
                    outs = np.zeros((R, m, Hq, v.shape[1]))
                    size = np.zeros((R, m, Hq, v.shape[1]))
                if last < 0:
                    continue
                x = k @ q[r, i, g] * scale
                top = x.max()
                e = np.exp(x - top)
                p = e / e.sum()
                lse[r, i, g] = top + math.log(e.sum())
                outs[r, i, g] = p @ v
                size[r, i, g] = p @ np.abs(v)
                logit[r, i, g] = (np.abs(k) @ np.abs(q[r, i, g])).max() * abs(scale)
    return outs, lse, size, logit


def rotate(x, positions, table, dim, interleaved, last):
    """x [T][heads][D] float64 with its rotated part turned by the table's angles."""
    y = x.copy()
    D = x.shape[-1]
    first = D - dim if last else 0
    half = dim // 2
    for t, p in enumerate(positions):
        if p < 0:
            continue
        for i in range(half):
            a, b = (first + 2 * i, first + 2 * i + 1) if interleaved else \
                (first + i, first + half + i)
            c, s = float(table[p, i]), float(table[p, half + i])
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def rotary_table(rows, dim, base, scaling=None):
    """Cosines and sines in 64 bits, by the formulas in the C header."""
    i = np.arange(dim // 2)
    s = scaling or {"kind": "none"}
    kind = s["kind"]
    if kind == "base":
        base = base * s["factor"] ** (dim / (dim - 2))
    w = base ** (-2.0 * i / dim)
    m = 1.0
    if kind == "linear":
        w = w / s["factor"]
    if kind in ("ramp", "bands"):
        fast, slow, n = s.get("beta_fast", 32.0), s.get("beta_slow", 1.0), s["original"]
        if kind == "ramp":
            def index(turns):
                return dim * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), dim - 1)
            if hi <= lo:
                hi = lo + 0.001
            keep = 1 - (i - lo) / (hi - lo)
            m = s.get("magnitude") or 1 + 0.1 * math.log(s["factor"])
        else:
            keep = (n * w / (2 * math.pi) - slow) / (fast - slow)
        keep = np.clip(keep, 0, 1)
        w = w * keep + w / s["factor"] * (1 - keep)
    angle = np.arange(rows)[:, None] * w
    return np.concatenate([m * np.cos(angle), m * np.sin(angle)], 1)
