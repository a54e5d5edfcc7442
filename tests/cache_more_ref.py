"""4-bit pools, capped and biased scores, weights and eviction, from their definitions (numpy; tests only)."""
from __future__ import annotations

import math

import numpy as np

import cache_ref

f32 = np.float32


def decode_e2m1(codes):
    """The number that each code (0 .. 15) stands for (float64)."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 1) & 3, c & 1
    v = np.where(e == 0, 0.5 * m, (2 + m) * np.exp2(e - 2.0))
    return np.where(c >= 8, -v, v)


def nearest(x, grid):
    """Index into an ascending grid of the number nearest to x; a tie to the even index."""
    grid = np.asarray(grid, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantize(x, s=f32(1)):
    """Rows [..., D] of float32 as (codes [..., D / 2], block scales [..., D / 16]) bytes, by the header's words."""
    x = np.asarray(x, dtype=f32)
    with np.errstate(all="ignore"):
        y = (x * (f32(1) / f32(s))).reshape(x.shape[:-1] + (-1, 16))
        top = np.max(np.abs(y), axis=-1)
        nan = np.isnan(y).any(-1)
        grid = cache_ref.decode_e4m3(np.arange(0x7F))           # 0 .. 448, ascending
        b = nearest(np.where(nan, 0, top * (f32(1) / f32(6))), grid)
        b = np.maximum(b, 1)
        inv = f32(1) / grid[b].astype(f32)
        q = y * inv[..., None]
        mag = nearest(np.abs(np.where(np.isnan(q), 0, q)), decode_e2m1(np.arange(8)))
        code = (mag + 8 * np.signbit(y)).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(nan, 0x7F, b).astype(np.uint8)


def values(codes, scales):
    """What bytes of codes and block scales stand for (float64)."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    return decode_e2m1(nib) * np.repeat(cache_ref.decode_e4m3(scales), 16, -1)


def rotate32(x, angles, table, dim, interleaved, last):
    """x [T][heads][D] float32, turned by the table's rows `angles`; each operation rounded to fp32."""
    y = x.copy()
    first, half = (x.shape[-1] - dim if last else 0), dim // 2
    for t, p in enumerate(angles):
        i = np.arange(half)
        a, b = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + half + i)
        c, s = table[p, :half].astype(f32), table[p, half:].astype(f32)
        y[t, :, a] = (x[t, :, a].T * c - x[t, :, b].T * s).T
        y[t, :, b] = (x[t, :, b].T * c + x[t, :, a].T * s).T
    return y


def scores(q, k, scale, cap=0.0, slopes=None, away=None):
    """Logits of one query over keys, float64, and how far fp32 may take them (a bound for each key)."""
    x = k @ q * scale
    off = (q.shape[0] / 16 + 1) * 2.0 ** -21 * (np.abs(k) @ np.abs(q)) * abs(scale) + 2.0 ** -20
    if cap:
        # |d tanh| <= 1; tanh itself to 2^-19 (a polynomial below 0.3, 1 - 2 / (1 + e^2u) above)
        x = cap * np.tanh(x / cap)
        off = off + 2.0 ** -19 * np.abs(x)
    if slopes is not None:
        # slope log2(e) rounded, its product with the distance and the sum one rounding
        x = x + slopes * away
        off = off + 2.0 ** -22 * np.abs(slopes * away) + 2.0 ** -23 * np.abs(x)
    return x, off


def attend(q, rows_of, lengths, scale, window=0, cap=0.0, slopes=None, width=None, group=1, lse_in=None):
    """q [R][m][Hq][D] float64; rows_of(r, g, j) -> (keys, values). Returns a dict: out, lse, size (sum of p |v|), total (of |v|),
    off (a row's largest logit error among keys that weigh anything), weights [R][Hq / group][width] by the
    given lse (or its own), and weights_off, a bound of their error."""
    R, m, Hq, D = q.shape
    out = size = total = None
    lse, off = np.full((R, m, Hq), -np.inf), np.zeros((R, m, Hq))
    w = np.zeros((R, Hq // group, width or max(max(lengths), 1)))
    w_off = np.zeros_like(w)
    for r in range(R):
        n = int(lengths[r])
        for g in range(Hq):
            k, v = rows_of(r, g, np.arange(max(n, 1)))
            if out is None:
                out, size, total = (np.zeros((R, m, Hq, v.shape[1])) for _ in range(3))
            for i in range(m):
                last = n - m + i
                if last < 0:
                    continue
                first = max(0, last - window + 1) if window else 0
                j = np.arange(first, last + 1)
                x, err = scores(q[r, i, g], k[j], scale, cap, None if slopes is None else float(slopes[g]), j - last)
                top = x.max()
                e = np.exp(x - top)
                p = e / e.sum()
                lse[r, i, g] = top + math.log(e.sum())
                off[r, i, g] = err[p > 2.0 ** -40].max()
                out[r, i, g] = p @ v[j]
                size[r, i, g] = p @ np.abs(v[j])
                total[r, i, g] = np.abs(v[j]).sum(0)
                z = lse[r, i, g] if lse_in is None else float(lse_in[r, i, g])
                pw = np.exp(x - z)
                w[r, g // group, j] += pw
                # the logit's error, lse's rounding in the exponent, ex2, and the sum
                w_off[r, g // group, j] += pw * (err + 2.0 ** -22 * (np.abs(x) + abs(z)) + 2.0 ** -20)
    return dict(out=out, lse=lse, size=size, total=total, off=off, weights=w, weights_off=w_off)


def kept_slots(w, n, keep, recent):
    """Slots that an eviction keeps of one head's n, ascending; w: float weights, NaN above all, ties to the lowest."""
    if n <= keep:
        return list(range(n))
    key = [(0 if np.isnan(x) else 1, 0.0 if np.isnan(x) else -float(x), j) for j, x in enumerate(w[:n - recent])]
    return sorted(t[2] for t in sorted(key)[:keep - recent]) + list(range(n - recent, n))
