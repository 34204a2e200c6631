"""Plain fp64 oracle of the 4-bit linear path and the sandwich norm (test
infrastructure, see h3_block's header). Formats (include/h3blk.h): e2m1 codes,
MX blocks of 32 with power-of-two scales, NV blocks of 16 with e4m3 scales and
a power-of-two scale per row."""
from __future__ import annotations

import math

import numpy as np

from .h3_block import TAG_PAD, f64, silu, sylvester_hadamard

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mx": 32, "nv": 16}


def _e4m3_table():
    """Every finite non-negative e4m3 value, ascending; index = code."""
    v = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        v += [(1 + m / 8) * 2.0 ** (e - 7) for m in range(8)]
    return np.array(v[:-1])  # the last code is NaN


E4M3 = _e4m3_table()


def nearest_even(a, table):
    """Index of the table entry nearest to a >= 0 (ties to the even index, saturating)."""
    a = np.asarray(a, dtype=np.float64)
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def rotate(x):
    """Unnormalised block-128 Walsh-Hadamard transform of each row."""
    n, k = x.shape
    return (x.reshape(n, k // 128, 128) @ np.sign(sylvester_hadamard(128))).reshape(n, k)


def quantize(x, fmt, rot=False):
    """[rows, K] -> codes (0..15, bit 3 the sign), block scale codes, row scales."""
    x = f64(x)
    if rot:
        with np.errstate(invalid="ignore"):
            x = rotate(x)
    n, k = x.shape
    b = x.reshape(n, -1, BLOCK[fmt])
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    row = np.ones(n)
    if fmt == "mx":
        e = np.array([[max(-126, _exponent(v, 7.0)) for v in r] for r in amax], dtype=np.int64).reshape(amax.shape)
        scale, code = 2.0 ** e, e + 127
        code = np.where(bad, 255, code)
    else:
        row = np.array([2.0 ** max(-126, _exponent(v, 2688.0)) if v > 0 else 1.0 for v in amax.max(-1)])
        code = nearest_even(amax / row[:, None] / 6.0, E4M3)
        scale = E4M3[code] * row[:, None]
        code = np.where(bad, 127, code)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(scale[..., None] > 0, np.abs(b) / scale[..., None], 0.0)
    codes = nearest_even(q, E2M1) + 8 * np.signbit(b)
    return codes.reshape(n, k), code, row / (math.sqrt(128.0) if rot else 1.0), bad


def _exponent(amax, top):
    """Smallest e with amax <= top * 2^e."""
    if amax == 0:
        return -126
    e = math.frexp(amax / top)[1]
    while amax <= top * 2.0 ** (e - 1):
        e -= 1
    while amax > top * 2.0 ** e:
        e += 1
    return e


def values(codes, scale_codes, row_scale, fmt):
    """What the 4-bit form stands for, fp64."""
    codes = np.asarray(codes)
    sc = np.asarray(scale_codes)
    if fmt == "mx":
        s = np.where(sc == 255, np.nan, 2.0 ** (sc.astype(np.float64) - 127))
    else:
        s = np.where(sc == 127, np.nan, E4M3[np.minimum(sc, 126)])
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    n, k = v.shape
    return (v.reshape(n, -1, BLOCK[fmt]) * s[..., None]).reshape(n, k) * f64(row_scale)[:, None]


def scale_offsets(rows, blocks):
    """Byte offset of the scale of (row, block) in the tiled scale buffer."""
    katoms = -(-blocks // 4)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    return ((r // 128) * katoms + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4


def product(a, b, swiglu=False):
    y = a @ b.T
    if swiglu:
        f = y.shape[1] // 2
        y = silu(y[:, :f]) * y[:, f:]
    return y


def sandwich(x, y, tag, tidx, table, branch, next_table=None, post_norm=True, post_gain=None, post_eps=1e-5,
             norm_eps=1e-5, branch_scale=1.0):
    """(x_out, h) of the sandwich norm, h None without a table for it."""
    x, y, table = f64(x), f64(y), f64(table)
    tag, tidx = np.asarray(tag), np.asarray(tidx)
    n_tags, n_t = table.shape[:2]
    ok = (tag != TAG_PAD) & (tag >= 0) & (tag < n_tags) & (tidx >= 0) & (tidx < n_t)
    def vec(t, i):
        m = np.zeros_like(x)
        m[ok] = f64(t)[tag[ok], tidx[ok], i]
        return m
    p = y
    if post_norm:
        p = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + post_eps)
        if post_gain is not None:
            p = p * f64(post_gain)
    x1 = x + branch_scale * vec(table, 5 if branch else 2) * p
    t, i = (next_table, 0) if branch else (table, 3)
    if t is None:
        return x1, None
    h = x1 / np.sqrt(np.mean(x1 * x1, -1, keepdims=True) + norm_eps)
    return x1, h * (1 + vec(t, i + 1)) + vec(t, i)
