"""fp64 oracle of the steps around the quantised heads: norm, 4-bit format, alternatives.

Plain numpy from the operators' definitions.
"""

from __future__ import annotations

import math

import numpy as np

from .fp8_head import AMAX_FLOOR, BLOCK, E4M3_MAX, e4m3

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------ norm

def bf16(y):
    """Nearest bf16 value (ties to even) of fp64 numbers in its normal range, or zero."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 1, -126) - 7)
    return np.rint(y / step) * step


def rmsnorm_fp8(x, weight, residual, eps):
    """(values of q, scale, x + residual or None) of finite fp64 [rows, cols].

    The row's factor is common to a block's values and its maximum, so q is taken
    without it, from products that fp64 holds exactly; blocks below the floor aside.
    """
    h = x if residual is None else bf16(x + residual)
    rows, cols = h.shape
    factor = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    u = h * weight
    n = -(-cols // BLOCK)
    q, scale = np.empty_like(h), np.empty((rows, n))
    for j in range(n):
        c = slice(j * BLOCK, (j + 1) * BLOCK)
        au = np.abs(u[:, c]).max(axis=1, keepdims=True)
        a = au * factor
        low = a < AMAX_FLOOR
        au = np.where(low, AMAX_FLOOR / factor, au)
        q[:, c] = e4m3(u[:, c] * E4M3_MAX / au)
        scale[:, j] = (np.maximum(a, AMAX_FLOOR) / E4M3_MAX)[:, 0]
    return q, scale, (None if residual is None else h)


# ------------------------------------------------------------------ microscaled e2m1

def e2m1_code(y):
    """Code (0 .. 15) of the nearest e2m1 value of fp64 numbers, ties to even, saturating."""
    y = np.asarray(y, np.float64)
    a = np.abs(y)[..., None]
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    odd = np.arange(7) % 2 == 1  # a tie between codes i and i + 1 goes up where i is odd
    code = (np.where(odd, a >= mid, a > mid)).sum(axis=-1)
    return code + 8 * np.signbit(y)


def mxfp4_byte(amax):
    """Scale byte of a block with finite largest magnitude amax (a bf16 value)."""
    if amax == 0:
        return 0
    m, e = math.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    b = e - 1 + (m >= 0.875) - 2 + 127
    return max(b, 0)


def mxfp4_quantize(x):
    """(codes [rows, cols], scale bytes [rows, cols / 32]) of fp64 x; a block that is not
    finite has byte 255 and codes 0 here (the codes say nothing)."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    amax = np.abs(b).max(axis=2)
    byte = np.array([[mxfp4_byte(v) if np.isfinite(v) else 255 for v in r] for r in amax])
    fine = (byte < 255)[:, :, None]
    y = np.where(fine, b, 0.0) * np.ldexp(1.0, 127 - np.where(byte < 255, byte, 127))[:, :, None]
    return e2m1_code(y).reshape(rows, cols), byte


def mxfp4_value(code, byte):
    """fp64 values of codes [rows, cols] and scale bytes [rows, cols / 32]."""
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, np.where(byte == 255, 127, byte) - 127))
    return v * np.repeat(s, 32, axis=1)


def unpack(q, scale, rows, cols):
    """(codes, bytes) from the packed elements and the scales' order in memory."""
    code = np.empty((rows, cols), np.int64)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    r, k = np.arange(rows)[:, None], np.arange(cols // 32)[None]
    return code, scale[r // 128, k // 4, r % 32, r // 32 % 4 * 4 + k % 4].astype(np.int64)


# ------------------------------------------------------------------ alternatives

def top_row(x, t, n, tokens=()):
    """(log-probs of tokens, entropy, top tokens, their log-probs) of one row of fp32 x."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64)) + 0.0
    V = x.size
    t = 1.0 if t == 0 else float(t)
    most = x.max()
    lp = np.full(V, -np.inf)
    entropy = 0.0
    if most > -np.inf:
        with np.errstate(over="ignore", invalid="ignore"):
            d = np.where(x == most, 0.0, (x - most) / t)
        w = np.exp(d)
        total = math.fsum(w)
        lp = d - math.log(total)
        kept = w > 0
        entropy = math.log(total) - math.fsum(w[kept] * d[kept]) / total
    order = np.lexsort((np.arange(V), -x))[:n]
    order = order[x[order] > -np.inf]
    top = np.full(n, -1, np.int64)
    top_lp = np.full(n, -np.inf)
    top[:order.size], top_lp[:order.size] = order, lp[order]
    got = np.array([lp[i] if 0 <= i < V else 0.0 for i in tokens])
    return got, entropy, top, top_lp
