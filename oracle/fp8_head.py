"""fp64 oracle of the fp8 head: block quantisation, block-scaled logits, sampling.

Plain numpy from the operators' definitions, row by row and block by block.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -60


def e4m3(y):
    """Nearest e4m3 value (ties to even) of fp64 numbers within +-448 after rounding."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(y / step) * step, -E4M3_MAX, E4M3_MAX)


def e4m3_values():
    """The value of every e4m3 bit pattern (index = bits); NaN at 0x7f and 0xff."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out[b] = math.nan if b & 0x7F == 0x7F else (-v if b & 0x80 else v)
    return out


def quantize(x, block_rows):
    """(values of q in fp64, scale in fp64) of finite fp64 x [rows, cols]."""
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // BLOCK)
    q = np.empty_like(x)
    scale = np.empty((nr, nc))
    for i in range(nr):
        r = slice(i * block_rows, (i + 1) * block_rows)
        for j in range(nc):
            c = slice(j * BLOCK, (j + 1) * BLOCK)
            a = max(float(np.abs(x[r, c]).max()), AMAX_FLOOR)
            scale[i, j] = a / E4M3_MAX
            q[r, c] = e4m3(x[r, c] * E4M3_MAX / a)
    return q, scale


def dequantize(q, scale, block_rows):
    s = np.repeat(np.repeat(scale, block_rows, 0), BLOCK, 1)
    return q * s[:q.shape[0], :q.shape[1]]


def sample_row(x, u, t, k=0, p=1.0, min_p=0.0, tol=0.0):
    """(tokens, logprobs) of one row of logits: every answer that masses known
    to a relative ``tol`` allow, in order of likelihood; one when tol is 0.

    x: fp32 values of the bf16 logits; t, p, min_p, u fp32.
    """
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(-np.inf), x) + np.float32(0)
    if not (x > -np.inf).any():
        return [-1], [0.0]
    order = np.lexsort((np.arange(x.size), -x))
    s = x[order]
    greedy = t == 0
    with np.errstate(over="ignore", invalid="ignore"):
        z = (s / np.float32(1 if greedy else t)).astype(np.float64)
        d = z - z[0]
        d[s == s[0]] = 0.0
        w = np.where(np.isnan(d), 0.0, np.exp(np.where(np.isnan(d), 0.0, d)))
    w[s == -np.inf] = 0.0
    total = math.fsum(w)
    if greedy:
        return [int(order[0])], [-math.log(total)]
    n_k = x.size if k <= 0 else min(int(k), x.size)
    cum = np.cumsum(w)

    def draw(off):
        n = n_k
        if p < 1:
            reach = float(p) * cum[n - 1] * (1 + off)
            n = min(n, int(np.searchsorted(cum[:n], reach, side="left")) + 1)
        if min_p > 0:
            n = min(n, max(1, int((w >= float(min_p) * (1 - off)).sum())))
        r = (float(u) + off) * cum[n - 1]
        return min(int(np.searchsorted(cum[:n], r, side="right")), n - 1)

    at = range(draw(-tol), draw(tol) + 1)
    return [int(order[j]) for j in at], [float(d[j]) - math.log(total) for j in at]
