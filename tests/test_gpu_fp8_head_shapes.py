"""The fp8 head at the shapes that real calls take, against the fp64 oracle.

Logits: tiles of 160 to 256 columns (two accumulators in TMEM, three or four
output boxes a promote group), several tiles of a CTA (ring, accumulator and
staging buffers carried from one to the next) and rasters of more than one group
of 16 m tiles. Quantisation: more tiles than the grid has CTAs. Sampling: rows
that are taken in windows, at every number of CTAs a row can get. Tolerances are
those of test_gpu_fp8_head.py.
"""

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
import workloads as W
from helpers import dev, to_dev
from test_gpu_fp8_head import LOWEST, check_logits, check_quantize, check_sample, logit_rows, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lmh.build()


def same_bits(a, b):
    import torch

    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_quantize_more_tiles_than_the_grid():
    check_quantize(W.random_bf16(17, (16400, 1296), 3.0), 128)


# T, H, V; on 152 SMs: tile columns, tiles
@pytest.mark.parametrize("T,H,V", [
    (64, 256, 32000),    # 224, 143
    (64, 272, 20000),    # 160, 125
    (1, 272, 39000),     # 160, 244: two tiles of a CTA, eight rows loaded
    (300, 272, 32003),   # 224, 429: odd rows
    (300, 256, 16500),   # 192, 258
    (2100, 400, 8200),   # 256, 561: two raster groups
    (2100, 272, 4099)])  # 256, 289: the same, odd rows
def test_logits_wide_tiles(T, H, V):
    ops = operands(T, H, V)
    check_logits(lmh.lmhead_logits_fp8(*ops), *ops)
    lmh.lmhead_device_status()


@pytest.mark.parametrize("H,V", [(400, 8200), (272, 32003)])
def test_logits_rows_do_not_depend_on_the_tile_width(H, V):
    # rows of 256-column tiles against the same rows of narrower ones
    h, hs, w, ws = operands(2100, H, V)
    whole = lmh.lmhead_logits_fp8(h, hs, w, ws)
    for a, b in [(0, 1), (2099, 2100), (5, 69), (1000, 1300), (1900, 2100), (77, 2000)]:
        part = lmh.lmhead_logits_fp8(h[a:b], hs[a:b], w, ws)
        assert same_bits(part, whole[a:b]), (a, b)


@pytest.mark.parametrize("T,V", [(300, 32003), (64, 20000), (2100, 4099)])
def test_logits_wide_tiles_at_any_address(T, V):
    import torch

    ops = operands(T, 144, V)
    ld8 = -(-V // 8) * 8
    aligned = torch.empty(T, ld8, dtype=torch.bfloat16, device=dev())[:, :V]
    lmh.lmhead_logits_fp8(*ops, out_logits=aligned)
    check_logits(aligned, *ops)
    for ld, off in [(V, 1), (V + 1, 0), (V + 1, 6), (ld8 + 2, 3), (ld8 + 8, 5), (ld8 + 8, 8)]:
        buf = torch.full((off + T * ld + 8,), 7.0, dtype=torch.bfloat16, device=dev())
        out = buf[off:off + T * ld].view(T, ld)[:, :V]
        lmh.lmhead_logits_fp8(*ops, out_logits=out)
        assert same_bits(out, aligned), (ld, off)
        out.fill_(7.0)
        assert (buf == 7.0).all(), (ld, off)


@pytest.mark.parametrize("T", [7, 30, 60, 120, 200, 400])
def test_sample_windows_at_every_split(T):
    # a third of the values tiny; all beyond the direct range; infinities; the lowest
    # value alone; all tiny. Cuts and draws fall in different windows of a row.
    import torch

    V = 2043
    x, g = logit_rows(T + 7, T, V)
    r = lambda v: W.bf16_bits_to_f32(W.f32_to_bf16_bits(np.float32(v)))  # noqa: E731
    t = np.full(T, 0.9, np.float32)
    for i in range(T):
        kind = i % 5
        if kind == 0:
            x[i, ::3] = r(1e-20 * g.normal(size=x[i, ::3].size))
            t[i] = 2.0
        elif kind == 1:
            x[i] = r(x[i] + 300.0)
        elif kind == 2:
            x[i, g.integers(0, V, 3)] = np.inf
        elif kind == 3:
            x[i] = LOWEST
        else:
            x[i] = r(x[i] * 1e-12)
            t[i] = 1e-12 if i % 2 else 1.0
    u = g.random(T, dtype=np.float32)
    k = g.choice([0, V // 3, 9 * V // 10], T).astype(np.int32)
    p = g.choice([1.0, 0.3, 0.8], T).astype(np.float32)
    m = g.choice([0.0, 0.01], T).astype(np.float32)
    tok, lp = check_sample(x, u, t, k, p, m)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    for i in range(0, T, 11):  # the same rows alone
        tk, l2 = lmh.lmhead_sample(lg[i:i + 1], to_dev(u[i:i + 1]), float(t[i]), top_k=int(k[i]),
                                   top_p=float(p[i]), min_p=float(m[i]))
        assert tk.item() == tok[i] and l2.item() == lp[i], i
