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


@pytest.mark.parametrize("V", [152064, 152061])
def test_offsets_past_2_31(V):
    # 2.2e9 logits, written by TMA and (odd rows) by the warps, then sampled
    import torch

    T = 14300
    h, hs, w, ws = operands(T, 16, V)
    lg = lmh.lmhead_logits_fp8(h, hs, w, ws)
    u = torch.rand(T, device=dev(), generator=torch.Generator(device=dev()).manual_seed(5))
    tok, lp = lmh.lmhead_sample(lg, u, 0.8, top_p=0.9)
    for a, b in [(0, 3), (14120, 14126), (T - 4, T)]:  # 2^31 / V is 14122.3
        part = lmh.lmhead_logits_fp8(h[a:b], hs[a:b], w, ws)
        check_logits(part, h[a:b], hs[a:b], w, ws)
        assert same_bits(part, lg[a:b]), (a, b)
        tk, l2 = lmh.lmhead_sample(part, u[a:b], 0.8, top_p=0.9)
        assert torch.equal(tk, tok[a:b]) and torch.equal(l2, lp[a:b]), (a, b)
    lmh.lmhead_device_status()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_offsets_past_2_31(block_rows):
    import torch

    g = torch.Generator(device=dev()).manual_seed(6)
    x = torch.randn(1024, 131072, device=dev(), generator=g).to(torch.bfloat16).repeat(17, 1)
    q, s = lmh.lmhead_quantize_fp8(x, block_rows)
    one, one_s = lmh.lmhead_quantize_fp8(x[:1024], block_rows)
    per = one_s.shape[0]
    for i in range(17):
        assert torch.equal(q[1024 * i:1024 * (i + 1)].view(torch.uint8), one.view(torch.uint8)), i
        assert torch.equal(s[per * i:per * (i + 1)], one_s), i


@pytest.mark.parametrize("V", [2 ** 19, 2 ** 19 + 1, 1000003])
def test_sample_large_vocabularies(V):
    # above 2^19 tokens a weight's unit grows with V
    x, g = logit_rows(V % 97, 6, V)
    u = g.random(6, dtype=np.float32)
    check_sample(x, u)
    check_sample(x, u, t=0.7, k=5000, p=0.95)
    check_sample(x, u, t=1.5, p=0.99, m=1e-4)
    # equal logits: the sums are exact, so the token is
    tok, _ = lmh.lmhead_sample(_flat(6, V), to_dev(u))
    assert tok.tolist() == [int(np.floor(np.float64(v) * V)) for v in u]


def _flat(T, V):
    import torch

    return torch.full((T, V), -3.0, dtype=torch.bfloat16, device=dev())


def test_empty_batches():
    import torch

    from invariant_lm_head_gb300.fp8_head import FP8Head

    for V in (1000, 1003):
        w = torch.randn(V, 256, device=dev()).to(torch.bfloat16)
        head, h, u = FP8Head(w), w[:0], torch.empty(0, device=dev())
        n = lmh.lmhead_kernel_launches()
        assert head.logits(h).shape == (0, V)
        tok, lp = head.sample(h, u, u.clone(), top_k=torch.empty(0, dtype=torch.int32, device=dev()))
        assert tok.shape == (0,) and lp.shape == (0,) and lmh.lmhead_kernel_launches() == n


def test_capture_of_a_split_not_launched_before():
    # a process whose only eager call was one row captures every other split
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, invariant_lm_head_gb300 as lmh
from invariant_lm_head_gb300.fp8_head import FP8Head
g = torch.Generator(device="cuda").manual_seed(1)
head = FP8Head(torch.randn(2003, 256, device="cuda", generator=g).to(torch.bfloat16))
h = torch.randn(400, 256, device="cuda", generator=g).to(torch.bfloat16)
u = torch.rand(400, device="cuda", generator=g)
head.sample(h[:1], u[:1])
torch.cuda.synchronize()
got = []
for T in (30, 60, 120, 200, 400):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = head.sample(h[:T], u[:T], 0.9, top_p=0.9)
    graph.replay()
    torch.cuda.synchronize()
    got.append((graph, T, out))
for graph, T, out in got:
    want = head.sample(h[:T], u[:T], 0.9, top_p=0.9)
    assert all(torch.equal(a, b) for a, b in zip(out, want)), T
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=root)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]
