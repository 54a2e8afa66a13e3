"""Around the quantised heads on the GPU, against the fp64 oracle.

Tolerances. Norm: q is the e4m3 value that exact arithmetic gives, equal; a scale is off
by its row's factor, whose sum of squares has at most 32 + 1 + 5 + 16 roundings on a
square's way (halved by the root), and by five more roundings: 32 of 2^-24. A block
below the floor, or outside fp32's usual range, takes rounded y: one e4m3 step.
4-bit quantisation is exact. Logits: one bf16 rounding (2^-8 of the value) and fp32 sums,
each of whose at most H / 64 steps adds 64 products with an error below 2^-21 of the sum
of the products' magnitudes (the tensor cores may truncate, and add in several parts).
Log-probs: with d = z - max z, c = log2(e) / t and its product are off by 2^-22 |d|, and
the sum by an exponential's few units of 2^-23 and one rounding for each of the at most
16 + V / 8192 + 13 additions on a weight's way, 2^-24 each: 3e-6 + 3e-7 |d| for V up to
200000. Entropy: the same relative errors of a sum of weights times |d|, 3e-6 (2 + 2 |h|).
"""

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
import workloads as W
from helpers import dev, to_dev, to_dev_bf16
from oracle import serving as o

pytestmark = pytest.mark.gpu

LOWEST = np.float32(-3.3895313892515355e38)


@pytest.fixture(scope="module", autouse=True)
def built():
    lmh.build()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def bf16_values(bits):
    return W.bf16_bits_to_f32(bits).astype(np.float64)


# ------------------------------------------------------------------ norm

def norm_inputs(rows, cols, seed=1):
    x = W.random_bf16(seed, (rows, cols), 1.0)
    r = W.random_bf16(seed + 1, (rows, cols), 4.0)
    w = W.f32_to_bf16_bits(1 + 0.3 * W.bf16_bits_to_f32(W.random_bf16(seed + 2, (1, cols), 1.0))[0])
    return x, r, w


def check_norm(got, x, r, w, eps=1e-6):
    q, s, out = got
    rq, rs, rr = o.rmsnorm_fp8(bf16_values(x), bf16_values(w), None if r is None else bf16_values(r),
                               eps)
    assert np.array_equal(f64(q), rq)
    assert (np.abs(f64(s) - rs) <= 32 * 2.0 ** -24 * rs).all()
    if out is not None:
        assert np.array_equal(f64(out), rr)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [
    (1, 16), (3, 128), (5, 400), (1, 4096), (200, 3600), (33, 4112), (7, 16384), (2, 16400),
    (2, 20000), (1, 32768), (2500, 272), (5000, 1296)])
def test_norm(rows, cols, residual):
    x, r, w = norm_inputs(rows, cols, rows + cols)
    r = r if residual else None
    got = lmh.lmhead_rmsnorm_fp8(to_dev_bf16(x), to_dev_bf16(w), None if r is None else to_dev_bf16(r))
    assert (got[2] is None) == (r is None)
    check_norm(got, x, r, w)


def test_norm_ties_and_small_numbers_of_bits():
    # few significant bits in x and w: many quotients are halfway between two e4m3 values
    g = np.random.default_rng(3)
    x = W.f32_to_bf16_bits(g.integers(-15, 16, (300, 512)).astype(np.float32))
    w = W.f32_to_bf16_bits(2.0 ** g.integers(-2, 3, 512).astype(np.float32))
    x[:, ::128] = W.f32_to_bf16_bits(np.float32(16.0))
    w[::128] = W.f32_to_bf16_bits(np.float32(4.0))
    check_norm(lmh.lmhead_rmsnorm_fp8(to_dev_bf16(x), to_dev_bf16(w)), x, None, w)


def test_norm_every_product_of_significands():
    # every pair of bf16 significands as a quotient's numerator, under several maxima
    m = np.arange(128, dtype=np.uint16)
    h = np.repeat(m, 128).reshape(128, 128) | np.uint16(126 << 7)
    w = np.tile(m, 128)[:128 * 128].reshape(128, 128)[0] | np.uint16(126 << 7)
    rows = []
    for top in range(0, 128, 3):
        r = h.copy()
        r[:, top] = np.uint16(127 << 7 | top)
        rows.append(r)
    x = np.concatenate(rows)
    check_norm(lmh.lmhead_rmsnorm_fp8(to_dev_bf16(x), to_dev_bf16(w)), x, None, w)


@pytest.mark.parametrize("scale", [1e-36, 1e-25, 1e-12, 1e12, 1e18, 1e25, 1e37])
def test_norm_magnitudes(scale):
    # sums of squares below and above fp32's range; eps far below the mean square
    import torch

    g = torch.Generator(device=dev()).manual_seed(5)
    x = (torch.randn(40, 384, device=dev(), generator=g) * scale).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(384, device=dev(), generator=g)).to(torch.bfloat16)
    q, s, _ = lmh.lmhead_rmsnorm_fp8(x, w, eps=1e-30)
    xd, wd = x.double(), w.double()
    y = xd * wd / torch.sqrt((xd * xd).mean(1, keepdim=True) + 1e-30)
    a = y.view(40, 3, 128).abs().amax(2).clamp_min(2.0 ** -60)
    if scale > 1e-20:
        assert ((s.double() - a / 448).abs() <= 32 * 2.0 ** -24 * a / 448).all()
        back = q.double().view(40, 3, 128) * s.double()[:, :, None]
        # half an e4m3 step of the value, or of the smallest normal number
        tol = (y.view(40, 3, 128).abs() * 2.0 ** -4).clamp_min(2.0 ** -10 / 448 * 1.001) * 1.00001
        tol = torch.maximum(tol, a[:, :, None] / 448 * 2.0 ** -10 * 1.001)
        assert ((back - y.view(40, 3, 128)).abs() <= tol).all()
    else:  # eps counts: only that the row is finite and no larger than the formula's
        assert torch.isfinite(q.float()).all() and torch.isfinite(s).all()
        assert ((s.double() - a / 448).abs() <= 1e-5 * a / 448).all()


def test_norm_of_the_largest_values():
    # every square past fp32, and their sum past what one scaling by 2^-64 would hold
    import torch

    big = float(-LOWEST)
    x = torch.full((3, 512), big, dtype=torch.bfloat16, device=dev())
    x[1, 7:] = 0
    x[2] *= (-1.0) ** torch.arange(512, device=dev())
    w = torch.full((512,), 2.0, dtype=torch.bfloat16, device=dev())
    q, s, _ = lmh.lmhead_rmsnorm_fp8(x, w)
    y = q.float() * s.repeat_interleave(128, 1)
    assert (y[0] / 2 - 1).abs().max() < 1e-5 and (y[2].abs() / 2 - 1).abs().max() < 1e-5
    assert (y[1, :7] / (2 * (512 / 7) ** 0.5) - 1).abs().max() < 1e-5 and (y[1, 7:] == 0).all()


def test_norm_zeros_floor_and_not_finite():
    import torch

    x = torch.zeros(6, 256, dtype=torch.bfloat16, device=dev())
    w = torch.ones(256, dtype=torch.bfloat16, device=dev())
    x[1] = 1.0
    x[1, 128:] = 1e-30  # a block below the floor beside one of ordinary size
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 2.0
    x[5, 0], x[5, 1] = 1.0, -0.0
    q, s, _ = lmh.lmhead_rmsnorm_fp8(x, w)
    q = q.float()
    floor = np.float32(2.0 ** -60 / 448)
    assert (q[0] == 0).all() and (s[0] == floor).all()
    assert (q[1, :128] == 448).all() and s[1, 1] == floor and (q[1, 128:] == 0).all()
    assert q[2].isnan().all() and s[2].isnan().all()
    assert (q[3, :128] == 0).all() and q[3, 128:].isnan().all() and s[3, 1].isnan()
    assert (q[4] == 448).all() and abs(float(s[4, 0]) * 448 - 1) < 1e-6
    assert q[5, 0] == 448 and (q[5, 1:] == 0).all() and torch.signbit(q[5, 1])


def test_norm_strides_in_place_and_alone():
    import torch

    x, r, w = norm_inputs(70, 400, 9)
    bx = torch.zeros(70, 640, dtype=torch.bfloat16, device=dev())
    br = torch.full((140, 408), 7.0, dtype=torch.bfloat16, device=dev())
    bx[:, 128:528] = to_dev_bf16(x)
    br[::2, :400] = to_dev_bf16(r)
    xs, rs, wd = bx[:, 128:528], br[::2, :400], to_dev_bf16(w)
    want = lmh.lmhead_rmsnorm_fp8(to_dev_bf16(x), wd, to_dev_bf16(r))
    check_norm(want, x, r, w)
    got = lmh.lmhead_rmsnorm_fp8(xs, wd, rs)
    same(got, want)
    none = lmh.lmhead_rmsnorm_fp8(xs, wd, rs, want_residual=False)
    assert none[2] is None
    same(none[:2], want[:2])
    for i in (0, 33, 69):  # a row alone
        same(lmh.lmhead_rmsnorm_fp8(xs[i:i + 1], wd, rs[i:i + 1]), [t[i:i + 1] for t in want])
    x0 = bx.clone()
    got = lmh.lmhead_rmsnorm_fp8(xs, wd, rs, out_residual=rs)  # the sum in the residual's place
    same(got, want)
    assert got[2].data_ptr() == rs.data_ptr() and torch.equal(bx, x0)
    assert (br[1::2] == 7).all() and (br[:, 400:] == 7).all()
    br[::2, :400] = to_dev_bf16(r)
    got = lmh.lmhead_rmsnorm_fp8(xs, wd, rs, out_residual=xs)  # and in x's
    same(got, want)
    assert (bx[:, :128] == 0).all() and (bx[:, 528:] == 0).all()


def same(got, want):
    import torch

    for a, b in zip(got, want, strict=True):
        if a is None or b is None:
            assert a is b
            continue
        t = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
        assert a.shape == b.shape and torch.equal(a.contiguous().view(t), b.contiguous().view(t))


# ------------------------------------------------------------------ 4-bit quantisation

def check_mxfp4(bits, x=None):
    x = to_dev_bf16(bits) if x is None else x
    q, s = lmh.lmhead_quantize_mxfp4(x)
    rows, cols = bits.shape
    code, byte = o.unpack(q.cpu().numpy(), s.cpu().numpy(), rows, cols)
    rc, rb = o.mxfp4_quantize(bf16_values(bits))
    assert np.array_equal(byte, rb)
    keep = np.repeat(rb < 255, 32, axis=1)
    assert np.array_equal(code[keep], rc[keep])
    sp = s.cpu().numpy()
    used = np.zeros(sp.shape, bool)
    r, k = np.meshgrid(np.arange(rows), np.arange(cols // 32), indexing="ij")
    used[r // 128, k // 4, r % 32, r // 32 % 4 * 4 + k % 4] = True
    assert (sp[~used] == 127).all()
    back = f64(lmh.lmhead_dequantize_mxfp4(q, s))
    ref = o.mxfp4_value(rc, rb)
    assert np.array_equal(back[keep], ref[keep]) and np.isnan(back[~keep]).all()
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 32), (2, 64), (31, 96), (128, 128), (129, 160), (300, 3616),
                                       (2500, 1312), (33, 4096)])
def test_quantize(rows, cols):
    check_mxfp4(W.random_bf16(rows * 3 + cols, (rows, cols), 2.0))


def test_quantize_every_value_under_every_maximum():
    # every finite bf16 as a block's largest, with values from 0 to it beside it
    top = np.arange(0x7F80, dtype=np.uint16)
    g = np.random.default_rng(1)
    drop = g.integers(0, 5 << 7, (top.size, 32))
    v = np.maximum(top[:, None].astype(np.int64) - drop, 0).astype(np.uint16)
    v |= g.integers(0, 2, v.shape).astype(np.uint16) << 15
    v[np.arange(top.size), g.integers(0, 32, top.size)] = top
    check_mxfp4_large(v.reshape(-1, 32 * 32))


def check_mxfp4_large(bits):
    # as check_mxfp4, but for values past bf16's largest, which come back infinite
    q, s = lmh.lmhead_quantize_mxfp4(to_dev_bf16(bits))
    code, byte = o.unpack(q.cpu().numpy(), s.cpu().numpy(), *bits.shape)
    rc, rb = o.mxfp4_quantize(bf16_values(bits))
    assert np.array_equal(byte, rb) and np.array_equal(code, rc)
    back, ref = f64(lmh.lmhead_dequantize_mxfp4(q, s)), o.mxfp4_value(rc, rb)
    big = np.abs(ref) > 3.4e38
    assert np.array_equal(back[~big], ref[~big]) and np.isinf(back[big]).all()


def test_quantize_ties_and_signs():
    y = np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, .125, .5, 1, 1.5, 2, 3, 4], np.float32)
    x = np.concatenate([y, -y]).reshape(1, 32)
    bits = np.concatenate([W.f32_to_bf16_bits(x * np.float32(2.0 ** e)) for e in (-100, -3, 0, 7, 90)])
    check_mxfp4(bits)


def test_quantize_not_finite():
    bits = W.random_bf16(3, (5, 128), 1.0)
    bits[1, 40], bits[2, 0], bits[3, 127], bits[4, 64] = 0x7F80, 0xFF80, 0x7FC0, 0xFFC1
    check_mxfp4(bits)


def test_quantize_strided_rows_and_outputs():
    import torch

    bits = W.random_bf16(11, (130, 512), 1.0)
    x = to_dev_bf16(bits)
    q, s = check_mxfp4(np.ascontiguousarray(bits[:, 128:416]), x[:, 128:416])
    check_mxfp4(np.ascontiguousarray(bits[::2, :256]), x[::2, :256])
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    got = lmh.lmhead_quantize_mxfp4(x[:, 128:416], out=q2, out_scale=s2)
    assert got[0] is q2 and got[1] is s2 and torch.equal(q, q2) and torch.equal(s, s2)
    out = torch.full((130, 512), 7.0, dtype=torch.bfloat16, device=dev())
    lmh.lmhead_dequantize_mxfp4(q, s, out=out[:, 8:296])
    assert torch.equal(out[:, 8:296], lmh.lmhead_dequantize_mxfp4(q, s))
    assert (out[:, :8] == 7).all() and (out[:, 296:] == 7).all()


def test_dequantize_every_code_under_every_scale():
    import torch

    q = torch.arange(256, dtype=torch.uint8, device=dev()).repeat(256, 1)  # 16 blocks a row
    rows, cols = 256, 512
    s = torch.zeros(2, 4, 32, 16, dtype=torch.uint8, device=dev())
    r, k = np.meshgrid(np.arange(rows), np.arange(cols // 32), indexing="ij")
    s[r // 128, k // 4, r % 32, r // 32 % 4 * 4 + k % 4] = to_dev(r.astype(np.uint8))
    back = f64(lmh.lmhead_dequantize_mxfp4(q, s))
    code, byte = o.unpack(q.cpu().numpy(), s.cpu().numpy(), rows, cols)
    ref = o.mxfp4_value(code, byte)
    big = np.abs(ref) > 3.4e38
    assert np.array_equal(np.isnan(back), np.isnan(ref)) and np.isinf(back[big]).all()
    rest = ~big & ~np.isnan(ref)
    assert np.array_equal(back[rest], ref[rest])


# ------------------------------------------------------------------ 4-bit logits

def operands(T, H, V, seed=1, spread=0):
    """spread: exponents of the blocks' sizes, up to 2^+-spread apart."""
    h, w = W.random_bf16(seed, (T, H), 1.0), W.random_bf16(seed + 1, (V, H), 0.02)
    if spread:
        g = np.random.default_rng(seed)
        for x in (h, w):
            e = np.repeat(g.integers(-spread, spread + 1, (x.shape[0], H // 32)), 32, axis=1)
            x[:] = W.f32_to_bf16_bits(W.bf16_bits_to_f32(x) * np.ldexp(np.float32(1), e))
    return (*lmh.lmhead_quantize_mxfp4(to_dev_bf16(h)), *lmh.lmhead_quantize_mxfp4(to_dev_bf16(w)))


def check_logits(out, hq, hs, wq, ws, rows=slice(None)):
    import torch

    h = lmh.lmhead_dequantize_mxfp4(hq, hs).double()[rows]
    w = lmh.lmhead_dequantize_mxfp4(wq, ws).double()
    ref, mag = h @ w.t(), h.abs() @ w.abs().t()
    tol = ref.abs() * 2.0 ** -8 + mag * (h.shape[1] / 64 + 1) * 2.0 ** -21
    assert torch.isfinite(out).all()
    assert ((out.double() - ref).abs() <= tol).all()


SHAPES = [(1, 32, 1), (1, 64, 7), (1, 128, 128), (2, 256, 130), (7, 160, 1000), (8, 3584, 4096),
          (9, 96, 31), (63, 416, 2047), (64, 4096, 2048), (65, 288, 8192), (127, 544, 999),
          (128, 512, 1024), (129, 512, 1025), (200, 3616, 3203), (256, 224, 4096), (257, 640, 513),
          (700, 1056, 2000), (1300, 384, 777), (300, 288, 40000), (2100, 416, 8200), (1, 288, 80000)]


@pytest.mark.parametrize("T,H,V", SHAPES)
def test_logits(T, H, V):
    ops = operands(T, H, V)
    check_logits(lmh.lmhead_logits_mxfp4(*ops), *ops)
    lmh.lmhead_device_status()


@pytest.mark.parametrize("T,H,V", [(5, 320, 300), (150, 1056, 700), (400, 512, 40000)])
def test_logits_scales_far_apart(T, H, V):
    ops = operands(T, H, V, 5, spread=30)
    check_logits(lmh.lmhead_logits_mxfp4(*ops), *ops)


def test_logits_each_scale_and_place():
    # one nonzero element a row: every (row, block) scale of both operands shows by itself
    import torch

    T, H, V = 130, 512, 300
    g = np.random.default_rng(2)
    for seed in range(3):
        h, w = np.zeros((T, H), np.float32), np.zeros((V, H), np.float32)
        col = g.integers(0, H, T)
        h[np.arange(T), col] = 2.0 ** g.integers(-20, 20, T)
        w[:] = g.choice(o.E2M1[1:], (V, H)) * np.repeat(2.0 ** g.integers(-20, 20, (V, H // 32)), 32, 1)
        x, y = (to_dev_bf16(W.f32_to_bf16_bits(v)) for v in (h, w))
        out = lmh.lmhead_logits_mxfp4(*lmh.lmhead_quantize_mxfp4(x), *lmh.lmhead_quantize_mxfp4(y))
        yq = f64(lmh.lmhead_dequantize_mxfp4(*lmh.lmhead_quantize_mxfp4(y)))
        want = h[np.arange(T), col][:, None].astype(np.float64) * yq.T[col]
        assert np.array_equal(f64(out), want)  # one product a logit: exact
    assert torch.isfinite(out).all()


def test_logits_do_not_depend_on_the_batch():
    import torch

    hq, hs, wq, ws = operands(300, 3616, 4100)
    h = to_dev_bf16(W.random_bf16(1, (300, 3616), 1.0))
    whole = lmh.lmhead_logits_mxfp4(hq, hs, wq, ws)
    for a, b in [(0, 1), (299, 300), (5, 12), (5, 69), (100, 228), (20, 149), (7, 300)]:
        part = lmh.lmhead_logits_mxfp4(*lmh.lmhead_quantize_mxfp4(h[a:b]), wq, ws)
        assert torch.equal(part.view(torch.int16), whole[a:b].view(torch.int16)), (a, b)
    # nor on the vocabulary around a column
    for a, b in [(0, 128), (128, 700), (3968, 4100)]:
        rows = slice(a // 128, -(-b // 128))
        part = lmh.lmhead_logits_mxfp4(hq, hs, wq[a:b].contiguous(), ws[rows].contiguous())
        assert torch.equal(part.view(torch.int16), whole[:, a:b].contiguous().view(torch.int16))


@pytest.mark.parametrize("T,V", [(1, 1003), (33, 2001), (130, 3203), (300, 4099), (5, 3)])
def test_logits_at_any_address(T, V):
    import torch

    ops = operands(T, 160, V)
    ld8 = -(-V // 8) * 8
    want = lmh.lmhead_logits_mxfp4(*ops, out_logits=torch.empty(T, ld8 + 8, dtype=torch.bfloat16,
                                                                device=dev())[:, :V])
    check_logits(want, *ops)
    for ld, off in [(V, 0), (V, 1), (V + 1, 6), (ld8, 0), (ld8 + 2, 3), (ld8 + 8, 5), (ld8 + 8, 8)]:
        buf = torch.full((off + T * ld + 8,), 7.0, dtype=torch.bfloat16, device=dev())
        out = buf[off:off + T * ld].view(T, ld)[:, :V]
        lmh.lmhead_logits_mxfp4(*ops, out_logits=out)
        assert torch.equal(out.contiguous().view(torch.int16), want.contiguous().view(torch.int16))
        out.fill_(7.0)
        assert (buf == 7.0).all(), (ld, off)


def test_logits_a_bad_block_stays_alone():
    import torch

    x = to_dev_bf16(W.random_bf16(1, (200, 288), 1.0))
    w = to_dev_bf16(W.random_bf16(2, (700, 288), 0.02))
    clean = lmh.lmhead_logits_mxfp4(*lmh.lmhead_quantize_mxfp4(x), *lmh.lmhead_quantize_mxfp4(w))
    x[3, 200], x[150, 0], w[333, 287] = float("inf"), float("nan"), float("nan")
    out = lmh.lmhead_logits_mxfp4(*lmh.lmhead_quantize_mxfp4(x), *lmh.lmhead_quantize_mxfp4(w))
    bad = torch.zeros(200, 700, dtype=torch.bool, device=dev())
    bad[[3, 150]] = True
    bad[:, 333] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("V", [152064, 152061])
def test_offsets_past_2_31(V):
    # 2.2e9 logits, written by TMA and (odd rows) by the warps, then looked at
    import torch

    T = 14300
    hq, hs, wq, ws = operands(T, 64, V)
    lg = lmh.lmhead_logits_mxfp4(hq, hs, wq, ws)
    ids = torch.arange(T, dtype=torch.int32, device=dev())
    lp, ent, tok, tlp = lmh.lmhead_top_logprobs(lg, ids, 0.8, top=6)
    for a, b in [(0, 3), (14120, 14126), (T - 4, T)]:  # 2^31 / V is 14122.3
        check_logits(lg[a:b], hq, hs, wq, ws, slice(a, b))
        got = lmh.lmhead_top_logprobs(lg[a:b].clone(), ids[a:b], 0.8, top=6)
        same(got, (lp[a:b], ent[a:b], tok[a:b], tlp[a:b]))
    lmh.lmhead_device_status()


def test_quantize_offsets_past_2_31():
    import torch

    g = torch.Generator(device=dev()).manual_seed(6)
    x = torch.randn(1024, 131072, device=dev(), generator=g).to(torch.bfloat16).repeat(17, 1)
    q, s = lmh.lmhead_quantize_mxfp4(x)
    one, one_s = lmh.lmhead_quantize_mxfp4(x[:1024])
    for i in range(17):
        assert torch.equal(q[1024 * i:1024 * (i + 1)], one), i
        assert torch.equal(s[8 * i:8 * (i + 1)], one_s), i
    back = lmh.lmhead_dequantize_mxfp4(q, s)
    assert torch.equal(back[-1024:], lmh.lmhead_dequantize_mxfp4(one, one_s))


def test_norm_offsets_past_2_31():
    import torch

    g = torch.Generator(device=dev()).manual_seed(7)
    x = torch.randn(1000, 32768, device=dev(), generator=g).to(torch.bfloat16)
    w = torch.randn(32768, device=dev(), generator=g).to(torch.bfloat16)
    one = lmh.lmhead_rmsnorm_fp8(x, w, x)
    xs = x.repeat(67, 1)
    got = lmh.lmhead_rmsnorm_fp8(xs, w, xs)
    for i in (0, 30, 65, 66):
        same([t[1000 * i:1000 * (i + 1)] for t in got], one)


# ------------------------------------------------------------------ alternatives

def logit_rows(seed, T, V, std=3.0):
    g = np.random.default_rng(seed)
    x = (g.normal(size=(T, V)) * std).astype(np.float32)
    x[np.arange(T)[:, None], g.integers(0, V, (T, min(V, 8)))] += 8
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(x)), g


def check_top(x, n, t=1.0, tokens=None, logits=None):
    import torch

    T, V = x.shape
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev()) if logits is None else logits
    x = lg.float().cpu().numpy()  # the bf16 values that the call gets
    ts = np.broadcast_to(np.float32(t), (T,))
    targ = float(t) if np.ndim(t) == 0 else to_dev(ts.copy())
    ids = np.zeros((T, 0), np.int32) if tokens is None else tokens
    got = lmh.lmhead_top_logprobs(lg, None if tokens is None else to_dev(ids), targ, top=n)
    lp, ent, tok, tlp = [None if v is None else v.cpu().numpy() for v in got]
    for i in range(T):
        rlp, rent, rtok, rtlp = o.top_row(x[i], ts[i], n, ids[i])
        assert np.array_equal(tok[i], rtok), (i, tok[i], rtok)
        near(tlp[i], rtlp)
        if tokens is not None:
            near(lp[i], rlp)
        assert abs(ent[i] - rent) <= 3e-6 * (2 + 2 * abs(rent)), i
    return got


def near(got, want):
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)  # -inf below fp32's range
    assert np.array_equal(np.isinf(got), np.isinf(want))
    fine = ~np.isinf(want)
    assert (np.abs(got[fine] - want[fine]) <= 3e-6 + 4e-7 * np.abs(want[fine])).all()


@pytest.mark.parametrize("V,n", [
    (1, 1), (1, 5), (2, 2), (7, 20), (8, 8), (9, 3), (255, 128), (2043, 20), (2048, 1), (8191, 64),
    (16384, 20), (16385, 20), (32003, 128), (65536, 5), (65537, 20), (152064, 20), (151937, 128),
    (300001, 7)])
def test_top(V, n):
    x, g = logit_rows(V + n, 5, V)
    ids = g.integers(0, V, (5, 3)).astype(np.int32)
    ids[0] = [-1, V, -100]
    check_top(x, n, 0.8, ids)
    check_top(x, n, np.array([0.0, 0.3, 1.0, 2.5, 40.0], np.float32), ids)


def test_top_of_none():
    x, _ = logit_rows(4, 3, 1000)
    lp, ent, tok, tlp = check_top(x, 0)
    assert lp is None and tok.shape == (3, 0) and tlp.shape == (3, 0)


def test_top_token_shapes():
    import torch

    x, _ = logit_rows(4, 6, 1000)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    one = lmh.lmhead_top_logprobs(lg, torch.arange(6, dtype=torch.int32, device=dev()))
    assert one[0].shape == (6,) and one[2].shape == (6, 20)
    # the same token twice, and more tokens than a CTA has threads
    ids = torch.randint(0, 1000, (6, 700), dtype=torch.int32, device=dev())
    ids[:, 1] = ids[:, 0]
    lp = lmh.lmhead_top_logprobs(lg, ids, top=0, want_entropy=False)
    assert lp[1] is None and lp[0].shape == (6, 700) and torch.equal(lp[0][:, 0], lp[0][:, 1])
    every = torch.arange(1000, dtype=torch.int32, device=dev()).repeat(6, 1)
    assert (lmh.lmhead_top_logprobs(lg, every)[0].exp().sum(1) - 1).abs().max() < 1e-5


@pytest.mark.parametrize("V", [300, 5000, 33000, 152061])
@pytest.mark.parametrize("kind", ["equal", "two", "few", "up", "down", "run", "zeros"])
def test_top_ties_go_by_index(V, kind):
    # more tokens than a list holds reach the n-th value; values that rise or fall with
    # the index; the largest ones all in one run
    g = np.random.default_rng(V)
    x = np.zeros((4, V), np.float32)
    if kind == "two":
        x[:] = g.integers(0, 2, x.shape)
    elif kind == "few":
        x[:] = g.integers(-3, 4, x.shape)
        x[1, V // 2] = 9
    elif kind == "up":
        x[:] = np.linspace(-5, 20, V)
    elif kind == "down":
        x[:] = np.linspace(20, -5, V)
    elif kind == "run":
        x[:] = g.normal(size=x.shape)
        x[:, V // 3:V // 3 + min(V // 2, 3000)] += 30
    elif kind == "zeros":
        x[:, ::2] = -0.0
        x[1, ::3] = -1.0
    x = W.bf16_bits_to_f32(W.f32_to_bf16_bits(x))
    check_top(x, 20)
    check_top(x, 128, 0.5)


@pytest.mark.parametrize("n", [1, 20, 128])
@pytest.mark.parametrize("V", [9001, 152064])
def test_top_of_crowded_levels(V, n):
    # more equal logits than a list holds, and the few above them where a search that
    # stops early would miss them; the n-th on the crowded level, and on one above it
    x = np.full((7, V), -3.0, np.float32)
    x[0, -5:] = 2.0, 1.0, 5.0, 1.0, 4.0
    x[1] = LOWEST
    x[1, -3:] = LOWEST / 2, 0.0, LOWEST / 4
    x[2, V // 2:] = -2.5  # a level of its own above the first
    x[2, -n // 2 - 1:] = 7.0
    x[3, ::7] = -2.984375  # the next number of the type
    x[4, ::7] = -2.984375
    x[4, -n:] = 8.0
    x[5] = -np.inf
    x[5, V // 3:V // 3 + 2000] = -1e30  # the only ones not masked
    x[6, np.random.default_rng(V).permutation(V)[:V // 2]] = -np.inf
    ids = np.array([[0, V - 1]] * 7, np.int32)
    check_top(x, n, 1.0, ids)
    logits = to_dev_bf16(W.f32_to_bf16_bits(x))
    many = lmh.lmhead_top_logprobs(logits.repeat(160, 1), to_dev(ids).repeat(160, 1), top=n)
    one = lmh.lmhead_top_logprobs(logits, to_dev(ids), top=n)
    for a, b in zip(many, one):
        assert all((a[i:i + 7] == b).all() for i in (0, 7 * 80, 7 * 159))


@pytest.mark.parametrize("V", [200, 9000, 70000])
def test_top_masks(V):
    g = np.random.default_rng(V)
    x, _ = logit_rows(V, 9, V)
    x[0] = -np.inf  # nothing left
    x[1] = np.nan
    x[2] = -np.inf
    x[2, V - 1] = -4.0  # one token left
    x[3] = -np.inf
    x[3, 30:37] = 1.0  # fewer than asked for, in one vector and the next
    x[4, g.random(V) < 0.99] = -np.inf
    x[5, ::2] = np.nan
    x[6] = LOWEST  # the type's lowest value as the mask, and alone
    x[7] = LOWEST
    x[7, [3, V // 2]] = 2.0, 2.5
    x[8, : V // 2] = -np.inf
    ids = g.integers(0, V, (9, 4)).astype(np.int32)
    ids[2, 0], ids[3, 1], ids[7, 0] = V - 1, 33, 5
    check_top(x, 20, 1.0, ids)
    check_top(x, 3, 0.7, ids)


def test_top_infinities_and_overflow():
    x, g = logit_rows(3, 6, 5000)
    x[0, 77] = np.inf
    x[1, [5, 4000]] = np.inf
    x[2, 9] = 3e38
    x[3] = W.bf16_bits_to_f32(W.f32_to_bf16_bits((x[3] * np.float32(1e37)).astype(np.float32)))
    x[4] = np.inf
    x[5, ::3] = -np.inf
    ids = g.integers(0, 5000, (6, 3)).astype(np.int32)
    ids[1, 0], ids[1, 1] = 4000, 6
    for t in (1.0, 1e-3, 1e-30, 1e30):
        check_top(x, 8, t, ids)


def test_top_of_tiny_temperatures_and_logits():
    x, g = logit_rows(5, 4, 3000)
    x = W.bf16_bits_to_f32(W.f32_to_bf16_bits(x * np.float32(1e-38)))
    check_top(x, 8, np.array([1e-38, 2e-39, 1.0, 3e38], np.float32), np.zeros((4, 1), np.int32))


def test_top_bad_temperatures_of_a_row():
    import torch

    x, _ = logit_rows(5, 6, 3000)
    nan, inf = float("nan"), float("inf")
    t = torch.tensor([1.0, -1.0, nan, inf, -inf, 1.0], device=dev())
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    ids = torch.tensor([1, 2, -1, 4, 5, 6], dtype=torch.int32, device=dev())
    lp, ent, tok, tlp = lmh.lmhead_top_logprobs(lg, ids, t, top=4)
    assert lp[1:5].isnan().all() and ent[1:5].isnan().all()
    assert (tok[1:5] == -1).all() and tlp[1:5].isnan().all()
    good = lmh.lmhead_top_logprobs(lg, ids, 1.0, top=4)
    same([v[[0, 5]] for v in (lp, ent, tok, tlp)], [v[[0, 5]] for v in good])


@pytest.mark.parametrize("V", [1003, 16385, 70001])
def test_top_at_any_address_and_alone(V):
    import torch

    T = 40
    x, g = logit_rows(V, T, V)
    ids = g.integers(0, V, (T, 2)).astype(np.int32)
    ld = -(-V // 8) * 8
    buf = torch.full((T, ld), 50.0, dtype=torch.bfloat16, device=dev())
    buf[:, :V] = torch.from_numpy(x).to(dev())
    want = check_top(x[:3], 20, 0.9, ids[:3], buf[:3, :V])
    want = lmh.lmhead_top_logprobs(buf[:, :V], to_dev(ids), 0.9)
    for stride, off in [(V, 0), (V, 1), (V + 1, 2), (V + 3, 7), (ld, 8), (ld, 3)]:
        flat = torch.full((off + T * stride,), 60.0, dtype=torch.bfloat16, device=dev())
        rows = flat[off:].view(T, stride)[:, :V]
        rows.copy_(buf[:, :V])
        same(lmh.lmhead_top_logprobs(rows, to_dev(ids), 0.9), want)
    for a, b in [(0, 1), (39, 40), (7, 20)]:
        same(lmh.lmhead_top_logprobs(buf[a:b, :V].clone(), to_dev(ids[a:b]), 0.9),
             [v[a:b] for v in want])


@pytest.mark.parametrize("T", [3, 60, 200])
def test_top_while_its_inputs_change(T):
    # A caller that forgets to order two streams gets senseless alternatives, nothing worse:
    # one reading of a temperature decides a CTA's way, and every index is bounded.
    import torch

    V = 40003
    x, g = logit_rows(T, T, V)
    good = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    wild = torch.randint(-32768, 32767, (T, V), device=dev(), dtype=torch.int16).view(torch.bfloat16)
    flat = torch.zeros_like(good)
    lg = good.clone()
    t = torch.full((T,), 0.9, device=dev())
    ts = [t.clone(), torch.full_like(t, 0.0), torch.full_like(t, float("nan")), torch.full_like(t, 1e-30)]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for i in range(200):
        with torch.cuda.stream(other):
            lg.copy_((wild, good, flat)[i % 3])
            t.copy_(ts[i % 4])
        lmh.lmhead_top_logprobs(lg, None, t, top=100)
    torch.cuda.synchronize()
    t.fill_(0.9)
    same(lmh.lmhead_top_logprobs(good, None, t, top=100), lmh.lmhead_top_logprobs(good, None, 0.9, top=100))


def test_top_many_rows():
    import torch

    x, g = logit_rows(9, 3000, 20003)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    lp, ent, tok, tlp = lmh.lmhead_top_logprobs(lg, None, 1.0, top=5)
    s, i = torch.sort(lg.float(), dim=1, descending=True, stable=True)
    assert torch.equal(tok.long(), i[:, :5])
    ref = torch.log_softmax(lg.double(), 1)
    assert (tlp.double() - ref.gather(1, i[:, :5])).abs().max() < 1e-5
    assert (ent.double() + (ref.exp() * ref).sum(1)).abs().max() < 5e-5


def test_top_agrees_with_the_sampler_and_the_formula():
    import torch

    x, g = logit_rows(71, 64, 32000)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    t = to_dev((0.5 + g.random(64)).astype(np.float32))
    t[:5] = 0.0
    tok, lp = lmh.lmhead_sample(lg, to_dev(g.random(64, dtype=np.float32)), t, top_p=0.9)
    got, ent, top, tlp = lmh.lmhead_top_logprobs(lg, tok, t)
    assert (got - lp).abs().max() < 1e-5 and torch.equal(top[:5, 0], tok[:5])
    ref, rent = lmh.logprob_from_logits_div(lg, tok, torch.where(t == 0, 1.0, t))[:2]
    assert (got - ref).abs().max() < 1e-5 and (ent - rent).abs().max() < 5e-5


# ------------------------------------------------------------------ together

def step_inputs(B=33, H=512, V=1500):
    h, r = to_dev_bf16(W.random_bf16(81, (B, H), 1.0)), to_dev_bf16(W.random_bf16(82, (B, H), 2.0))
    w = to_dev_bf16(W.random_bf16(83, (V, H), 0.05))
    g = to_dev_bf16(W.f32_to_bf16_bits(np.linspace(0.5, 1.5, H, dtype=np.float32)))
    return h, r, w, g


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_a_step_on_streams_and_in_a_graph(kind):
    import torch

    from invariant_lm_head_gb300.fp4_head import FP4Head
    from invariant_lm_head_gb300.fp8_head import FP8Head

    h, r, w, g = step_inputs()
    u = torch.rand(33, device=dev())
    head = FP8Head(w, g) if kind == "fp8" else FP4Head(w)
    more = {"residual": r} if kind == "fp8" else {}

    def step():
        out = torch.empty(33, 1504, dtype=torch.bfloat16, device=dev())[:, :1500]
        tok, lp = head.sample(h, u, 0.8, top_p=0.9, out_logits=out, **more)
        return (tok, lp, *lmh.lmhead_top_logprobs(out, tok, 0.8, top=5))

    want = step()
    assert (want[1] - want[2]).abs().max() < 1e-5
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    same(got, want)
    graphs = []
    for _ in range(2):  # two captures, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for graph, out in graphs * 2:
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(out, want)
    h.copy_(to_dev_bf16(W.random_bf16(84, (33, 512), 1.0)))  # new inputs, same graph
    graphs[0][0].replay()
    torch.cuda.synchronize()
    same(graphs[0][1], step())
    lmh.lmhead_device_status()


def test_calls_on_a_given_stream():
    import torch

    h, r, w, g = step_inputs()
    q, s = lmh.lmhead_quantize_mxfp4(h)
    wq, ws = lmh.lmhead_quantize_mxfp4(w)
    lg = lmh.lmhead_logits_mxfp4(q, s, wq, ws)
    ids = torch.arange(33, dtype=torch.int32, device=dev())
    calls = [lambda **k: lmh.lmhead_rmsnorm_fp8(h, g, r, **k),
             lambda **k: lmh.lmhead_quantize_mxfp4(h, **k),
             lambda **k: (lmh.lmhead_dequantize_mxfp4(q, s, **k),),
             lambda **k: (lmh.lmhead_logits_mxfp4(q, s, wq, ws, **k),),
             lambda **k: lmh.lmhead_top_logprobs(lg, ids, 0.9, **k)]
    other = torch.cuda.Stream()
    busy = torch.randn(3000, 3000, device=dev())
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        old = [torch.empty_like(t) for t in want for _ in range(8)]
        for _ in range(10):
            busy @ busy
        for t in old:
            t.view(torch.uint8).fill_(85)
        del old, t
        got = call(stream=other)
        torch.cuda.synchronize()
        same(got, want)


def test_two_calls_at_once():
    # two streams, different inputs, many times: nothing is shared between calls
    import torch

    ops = [operands(200, 288, 9000, s) for s in (1, 5)]
    want = [lmh.lmhead_logits_mxfp4(*p) for p in ops]
    tops = [lmh.lmhead_top_logprobs(w, None, 1.0) for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, p, w in zip(streams, ops, want):
            with torch.cuda.stream(s):
                got.append((lmh.lmhead_logits_mxfp4(*p), lmh.lmhead_top_logprobs(w, None, 1.0)))
    torch.cuda.synchronize()
    for i, (lg, top) in enumerate(got):
        same((lg,), (want[i % 2],))
        same(top, tops[i % 2])


def test_empty_batches():
    import torch

    from invariant_lm_head_gb300.fp4_head import FP4Head

    w = torch.randn(1003, 256, device=dev()).to(torch.bfloat16)
    head, h, u = FP4Head(w), w[:0], torch.empty(0, device=dev())
    n = lmh.lmhead_kernel_launches()
    assert head.logits(h).shape == (0, 1003)
    tok, lp = head.sample(h, u)
    assert tok.shape == (0,) and lp.shape == (0,)
    q, s, r = lmh.lmhead_rmsnorm_fp8(h, w[0], h)
    assert q.shape == (0, 256) and s.shape == (0, 2) and r.shape == (0, 256)
    got = lmh.lmhead_top_logprobs(torch.empty(0, 1003, dtype=torch.bfloat16, device=dev()), tok)
    assert [t.shape[0] for t in got] == [0] * 4 and lmh.lmhead_kernel_launches() == n


def test_fp4_head():
    import torch

    from invariant_lm_head_gb300.fp4_head import FP4Head

    w = to_dev_bf16(W.random_bf16(91, (2007, 384), 0.05))
    h = to_dev_bf16(W.random_bf16(92, (9, 384), 1.0))
    u = torch.rand(9, device=dev())
    head = FP4Head(w)
    assert (head.vocab_size, head.hidden_size) == (2007, 384)
    lg = head.logits(h)
    check_logits(lg, *lmh.lmhead_quantize_mxfp4(h), head.weight_q, head.weight_scale)
    assert torch.equal(head.weight(), lmh.lmhead_dequantize_mxfp4(head.weight_q, head.weight_scale))
    full = h.double() @ w.double().t()
    assert (lg.double() - full).norm() / full.norm() < 0.2  # 0.112 each for normal values, and slack
    tok, lp = head.sample(h, u, 0.8, top_k=40)
    same((tok, lp), lmh.lmhead_sample(lg, u, 0.8, top_k=40))
    mask = torch.ones(2007, dtype=torch.bool, device=dev())
    mask[[3, 77]] = False
    out = torch.empty(9, 2008, dtype=torch.bfloat16, device=dev())[:, :2007]
    tok, lp = head.sample(h, u, mask=mask, out_logits=out)
    assert set(tok.tolist()) <= {3, 77}
    got = lmh.lmhead_top_logprobs(out, tok, top=4)
    assert (got[0] - lp).abs().max() < 1e-5 and (got[2][:, 2:] == -1).all()
    w2 = to_dev_bf16(W.random_bf16(93, (2007, 384), 0.05))
    q0 = head.weight_q.data_ptr()
    head.refresh(w2)
    assert head.weight_q.data_ptr() == q0
    assert torch.equal(head.logits(h), FP4Head(w2).logits(h))


def test_fp8_head_with_its_norm():
    import torch

    from invariant_lm_head_gb300.fp8_head import FP8Head

    h, r, w, g = step_inputs()
    head = FP8Head(w, g, 1e-5)
    q, s, _ = lmh.lmhead_rmsnorm_fp8(h, g, r, eps=1e-5)
    assert torch.equal(head.logits(h, residual=r),
                       lmh.lmhead_logits_fp8(q, s, head.weight_q, head.weight_scale))
    q, s, none = lmh.lmhead_rmsnorm_fp8(h, g, eps=1e-5)
    assert none is None and torch.equal(head.logits(h),
                                        lmh.lmhead_logits_fp8(q, s, head.weight_q, head.weight_scale))
    x = (h.double() + r.double())
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5) * g.double()
    full = y @ w.double().t()
    assert (head.logits(h, residual=r).double() - full).norm() / full.norm() < 0.1


def test_capture_before_any_other_call():
    # a process whose first calls of each kind but one are captured ones
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, invariant_lm_head_gb300 as lmh
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(300, 256, device="cuda", generator=g).to(torch.bfloat16)
w = torch.randn(70000, 256, device="cuda", generator=g).to(torch.bfloat16)
n = torch.ones(256, device="cuda").to(torch.bfloat16)
lmh.lmhead_quantize_fp8(x)
def step(V):
    q = lmh.lmhead_quantize_mxfp4(x)
    lg = lmh.lmhead_logits_mxfp4(*q, *lmh.lmhead_quantize_mxfp4(w[:V]))
    return (lg, lmh.lmhead_dequantize_mxfp4(*q), *lmh.lmhead_rmsnorm_fp8(x, n, x),
            *lmh.lmhead_top_logprobs(lg, None, 0.7)[1:])
torch.cuda.synchronize()
got = []
for V in (1000, 20003, 70000):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(V)
    graph.replay()
    torch.cuda.synchronize()
    got.append([t.clone() for t in out])
for V, a in zip((1000, 20003, 70000), got):
    for s, t in zip(a, step(V)):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_example_runs(kind):
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "serve_alternatives.py"),
                        "--head", kind, "--batch", "5", "--hidden", "256", "--vocab", "1003",
                        "--steps", "8"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens/s" in r.stdout


@pytest.mark.parametrize("where", ["stream", "graph"])
def test_calls_that_depend_on_each_other_back_to_back(where):
    # each call begins while the one ahead ends: it must see all that one wrote, and
    # must not write what that one still reads
    import torch

    B, H, V = 300, 512, 9001
    h, r0, w, g = step_inputs(B, H, V)
    r, q, s = r0.clone(), *lmh.lmhead_quantize_mxfp4(h)
    wq, ws = lmh.lmhead_quantize_mxfp4(w)
    x = h.clone()
    logits = torch.empty(B, 9008, dtype=torch.bfloat16, device=dev())[:, :V]
    n = 40

    def chain(sync):
        # the residual in place, a 4-bit round trip of it as the next input, its logits
        # into one buffer, and what is read there
        wait = torch.cuda.synchronize if sync else lambda: None
        out = []
        for _ in range(n):
            nq, ns, _ = lmh.lmhead_rmsnorm_fp8(x, g, r, out_residual=r)
            wait()
            lmh.lmhead_quantize_mxfp4(r, out=q, out_scale=s)
            wait()
            lmh.lmhead_dequantize_mxfp4(q, s, out=x)
            wait()
            x.mul_(-0.25)
            wait()
            lmh.lmhead_logits_mxfp4(q, s, wq, ws, out_logits=logits)
            wait()
            out += [nq, ns, *lmh.lmhead_top_logprobs(logits, None, 0.8, top=4)[1:]]
            wait()
        return out

    def start():
        r.copy_(r0)
        x.copy_(h)

    want = [t.clone() for t in chain(True)]
    end = r.clone()
    assert not torch.equal(end, r0)
    if where == "stream":
        for _ in range(3):
            start()
            got = chain(False)
            torch.cuda.synchronize()
            same(got, want)
            assert torch.equal(r, end)
        return
    graph = torch.cuda.CUDAGraph()
    start()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = chain(False)
    for _ in range(3):
        start()
        graph.replay()
        torch.cuda.synchronize()
        same(got, want)
        assert torch.equal(r, end)


@pytest.mark.parametrize("where", ["streams", "graph"])
def test_calls_behind_two_streams(where):
    # a call that begins early on one stream also waits for what it was told to on another
    import torch

    x = [to_dev_bf16(W.random_bf16(60 + i, (300, 512), 1.0)) for i in range(2)]
    w = [to_dev_bf16(W.random_bf16(70 + i, (40000, 512), 0.05)) for i in range(2)]
    want = [lmh.lmhead_logits_mxfp4(*lmh.lmhead_quantize_mxfp4(a), *lmh.lmhead_quantize_mxfp4(b))
            for a, b in zip(x, w)]
    h, m = torch.empty_like(x[0]), torch.empty_like(w[0])
    hq, wq = lmh.lmhead_quantize_mxfp4(x[0]), lmh.lmhead_quantize_mxfp4(w[0])
    out = torch.empty_like(want[0])
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lmh.lmhead_quantize_mxfp4(m, out=wq[0], out_scale=wq[1])
        lmh.lmhead_quantize_mxfp4(h, out=hq[0], out_scale=hq[1])
        torch.cuda.current_stream().wait_stream(side)
        lmh.lmhead_logits_mxfp4(*hq, *wq, out_logits=out)
        return lmh.lmhead_top_logprobs(out, None, 1.0, top=3)

    tops = [lmh.lmhead_top_logprobs(v, None, 1.0, top=3) for v in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if where == "graph":
        with torch.cuda.graph(graph):
            got = step()
    for i in range(30):
        with torch.cuda.stream(main):
            h.copy_(x[i % 2])
            m.copy_(w[i % 2])
            if where == "graph":
                graph.replay()
            else:
                got = step()
        torch.cuda.synchronize()
        same((out,), (want[i % 2],))
        same(got, tops[i % 2])
