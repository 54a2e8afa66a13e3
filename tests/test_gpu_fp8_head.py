"""The fp8 head on the GPU against the fp64 oracle.

Tolerances. Quantisation is exact: q is the correctly rounded e4m3 value and
scale the correctly rounded fp32 one. Logits: one bf16 rounding (2^-8 of the
value) and the fp32 sums, each of whose at most 128 + KB + 2 roundings is below
2^-23 of the sum of the products' magnitudes (2^-23 rather than 2^-24: the
tensor cores may truncate). Tokens: one of those that the oracle allows when
every border moves by 1e-6, relatively (nearly always exactly one token): a
weight is off by the exponential's few units of 2^-24 and one unit of 2^-44. log-probs: 2^-23 of
the value (its rounding and the difference's), and 1e-6 for the logarithm of a
sum of such weights.
"""

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
import workloads as W
from helpers import dev, to_dev, to_dev_bf16
from oracle import fp8_head as o

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lmh.build()


def bf16_values(bits):
    return W.bf16_bits_to_f32(bits).astype(np.float64)


# ------------------------------------------------------------------ quantisation

def check_quantize(bits, block_rows, x=None):
    x = to_dev_bf16(bits) if x is None else x
    q, s = lmh.lmhead_quantize_fp8(x, block_rows)
    rq, rs = o.quantize(bf16_values(bits), block_rows)
    assert np.array_equal(q.float().cpu().numpy().astype(np.float64), rq)
    assert np.array_equal(s.cpu().numpy(), rs.astype(np.float32))
    return q, s


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (127, 272), (128, 256),
                                       (129, 400), (300, 3600), (2500, 1296)])
def test_quantize(rows, cols, block_rows):
    check_quantize(W.random_bf16(rows * 7 + cols, (rows, cols), 3.0), block_rows)


def test_quantize_every_quotient():
    # every bf16 significand over every maximum's, down to where q rounds to zero
    amax = np.arange(128, dtype=np.uint16) | (127 << 7)
    mags = np.arange((127 - 19) << 7, 128 << 7, dtype=np.uint16)
    per = 127
    n = -(-mags.size // per)
    vals = np.zeros(n * per, np.uint16)
    vals[:mags.size] = mags
    vals[::3] |= 0x8000
    blocks = np.zeros((128, n, 128), np.uint16)
    blocks[:, :, 0] = amax[:, None]
    v = np.broadcast_to(vals.reshape(1, n, per), (128, n, per)).copy()
    v[(v & 0x7FFF) > amax[:, None, None]] = 0
    blocks[:, :, 1:] = v
    check_quantize(blocks.reshape(128, n * 128), 1)


@pytest.mark.parametrize("shift", [-126, -70, -60, -59, 60, 126, 127])
def test_quantize_magnitudes(shift):
    bits = W.random_bf16(5, (64, 256), 0.3)
    e = (bits >> 7) & 0xFF
    e2 = e.astype(np.int32) + shift
    bits = np.where((e2 > 0) & (e2 < 255), (bits & 0x807F) | (np.clip(e2, 0, 254) << 7), 0)
    check_quantize(bits.astype(np.uint16), 1)


def test_quantize_zeros_and_not_finite():
    import torch

    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=dev())
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3, 3] = -2.0
    q, s = lmh.lmhead_quantize_fp8(x)
    q = q.float()
    assert (q[0] == 0).all() and (s[0] == 2.0 ** -60 / 448).all()
    assert q[1, :128].isnan().all() and s[1, 0].isnan() and (q[1, 128:] == 0).all()
    assert q[2, 128:].isnan().all() and s[2, 1].isinf() and (q[2, :128] == 0).all()
    assert q[3, 3] == -448 and s[3, 0] == np.float32(2.0 / 448)


def test_quantize_strided_rows():
    bits = W.random_bf16(11, (130, 512), 1.0)
    x = to_dev_bf16(bits)
    check_quantize(np.ascontiguousarray(bits[:, 128:400]), 1, x[:, 128:400])
    check_quantize(np.ascontiguousarray(bits[::2, :256]), 128, x[::2, :256])


# ------------------------------------------------------------------ logits

def operands(T, H, V, seed=1):
    h, hs = lmh.lmhead_quantize_fp8(to_dev_bf16(W.random_bf16(seed, (T, H), 1.0)), 1)
    w, ws = lmh.lmhead_quantize_fp8(to_dev_bf16(W.random_bf16(seed + 1, (V, H), 0.02)), 128)
    return h, hs, w, ws


def check_logits(out, h, hs, w, ws):
    import torch

    hd = h.double() * hs.double().repeat_interleave(128, 1)[:, :h.shape[1]]
    wd = w.double() * ws.double().repeat_interleave(128, 0)[:w.shape[0]] \
        .repeat_interleave(128, 1)[:, :w.shape[1]]
    ref, mag = hd @ wd.t(), hd.abs() @ wd.abs().t()
    tol = ref.abs() * 2.0 ** -8 + mag * (128 + hs.shape[1] + 2) * 2.0 ** -23
    assert torch.isfinite(out).all()
    assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,H,V", [
    (1, 16, 1), (1, 128, 128), (2, 256, 130), (7, 144, 1000), (8, 3584, 4096), (63, 400, 2047),
    (64, 4096, 2048), (65, 256, 8192), (127, 272, 999), (128, 512, 1024), (129, 512, 1025),
    (200, 3600, 3203), (256, 256, 4096), (257, 640, 513), (700, 1040, 2000), (1300, 384, 777)])
def test_logits(T, H, V):
    ops = operands(T, H, V)
    check_logits(lmh.lmhead_logits_fp8(*ops), *ops)
    lmh.lmhead_device_status()


def test_logits_rows_do_not_depend_on_the_batch():
    import torch

    h, hs, w, ws = operands(600, 1296, 2056)
    whole = lmh.lmhead_logits_fp8(h, hs, w, ws)
    for a, b in [(0, 1), (5, 6), (3, 67), (100, 228), (100, 229), (87, 343), (599, 600), (1, 600)]:
        part = lmh.lmhead_logits_fp8(h[a:b], hs[a:b], w, ws)
        assert torch.equal(part.view(torch.int16), whole[a:b].view(torch.int16)), (a, b)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("ld,off", [(1300, 0), (1301, 0), (1304, 0), (1304, 3), (1296, 8)])
def test_logits_into_strided_rows(T, ld, off):
    import torch

    V = 1288
    ops = operands(T, 256, V)
    buf = torch.full((T * ld + off + 8,), 7.0, dtype=torch.bfloat16, device=dev())
    out = buf[off:off + T * ld].view(T, ld)[:, :V]
    lmh.lmhead_logits_fp8(*ops, out_logits=out)
    check_logits(out, *ops)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[off:off + T * ld].view(T, ld)[:, :V] = False
    assert (buf[rest] == 7.0).all()  # nothing outside the logits is written


@pytest.mark.parametrize("V", [5, 33, 250, 1003])
def test_logits_rows_at_any_address(V):
    # whatever a row's offset in 16 bytes, and wherever the vocabulary ends in it
    import torch

    T = 45
    ops = operands(T, 256, V)
    ld8 = -(-V // 8) * 8
    aligned = torch.empty(T, ld8, dtype=torch.bfloat16, device=dev())[:, :V]
    lmh.lmhead_logits_fp8(*ops, out_logits=aligned)
    check_logits(aligned, *ops)
    for ld in (V, V + 1, ld8 + 2, ld8 + 4):
        for off in range(8):
            buf = torch.full((off + T * ld + 8,), 7.0, dtype=torch.bfloat16, device=dev())
            out = buf[off:off + T * ld].view(T, ld)[:, :V]
            lmh.lmhead_logits_fp8(*ops, out_logits=out)
            assert torch.equal(out.view(torch.int16), aligned.view(torch.int16)), (ld, off)
            out.fill_(7.0)
            assert (buf == 7.0).all(), (ld, off)


def test_logits_a_bad_row_stays_alone():
    import torch

    h, hs, w, ws = operands(40, 256, 300)
    want = lmh.lmhead_logits_fp8(h, hs, w, ws)
    hs2 = hs.clone()
    hs2[7, 1] = float("nan")
    got = lmh.lmhead_logits_fp8(h, hs2, w, ws)
    keep = torch.arange(40, device=dev()) != 7
    assert got[7].isnan().all() and torch.equal(got[keep], want[keep])


# ------------------------------------------------------------------ sampling

TOL = 1e-6


def check_sample(x, u, t=1.0, k=0, p=1.0, m=0.0, logits=None):
    """x: fp32 values that bf16 holds, [T, V]; u and settings scalars or [T] arrays."""
    import torch

    T = x.shape[0]
    if logits is None:
        logits = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).to(dev())
    u = np.broadcast_to(np.asarray(u, np.float32), (T,))

    def arg(v, dtype):
        return to_dev(np.asarray(v, dtype)) if isinstance(v, np.ndarray) else v

    tok, lp = lmh.lmhead_sample(logits, to_dev(u), arg(t, np.float32), top_k=arg(k, np.int32),
                                top_p=arg(p, np.float32), min_p=arg(m, np.float32))
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
    row = lambda v, i: np.float32(v[i] if isinstance(v, np.ndarray) else v)  # noqa: E731
    for i in range(T):
        toks, lps = o.sample_row(x[i], u[i], row(t, i), int(row(k, i)), row(p, i), row(m, i), TOL)
        assert tok[i] in toks, (i, tok[i], toks)
        ref = lps[toks.index(tok[i])]
        assert abs(lp[i] - ref) <= 1e-6 + 2.0 ** -23 * abs(ref), (i, lp[i], ref)
    return tok, lp


def logit_rows(seed, T, V, std=2.0):
    bits = W.random_bf16(seed, (T, V), std)
    x = W.bf16_bits_to_f32(bits).copy()
    g = np.random.Generator(np.random.PCG64(seed))
    for i in range(T):  # some likely tokens
        at = g.integers(0, V, size=min(V, 24))
        x[i, at] = W.bf16_bits_to_f32(W.f32_to_bf16_bits(x[i, at] + g.normal(8, 3, at.size)))
    return x, g


@pytest.mark.parametrize("V", [1, 2, 7, 8, 33, 1000, 4096, 4097, 32003])
@pytest.mark.parametrize("mode", ["plain", "top_k", "top_p", "min_p", "all", "rows"])
def test_sample(V, mode):
    T = 48
    x, g = logit_rows(V, T, V)
    u = g.random(T, dtype=np.float32)
    kw = {"plain": {}, "top_k": dict(k=5, t=0.7), "top_p": dict(p=0.9, t=1.3),
          "min_p": dict(m=0.05), "all": dict(k=40, p=0.8, m=0.02, t=0.6),
          "rows": dict(t=np.where(g.random(T) < 0.2, 0, 0.2 + 2 * g.random(T)).astype(np.float32),
                       k=np.where(g.random(T) < 0.3, 0, g.integers(1, 2 * V + 2, T)),
                       p=np.where(g.random(T) < 0.3, 1, g.random(T) + 1e-3).astype(np.float32),
                       m=np.where(g.random(T) < 0.3, 0, 0.3 * g.random(T)).astype(np.float32))}
    check_sample(x, u, **kw[mode])


def test_sample_full_vocabulary():
    x, g = logit_rows(3, 24, 152064)
    u = g.random(24, dtype=np.float32)
    check_sample(x, u)
    check_sample(x, u, t=0.7, p=0.95)
    check_sample(x, u, t=1.5, k=1000, m=0.001)


@pytest.mark.parametrize("u", [0.0, 1.0])
def test_sample_ends(u):
    x, _ = logit_rows(9, 16, 2000)
    check_sample(x, u)
    check_sample(x, u, k=7)
    check_sample(x, u, p=0.5)
    check_sample(x, u, k=3000, p=1.0)


def test_sample_ties_go_by_index():
    g = np.random.Generator(np.random.PCG64(4))
    u = (np.arange(64, dtype=np.float32) + 0.5) / 64
    x = np.full((64, 64), 1.5, np.float32)
    assert check_sample(x, u)[0].tolist() == list(range(64))
    assert check_sample(x, u, k=16)[0].tolist() == [i // 4 for i in range(64)]
    assert check_sample(x, u, t=0.0)[0].tolist() == [0] * 64
    zeros = np.where(g.random((64, 999)) < 0.5, np.float32(-0.0), np.float32(0.0))
    check_sample(zeros, u)
    check_sample(zeros, u, p=0.37)
    check_sample(g.integers(-2, 3, (64, 5000)).astype(np.float32), u, k=1234, p=0.77)


LOWEST = -3.3895313892515355e38


@pytest.mark.parametrize("mask", [-np.inf, LOWEST, np.nan])
@pytest.mark.parametrize("share", [0.5, 0.999, 1.0])
def test_sample_masks(mask, share):
    x, g = logit_rows(21, 32, 3001)
    x[g.random(x.shape) < share] = mask
    if mask == LOWEST or share < 1:
        check_sample(x, g.random(32, dtype=np.float32), t=0.8, p=0.9)
        check_sample(x, g.random(32, dtype=np.float32), t=0.3)
    else:
        tok, lp = check_sample(x, 0.5)
        assert (tok == -1).all() and (lp == 0).all()
    check_sample(x, 0.5, t=0.0)


def test_sample_values_outside_the_usual_range():
    x, g = logit_rows(33, 40, 2500)
    u = g.random(40, dtype=np.float32)
    r = lambda v: W.bf16_bits_to_f32(W.f32_to_bf16_bits(v.astype(np.float32)))  # noqa: E731
    check_sample(r(x * 1e-12), u)                     # all tiny: flat rows
    check_sample(r(x * 1e-12), u, t=1e-12, p=0.9)     # and peaked ones
    check_sample(r(x * 1e30), u, t=1e30, k=50)
    check_sample(r(x + 300.0), u, t=0.9, p=0.95)
    check_sample(r(x - 500.0), u)
    check_sample(r(x * 300.0), u, t=300.0, p=0.9, m=0.01)
    y = x.copy()
    y[:, ::3] = r(1e-20 * g.normal(size=y[:, ::3].shape))
    check_sample(y, u, t=2.0)
    y[:, 5] = np.inf
    y[::2, 9] = np.inf
    tok, _ = check_sample(y, u)
    assert (tok[1::2] == 5).all() and set(tok[::2]) <= {5, 9}
    check_sample(np.full((40, 7), LOWEST, np.float32), u, t=0.5)   # z overflows
    check_sample(np.full((40, 7), -LOWEST, np.float32), u, t=0.5)


def test_sample_strides_and_offsets():
    import torch

    x, g = logit_rows(41, 20, 1003)
    u = g.random(20, dtype=np.float32)
    for ld, off in [(1003, 0), (1003, 1), (1008, 5), (1200, 8)]:
        buf = torch.full((20 * ld + off,), 30.0, dtype=torch.bfloat16, device=dev())
        view = buf[off:off + 20 * ld].view(20, ld)[:, :1003]
        view.copy_(torch.from_numpy(x))
        check_sample(x, u, p=0.9, logits=view)


def test_sample_bad_settings_of_a_row():
    import torch

    x, g = logit_rows(51, 12, 500)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    f = lambda *v: torch.tensor(v, device=dev())  # noqa: E731
    nan, inf = float("nan"), float("inf")
    t = f(1., -1., nan, inf, 1., 1., 1., 1., 1., 1., 1., 0.)
    k = torch.tensor([0, 0, 0, 0, -1, 0, 0, 0, 0, 0, 0, 0], dtype=torch.int32, device=dev())
    p = f(1., 1., 1., 1., 1., 0., nan, 1., 1., 1., 1., 2.)
    m = f(0., 0., 0., 0., 0., 0., 0., 1.5, nan, 0., 0., -1.)
    u = f(.5, .5, .5, .5, .5, .5, .5, .5, .5, nan, 1.5, .5)
    tok, lp = lmh.lmhead_sample(lg, u, t, top_k=k, top_p=p, min_p=m)
    assert (tok[1:11] == -1).all() and lp[1:11].isnan().all()
    assert tok[0] >= 0 and tok[11] == lg[11].float().argmax()


def test_sample_does_not_depend_on_the_batch():
    import torch

    x, g = logit_rows(61, 300, 5000)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    u = to_dev(g.random(300, dtype=np.float32))
    tok, lp = lmh.lmhead_sample(lg, u, 0.9, top_p=0.97)
    for a, b in [(0, 1), (7, 8), (10, 30), (100, 299), (0, 300)]:
        tk, l2 = lmh.lmhead_sample(lg[a:b], u[a:b], 0.9, top_p=0.97)
        assert torch.equal(tk, tok[a:b]) and torch.equal(l2, lp[a:b])


def test_sample_logprob_is_the_sampler_formula():
    # the trainer's log-prob of the drawn token, within its own tolerance
    import torch

    x, g = logit_rows(71, 64, 32000)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    t = to_dev((0.5 + g.random(64)).astype(np.float32))
    tok, lp = lmh.lmhead_sample(lg, to_dev(g.random(64, dtype=np.float32)), t, top_p=0.9)
    ref = lmh.logprob_from_logits_div(lg, tok, t)[0]
    assert (lp - ref).abs().max() < 1e-5


# ------------------------------------------------------------------ together

def test_streams_and_graphs():
    import torch

    h = to_dev_bf16(W.random_bf16(81, (33, 512), 1.0))
    w, ws = lmh.lmhead_quantize_fp8(to_dev_bf16(W.random_bf16(82, (1500, 512), 0.05)), 128)
    u = torch.rand(33, device=dev())

    def step():
        hq, hs = lmh.lmhead_quantize_fp8(h)
        lg = lmh.lmhead_logits_fp8(hq, hs, w, ws)
        return (lg, *lmh.lmhead_sample(lg, u, 0.8, top_p=0.9))

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for o_ in out:
        o_.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    h.copy_(to_dev_bf16(W.random_bf16(83, (33, 512), 1.0)))  # new inputs, same graph
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    lmh.lmhead_device_status()


def test_head_class():
    import torch

    from invariant_lm_head_gb300.fp8_head import FP8Head

    w = to_dev_bf16(W.random_bf16(91, (2007, 384), 0.05))
    h = to_dev_bf16(W.random_bf16(92, (9, 384), 1.0))
    u = torch.rand(9, device=dev())
    head = FP8Head(w)
    assert (head.vocab_size, head.hidden_size) == (2007, 384)
    lg = head.logits(h)
    check_logits(lg, *lmh.lmhead_quantize_fp8(h), head.weight_q, head.weight_scale)
    tok, lp = head.sample(h, u, 0.8, top_k=40)
    want = lmh.lmhead_sample(lg, u, 0.8, top_k=40)
    assert torch.equal(tok, want[0]) and torch.equal(lp, want[1])
    mask = torch.ones(2007, dtype=torch.bool, device=dev())
    mask[[3, 77]] = False
    out = torch.empty(9, 2008, dtype=torch.bfloat16, device=dev())[:, :2007]
    tok, lp = head.sample(h, u, mask=mask, out_logits=out)
    assert set(tok.tolist()) <= {3, 77} and (out[:, 4] == float("-inf")).all()
    w2 = to_dev_bf16(W.random_bf16(93, (2007, 384), 0.05))
    q0 = head.weight_q.data_ptr()
    head.refresh(w2)
    assert head.weight_q.data_ptr() == q0
    assert torch.equal(head.logits(h), FP8Head(w2).logits(h))


def test_example_runs():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "serve_fp8_head.py"),
                        "--batch", "5", "--hidden", "256", "--vocab", "1003", "--steps", "8"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens/s" in r.stdout


@pytest.mark.parametrize("T", [1, 19, 38, 39, 76, 77, 152, 153, 400])
def test_sample_every_split_of_a_row(T):
    # rows go to 8, 4, 2 or 1 CTAs by their number; each must give the oracle's token every time
    import torch

    V = 2043
    x, g = logit_rows(T, T, V)
    u = g.random(T, dtype=np.float32)
    tok, lp = check_sample(x, u, t=0.9, p=0.95, k=500)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    for _ in range(20):
        t2, l2 = lmh.lmhead_sample(lg, to_dev(u), 0.9, top_k=500, top_p=0.95)
        assert np.array_equal(t2.cpu().numpy(), tok) and np.array_equal(l2.cpu().numpy(), lp)


@pytest.mark.parametrize("T", [3, 60, 120, 200])
def test_sample_while_its_inputs_change(T):
    # A caller that forgets to order two streams gets senseless tokens, nothing worse:
    # every thread follows one copy of what decides its way, and every index is bounded.
    import torch

    V = 3003
    x, g = logit_rows(T, T, V)
    good = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    wild = torch.randint(-32768, 32767, (T, V), device=dev(), dtype=torch.int16).view(torch.bfloat16)
    lg, u = good.clone(), torch.rand(T, device=dev())
    t = torch.full((T,), 0.9, device=dev())
    ts = [t.clone(), torch.full_like(t, 0.0), torch.full_like(t, float("nan")),
          torch.full_like(t, 1e-30)]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for i in range(200):
        with torch.cuda.stream(other):
            lg.copy_(wild if i % 2 else good)
            t.copy_(ts[i % 4])
        lmh.lmhead_sample(lg, u, t, top_p=0.9, top_k=1000)
    torch.cuda.synchronize()
    uu = u.cpu().numpy()
    check_sample(x, uu, t=0.9, p=0.9, k=1000, logits=good)
