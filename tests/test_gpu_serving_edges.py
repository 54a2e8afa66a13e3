"""Around the quantised heads on the GPU: edges of rows, batches, grids and arguments.

Tolerances are those of test_gpu_serving.py, where they are derived.
"""

import ctypes

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
import workloads as W
from helpers import dev, to_dev, to_dev_bf16
from oracle import serving as o
from test_gpu_serving import (LOWEST, check_logits, f64, logit_rows, near, norm_inputs, operands,
                              same, step_inputs)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lmh.build()


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("eps", [1e-37, 1e-39, 1e-42, 2.0 ** -149])
@pytest.mark.parametrize("cols", [272, 8000, 20000])
def test_norm_with_an_eps_near_the_squares(cols, eps):
    # squares at and below the smallest fp32 numbers, beside an eps that is no larger
    x = W.random_bf16(3, (12, cols), 1.0)
    size = np.float32([1e-19, 1e-20, 1e-21, 3e-22, 1e-22, 3e-23, 1e-23, 1e-24, 1e-26, 1.0, 1e-35, 0.0])
    x = W.f32_to_bf16_bits(W.bf16_bits_to_f32(x) * size[:, None])
    w = W.random_bf16(4, (1, cols), 1.0)[0]
    q, s, _ = lmh.lmhead_rmsnorm_fp8(to_dev_bf16(x), to_dev_bf16(w), eps=eps)
    eps = float(np.float32(eps))
    rq, rs, _ = o.rmsnorm_fp8(W.bf16_bits_to_f32(x).astype(np.float64),
                              W.bf16_bits_to_f32(w).astype(np.float64), None, eps)
    assert (np.abs(f64(s) - rs) <= 32 * 2.0 ** -24 * rs).all()
    usual = np.arange(12) != 10  # its products are below 2^-100 and take the rounded y
    assert np.array_equal(f64(q)[usual], rq[usual])


def check_rounded(q, quotient):
    """q is the e4m3 value next to the quotient that the kernel has: off by half a step, by the
    row's factor's 2^-19 and by the four roundings of y and of the block's largest y."""
    _, e = np.frexp(np.abs(quotient))
    half = np.ldexp(0.5, np.maximum(e - 1, -6) - 3)
    assert (np.abs(q - quotient) <= half + (2.0 ** -19 + 2.0 ** -22) * np.abs(quotient)).all()


@pytest.mark.parametrize("cols", [400, 4096, 8192, 16400])
@pytest.mark.parametrize("scale", [1e-36, 5e-32, 1e-25, 1e-12])
def test_norm_values_of_small_rows(scale, cols):
    # rows of which every block is below the floor (1e-36), or above it with products too
    # small to be exact (5e-32), or exact
    eps = float(np.float32(1e-30))
    x = W.random_bf16(11, (9, cols), 1.0)
    x = W.f32_to_bf16_bits(W.bf16_bits_to_f32(x) * np.float32(scale))
    w = norm_inputs(1, cols)[2]
    q, s, _ = lmh.lmhead_rmsnorm_fp8(to_dev_bf16(x), to_dev_bf16(w), eps=eps)
    xv, wv = (W.bf16_bits_to_f32(v).astype(np.float64) for v in (x, w))
    rq, rs, _ = o.rmsnorm_fp8(xv, wv, None, eps)
    assert (np.abs(f64(s) - rs) <= 32 * 2.0 ** -24 * rs).all()
    if scale > 1e-30:
        assert np.array_equal(f64(q), rq)
    else:
        y = xv * wv / np.sqrt((xv * xv).mean(1, keepdims=True) + eps)
        check_rounded(f64(q), y / np.repeat(rs, 128, 1)[:, :cols])
    assert (np.abs(f64(q)).max(1) >= 0.25).all()  # 1e-36: 1e-21 * 448 / 2^-60 is about a half


@pytest.mark.parametrize("cols", [640, 4096, 8192, 20000])
def test_norm_blocks_below_the_floor_beside_others(cols):
    # blocks of ordinary size, below the floor with values that do not vanish there, and
    # all zero, in the same warps
    x = W.bf16_bits_to_f32(W.random_bf16(12, (20, cols), 1.0))
    block = np.arange(cols) // 128
    size = np.float32([1.0, 2.0 ** -62, 2.0 ** -66, 1.0, 0.0])
    rows = np.arange(20)[:, None]
    x = W.f32_to_bf16_bits(x * size[(block[None] + rows) % 5])
    w = norm_inputs(1, cols)[2]
    q, s, _ = lmh.lmhead_rmsnorm_fp8(to_dev_bf16(x), to_dev_bf16(w))
    xv, wv = (W.bf16_bits_to_f32(v).astype(np.float64) for v in (x, w))
    rq, rs, _ = o.rmsnorm_fp8(xv, wv, None, float(np.float32(1e-6)))
    assert (np.abs(f64(s) - rs) <= 32 * 2.0 ** -24 * rs).all()
    q, kind = f64(q), (block[None] + rows) % 5
    ordinary = (kind == 0) | (kind == 3)
    assert np.array_equal(q[ordinary], rq[ordinary])
    y = xv * wv / np.sqrt((xv * xv).mean(1, keepdims=True) + float(np.float32(1e-6)))
    check_rounded(q, y / np.repeat(rs, 128, 1)[:, :cols])
    for k in (1, 2):
        assert (q[kind == k] != 0).any()
    assert (q[kind == 4] == 0).all()


# ------------------------------------------------------------------ 4-bit logits

@pytest.mark.parametrize("step", [16, 8])
@pytest.mark.parametrize("T,V", [(1, 78003), (33, 78100), (97, 40017), (141, 39999), (300, 20250)])
def test_logits_where_the_lanes_of_a_warp_part(T, V, step):
    # rows past T and a vocabulary that ends inside a box, each followed by reads of the
    # boxes behind it and of the CTA's next tiles; rows on 32 and on 16 bytes
    import torch

    ops = operands(T, 96, V)
    ld = -(-V // 16) * 16 + step
    buf = torch.full((T, ld), 7.0, dtype=torch.bfloat16, device=dev())
    out = lmh.lmhead_logits_mxfp4(*ops, out_logits=buf[:, :V])
    check_logits(out, *ops)
    assert (buf[:, V:] == 7.0).all()
    lmh.lmhead_device_status()


# ------------------------------------------------------------------ alternatives

def rows_of_every_kind(T, V):
    """(logits as bf16 values in fp32, temperatures, tokens): plain rows, and at the start
    ties past the list, masks, infinities and temperatures far from 1."""
    x, g = logit_rows(T + V, T, V)
    x[0] = 0.25  # all equal
    x[1] = LOWEST
    x[1, V - 3:] = 2.0, 1.0, 1.0
    x[2] = -np.inf
    x[2, V - 1] = -4.0
    x[3] = -np.inf
    x[4, ::2] = np.nan
    x[5, V - 6000:V - 2000] = 30.0  # the largest in one run, behind the middle
    x[6, V - 9] = np.inf
    x[7, [3, V // 2, V - 2]] = np.inf
    x[8] *= np.float32(1e37)
    x[12, g.random(V) < 0.98] = -np.inf
    x[13, V // 4:] = -np.inf  # nothing behind the first quarter
    x[14, :3 * V // 4] = np.nan  # nothing before the last
    x[15, ::3] = -2.984375  # more on one level than a list holds, a few above
    x[16] = np.round(x[16])
    t = (0.5 + g.random(T)).astype(np.float32)
    t[9], t[10], t[11], t[17] = 1e-30, 1e30, 0.0, 2e-39
    ids = g.integers(0, V, (T, 3)).astype(np.int32)
    ids[:20, 0] = V - 1
    ids[3:6, 1] = -1, V, 2 ** 31 - 1
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(x)), t, ids


def batch_of_two_ctas(which):
    """77, 100 and 152 rows where the device has 152 SMs: rows that two CTAs share."""
    import torch

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return {"first": sms // 2 + 1, "middle": 2 * sms // 3, "last": sms}[which]


@pytest.mark.parametrize("n", [1, 20, 128])
@pytest.mark.parametrize("V", [32003, 70000, 152064])
@pytest.mark.parametrize("which", ["first", "middle", "last"])
def test_top_of_rows_that_two_ctas_share(which, V, n):
    # against the formula; and the bits of the rows alone, in a batch of one CTA a row, and
    # at addresses that are not on 16 bytes
    import torch

    T = batch_of_two_ctas(which)
    x, t, ids = rows_of_every_kind(T, V)
    lg = torch.from_numpy(x).to(dev()).to(torch.bfloat16)
    ts, tokens = to_dev(t), to_dev(ids)
    got = lmh.lmhead_top_logprobs(lg, tokens, ts, top=n)
    lp, ent, tok, tlp = [v.cpu().numpy() for v in got]
    for i in [*range(20), T // 2, T - 1]:
        rlp, rent, rtok, rtlp = o.top_row(x[i], t[i], n, ids[i])
        assert np.array_equal(tok[i], rtok), (i, tok[i], rtok)
        near(tlp[i], rtlp)
        near(lp[i], rlp)
        assert abs(ent[i] - rent) <= 3e-6 * (2 + 2 * abs(rent)), i
    for a, b in [(0, 12), (12, 40), (T - 1, T)]:
        alone = lmh.lmhead_top_logprobs(lg[a:b], tokens[a:b], ts[a:b], top=n)
        same(alone, [v[a:b] for v in got])
    many = [v.repeat(6, *[1] * (v.dim() - 1)) for v in (lg, tokens, ts)]
    whole = lmh.lmhead_top_logprobs(many[0], many[1], many[2], top=n)
    for i in (0, 5):
        same([v[i * T:(i + 1) * T] for v in whole], got)
    for stride, off in [(V + 1, 1), (V + 5, 4)]:
        flat = torch.full((off + T * stride,), 60.0, dtype=torch.bfloat16, device=dev())
        odd = flat[off:].view(T, stride)[:, :V]
        odd.copy_(lg)
        same(lmh.lmhead_top_logprobs(odd, tokens, ts, top=n), got)
    lmh.lmhead_device_status()


@pytest.mark.parametrize("V", [32003, 152064])
@pytest.mark.parametrize("T", [3, 100])
def test_top_bad_temperatures_of_rows_that_ctas_share(T, V):
    import torch

    x, g = logit_rows(T, T, V)
    lg = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    ids = to_dev(np.stack([g.integers(0, V, T), np.full(T, -1)], 1).astype(np.int32))
    t = torch.ones(T, device=dev())
    for bad in (-1.0, float("nan"), float("inf"), -float("inf")):
        t[1::2] = bad
        lp, ent, tok, tlp = lmh.lmhead_top_logprobs(lg, ids, t, top=30)
        assert lp[1::2].isnan().all() and ent[1::2].isnan().all()
        assert (tok[1::2] == -1).all() and tlp[1::2].isnan().all()
        good = lmh.lmhead_top_logprobs(lg, ids, 1.0, top=30)
        same([v[::2] for v in (lp, ent, tok, tlp)], [v[::2] for v in good])


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launched_grids(call):
    """The grids of the kernels that a call launches, from a graph that it is captured into."""
    import torch

    cuda = ctypes.CDLL("libcuda.so.1")
    stream, graph, n = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        handle = ctypes.c_void_p(stream.cuda_stream)
        assert cuda.cuStreamBeginCapture_v2(handle, 2) == 0
        try:
            call()
        finally:
            assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert cuda.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes, grids = (ctypes.c_void_p * n.value)(), []
    assert cuda.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        p = KernelNode()
        assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        grids.append(tuple(p.grid))
    assert cuda.cuGraphDestroy(graph) == 0
    return grids


@pytest.mark.parametrize("V", [5, 8192, 8193, 9001, 16000, 16384, 16385, 24576, 24577, 32003, 152064])
@pytest.mark.parametrize("T", [1, 48, 100, 400])
def test_top_launches_no_idle_half(T, V):
    # of the CTAs that share a row, more than half have a part of it; the row's bits are
    # those of any other batch
    import torch

    lg = torch.randn(T, V, device=dev(), generator=torch.Generator(device=dev()).manual_seed(V)).to(torch.bfloat16)
    outs = dict(out_entropy=torch.empty(T, device=dev()),
                out_top_token=torch.empty(T, 5, dtype=torch.int32, device=dev()),
                out_top_logprob=torch.empty(T, 5, device=dev()))
    lmh.lmhead_top_logprobs(lg, top=5, **outs)
    got = [v.clone() for v in outs.values()]
    grids = launched_grids(lambda: lmh.lmhead_top_logprobs(lg, top=5, **outs))
    assert len(grids) == 1 and grids[0][0] % T == 0
    ctas = grids[0][0] // T
    assert ctas in (1, 2, 4)
    vectors = -(-V // 8)  # a slice: a quarter of the row in whole runs of 32, 1024 at least
    slices = -(-vectors // max(1024, -(-(-(-vectors // 4)) // 32) * 32))
    assert ctas == 1 or 2 * -(-slices * ctas // 4) > ctas
    same(lmh.lmhead_top_logprobs(lg[T - 1:], top=5)[1:], [v[T - 1:] for v in got])


# ------------------------------------------------------------------ heads

def test_fp8_head_takes_over_a_new_norm():
    # in a captured graph too; a trainer's parameter as the norm's weight, and updates in place
    import torch

    from invariant_lm_head_gb300.fp8_head import FP8Head

    h, r, w, g = step_inputs()
    w2, g2 = w.flip(0).contiguous(), (g.float() * 1.5 + 0.25).to(torch.bfloat16)
    norm = torch.nn.Parameter(g.clone())
    head = FP8Head(w, norm, 1e-5)
    at = norm.data_ptr()
    head.logits(h, residual=r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = head.logits(h, residual=r)

    def expect(weight, norm_weight):
        want = FP8Head(weight, norm_weight, 1e-5).logits(h, residual=r)
        graph.replay()
        assert torch.equal(head.logits(h, residual=r), want) and torch.equal(out, want)

    expect(w, g)
    head.refresh(w2, torch.nn.Parameter(g2))
    assert head.norm_weight.data_ptr() == at
    expect(w2, g2)
    head.refresh(w)  # the norm's stays
    expect(w, g2)
    with torch.no_grad():
        norm.copy_(g)  # the tensor that the head holds
    expect(w, g)
    head.refresh(w2, norm)
    expect(w2, g)
