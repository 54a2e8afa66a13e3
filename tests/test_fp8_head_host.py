"""Host-side checks of the fp8 head: the oracle's pins, and refusals before any device use."""

import math

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
from oracle import fp8_head as o


@pytest.fixture(scope="module")
def lib():
    lmh.build()
    return lmh.library()


def test_e4m3_rounding_against_every_value():
    vals = np.sort(o.e4m3_values()[np.isfinite(o.e4m3_values())])
    assert vals.max() == 448 and vals[vals > 0].min() == 2.0 ** -9
    assert np.array_equal(o.e4m3(vals), vals)
    pos = np.unique(np.abs(vals))
    mid = (pos[1:] + pos[:-1]) / 2
    for eps, want in ((-1e-9, pos[:-1]), (1e-9, pos[1:])):
        assert np.array_equal(o.e4m3(mid * (1 + eps)), want)
    # ties go to the even code: code i is between codes i and i + 1
    even = np.where(np.arange(mid.size) % 2 == 0, pos[:-1], pos[1:])
    assert np.array_equal(o.e4m3(mid), even)


def test_sample_row_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3], np.float32))
    pick = lambda u, **kw: o.sample_row(x, u, 1.0, **kw)[0][0]  # noqa: E731
    assert [pick(u) for u in (0.0, 0.39, 0.41, 0.69, 0.71, 0.89, 0.91, 1.0)] == \
        [1, 1, 3, 3, 2, 2, 0, 0]
    assert [pick(u, k=2) for u in (0.0, 0.56, 0.58, 1.0)] == [1, 1, 3, 3]
    assert [pick(u, p=0.6) for u in (0.56, 0.58, 1.0)] == [1, 3, 3]
    assert pick(0.999, p=0.01) == 1 and pick(0.999, min_p=0.7) == 3 and pick(0.9, k=1) == 1
    tok, lp = o.sample_row(x, 0.5, 1.0)
    assert tok == [3] and lp[0] == pytest.approx(math.log(0.3), abs=1e-7)
    assert o.sample_row(x, 0.99, 0.0)[0] == [1]
    assert o.sample_row(np.full(3, -np.inf), 0.5, 1.0) == ([-1], [0.0])
    assert o.sample_row(x, 0.5, 1.0, tol=1e-6)[0] == [3]
    assert o.sample_row(x, 0.4, 1.0, tol=1e-6)[0] == [1, 3]  # on a border: either
    ties = np.zeros(4, np.float32)
    assert [o.sample_row(ties, u, 1.0)[0][0] for u in (0.0, 0.25, 0.5, 0.99)] == [0, 1, 2, 3]


def test_quantize_refusals(lib):
    before = lib.lmhead_kernel_launches()
    f = lib.lmhead_quantize_fp8
    ok = dict(x=16, rows=4, cols=256, ld=256, br=1, q=16, s=16)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["x"], a["rows"], a["cols"], a["ld"], a["br"], a["q"], a["s"], None)

    for bad in (dict(rows=-1), dict(cols=0), dict(rows=2147483393), dict(cols=2147483393),
                dict(br=0), dict(br=64), dict(ld=255), dict(x=None), dict(q=None), dict(s=None)):
        assert call(**bad) == lmh.LMH_ERR_INVALID_ARG, bad
    for bad in (dict(cols=8), dict(cols=100, ld=104), dict(ld=260), dict(x=24), dict(q=24),
                dict(s=18)):
        assert call(**bad) == lmh.LMH_ERR_ALIGNMENT, bad
    assert call(rows=0, x=None, q=None, s=None) == lmh.LMH_OK
    assert lib.lmhead_kernel_launches() == before


def test_logits_refusals(lib):
    before = lib.lmhead_kernel_launches()
    ok = dict(hq=16, hs=16, wq=16, ws=16, T=4, H=256, V=1000, out=16, ld=1000)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.lmhead_logits_fp8(a["hq"], a["hs"], a["wq"], a["ws"], a["T"], a["H"], a["V"],
                                     a["out"], a["ld"], None)

    for bad in (dict(T=-1), dict(V=0), dict(H=0), dict(T=2147483393), dict(ld=999), dict(hq=None),
                dict(hs=None), dict(wq=None), dict(ws=None), dict(out=None),
                dict(T=2147483392, V=2147483392, ld=2147483392)):
        assert call(**bad) == lmh.LMH_ERR_INVALID_ARG, bad
    for bad in (dict(H=200), dict(hq=8), dict(wq=24), dict(hs=18), dict(ws=2), dict(out=17)):
        assert call(**bad) == lmh.LMH_ERR_ALIGNMENT, bad
    assert call(T=0, hq=None, hs=None, out=None) == lmh.LMH_OK
    assert lib.lmhead_kernel_launches() == before


def test_sample_refusals(lib):
    before = lib.lmhead_kernel_launches()
    ok = dict(x=2, T=4, V=1000, ld=1000, t=1.0, rt=None, k=0, rk=None, p=1.0, rp=None, m=0.0,
              rm=None, u=16, tok=16, lp=16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.lmhead_sample(a["x"], a["T"], a["V"], a["ld"], a["t"], a["rt"], a["k"], a["rk"],
                                 a["p"], a["rp"], a["m"], a["rm"], a["u"], a["tok"], a["lp"], None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(T=-1), dict(T=2147483392 // 8 + 1), dict(V=0), dict(V=2147483393),
                dict(ld=999), dict(t=-1.0), dict(t=nan),
                dict(t=inf), dict(k=-1), dict(p=0.0), dict(p=1.5), dict(p=nan), dict(m=-0.1),
                dict(m=1.1), dict(m=nan), dict(x=None), dict(u=None), dict(tok=None)):
        assert call(**bad) == lmh.LMH_ERR_INVALID_ARG, bad
    for bad in (dict(x=3), dict(u=18), dict(tok=18), dict(lp=18), dict(rt=18), dict(rk=18),
                dict(rp=18), dict(rm=18)):
        assert call(**bad) == lmh.LMH_ERR_ALIGNMENT, bad
    assert call(T=0, x=None, u=None, tok=None, lp=None) == lmh.LMH_OK
    assert lib.lmhead_kernel_launches() == before


def test_binding_refusals(lib):
    torch = pytest.importorskip("torch")
    bf, f8, f32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
    x = torch.zeros(4, 256, dtype=bf)
    with pytest.raises(TypeError):
        lmh.lmhead_quantize_fp8(x.float())
    with pytest.raises(ValueError):
        lmh.lmhead_quantize_fp8(x, 64)
    with pytest.raises(ValueError):
        lmh.lmhead_quantize_fp8(x.t())
    with pytest.raises(ValueError):
        lmh.lmhead_quantize_fp8(x[:1].expand(4, 256))
    with pytest.raises(ValueError):
        lmh.lmhead_quantize_fp8(x, out_scale=torch.zeros(4, 3))
    hq, wq = torch.zeros(4, 256, dtype=f8), torch.zeros(1000, 256, dtype=f8)
    hs, ws = torch.zeros(4, 2), torch.zeros(8, 2)
    with pytest.raises(TypeError):
        lmh.lmhead_logits_fp8(x, hs, wq, ws)
    with pytest.raises(ValueError):
        lmh.lmhead_logits_fp8(hq, hs, wq, ws[:7])
    with pytest.raises(ValueError):
        lmh.lmhead_logits_fp8(hq, hs[:, :1].contiguous(), wq, ws)
    with pytest.raises(ValueError):
        lmh.lmhead_logits_fp8(hq[:, :128].contiguous(), hs, wq, ws)
    with pytest.raises(ValueError):
        lmh.lmhead_logits_fp8(hq, hs, wq, ws, out_logits=torch.zeros(4, 999, dtype=bf))
    u = torch.zeros(4, dtype=f32)
    with pytest.raises(TypeError):
        lmh.lmhead_sample(x, u.double())
    with pytest.raises(ValueError):
        lmh.lmhead_sample(x, u[:3])
    with pytest.raises(ValueError):
        lmh.lmhead_sample(x, u, torch.ones(3))
    with pytest.raises(TypeError):
        lmh.lmhead_sample(x, u, top_k=torch.ones(4))
    with pytest.raises(ValueError):
        lmh.lmhead_sample(x, u, top_k=-1)


def test_binding_refuses_host_tensors(lib):
    # a host pointer must never reach a kernel, whatever else is right
    torch = pytest.importorskip("torch")
    before = lib.lmhead_kernel_launches()
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    hq, wq = (torch.zeros(n, 256, dtype=torch.float8_e4m3fn) for n in (4, 1000))
    hs, ws = torch.zeros(4, 2), torch.zeros(8, 2)
    for call in (lambda: lmh.lmhead_quantize_fp8(x), lambda: lmh.lmhead_quantize_fp8(x, 128),
                 lambda: lmh.lmhead_logits_fp8(hq, hs, wq, ws),
                 lambda: lmh.lmhead_sample(x, torch.zeros(4))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    assert lib.lmhead_kernel_launches() == before
