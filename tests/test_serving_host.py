"""Host-side checks around the quantised heads: the oracle's pins, and refusals before any device use."""

import math

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
import invariant_lm_head_gb300.fp4_head as fp4_head
import invariant_lm_head_gb300.fp8_head as fp8_head
from oracle import serving as o

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    lmh.build()
    return lmh.library()


# ------------------------------------------------------------------ the oracle

def test_e2m1_codes_by_hand():
    y = [0, .25, .26, .74, .75, 1, 1.25, 1.26, 1.75, 2.5, 2.51, 3.49, 3.5, 5, 5.01, 6, 7, 100]
    want = [0, 0, 1, 1, 2, 2, 2, 3, 4, 4, 5, 5, 6, 6, 7, 7, 7, 7]
    assert o.e2m1_code(np.array(y)).tolist() == want
    assert o.e2m1_code(-np.array(y)).tolist() == [c + 8 for c in want]
    assert o.e2m1_code(np.concatenate([o.E2M1, -o.E2M1])).tolist() == list(range(16))


def test_scale_byte_leaves_the_largest_between_3_5_and_7():
    for b in range(1, 0x7F80):  # every positive bf16
        a = float(np.uint32(b << 16).view(np.float32))
        byte = o.mxfp4_byte(a)
        r = a / 2.0 ** (byte - 127)
        assert 0 <= byte <= 253 and r < 7 and (r >= 3.5 or byte == 0), b


def test_pack_order():
    rows, cols = 130, 160
    s = np.arange(2 * 2 * 32 * 16).reshape(2, 2, 32, 16)
    _, b = o.unpack(np.zeros((rows, cols // 2), np.uint8), s, rows, cols)
    assert b[0, 0] == 0 and b[1, 0] == 16 and b[32, 0] == 4 and b[33, 2] == 22
    assert b[0, 4] == 512 and b[128, 0] == 1024 and b[129, 4] == 1024 + 512 + 16


def test_norm_by_hand():
    x = np.array([[3.0, 4.0] * 8])
    q, s, r = o.rmsnorm_fp8(x, np.ones(16), None, 1e-9)
    assert r is None and q[0, 1] == 448 and q[0, 0] == 320  # 336 is a tie, to the even fraction
    assert s[0, 0] == pytest.approx(4 / math.sqrt(12.5) / 448, rel=1e-9)
    q, s, r = o.rmsnorm_fp8(x, np.ones(16), -x, 1e-9)
    assert (q == 0).all() and (r == 0).all() and s[0, 0] == 2.0 ** -60 / 448


def test_top_row_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    lp, h, tok, tlp = o.top_row(x, 1.0, 3, (0, 2, -1, 4))
    assert np.allclose(lp, [math.log(0.1), math.log(0.2), 0, 0])
    assert tok.tolist() == [1, 3, 2] and np.allclose(tlp, np.log([.4, .3, .2]))
    assert h == pytest.approx(-sum(p * math.log(p) for p in (.1, .4, .2, .3)))
    inf = np.inf
    lp, h, tok, tlp = o.top_row(np.array([0, -inf, 0, np.nan]), 0.0, 4, (1, 2))
    assert tok.tolist() == [0, 2, -1, -1] and h == pytest.approx(math.log(2))
    assert lp[0] == -inf and lp[1] == pytest.approx(-math.log(2)) and tlp[2] == -inf
    assert o.top_row(np.full(3, -inf), 1.0, 2, (0,))[1:3][0] == 0
    lp, h, tok, tlp = o.top_row(np.array([1, inf, inf, 3]), 1.0, 3, (1, 3))
    assert tok.tolist() == [1, 2, 3] and lp[0] == pytest.approx(-math.log(2)) and lp[1] == -inf


# ------------------------------------------------------------------ refusals of the C entries

NAN, INF, BIG = float("nan"), float("inf"), 2147483393


def refused(lib, call, invalid, misaligned, fine):
    before = lib.lmhead_kernel_launches()
    for bad in invalid:
        assert call(**bad) == lmh.LMH_ERR_INVALID_ARG, bad
        assert lib.lmhead_last_error_string() != b""
    for bad in misaligned:
        assert call(**bad) == lmh.LMH_ERR_ALIGNMENT, bad
    for good in fine:
        assert call(**good) == lmh.LMH_OK, good
    assert lib.lmhead_kernel_launches() == before


def test_norm_refusals(lib):
    ok = dict(x=16, r=16, w=16, rows=4, cols=256, ldx=256, ldr=256, eps=1e-6, out=16, ldo=256, q=16,
              s=16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.lmhead_rmsnorm_fp8(a["x"], a["r"], a["w"], a["rows"], a["cols"], a["ldx"],
                                      a["ldr"], a["eps"], a["out"], a["ldo"], a["q"], a["s"], None)

    refused(lib, call,
            [dict(rows=-1), dict(rows=BIG), dict(cols=0), dict(cols=32784, ldx=32784), dict(eps=0.0),
             dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(ldx=255), dict(ldr=255),
             dict(ldo=255), dict(r=None), dict(x=None), dict(w=None), dict(q=None), dict(s=None)],
            [dict(cols=24), dict(ldx=260), dict(ldr=260), dict(ldo=260), dict(x=24), dict(r=24),
             dict(w=8), dict(out=24), dict(q=8), dict(s=18)],
            [dict(rows=0, x=None, w=None, q=None, s=None)])


def test_quantize_refusals(lib):
    ok = dict(x=16, rows=4, cols=256, ld=256, q=16, s=16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.lmhead_quantize_mxfp4(a["x"], a["rows"], a["cols"], a["ld"], a["q"], a["s"], None)

    def back(**kw):
        a = dict(ok, **kw)
        return lib.lmhead_dequantize_mxfp4(a["q"], a["s"], a["rows"], a["cols"], a["x"], a["ld"],
                                           None)

    for f in (call, back):
        refused(lib, f,
                [dict(rows=-1), dict(rows=BIG), dict(cols=0), dict(cols=BIG), dict(ld=255),
                 dict(x=None), dict(q=None), dict(s=None)],
                [dict(cols=16), dict(cols=144), dict(ld=260), dict(x=24), dict(q=24), dict(s=8)],
                [dict(rows=0, x=None, q=None, s=None)])


def test_logits_refusals(lib):
    ok = dict(hq=16, hs=16, wq=16, ws=16, T=4, H=256, V=1000, out=16, ld=1000)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.lmhead_logits_mxfp4(a["hq"], a["hs"], a["wq"], a["ws"], a["T"], a["H"], a["V"],
                                       a["out"], a["ld"], None)

    refused(lib, call,
            [dict(T=-1), dict(V=0), dict(H=0), dict(T=BIG), dict(ld=999), dict(hq=None),
             dict(hs=None), dict(wq=None), dict(ws=None), dict(out=None),
             dict(T=BIG - 1, V=BIG - 1, ld=BIG - 1)],
            [dict(H=48), dict(hq=8), dict(wq=24), dict(hs=8), dict(ws=4), dict(out=17)],
            [dict(T=0, hq=None, hs=None, out=None)])


def test_top_refusals(lib):
    ok = dict(x=2, T=4, V=1000, ld=1000, t=1.0, rt=None, ids=16, k=1, n=5, lp=16, h=16, tok=16,
              tlp=16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.lmhead_top_logprobs(a["x"], a["T"], a["V"], a["ld"], a["t"], a["rt"], a["ids"],
                                       a["k"], a["n"], a["lp"], a["h"], a["tok"], a["tlp"], None)

    refused(lib, call,
            [dict(T=-1), dict(T=2147483392 // 8 + 1), dict(V=0), dict(V=BIG), dict(ld=999),
             dict(t=-1.0), dict(t=NAN), dict(t=INF), dict(k=-1), dict(n=-1), dict(n=129),
             dict(x=None), dict(ids=None), dict(lp=None), dict(tok=None), dict(tlp=None)],
            [dict(x=3), dict(rt=18), dict(ids=18), dict(lp=18), dict(h=18), dict(tok=18),
             dict(tlp=18)],
            [dict(T=0, x=None, ids=None, lp=None, tok=None, tlp=None)])


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refusals(lib):
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    before = lib.lmhead_kernel_launches()
    x, w = torch.zeros(4, 256, dtype=bf), torch.zeros(256, dtype=bf)
    hq, wq = torch.zeros(4, 128, dtype=u8), torch.zeros(1000, 128, dtype=u8)
    hs, ws = torch.zeros(1, 2, 32, 16, dtype=u8), torch.zeros(8, 2, 32, 16, dtype=u8)
    ids, t = torch.zeros(4, dtype=i32), torch.ones(4)
    wrong_type = [
        lambda: lmh.lmhead_rmsnorm_fp8(x.float(), w),
        lambda: lmh.lmhead_rmsnorm_fp8(x, w.float()),
        lambda: lmh.lmhead_rmsnorm_fp8(x, w, x.float()),
        lambda: lmh.lmhead_rmsnorm_fp8(x, w, out=torch.zeros(4, 256, dtype=u8)),
        lambda: lmh.lmhead_quantize_mxfp4(x.half()),
        lambda: lmh.lmhead_quantize_mxfp4(x, out_scale=hs.int()),
        lambda: lmh.lmhead_dequantize_mxfp4(x, hs),
        lambda: lmh.lmhead_logits_mxfp4(x, hs, wq, ws),
        lambda: lmh.lmhead_logits_mxfp4(hq, hs.float(), wq, ws),
        lambda: lmh.lmhead_top_logprobs(x.float()),
        lambda: lmh.lmhead_top_logprobs(x, ids.long()),
        lambda: lmh.lmhead_top_logprobs(x, ids, t.double()),
    ]
    wrong_shape = [
        lambda: lmh.lmhead_rmsnorm_fp8(x, w[:128]),
        lambda: lmh.lmhead_rmsnorm_fp8(x, w, x[:3]),
        lambda: lmh.lmhead_rmsnorm_fp8(x.t(), w),
        lambda: lmh.lmhead_rmsnorm_fp8(x, w, out_residual=x),
        lambda: lmh.lmhead_rmsnorm_fp8(x, w, out_scale=torch.zeros(4, 3)),
        lambda: lmh.lmhead_quantize_mxfp4(x[:1].expand(4, 256)),
        lambda: lmh.lmhead_quantize_mxfp4(x, out=torch.zeros(4, 256, dtype=u8)),
        lambda: lmh.lmhead_quantize_mxfp4(x, out_scale=ws),
        lambda: lmh.lmhead_dequantize_mxfp4(hq, ws),
        lambda: lmh.lmhead_dequantize_mxfp4(hq, hs, out=x[:3]),
        lambda: lmh.lmhead_logits_mxfp4(hq, ws, wq, ws),
        lambda: lmh.lmhead_logits_mxfp4(hq, hs, wq, hs),
        lambda: lmh.lmhead_logits_mxfp4(hq[:, :64].contiguous(), hs, wq, ws),
        lambda: lmh.lmhead_logits_mxfp4(hq, hs, wq, ws, out_logits=torch.zeros(4, 999, dtype=bf)),
        lambda: lmh.lmhead_top_logprobs(x, ids[:3]),
        lambda: lmh.lmhead_top_logprobs(x, ids.view(1, 1, 4)),
        lambda: lmh.lmhead_top_logprobs(x, ids, t[:3]),
        lambda: lmh.lmhead_top_logprobs(x, ids, top=129),
        lambda: lmh.lmhead_top_logprobs(x, ids, top=-1),
        lambda: lmh.lmhead_top_logprobs(x, ids, top=5, out_top_token=torch.zeros(4, 4, dtype=i32)),
        lambda: lmh.lmhead_top_logprobs(x, out_logprob=t),
        lambda: lmh.lmhead_top_logprobs(x, ids, out_logprob=t.view(4, 1)),
    ]
    for f in wrong_type:
        with pytest.raises(TypeError):
            f()
    for f in wrong_shape:
        with pytest.raises(ValueError):
            f()
    assert lib.lmhead_kernel_launches() == before


class Elsewhere(torch.Tensor):
    """A host tensor that says it is on cuda:1."""

    device = property(lambda self: torch.device("cuda:1"))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.device.index


class Here(Elsewhere):
    device = property(lambda self: torch.device("cuda:0"))


class OtherStream:
    device = torch.device("cuda:1")
    cuda_stream = 0


def calls(kind):
    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(kind)

    bf, u8 = torch.bfloat16, torch.uint8
    x, w, lg, ids = t(4, 256, dtype=bf), t(256, dtype=bf), t(4, 1000, dtype=bf), t(4, dtype=torch.int32)
    hq, wq = t(4, 128, dtype=u8), t(1000, 128, dtype=u8)
    hs, ws = t(1, 2, 32, 16, dtype=u8), t(8, 2, 32, 16, dtype=u8)
    return {
        "norm": lambda **k: lmh.lmhead_rmsnorm_fp8(x, w, x, **k),
        "quantize": lambda **k: lmh.lmhead_quantize_mxfp4(x, **k),
        "dequantize": lambda **k: lmh.lmhead_dequantize_mxfp4(hq, hs, **k),
        "logits": lambda **k: lmh.lmhead_logits_mxfp4(hq, hs, wq, ws, **k),
        "top": lambda **k: lmh.lmhead_top_logprobs(lg, ids, t(4), **k),
    }


@pytest.mark.parametrize("name", list(calls(Elsewhere)))
def test_other_devices_are_refused(name, lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    before = lib.lmhead_kernel_launches()
    with pytest.raises(ValueError, match="current device is cuda:0"):
        calls(Elsewhere)[name]()
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        calls(Here)[name](stream=OtherStream())
    with pytest.raises(ValueError, match="CUDA device"):
        calls(torch.Tensor)[name]()
    assert lib.lmhead_kernel_launches() == before


def test_heads_refuse_a_residual_without_a_norm(lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for kind in (fp4_head.FP4Head, fp8_head.FP8Head):
        head = kind.__new__(kind)
        head.norm_weight = None
        with pytest.raises(ValueError, match="norm"):
            head.logits(x, residual=x)
