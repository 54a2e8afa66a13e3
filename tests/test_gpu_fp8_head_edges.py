"""Edges of the fp8 head on the GPU."""

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
import workloads as W
from helpers import dev, to_dev_bf16
from oracle import fp8_head as o
from test_gpu_fp8_head import bf16_values, check_logits, logit_rows, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lmh.build()


@pytest.mark.parametrize("V", [1, 5, 8, 9, 33, 1003, 1004, 1006, 20007, 32003])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_logits_nothing_past_the_vocabulary_is_written(T, V):
    # rows on 16-byte boundaries, the vocabulary ending inside 16 bytes or on them
    import torch

    ops = operands(T, 256, V)
    ld = -(-V // 8) * 8 + 8
    for off, gap in [(0, ld), (8, ld), (0, ld + 8)]:
        buf = torch.full((off + (T + 1) * gap,), 7.0, dtype=torch.bfloat16, device=dev())
        out = buf[off:off + T * gap].view(T, gap)[:, :V]
        lmh.lmhead_logits_fp8(*ops, out_logits=out)
        check_logits(out, *ops)
        out.fill_(7.0)
        assert (buf == 7.0).all(), (off, gap)


def test_logits_of_one_row_leave_the_next_alone():
    import torch

    ops = operands(1, 256, 1003)
    buf = torch.full((9, 1003), 7.0, dtype=torch.bfloat16, device=dev())
    for i in (0, 8):  # rows that start on 16 bytes
        lmh.lmhead_logits_fp8(*ops, out_logits=buf[i:i + 1])
        check_logits(buf[i:i + 1], *ops)
    assert (buf[1:8] == 7.0).all()


@pytest.mark.parametrize("T", [3, 60, 120, 200])
def test_sample_writes_every_token(T):
    # Rows that another stream rewrites during the call, between values inside and
    # outside the direct range: a senseless token, but always a token or -1.
    import torch

    V = 3003
    x, _ = logit_rows(T, T, V)
    good = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    wild = torch.randint(-32768, 32767, (T, V), device=dev(), dtype=torch.int16).view(torch.bfloat16)
    lg, u = good.clone(), torch.rand(T, device=dev())
    tok = torch.empty(T, dtype=torch.int32, device=dev())
    bad = torch.zeros((), dtype=torch.int64, device=dev())
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(200):
        with torch.cuda.stream(other):
            lg.copy_(wild if i % 2 else good)
        tok.fill_(1 << 30)
        lmh.lmhead_sample(lg, u, 0.9, top_p=0.9, top_k=1000, out_token=tok)
        bad += ((tok < -1) | (tok >= V)).sum()
    torch.cuda.synchronize()
    assert bad.item() == 0


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_keeps_the_sign_of_zero(block_rows):
    # x * 448 / a rounded once has x's sign, in -0 and in what rounds to it
    bits = W.random_bf16(3, (130, 400), 1.0)
    bits[:, ::3] = 0x8000
    bits[:, 1::9] = 0x0000
    bits[:, 2::9] = 0x8001  # the smallest of all, to -0
    bits[:, 4::9] = 0x0001
    bits[5] = 0x8000        # blocks of nothing else (of 1 x 128)
    q, _ = lmh.lmhead_quantize_fp8(to_dev_bf16(bits), block_rows)
    rq, _ = o.quantize(bf16_values(bits), block_rows)
    got = q.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(got, rq) and np.array_equal(np.signbit(got), np.signbit(rq))
    assert np.array_equal(np.signbit(got), bits >= 0x8000)
