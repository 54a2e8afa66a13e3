"""Edges of the fp8 head on the GPU."""

import pytest

import invariant_lm_head_gb300 as lmh
from helpers import dev
from test_gpu_fp8_head import check_logits, logit_rows, operands

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
