"""Edges of the fp8 head on the GPU."""

import pytest

import invariant_lm_head_gb300 as lmh
from helpers import dev
from test_gpu_fp8_head import check_logits, operands

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
