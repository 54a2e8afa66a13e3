"""Around the quantised heads on the GPU: edges of rows, batches, grids and arguments.

Tolerances are those of test_gpu_serving.py, where they are derived.
"""

import numpy as np
import pytest

import invariant_lm_head_gb300 as lmh
from helpers import dev
from test_gpu_serving import check_logits, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lmh.build()


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
