"""Arguments of the calls around the quantised heads that need no GPU to be refused."""

import pytest
import torch

import invariant_lm_head_gb300 as lmh
from invariant_lm_head_gb300.fp8_head import FP8Head
from test_serving_host import Here, lib  # noqa: F401  (a fixture)


@pytest.mark.parametrize("kind", [torch.Tensor, Here])
def test_what_is_no_tensor_is_a_type_error(kind, lib, monkeypatch):  # noqa: F811
    # on the host, and where the other arguments are on the current device
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(kind)

    bf, u8 = torch.bfloat16, torch.uint8
    x, w, lg = t(4, 256, dtype=bf), t(256, dtype=bf), t(4, 1000, dtype=bf)
    hq, wq = t(4, 128, dtype=u8), t(1000, 128, dtype=u8)
    hs, ws = t(1, 2, 32, 16, dtype=u8), t(8, 2, 32, 16, dtype=u8)
    before = lib.lmhead_kernel_launches()
    for no in ([1.0] * 256, (1, 2), 1.0, "w", w.as_subclass(torch.Tensor).float().numpy()):
        for call in (lambda: lmh.lmhead_rmsnorm_fp8(x, no),
                     lambda: lmh.lmhead_rmsnorm_fp8(x, w, no),
                     lambda: lmh.lmhead_dequantize_mxfp4(hq, no),
                     lambda: lmh.lmhead_logits_mxfp4(hq, no, wq, ws),
                     lambda: lmh.lmhead_logits_mxfp4(hq, hs, no, ws),
                     lambda: lmh.lmhead_logits_mxfp4(hq, hs, wq, no),
                     lambda: lmh.lmhead_top_logprobs(lg, no)):
            with pytest.raises(TypeError, match="must be a torch.Tensor"):
                call()
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        lmh.lmhead_rmsnorm_fp8(x, None)
    assert lib.lmhead_kernel_launches() == before


def test_refresh_refuses_another_norm_before_it_writes():
    w, g = torch.zeros(1000, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    head = FP8Head.__new__(FP8Head)
    head.norm_weight = None
    with pytest.raises(ValueError, match="needs a head with a norm"):
        head.refresh(w, g)
    head.norm_weight = g.clone()
    for bad, error in ((g[:128], ValueError), (g[:1], ValueError), (g.float(), TypeError),
                       ([1.0] * 256, TypeError), (g.view(1, 256), ValueError)):
        with pytest.raises(error, match="norm_weight"):
            head.refresh(w, bad)
    assert torch.equal(head.norm_weight, g)
