"""An 8-bit LM head for serving: the weight held in e4m3, logits and tokens from it.

The three operators it joins are lmhead_quantize_fp8, lmhead_logits_fp8 and
lmhead_sample (include/lmhead.h has their formulas). A token's bits, its
log-prob's and its logits' do not depend on the batch its row arrives in.

    head = FP8Head(weight)                      # bf16 [V, H], e.g. the trainer's
    token, logprob = head.sample(hidden, uniform, 0.7, top_p=0.95)
    head.refresh(weight)                        # after a training step

With the model's last norm in it (lmhead_rmsnorm_fp8, in place of the quantisation), the
head takes the last layer's output and the residual stream:

    head = FP8Head(weight, norm_weight, norm_eps=1e-6)
    token, logprob = head.sample(hidden, uniform, residual=residual)
    head.refresh(weight, norm_weight)           # after a training step

The norm's weight is not quantised, and so not copied: the head reads the tensor that it
was given, and writes a refresh's norm_weight into it.

Every call runs on the current stream and can be captured into a CUDA graph
(after a first call outside of one). The head holds one byte per weight
element, and four per 128 x 128 block.
"""

from __future__ import annotations

import invariant_lm_head_gb300 as lmh

from .quantized_head import QuantizedHead


class FP8Head(QuantizedHead):
    """A head whose weight [V, H] is held in e4m3 with one scale per 128 x 128 block."""

    def __init__(self, weight, norm_weight=None, norm_eps: float = 1e-6):
        self.weight_q, self.weight_scale = lmh.lmhead_quantize_fp8(weight, 128)
        self.norm_weight, self.norm_eps = norm_weight, norm_eps

    @property
    def vocab_size(self) -> int:
        return self.weight_q.shape[0]

    @property
    def hidden_size(self) -> int:
        return self.weight_q.shape[1]

    def refresh(self, weight, norm_weight=None) -> None:
        """Quantise a new weight of the same shape in place (graphs stay valid).

        norm_weight: the norm's new weight, written into the tensor that the head holds;
        without one that tensor stays as it is.
        """
        held = self.norm_weight
        if norm_weight is not None:
            if held is None:
                raise ValueError("norm_weight needs a head with a norm")
            lmh._need_out(norm_weight, "norm_weight", held.dtype, held.device, tuple(held.shape))
        lmh.lmhead_quantize_fp8(weight, 128, out=self.weight_q, out_scale=self.weight_scale)
        if norm_weight is not None:
            held.detach().copy_(norm_weight.detach())

    def logits(self, hidden, *, residual=None, out_logits=None):
        """bf16 logits [T, V] of hidden bf16 [T, H] (rows may be strided).

        A head with a norm takes hidden states before it, and adds residual (or None).
        """
        if self.norm_weight is not None:
            hidden_q, hidden_scale, _ = lmh.lmhead_rmsnorm_fp8(
                hidden, self.norm_weight, residual, eps=self.norm_eps, want_residual=False)
        elif residual is not None:
            raise ValueError("residual needs a head with a norm")
        else:
            hidden_q, hidden_scale = lmh.lmhead_quantize_fp8(hidden)
        return lmh.lmhead_logits_fp8(hidden_q, hidden_scale, self.weight_q, self.weight_scale,
                                     out_logits=out_logits)
