"""A 4-bit LM head for serving: the weight held in microscaled e2m1.

    head = FP4Head(weight)                      # bf16 [V, H], e.g. the trainer's
    token, logprob = head.sample(hidden, uniform, 0.7, top_p=0.95)
    head.refresh(weight)                        # after a training step

The interface is FP8Head's; half its memory, and half its time where reading the
weight is what counts. The hidden states are quantised to 4 bits as well: logits of
normal values are some 16 % off (2-norm), 4 % with the 8-bit head. Every call runs on
the current stream and can be captured into a CUDA graph (after a first call outside of
one). The head holds 17/32 bytes per weight element.
"""

from __future__ import annotations

import invariant_lm_head_gb300 as lmh

from .quantized_head import QuantizedHead


class FP4Head(QuantizedHead):
    """A head whose weight [V, H] is held in e2m1 with a power of two per 32 elements."""

    def __init__(self, weight):
        self.weight_q, self.weight_scale = lmh.lmhead_quantize_mxfp4(weight)

    @property
    def vocab_size(self) -> int:
        return self.weight_q.shape[0]

    @property
    def hidden_size(self) -> int:
        return 2 * self.weight_q.shape[1]

    def refresh(self, weight) -> None:
        """Quantise a new weight of the same shape in place (graphs stay valid)."""
        lmh.lmhead_quantize_mxfp4(weight, out=self.weight_q, out_scale=self.weight_scale)

    def weight(self):
        """The bf16 weight [V, H] that the held values stand for."""
        return lmh.lmhead_dequantize_mxfp4(self.weight_q, self.weight_scale)

    def logits(self, hidden, *, residual=None, out_logits=None):
        """bf16 logits [T, V] of hidden bf16 [T, H] (rows may be strided)."""
        if residual is not None:
            raise ValueError("the 4-bit head takes hidden states after their norm")
        hidden_q, hidden_scale = lmh.lmhead_quantize_mxfp4(hidden)
        return lmh.lmhead_logits_mxfp4(hidden_q, hidden_scale, self.weight_q, self.weight_scale,
                                       out_logits=out_logits)
