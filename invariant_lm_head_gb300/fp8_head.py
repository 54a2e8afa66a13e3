"""An 8-bit LM head for serving: the weight held in e4m3, logits and tokens from it.

The three operators it joins are lmhead_quantize_fp8, lmhead_logits_fp8 and
lmhead_sample (include/lmhead.h has their formulas). A token's bits, its
log-prob's and its logits' do not depend on the batch its row arrives in.

    head = FP8Head(weight)                      # bf16 [V, H], e.g. the trainer's
    token, logprob = head.sample(hidden, uniform, 0.7, top_p=0.95)
    head.refresh(weight)                        # after a training step

Every call runs on the current stream and can be captured into a CUDA graph
(after a first call outside of one). The head holds one byte per weight
element, and four per 128 x 128 block.
"""

from __future__ import annotations

import invariant_lm_head_gb300 as lmh


class FP8Head:
    """A head whose weight [V, H] is held in e4m3 with one scale per 128 x 128 block."""

    def __init__(self, weight):
        self.weight_q, self.weight_scale = lmh.lmhead_quantize_fp8(weight, 128)

    @property
    def vocab_size(self) -> int:
        return self.weight_q.shape[0]

    @property
    def hidden_size(self) -> int:
        return self.weight_q.shape[1]

    def refresh(self, weight) -> None:
        """Quantise a new weight of the same shape in place (graphs stay valid)."""
        lmh.lmhead_quantize_fp8(weight, 128, out=self.weight_q, out_scale=self.weight_scale)

    def logits(self, hidden, *, out_logits=None):
        """bf16 logits [T, V] of hidden bf16 [T, H] (rows may be strided)."""
        hidden_q, hidden_scale = lmh.lmhead_quantize_fp8(hidden)
        return lmh.lmhead_logits_fp8(hidden_q, hidden_scale, self.weight_q, self.weight_scale,
                                     out_logits=out_logits)

    def sample(self, hidden, uniform, temperature=1.0, *, top_k=0, top_p=1.0, min_p=0.0,
               mask=None, out_logits=None):
        """(token int32 [T], logprob f32 [T]) of hidden bf16 [T, H].

        uniform f32 [T] in [0, 1]; the settings are those of lmhead_sample. mask
        (bool [T, V] or [V]) marks tokens that must not be drawn; they drop out of
        the log-prob's distribution too. out_logits receives the (masked) logits.
        """
        if out_logits is None and self.vocab_size % 8:
            # rows of their own that start on 16 bytes, for wide stores and loads
            V = self.vocab_size
            out_logits = hidden.new_empty((hidden.shape[0], -(-V // 8) * 8))[:, :V]
        logits = self.logits(hidden, out_logits=out_logits)
        if mask is not None:
            logits.masked_fill_(mask, float("-inf"))
        return lmh.lmhead_sample(logits, uniform, temperature, top_k=top_k, top_p=top_p,
                                 min_p=min_p)
