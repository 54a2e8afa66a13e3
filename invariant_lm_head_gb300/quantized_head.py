"""What the quantised heads share: sampling from their logits."""

from __future__ import annotations

import invariant_lm_head_gb300 as lmh


class QuantizedHead:
    """A head with ``vocab_size`` and ``logits(hidden, residual=, out_logits=)``."""

    def sample(self, hidden, uniform, temperature=1.0, *, top_k=0, top_p=1.0, min_p=0.0,
               mask=None, residual=None, out_logits=None):
        """(token int32 [T], logprob f32 [T]) of hidden bf16 [T, H].

        uniform f32 [T] in [0, 1]; the settings are those of lmhead_sample. mask
        (bool [T, V] or [V]) marks tokens that must not be drawn; they drop out of
        the log-prob's distribution too. out_logits receives the (masked) logits, for
        lmhead_top_logprobs, say. residual: see the head's logits.
        """
        if out_logits is None and self.vocab_size % 8:
            # rows of their own that start on 16 bytes, for wide stores and loads
            V = self.vocab_size
            out_logits = hidden.new_empty((hidden.shape[0], -(-V // 8) * 8))[:, :V]
        logits = self.logits(hidden, residual=residual, out_logits=out_logits)
        if mask is not None:
            logits.masked_fill_(mask, float("-inf"))
        return lmh.lmhead_sample(logits, uniform, temperature, top_k=top_k, top_p=top_p,
                                 min_p=min_p)
