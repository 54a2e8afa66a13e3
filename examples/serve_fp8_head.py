"""Decoding with an 8-bit head, captured into one CUDA graph per step.

A batch of synthetic sequences decodes a number of tokens: hidden states come
from a random embedding of the last token (the place of a transformer), the head
is an e4m3 copy of a bf16 weight, and each request has its own sampling settings.
At the end the drawn tokens' log-probs are compared with what the bf16 head gives
for the same tokens, and the graph with calls made one by one.

    python examples/serve_fp8_head.py [--batch 64] [--hidden 4096] [--vocab 32000]
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import invariant_lm_head_gb300 as lmh  # noqa: E402
from invariant_lm_head_gb300.fp8_head import FP8Head  # noqa: E402


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    lmh.build()
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(7)
    B, H, V = a.batch, a.hidden, a.vocab
    weight = (torch.randn(V, H, device=dev, generator=g) * 2 / H ** 0.5).to(torch.bfloat16)
    embed = torch.randn(V, H, device=dev, generator=g).to(torch.bfloat16)
    temperature = 0.5 + torch.rand(B, device=dev, generator=g)
    top_p = 0.8 + 0.2 * torch.rand(B, device=dev, generator=g)
    uniform = torch.rand(a.steps, B, device=dev, generator=g)
    start = torch.randint(V, (B,), device=dev, generator=g, dtype=torch.int32)

    head = FP8Head(weight)
    token, u = start.clone(), uniform[0].clone()
    logprob = torch.empty(B, device=dev)

    def step():
        t, lp = head.sample(embed[token.long()], u, temperature, top_p=top_p)
        token.copy_(t)
        logprob.copy_(lp)

    def run(one):
        token.copy_(start)
        tokens, logprobs = [], []
        for i in range(a.steps):
            u.copy_(uniform[i])
            one()
            tokens.append(token.clone())
            logprobs.append(logprob.clone())
        return torch.stack(tokens), torch.stack(logprobs)

    tokens, logprobs = run(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    again, logprobs_again = run(graph.replay)
    assert torch.equal(tokens, again) and torch.equal(logprobs, logprobs_again)
    # a sequence alone draws the same tokens as in the batch
    lg = head.logits(embed[start[:1].long()])
    alone = lmh.lmhead_sample(lg, uniform[0, :1], temperature[:1].clone(), top_p=top_p[:1].clone())
    assert torch.equal(alone[0], tokens[0, :1]) and torch.equal(alone[1], logprobs[0, :1])

    before = torch.cat([start[None], tokens[:-1]]).reshape(-1)
    bf16_logits = embed[before.long()] @ weight.t()
    t = temperature.repeat(a.steps)
    bf16 = lmh.logprob_from_logits_div(bf16_logits, tokens.reshape(-1).contiguous(), t)[0]
    diff = (bf16 - logprobs.reshape(-1)).abs()

    torch.cuda.synchronize()
    t0 = time.perf_counter()
    run(graph.replay)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / a.steps
    print(f"{B} sequences, H={H}, V={V}: {dt * 1e6:.1f} us a step, {B / dt:.0f} tokens/s; "
          f"log-prob against the bf16 head: mean |d| {diff.mean():.4f}, max {diff.max():.4f}")


if __name__ == "__main__":
    main()
