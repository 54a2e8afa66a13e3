"""A decode step from the last layer's output to what a server reports, in one CUDA graph.

A batch of synthetic sequences decodes a number of tokens. Each step adds the residual
and norms (inside the 8-bit head; before the 4-bit one), computes logits, draws a token
with the request's own settings, and reports its log-prob, the distribution's entropy
and the likeliest alternatives. At the end the graph is compared with calls made one
by one, and the log-probs with those of the unquantised head.

    python examples/serve_alternatives.py [--head fp8|fp4] [--batch 64] [--hidden 4096] [--vocab 32000]
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import invariant_lm_head_gb300 as lmh  # noqa: E402
from invariant_lm_head_gb300.fp4_head import FP4Head  # noqa: E402
from invariant_lm_head_gb300.fp8_head import FP8Head  # noqa: E402


def norm(x, weight, eps=1e-6):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()).to(torch.bfloat16)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--head", choices=("fp8", "fp4"), default="fp8")
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--top", type=int, default=5)
    a = ap.parse_args()
    lmh.build()
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(7)
    B, H, V = a.batch, a.hidden, a.vocab
    weight = (torch.randn(V, H, device=dev, generator=g) * 2 / H ** 0.5).to(torch.bfloat16)
    norm_weight = (1 + 0.1 * torch.randn(H, device=dev, generator=g)).to(torch.bfloat16)
    # a layer's output and the residual stream, by the last token (the place of a transformer)
    embed = torch.randn(V, H, device=dev, generator=g).to(torch.bfloat16)
    stream = (3 * torch.randn(V, H, device=dev, generator=g)).to(torch.bfloat16)
    temperature = 0.5 + torch.rand(B, device=dev, generator=g)
    uniform = torch.rand(a.steps, B, device=dev, generator=g)
    start = torch.randint(V, (B,), device=dev, generator=g, dtype=torch.int32)

    head = FP8Head(weight, norm_weight) if a.head == "fp8" else FP4Head(weight)
    logits = torch.empty(B, -(-V // 8) * 8, dtype=torch.bfloat16, device=dev)[:, :V]
    token, u = start.clone(), uniform[0].clone()
    report = [torch.empty(B, device=dev), torch.empty(B, device=dev),
              torch.empty(B, a.top, dtype=torch.int32, device=dev), torch.empty(B, a.top, device=dev)]

    def step():
        at = token.long()
        if a.head == "fp8":
            t, _ = head.sample(embed[at], u, temperature, top_p=0.9, residual=stream[at],
                               out_logits=logits)
        else:
            t, _ = head.sample(norm(embed[at] + stream[at], norm_weight), u, temperature, top_p=0.9,
                               out_logits=logits)
        lmh.lmhead_top_logprobs(logits, t, temperature, top=a.top, out_logprob=report[0],
                                out_entropy=report[1], out_top_token=report[2],
                                out_top_logprob=report[3])
        token.copy_(t)

    def run(one):
        token.copy_(start)
        got = []
        for i in range(a.steps):
            u.copy_(uniform[i])
            one()
            got.append([token.clone(), *(t.clone() for t in report)])
        return [torch.stack(t) for t in zip(*got)]

    first = run(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    again = run(graph.replay)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    tokens, logprob, entropy, top_token, top_logprob = first
    listed = top_token == tokens[:, :, None]
    assert (torch.where(listed, top_logprob - logprob[:, :, None], 0.0) == 0).all()

    before = torch.cat([start[None], tokens[:-1]]).reshape(-1).long()
    full = norm(embed[before] + stream[before], norm_weight) @ weight.t()
    exact = lmh.logprob_from_logits_div(full, tokens.reshape(-1).contiguous(),
                                        temperature.repeat(a.steps))[0]
    diff = (exact - logprob.reshape(-1)).abs()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    run(graph.replay)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / a.steps
    print(f"{a.head} head, {B} sequences, H={H}, V={V}: {dt * 1e6:.1f} us a step, {B / dt:.0f} tokens/s; "
          f"entropy {entropy.mean():.3f}; drawn token listed {listed.any(2).float().mean():.2f}; "
          f"log-prob against the bf16 head: mean |d| {diff.mean():.4f}, max {diff.max():.4f}")


if __name__ == "__main__":
    main()
