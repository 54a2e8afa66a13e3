"""Measured cases of the fp8 head: block quantisation, the fp8 logits and the sampler.

Three operators that a server runs one after the other on each step:

* ``quantize``: bf16 -> e4m3 with one fp32 scale per block, 1 x 128 for
  activations, 128 x 128 for the head's weight;
* ``logits``: bf16 logits of an e4m3 hidden and an e4m3 weight with those scales;
* ``sample``: one token per row of bf16 logits from a given uniform number,
  with temperature, top-k, top-p and min-p, and its log-prob.

``own`` chooses between the plain form in elementary torch operations and the
library's entry points. ``exact`` restates each operator in 64 bits.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -60  # blocks of (almost) zeros quantise with this maximum


def listed():
    return [
        # a decode step's hidden states, 64 sequences
        {"name": "quantize decode 64x3584", "op": "quantize", "rows": 64, "cols": 3584, "block_rows": 1},
        # a long packed prefill or rollout scored at once
        {"name": "quantize prefill 16384x5120", "op": "quantize", "rows": 16384, "cols": 5120, "block_rows": 1},
        # the head's weight after a training step, before serving goes on
        {"name": "quantize weight 152064x3584", "op": "quantize", "rows": 152064, "cols": 3584, "block_rows": 128},
        # one sequence's next token: the weight is read once, nothing else counts
        {"name": "logits T1 H3584 V152064", "op": "logits", "T": 1, "H": 3584, "V": 152064},
        # a decode batch over a small vocabulary
        {"name": "logits T64 H4096 V32000", "op": "logits", "T": 64, "H": 4096, "V": 32000},
        # ragged everywhere: a short last block of H, an odd vocabulary, T off every tile
        {"name": "logits T200 H3600 V32003", "op": "logits", "T": 200, "H": 3600, "V": 32003},
        # whole sequences scored in one call
        {"name": "logits T2048 H3584 V152064", "op": "logits", "T": 2048, "H": 3584, "V": 152064},
        # one sequence, nucleus sampling
        {"name": "sample T1 V152064 top-p", "op": "sample", "T": 1, "V": 152064, "mode": "top_p", "masked": 0.0},
        # a decode batch whose requests each bring their own settings, some greedy
        {"name": "sample T64 V32000 mixed", "op": "sample", "T": 64, "V": 32000, "mode": "mixed", "masked": 0.0},
        # constrained decoding: a grammar masks most of an odd vocabulary
        {"name": "sample T48 V32003 masked", "op": "sample", "T": 48, "V": 32003, "mode": "top_k", "masked": 0.9},
        # a large serving batch with mixed settings
        {"name": "sample T256 V152064 mixed", "op": "sample", "T": 256, "V": 152064, "mode": "mixed", "masked": 0.0},
        # a rollout batch: plain sampling from the whole distribution
        {"name": "sample T1024 V152064 plain", "op": "sample", "T": 1024, "V": 152064, "mode": "plain", "masked": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "logits", "sample"])
    if op == "quantize":
        weight = rng.random() < 0.3
        rows = _log_int(rng, 1000, 152064) if weight else _log_int(rng, 1, 16384)
        cols = 16 * _log_int(rng, 16, 224 if weight else 320)
        return {"op": op, "rows": rows, "cols": cols, "block_rows": BLOCK if weight else 1}
    V = _log_int(rng, 1000, 152064)
    if op == "logits":
        return {"op": op, "T": _log_int(rng, 1, 2048), "H": 16 * _log_int(rng, 16, 224), "V": V}
    mode = rng.choice(["plain", "top_k", "top_p", "mixed"])
    return {"op": op, "T": _log_int(rng, 1, 1024), "V": V, "mode": mode,
            "masked": rng.choice([0.0, 0.0, 0.5, 0.98])}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _quantized(rows, cols, block_rows, std, g):
    """Block-quantised normal values, made here so that both sides get the same bits."""
    x = (torch.randn(rows, cols, device="cuda", generator=g) * std).to(torch.bfloat16)
    return _plain_quantize(x, block_rows)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "quantize":
        rows, cols, weight = case["rows"], case["cols"], case["block_rows"] > 1
        x = torch.randn(rows, cols, device="cuda", generator=g)
        if weight:
            x *= 0.02
        else:  # a few channels of hidden states are far larger than the rest
            x *= torch.exp(0.5 * torch.randn(1, cols, device="cuda", generator=g))
            x[:, torch.randint(cols, (max(1, cols // 500),), device="cuda", generator=g)] *= 30.0
        return {"op": op, "x": x.to(torch.bfloat16), "block_rows": case["block_rows"]}
    if op == "logits":
        T, H, V = case["T"], case["H"], case["V"]
        hq, hs = _quantized(T, H, 1, 1.0, g)
        wq, ws = _quantized(V, H, BLOCK, 0.02, g)
        return {"op": op, "hq": hq, "hs": hs, "wq": wq, "ws": ws}
    T, V, mode = case["T"], case["V"], case["mode"]
    # a wide bulk, a row offset, and some tens of likely tokens well above it
    x = 2.0 * torch.randn(T, V, device="cuda", generator=g) + torch.randn(T, 1, device="cuda", generator=g)
    hot = torch.randint(V, (T, min(V, 64)), device="cuda", generator=g)
    x.scatter_add_(1, hot, 8.0 + 3.0 * torch.randn(hot.shape, device="cuda", generator=g))
    if case["masked"] > 0:
        x.masked_fill_(torch.rand(T, V, device="cuda", generator=g) < case["masked"], -math.inf)
        x[::7, 0] = -1.0  # a few rows where one token stays for sure
    state = {"op": op, "logits": x.to(torch.bfloat16), "u": torch.rand(T, device="cuda", generator=g),
             "temperature": 0.7 if mode == "top_p" else 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0}
    if mode == "top_p":
        state["top_p"] = 0.95
    elif mode == "top_k":
        state["top_k"], state["min_p"] = 50, 0.01
    elif mode == "mixed":
        pick = torch.rand(4, T, device="cuda", generator=g)
        t = 0.3 + 1.2 * torch.rand(T, device="cuda", generator=g)
        state["temperature"] = torch.where(pick[0] < 0.1, 0.0, t)
        k = torch.randint(1, 200, (T,), device="cuda", generator=g, dtype=torch.int32)
        state["top_k"] = torch.where(pick[1] < 0.5, 0, k).to(torch.int32)
        p = 0.5 + 0.5 * torch.rand(T, device="cuda", generator=g)
        state["top_p"] = torch.where(pick[2] < 0.3, 1.0, p)
        q = 0.2 * torch.rand(T, device="cuda", generator=g)
        state["min_p"] = torch.where(pick[3] < 0.5, 0.0, q)
    return state


# ------------------------------------------------------------------ plain forms

def _blocks(x, block_rows):
    """x padded with zeros to whole blocks, as [row block, block_rows, column block, 128]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % block_rows))
    return x.view(x.shape[0] // block_rows, block_rows, x.shape[1] // BLOCK, BLOCK)


def _plain_quantize(x, block_rows):
    rows, cols = x.shape
    b = _blocks(x.float(), block_rows)
    amax = b.abs().amax(dim=(1, 3), keepdim=True).clamp_min(AMAX_FLOOR)
    # the product is exact and one division follows, so a quotient halfway between
    # two e4m3 values stays halfway and nothing else crosses such a point
    q = (b * E4M3_MAX / amax).to(torch.float8_e4m3fn)
    q = q.view(b.shape[0] * block_rows, -1)[:rows, :cols].contiguous()
    return q, (amax / E4M3_MAX)[:, 0, :, 0].contiguous()


def _dequantized(q, scale, dtype):
    block_rows = 1 if q.shape[0] == scale.shape[0] else BLOCK
    s = scale.to(dtype).repeat_interleave(block_rows, 0)[:q.shape[0]]
    return q.to(dtype) * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _plain_logits(hq, hs, wq, ws):
    h = _blocks(hq.float(), 1).squeeze(1) * hs[:, :, None]
    w = _blocks(wq.float(), BLOCK) * ws[:, None, :, None]
    h = h.view(h.shape[0], -1)
    w = w.view(-1, h.shape[1])[:wq.shape[0]]
    return (h @ w.t()).to(torch.bfloat16)


def _column(v, rows, dtype):
    if isinstance(v, torch.Tensor):
        return v.to(dtype).view(rows, 1)
    return torch.full((rows, 1), v, dtype=dtype, device="cuda")


def _plain_sample(logits, u, temperature, top_k, top_p, min_p):
    T, V = logits.shape
    t = _column(temperature, T, torch.float32)
    greedy = t == 0
    k = _column(top_k, T, torch.int64)
    p = _column(top_p, T, torch.float32).double()
    floor = _column(min_p, T, torch.float32).double()
    x = logits.float() + 0.0
    x = torch.where(x.isnan(), -math.inf, x)
    x, index = torch.sort(x, dim=1, descending=True, stable=True)
    z = x / torch.where(greedy, 1.0, t)
    d = z.double() - z[:, :1].double()
    d = torch.where(x == x[:, :1], 0.0, d)
    w = torch.where((x == -math.inf) | d.isnan(), 0.0, torch.exp(d))
    cum = torch.cumsum(w, dim=1)
    rank = torch.arange(V, device="cuda").view(1, V)
    last = torch.where(k > 0, k, V).clamp(max=V) - 1
    reach = p * cum.gather(1, last)
    before = torch.cat([torch.zeros(T, 1, dtype=cum.dtype, device="cuda"), cum[:, :-1]], dim=1)
    keep = (rank <= last) & ((before < reach) | (p >= 1)) & (w >= floor)
    kept = torch.where(keep, cum, 0.0).amax(dim=1, keepdim=True)
    at = (keep & (cum <= u.double().view(T, 1) * kept)).sum(dim=1, keepdim=True)
    at = torch.minimum(at, keep.sum(dim=1, keepdim=True) - 1).clamp(min=0)
    at = torch.where(greedy, 0, at)
    nothing = cum[:, -1:] == 0
    token = torch.where(nothing, -1, index.gather(1, at)).to(torch.int32)
    logprob = torch.where(nothing, 0.0, d.gather(1, at) - cum[:, -1:].log()).float()
    return token.view(T), logprob.view(T)


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["op"]
    if own:
        import invariant_lm_head_gb300 as lmh
    if op == "quantize":
        if own:
            return lmh.lmhead_quantize_fp8(state["x"], state["block_rows"])
        return _plain_quantize(state["x"], state["block_rows"])
    if op == "logits":
        args = state["hq"], state["hs"], state["wq"], state["ws"]
        if own:
            return lmh.lmhead_logits_fp8(*args)
        return _plain_logits(*args)
    if own:
        return lmh.lmhead_sample(state["logits"], state["u"], state["temperature"], top_k=state["top_k"],
                                 top_p=state["top_p"], min_p=state["min_p"])
    return _plain_sample(state["logits"], state["u"], state["temperature"], state["top_k"], state["top_p"],
                         state["min_p"])


def work(case):
    ceil = lambda a, b: -(-a // b)  # noqa: E731
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        scales = ceil(case["rows"], case["block_rows"]) * ceil(case["cols"], BLOCK)
        return {"bytes": 3 * n + 4 * scales, "flops": 2 * n}
    if case["op"] == "logits":
        T, H, V = case["T"], case["H"], case["V"]
        scales = (T + ceil(V, BLOCK)) * ceil(H, BLOCK)
        return {"bytes": T * H + V * H + 2 * T * V + 4 * scales, "flops": 2 * T * H * V}
    T, V = case["T"], case["V"]
    settings = 12 * T if case["mode"] == "mixed" else 0
    return {"bytes": 2 * T * V + 12 * T + 4 * settings // 3, "flops": 4 * T * V}


# ------------------------------------------------------------------ in 64 bits

def _e4m3(y):
    """Nearest e4m3 value, ties to even: three fraction bits, exponents from -6."""
    fraction, _ = torch.frexp(y)  # y / fraction is the power of two above |y|, exactly
    step = (torch.where(y == 0, 0.0, y / fraction) / 16).clamp_min(2.0 ** -9)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_row(x, u, t, k, p, floor):
    """One row's token and log-prob from the list of its tokens in order of likelihood."""
    x = np.where(np.isnan(x), -np.inf, x)
    if not (x > -np.inf).any():
        return -1, 0.0
    order = np.lexsort((np.arange(x.size), -x))
    x = x[order]
    z = x / (t if t > 0 else 1.0)
    d = np.zeros_like(z)
    lower = x < x[0]
    d[lower] = z[lower] - z[0]
    w = np.exp(d)
    total = math.fsum(w)
    if t == 0:
        return order[0], -math.log(total)
    n = min(k, x.size) if k > 0 else x.size
    cum = np.cumsum(w[:n])
    if p < 1:
        n = min(n, int(np.searchsorted(cum, p * cum[-1], side="left")) + 1)
    n = max(1, min(n, int((w >= floor).sum())))
    j = min(int(np.searchsorted(cum[:n], u * cum[n - 1], side="right")), n - 1)
    return order[j], d[j] - math.log(total)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        b = _blocks(s["x"].double(), s["block_rows"])
        amax = b.abs().amax(dim=(1, 3), keepdim=True).clamp_min(AMAX_FLOOR)
        q = _e4m3(b * E4M3_MAX / amax).flatten(2).flatten(0, 1)[:case["rows"], :case["cols"]]
        return q, (amax / E4M3_MAX).squeeze(3).squeeze(1)
    if case["op"] == "logits":
        h = _dequantized(s["hq"], s["hs"], torch.float64)
        return h @ _dequantized(s["wq"], s["ws"], torch.float64).t()
    T, V = case["T"], case["V"]
    if T * V > 40_000_000:
        return None
    x = s["logits"].double().cpu().numpy()
    # the operator divides in fp32: each row's values as that division gives them
    ts, ks, ps, fs = (torch.as_tensor(s[n]).double().cpu().numpy() * np.ones(T)
                      for n in ("temperature", "top_k", "top_p", "min_p"))
    us = s["u"].double().cpu().numpy()
    rows = [_exact_row(x[i], us[i], ts[i], int(ks[i]), ps[i], fs[i]) for i in range(T)]
    return np.array([r[0] for r in rows], np.int32), np.array([r[1] for r in rows], np.float64)
