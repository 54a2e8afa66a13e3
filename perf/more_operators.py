"""Measured cases of the steps around a quantised head: norm, 4-bit logits, alternatives.

Operators that a server runs before, in place of and after the fp8 head's:

* ``norm``: the model's last RMS norm with the residual's addition, its output in
  e4m3 with one fp32 scale per 1 x 128 block, as the fp8 logits take it;
* ``quantize``: bf16 -> microscaled 4-bit floating point (e2m1, one power of two per
  32 elements of a row) and back to the bf16 values that it stands for;
* ``logits``: bf16 logits of a hidden and a weight in that format;
* ``top``: log-probs of given tokens of bf16 logits, the entropy, and the likeliest
  alternatives with theirs.

``own`` chooses between the plain form in elementary torch operations and the
library's entry points. ``exact`` restates each operator in 64 bits.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -60  # 8-bit blocks of (almost) zeros quantise with this maximum
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes, by code


def listed():
    return [
        # one sequence's hidden state before the head of a decode step
        {"name": "norm T1 H4096", "op": "norm", "rows": 1, "cols": 4096, "residual": True},
        # a decode batch whose residual was added before
        {"name": "norm T200 H3600 plain", "op": "norm", "rows": 200, "cols": 3600, "residual": False},
        # a long packed prefill or rollout scored at once
        {"name": "norm T16384 H5120", "op": "norm", "rows": 16384, "cols": 5120, "residual": True},
        # a decode step's hidden states, 64 sequences
        {"name": "quantize 64x3584", "op": "quantize", "rows": 64, "cols": 3584, "std": 1.0},
        # the head's weight after a training step, and what the server then holds
        {"name": "quantize 152064x3584", "op": "quantize", "rows": 152064, "cols": 3584, "std": 0.02},
        # one sequence's next token: the weight is read once, nothing else counts
        {"name": "logits T1 H3584 V152064", "op": "logits", "T": 1, "H": 3584, "V": 152064},
        # a decode batch over a small vocabulary
        {"name": "logits T64 H4096 V32000", "op": "logits", "T": 64, "H": 4096, "V": 32000},
        # ragged everywhere: a short end of H, an odd vocabulary, T off every tile
        {"name": "logits T200 H3616 V32003", "op": "logits", "T": 200, "H": 3616, "V": 32003},
        # whole sequences scored in one call
        {"name": "logits T2048 H3584 V152064", "op": "logits", "T": 2048, "H": 3584, "V": 152064},
        # one sequence's drawn token and the twenty alternatives that a client asked for
        {"name": "top T1 V152064", "op": "top", "T": 1, "V": 152064, "tokens": 1, "top": 20, "masked": 0.0},
        # constrained decoding over an odd vocabulary: four candidate answers scored, five listed
        {"name": "top T48 V32003 masked", "op": "top", "T": 48, "V": 32003, "tokens": 4, "top": 5, "masked": 0.9},
        # a rollout batch: the drawn tokens' log-probs, with alternatives for the trainer
        {"name": "top T1024 V152064", "op": "top", "T": 1024, "V": 152064, "tokens": 1, "top": 20, "masked": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "logits", "top"])
    if op == "norm":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": 16 * _log_int(rng, 16, 320),
                "residual": rng.random() < 0.7}
    if op == "quantize":
        weight = rng.random() < 0.4
        return {"op": op, "rows": _log_int(rng, 1000, 152064) if weight else _log_int(rng, 1, 16384),
                "cols": 32 * _log_int(rng, 8, 112), "std": 0.02 if weight else 1.0}
    V = _log_int(rng, 1000, 152064)
    if op == "logits":
        return {"op": op, "T": _log_int(rng, 1, 2048), "H": 32 * _log_int(rng, 8, 112), "V": V}
    return {"op": op, "T": _log_int(rng, 1, 1024), "V": V, "tokens": rng.choice([1, 1, 2, 5]),
            "top": _log_int(rng, 1, 64), "masked": rng.choice([0.0, 0.0, 0.5, 0.98])}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6421 + 29)


def _hidden(rows, cols, std, g):
    """Normal values; a few channels of hidden states are far larger than the rest."""
    x = torch.randn(rows, cols, device="cuda", generator=g) * std
    if std >= 1.0:
        x *= torch.exp(0.5 * torch.randn(1, cols, device="cuda", generator=g))
        x[:, torch.randint(cols, (max(1, cols // 500),), device="cuda", generator=g)] *= 30.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        w = (1.0 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(torch.bfloat16)
        x = _hidden(rows, cols, 1.0, g)
        r = _hidden(rows, cols, 2.0, g) if case["residual"] else None
        return {"op": op, "x": x, "residual": r, "weight": w}
    if op == "quantize":
        return {"op": op, "x": _hidden(case["rows"], case["cols"], case["std"], g)}
    if op == "logits":
        hq, hs = _pack(_hidden(case["T"], case["H"], 1.0, g))
        wq, ws = _pack(_hidden(case["V"], case["H"], 0.02, g))
        return {"op": op, "hq": hq, "hs": hs, "wq": wq, "ws": ws}
    T, V = case["T"], case["V"]
    # a wide bulk, a row offset, and some tens of likely tokens well above it
    x = 2.0 * torch.randn(T, V, device="cuda", generator=g) + torch.randn(T, 1, device="cuda", generator=g)
    hot = torch.randint(V, (T, min(V, 64)), device="cuda", generator=g)
    x.scatter_add_(1, hot, 8.0 + 3.0 * torch.randn(hot.shape, device="cuda", generator=g))
    if case["masked"] > 0:
        x.masked_fill_(torch.rand(T, V, device="cuda", generator=g) < case["masked"], -math.inf)
        x[::7, 0] = -1.0  # a few rows where one token stays for sure
    # the tokens to score: mostly likely ones, some anywhere
    tokens = torch.randint(V, (T, case["tokens"]), device="cuda", generator=g)
    likely = hot[:, :case["tokens"]]
    tokens = torch.where(torch.rand(tokens.shape, device="cuda", generator=g) < 0.8, likely, tokens)
    t = 0.5 + torch.rand(T, device="cuda", generator=g)
    return {"op": op, "logits": x.to(torch.bfloat16), "tokens": tokens.to(torch.int32), "temperature": t,
            "top": min(case["top"], V)}


# ------------------------------------------------------------------ plain forms

def _plain_norm(x, residual, weight):
    r = None if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    h = (x if r is None else r).float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * weight.float()
    rows, cols = y.shape
    b = torch.nn.functional.pad(y, (0, -cols % 128)).view(rows, -1, 128)
    amax = b.abs().amax(dim=2, keepdim=True).clamp_min(AMAX_FLOOR)
    q = (b * E4M3_MAX / amax).to(torch.float8_e4m3fn).view(rows, -1)[:, :cols].contiguous()
    scale = (amax / E4M3_MAX).squeeze(2)
    return (q, scale) if r is None else (q, scale, r)


def _two(e, dtype):
    """2^e from the bits, for exponents of normal numbers (an underflow is 0)."""
    if dtype == torch.float64:
        return (e.long() + 1023 << 52).view(dtype)
    return (e.int() + 127 << 23).view(dtype)


def _shares(x):
    """Codes (0 .. 15) of x's elements and biased exponents of the 32-blocks' scales.

    A scale is the power of two that leaves a block's largest magnitude in [3.5, 7): the
    largest element is then off by half a step at most, like every other.
    """
    rows, cols = x.shape
    bits = x.view(torch.int16).to(torch.int32) & 0x7FFF
    e = (bits.view(rows, cols // 32, 32).amax(dim=2) + 0x20 >> 7) - 2
    e = e.clamp_min(0)
    y = x.float().view(rows, -1, 32) * _two(127 - e, torch.float32)[:, :, None]
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (y < 0).byte()
    return code.view(rows, cols), e


def _pack(x):
    """The format in memory: two codes a byte (the first in the low half), and the
    exponents of 128 rows x 4 blocks together, [row % 32][row // 32 % 4][block % 4]."""
    code, e = _shares(x)
    rows, blocks = e.shape
    q = code[:, 0::2] | code[:, 1::2] << 4
    e = torch.nn.functional.pad(e.to(torch.uint8), (0, -blocks % 4, 0, -rows % 128), value=127)
    s = e.view(e.shape[0] // 128, 4, 32, e.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return q.contiguous(), s.reshape(s.shape[0], s.shape[1], 32, 16).contiguous()


def _values(code, e, dtype):
    """What codes and exponents stand for."""
    rows, cols = code.shape
    v = torch.tensor(E2M1 + tuple(-m for m in E2M1), dtype=dtype, device=code.device)[code.int()]
    return (v.view(rows, -1, 32) * _two(e.int() - 127, dtype)[:, :, None]).view(rows, cols)


def _unpack(q, s):
    rows, half = q.shape
    code = torch.stack([q & 15, q >> 4], dim=2).view(rows, 2 * half)
    e = s.view(s.shape[0], s.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4)
    return code, e.reshape(s.shape[0] * 128, s.shape[1] * 4)[:rows, :half // 16]


def _plain_logits(hq, hs, wq, ws):
    h = _values(*_unpack(hq, hs), torch.float32)
    w = _values(*_unpack(wq, ws), torch.float32)
    return (h @ w.t()).to(torch.bfloat16)


def _plain_top(logits, tokens, temperature, top):
    V = logits.shape[1]
    x = logits.float() + 0.0
    x = torch.where(x.isnan(), -math.inf, x)
    x, index = torch.sort(x, dim=1, descending=True, stable=True)
    z = x / temperature[:, None]
    d = torch.where(x == x[:, :1], 0.0, z - z[:, :1])
    w = torch.where(x == -math.inf, 0.0, torch.exp(d))
    total = w.sum(dim=1, keepdim=True)
    lse = total.log()
    entropy = (lse - torch.where(w > 0, w * d, 0.0).sum(dim=1, keepdim=True) / total).squeeze(1)
    none = x[:, :top] == -math.inf
    top_token = torch.where(none, -1, index[:, :top]).to(torch.int32)
    top_logprob = torch.where(none, -math.inf, d[:, :top] - lse)
    chosen = logits.float().gather(1, tokens.long().clamp(0, V - 1))
    dt = torch.where(chosen == x[:, :1], 0.0, chosen / temperature[:, None] - z[:, :1])
    valid = (tokens >= 0) & (tokens < V)
    return torch.where(valid, dt - lse, 0.0), entropy, top_token, top_logprob


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["op"]
    if own:
        import invariant_lm_head_gb300 as lmh
    if op == "norm":
        if own:
            q, scale, r = lmh.lmhead_rmsnorm_fp8(state["x"], state["weight"], state["residual"], eps=EPS)
            return (q, scale) if r is None else (q, scale, r)
        return _plain_norm(state["x"], state["residual"], state["weight"])
    if op == "quantize":
        if own:
            return lmh.lmhead_dequantize_mxfp4(*lmh.lmhead_quantize_mxfp4(state["x"]))
        return _values(*_unpack(*_pack(state["x"])), torch.float32).to(torch.bfloat16)
    if op == "logits":
        args = state["hq"], state["hs"], state["wq"], state["ws"]
        if own:
            return lmh.lmhead_logits_mxfp4(*args)
        return _plain_logits(*args)
    if own:
        return lmh.lmhead_top_logprobs(state["logits"], state["tokens"], state["temperature"], top=state["top"])
    return _plain_top(state["logits"], state["tokens"], state["temperature"], state["top"])


def work(case):
    ceil = lambda a, b: -(-a // b)  # noqa: E731
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        scales = case["rows"] * ceil(case["cols"], 128)
        return {"bytes": (7 if case["residual"] else 3) * n + 4 * scales + 2 * case["cols"], "flops": 6 * n}
    if op == "quantize":  # the values in, the packed form out, the values out
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * n + n // 2 + n // 32, "flops": 2 * n}
    T, V = case["T"], case["V"]
    if op == "logits":
        H = case["H"]
        return {"bytes": (T + V) * (H // 2 + H // 32) + 2 * T * V, "flops": 2 * T * H * V}
    return {"bytes": 2 * T * V + T * (8 + 8 * case["tokens"] + 8 * min(case["top"], V)), "flops": 5 * T * V}


# ------------------------------------------------------------------ in 64 bits

def _nearest(y, fraction_bits, lowest_exponent, largest):
    """Nearest floating value with that many fraction bits, ties to even, saturating."""
    _, e = torch.frexp(y)
    step = _two((e - 1).clamp_min(lowest_exponent) - fraction_bits, y.dtype)
    return (torch.round(y / step) * step).clamp(-largest, largest)


def _exact_blocks(x):
    """e2m1 values and scales of 64-bit x [rows, cols], from the format's definition."""
    b = x.view(x.shape[0], -1, 32)
    amax = b.abs().amax(dim=2, keepdim=True)
    # the exponent of the largest magnitude, rounded to two significant bits, less two
    _, e = torch.frexp(amax)
    e = e - 1 + (amax >= 1.75 * _two(e - 1, amax.dtype)).to(e.dtype) - 2
    scale = torch.where(amax == 0, 2.0 ** -127, _two(e.clamp_min(-127), amax.dtype))
    return _nearest(b / scale, 1, 0, 6.0), scale


def _exact_operand(q, s):
    """The value [rows, cols] of each code without its scale, and the scales [rows, cols / 32]."""
    byte = q.to(torch.int64)
    code = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=q.device)
    code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
    m, e = code % 2, code // 2 % 4
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _two(e - 1, torch.float64))
    row = torch.arange(q.shape[0], device=q.device)[:, None]
    blk = torch.arange(q.shape[1] // 16, device=q.device)[None]
    b = s[row // 128, blk // 4, row % 32, row // 32 % 4 * 4 + blk % 4]
    return torch.where(code >= 8, -v, v), _two(b.long() - 127, torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h, r = s["x"].double(), None
        if s["residual"] is not None:
            r = (h + s["residual"].double()).to(torch.bfloat16)
            h = r.double()
        y = h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].double()
        q, scale = [], []
        for b in y.split(128, dim=1):
            a = b.abs().amax(dim=1, keepdim=True).clamp_min(AMAX_FLOOR)
            q.append(_nearest(b * E4M3_MAX / a, 3, -6, E4M3_MAX))
            scale.append(a / E4M3_MAX)
        out = torch.cat(q, dim=1), torch.cat(scale, dim=1)
        return out if r is None else (*out, r.double())
    if op == "quantize":
        rows = []
        for part in s["x"].split(16384):  # in pieces, for memory
            v, scale = _exact_blocks(part.double())
            rows.append((v * scale).view(part.shape))
        return torch.cat(rows)
    if op == "logits":
        hv, hs = _exact_operand(s["hq"], s["hs"])
        wv, ws = _exact_operand(s["wq"], s["ws"])
        out = torch.zeros(case["T"], case["V"], dtype=torch.float64, device="cuda")
        for k in range(hs.shape[1]):
            # a block's products are multiples of 1/4 and their sum is at most 32 * 36: exact in 32 bits
            cols = slice(32 * k, 32 * k + 32)
            part = hv[:, cols].float() @ wv[:, cols].float().t()
            out += part * hs[:, k, None] * ws[None, :, k]
        return out
    V, top = s["logits"].shape[1], s["top"]
    entropy, chosen, tokens, logprobs = [], [], [], []
    for x, t, ids in zip(s["logits"].split(64), s["temperature"].split(64), s["tokens"].long().split(64)):
        z = x.double() / t.double()[:, None]
        lp = torch.log_softmax(z, dim=1)
        p = torch.exp(lp)
        entropy.append(-torch.where(p > 0, p * lp, 0.0).sum(dim=1))
        chosen.append(lp.gather(1, ids))
        # one integer a token, in the order of the list: the logit's bits made monotonic, then the index
        b = (x + 0.0).view(torch.int16).long() & 0xFFFF
        key = torch.where(b >= 0x8000, 0xFFFF - b, b + 0x8000) * 2 ** 32 - torch.arange(V, device="cuda")
        at = torch.topk(key, top, dim=1, sorted=True).indices
        logprobs.append(lp.gather(1, at))
        tokens.append(torch.where(x.gather(1, at) == -math.inf, -1, at).to(torch.int32))
    return torch.cat(chosen), torch.cat(entropy), torch.cat(tokens), torch.cat(logprobs)
