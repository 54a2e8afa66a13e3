"""The binding's stream= argument: what a call allocates belongs to that stream.

Each test keeps the current stream behind (or busy) with matrix products, frees or
drops a tensor whose memory the call could be given, and compares the results
with those of a call on the current stream.
"""

import pytest

import invariant_lm_head_gb300 as lmh
import workloads as W
from helpers import dev, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lmh.build()


@pytest.fixture(scope="module")
def delay():
    """A function that gives the current stream some 20 ms of work."""
    import torch

    a = torch.randn(4096, 4096, device=dev())
    b = torch.empty_like(a)

    def run():
        for _ in range(10):
            torch.mm(a, a, out=b)

    run()
    torch.cuda.synchronize()
    return run


def head_inputs(T, H, V, seed):
    h, hs = lmh.lmhead_quantize_fp8(to_dev_bf16(W.random_bf16(seed, (T, H), 1.0)))
    w, ws = lmh.lmhead_quantize_fp8(to_dev_bf16(W.random_bf16(seed + 1, (V, H), 0.05)), 128)
    return h, hs, w, ws


def bits(t):
    import torch

    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def calls():
    """name -> a call with a stream, on inputs made beforehand."""
    x = to_dev_bf16(W.random_bf16(1, (2000, 1024), 1.0))
    ops = head_inputs(300, 256, 8200, 2)
    logits = lmh.lmhead_logits_fp8(*ops)
    u = to_dev(W.random_f32(4, 300)).abs() % 1.0
    labels = to_dev(W.random_labels(5, 300, 8200))
    h = to_dev_bf16(W.random_bf16(6, (1000, 256), 1.0))
    w = to_dev_bf16(W.random_bf16(7, (8192, 256), 0.05))
    lab = to_dev(W.random_labels(8, 1000, 8192))
    g = to_dev(W.random_f32(9, 1000))
    return {
        "quantize": lambda s: lmh.lmhead_quantize_fp8(x, stream=s),
        "logits": lambda s: (lmh.lmhead_logits_fp8(*ops, stream=s),),
        "sample": lambda s: lmh.lmhead_sample(logits, u, 0.9, top_p=0.9, stream=s),
        "logits path": lambda s: lmh.logprob_from_logits(logits, labels, want_lse=True, stream=s),
        "forward": lambda s: lmh.lmhead_logprob_fwd(h, w, lab, want_lse=True, stream=s),
        "backward": lambda s: lmh.lmhead_logprob_bwd(h, w, lab, g, stream=s),
        "chunked": lambda s: lmh.lmhead_logprob_bwd_chunked(h, w, lab, g, row_chunk=512, stream=s),
    }


NAMES = ["quantize", "logits", "sample", "logits path", "forward", "backward", "chunked"]


@pytest.fixture(scope="module")
def ready():
    import torch

    c = calls()
    want = {n: [t.clone() for t in f(None)] for n, f in c.items()}
    torch.cuda.synchronize()
    return c, want


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_memory_that_the_current_stream_still_writes(name, ready, delay):
    import torch

    call, want = ready[0][name], ready[1][name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want for _ in range(16)]
    delay()
    for t in old:
        bits(t).fill_(85)
    del old, t
    got = call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_dropped_outputs_stay_until_the_current_stream_has_read_them(name, ready, delay):
    import torch

    call, want = ready[0][name], ready[1][name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    delay()
    copies = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(s):
        for shape, dtype in shapes:
            bits(torch.empty(shape, dtype=dtype, device=dev())).fill_(85)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(copies, want))


@pytest.mark.parametrize("name", ["forward", "backward", "chunked"])
def test_the_workspace_stays_the_calls_own(name, ready, delay):
    # the current stream allocates and writes while the call has yet to run
    import torch

    call, want = ready[0][name], ready[1][name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        delay()
    got = call(s)
    if name == "chunked":
        size = lmh.lmhead_workspace_size_bwd(1000, 256, 8192, 512)
    else:
        size = lmh.lmhead_workspace_size(
            lmh.LMH_OP_FWD if name == "forward" else lmh.LMH_OP_BWD, 1000, 256, 8192)
    end = torch.cuda.Event()
    over = torch.empty(size, dtype=torch.uint8, device=dev())
    while True:  # keep writing until the call has ended
        end.record(s)
        for _ in range(50):
            over.fill_(85)
        torch.cuda.current_stream().synchronize()
        if end.query():
            break
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))


def test_the_current_stream_given_by_name(ready):
    import torch

    for name in NAMES:
        got = ready[0][name](torch.cuda.current_stream())
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, ready[1][name])), name
