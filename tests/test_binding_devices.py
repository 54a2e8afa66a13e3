"""The binding refuses what does not belong to the current device, before any launch.

Tensors and streams of a second GPU are stand-ins that only say so: no GPU is used.
"""

import pytest

import invariant_lm_head_gb300 as lmh
import invariant_lm_head_gb300.fp8_head as fp8_head

torch = pytest.importorskip("torch")


class Elsewhere(torch.Tensor):
    """A host tensor that says it is on cuda:1."""

    device = property(lambda self: torch.device("cuda:1"))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.device.index


class Here(Elsewhere):
    device = property(lambda self: torch.device("cuda:0"))


class OtherStream:
    device = torch.device("cuda:1")
    cuda_stream = 0


def calls(kind):
    """name -> a call that is right but for its tensors' device."""
    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(kind)

    bf, f8, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
    h, w, lab, g = t(4, 256, dtype=bf), t(1024, 256, dtype=bf), t(4, dtype=i32), t(4)
    hq, wq, lg = t(4, 256, dtype=f8), t(1024, 256, dtype=f8), t(4, 1024, dtype=bf)
    hs, ws, plane, u = t(4, 2), t(8, 2), t(1, 4), t(4)
    host = [torch.zeros_like(x.as_subclass(torch.Tensor)) for x in (h, w, lab)]
    return {
        "quantize": lambda **k: lmh.lmhead_quantize_fp8(h, **k),
        "quantize weight": lambda **k: lmh.lmhead_quantize_fp8(w, 128, **k),
        "logits": lambda **k: lmh.lmhead_logits_fp8(hq, hs, wq, ws, **k),
        "sample": lambda **k: lmh.lmhead_sample(lg, u, u, **k),
        "fwd": lambda **k: lmh.lmhead_logprob_fwd(h, w, lab, **k),
        "fwd stats": lambda **k: lmh.lmhead_logprob_fwd_stats(h, w, lab, **k),
        "fwd host": lambda **k: lmh.lmhead_logprob_fwd_host(*host, hidden=h, weight=w, labels=lab,
                                                            **k),
        "bwd": lambda **k: lmh.lmhead_logprob_bwd(h, w, lab, g, **k),
        "entropy bwd": lambda **k: lmh.lmhead_logprob_entropy_bwd(h, w, lab, g, g, **k),
        "chunked": lambda **k: lmh.lmhead_logprob_bwd_chunked(h, w, lab, g, row_chunk=128, **k),
        "shard": lambda **k: lmh.lmhead_logprob_bwd_shard(h, w, lab, g, g, 0, **k),
        "sum ranks": lambda **k: lmh.lmhead_sum_ranks_bf16(t(2, 8), **k),
        "logits path": lambda **k: lmh.logprob_from_logits(lg, lab, **k),
        "division": lambda **k: lmh.logprob_from_logits_div(lg, lab, u, **k),
        "partials": lambda **k: lmh.lmhead_logprob_fwd_partials(
            h, w, lab, 0, part_m=plane, part_s=plane, part_u=plane, label_logit=g, **k),
        "merge": lambda **k: lmh.lmhead_logprob_merge(plane, plane, plane, g, lab, 1024, **k),
        "engine": lambda **k: lmh.lmhead_engine_gemm(h, w, **k),
    }


NAMES = list(calls(Elsewhere))


@pytest.fixture
def launches(monkeypatch):
    lmh.build()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    n = lmh.lmhead_kernel_launches()
    yield
    assert lmh.lmhead_kernel_launches() == n


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(name, launches):
    with pytest.raises(ValueError, match="current device is cuda:0"):
        calls(Elsewhere)[name]()


@pytest.mark.parametrize("name", NAMES)
def test_streams_of_another_device_are_refused(name, launches):
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        calls(Here)[name](stream=OtherStream())


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_are_refused(name, launches):
    with pytest.raises(ValueError, match="CUDA device"):
        calls(torch.Tensor)[name]()


def test_a_head_of_another_device_is_refused(launches):
    w = torch.zeros(1024, 256, dtype=torch.bfloat16).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        fp8_head.FP8Head(w)
