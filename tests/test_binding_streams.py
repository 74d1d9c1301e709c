"""Where the binding allocates an output that the caller did not give: for a kernel on another stream,
of that stream's memory (a block freed on the current stream may still be in use there), and
recorded for the current stream, which reads the result.  On the CPU, with stand-ins for the
allocator and the streams."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth


@pytest.fixture
def allocations(monkeypatch):
    """[(stream the block belongs to, streams recorded)] of every torch.empty."""
    now, seen = ["current"], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream.name)
        yield
        now.pop()

    class Tensor:
        def __init__(self, shape):
            self.shape, self.recorded = shape, []
            seen.append((now[-1], self.recorded))

        def record_stream(self, stream):
            self.recorded.append(stream.name)

        def data_ptr(self):
            return 0x10000

    class Library:
        def __getattr__(self, name):
            return lambda *args: 0

    monkeypatch.setattr(torch, "empty", lambda shape, **kw: Tensor(shape))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(name=now[-1], cuda_stream=0))
    monkeypatch.setattr(bsq, "_lib", Library())
    monkeypatch.setattr(bsq, "_raw_stream", lambda stream, like: 0)
    monkeypatch.setattr(bsq, "_current_device", lambda: 0, raising=False)
    return seen


class Operand(torch.Tensor):
    """A CPU tensor that calls itself a CUDA one."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def operand(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Operand)


SIDE = SimpleNamespace(name="side", cuda_stream=1)


def calls():
    x = operand(4, 256, dtype=torch.bfloat16)
    codes, scale = operand(4, 256, dtype=torch.uint8), operand(4, 2)
    w = synth.Packed(synth.FMT_FP8, operand(1, 256, 256, dtype=torch.uint8), operand(1, 2, 2), None, 1, 256, 256)
    offs = operand(1, dtype=torch.int32)
    return {
        "quantize_e4m3": lambda s: bsq.quantize_e4m3(x, stream=s),
        "fp8_forward": lambda s: bsq.fp8_forward(codes, scale, w, stream=s),
        "fp8_dgrad": lambda s: bsq.fp8_dgrad(codes, scale, w, stream=s),
        "fp8_grouped_forward": lambda s: bsq.fp8_grouped_forward(codes, scale, w, offs, stream=s),
        "fp8_grouped_dgrad": lambda s: bsq.fp8_grouped_dgrad(codes, scale, w, offs, stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_outputs_are_the_launching_streams(allocations, name):
    call = calls()[name]
    call(SIDE)
    assert allocations and all(a == ("side", ["current"]) for a in allocations), allocations
    del allocations[:]
    call(None)
    assert allocations and all(a == ("current", []) for a in allocations), allocations


def decoding_calls():
    """The entry points that decode their operands, temporaries of the backward on E5M2 codes included."""
    g = operand(4, 256, dtype=torch.bfloat16)
    w = synth.Packed(synth.FMT_FP8, operand(1, 256, 256, dtype=torch.uint8), operand(1, 2, 2), None, 1, 256, 256)
    x = synth.Packed(synth.FMT_FP8, operand(1, 4, 256, dtype=torch.uint8), operand(1, 1, 2), None, 1, 4, 256)
    offs = operand(1, dtype=torch.int32)
    return {
        "dequant": lambda s: bsq.dequant(w, stream=s),
        "linear_dgrad": lambda s: bsq.linear_dgrad(g, w, stream=s),
        "linear_dgrad_smallm_noalloc": lambda s: bsq.linear_dgrad_smallm_noalloc(g, w, stream=s),
        "linear_wgrad": lambda s: bsq.linear_wgrad(g, x, stream=s),
        "linear_backward": lambda s: bsq.linear_backward(g, w, x, stream=s),
        "quantize_e5m2": lambda s: bsq.quantize_e5m2(g, stream=s),
        "linear_backward_e5m2": lambda s: bsq.linear_backward_e5m2(g, w, x, stream=s),
        "linear_forward": lambda s: bsq.linear_forward(x, w, stream=s),
        "grouped_dgrad": lambda s: bsq.grouped_dgrad(g, w, offs, stream=s),
        "grouped_wgrad": lambda s: bsq.grouped_wgrad(g, x, offs, 1, stream=s),
    }


@pytest.mark.parametrize("name", list(decoding_calls()))
def test_outputs_of_decoding_calls_are_the_launching_streams(allocations, monkeypatch, name):
    monkeypatch.setattr(bsq, "_stream", lambda stream: 0)
    call = decoding_calls()[name]
    call(SIDE)
    assert allocations and all(a == ("side", ["current"]) for a in allocations), allocations
    del allocations[:]
    call(None)
    assert allocations and all(a == ("current", []) for a in allocations), allocations
