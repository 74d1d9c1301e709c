"""The binding of the router, the operators between tokens and rows and the 4-bit products: devices,
streams' memory and shapes, on the CPU with tensors that say which device they are on and a
library that records its calls."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth

BF16, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


class Operand(torch.Tensor):
    """A CPU tensor that calls itself one of CUDA device `index`."""
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


def operand(index, *shape, dtype=F32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Operand)
    t.index = index
    return t


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(bsq, "_lib", L)
    monkeypatch.setattr(bsq, "_raw_stream", lambda stream, like: 0)
    monkeypatch.setattr(bsq, "_current_device", lambda: 0)
    return L


def weight(d, E=1, fmt=synth.FMT_NVFP4):
    return synth.Packed(fmt, operand(d, E, 64, 128, dtype=U8), operand(d, E, 64, 256 // (16 if fmt == synth.FMT_NVFP4 else 32), dtype=U8),
                        operand(d, E), E, 64, 256)


def calls(d, o=None, stream=None, outs=True):
    """Every entry point with operands on device d, and outputs on device o (outs=False: none given)."""
    o = d if o is None else o
    out = lambda *shape, dtype: operand(o, *shape, dtype=dtype) if outs else None  # noqa: E731
    logits, ids = operand(d, 4, 8, dtype=BF16), operand(d, 4, 2, dtype=I32)
    w, x, y = operand(d, 4, 2), operand(d, 4, 256, dtype=BF16), operand(d, 8, 256, dtype=BF16)
    rows_out = dict(codes=out(8, 256, dtype=U8), scale=out(8, 2, dtype=F32), e4m3=True, stream=stream)
    return {
        "route": lambda: bsq.route(logits, 2, bias=operand(d, 8), ids=out(4, 2, dtype=I32), weights=out(4, 2, dtype=F32), stream=stream),
        "route_backward": lambda: bsq.route_backward(logits, ids, w, out=out(4, 8, dtype=BF16), stream=stream),
        "sort_experts": lambda: bsq.sort_experts(ids, 8, offsets=out(8, dtype=I32), rows=out(4, 2, dtype=I32), slots=out(8, dtype=I32), stream=stream),
        "dispatch": lambda: bsq.dispatch(x, ids, w, out=out(8, 256, dtype=BF16), **rows_out),
        "combine": lambda: bsq.combine(y, ids, w, out=out(4, 256, dtype=BF16), stream=stream),
        "combine_backward": lambda: bsq.combine_backward(x, y, ids, w, grad_y=out(8, 256, dtype=BF16), grad_weights=out(4, 2, dtype=F32), **rows_out),
        "fp4_forward": lambda: bsq.fp4_forward(x, weight(d), out=out(4, 64, dtype=BF16), stream=stream),
        "fp4_grouped_forward": lambda: bsq.fp4_grouped_forward(x, weight(d, 3), operand(d, 3, dtype=I32), out=out(4, 64, dtype=BF16), stream=stream),
    }


NAMES = list(calls(0))


@pytest.mark.parametrize("name", NAMES)
def test_the_current_device_is_taken(library, name):
    calls(0)[name]()
    assert library.calls == ["bsq_" + name]


@pytest.mark.parametrize("name", NAMES)
def test_another_device_is_refused(library, name):
    with pytest.raises(ValueError, match="cuda:1"):
        calls(1)[name]()
    assert not library.calls


@pytest.mark.parametrize("name", NAMES)
def test_outputs_elsewhere_are_refused(library, name):
    with pytest.raises(ValueError, match="cuda:1"):
        calls(0, 1)[name]()
    assert not library.calls


def test_operands_elsewhere_are_refused(library):
    here = lambda *s, dtype=F32: operand(0, *s, dtype=dtype)  # noqa: E731
    there = lambda *s, dtype=F32: operand(1, *s, dtype=dtype)  # noqa: E731
    w = weight(0)
    for call in (lambda: bsq.route(here(4, 8), 2, bias=there(8)),
                 lambda: bsq.route_backward(here(4, 8), there(4, 2, dtype=I32), here(4, 2)),
                 lambda: bsq.route_backward(here(4, 8), here(4, 2, dtype=I32), there(4, 2)),
                 lambda: bsq.dispatch(here(4, 256, dtype=BF16), there(4, 2, dtype=I32)),
                 lambda: bsq.dispatch(here(4, 256, dtype=BF16), here(4, 2, dtype=I32), there(4, 2)),
                 lambda: bsq.combine(here(8, 256, dtype=BF16), there(4, 2, dtype=I32)),
                 lambda: bsq.combine(here(8, 256, dtype=BF16), here(4, 2, dtype=I32), there(4, 2)),
                 lambda: bsq.combine_backward(here(4, 256, dtype=BF16), there(8, 256, dtype=BF16), here(4, 2, dtype=I32)),
                 lambda: bsq.fp4_forward(there(4, 256, dtype=BF16), w),
                 lambda: bsq.fp4_forward(here(4, 256, dtype=BF16), synth.Packed(w.fmt, there(1, 64, 128, dtype=U8), w.scale, w.tensor_scale, 1, 64, 256)),
                 lambda: bsq.fp4_forward(here(4, 256, dtype=BF16), synth.Packed(w.fmt, w.data, w.scale, there(1), 1, 64, 256)),
                 lambda: bsq.fp4_grouped_forward(here(4, 256, dtype=BF16), weight(0, 3), there(3, dtype=I32))):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert not library.calls


def test_shapes_and_types_are_refused(library):
    o = lambda *s, dtype=F32: operand(0, *s, dtype=dtype)  # noqa: E731
    x, ids, w, y = o(4, 256, dtype=BF16), o(4, 2, dtype=I32), o(4, 2), o(8, 256, dtype=BF16)
    p = weight(0)
    for call in (lambda: bsq.route(o(8), 2), lambda: bsq.route(o(4, 8, dtype=torch.float16), 2), lambda: bsq.route(o(8, 4).t(), 2),
                 lambda: bsq.route(o(4, 8), 2, gate="relu"), lambda: bsq.route(o(4, 8), 2, bias=o(7)), lambda: bsq.route(None, 2),
                 lambda: bsq.route(o(4, 8), 2, ids=o(4, 3, dtype=I32)), lambda: bsq.route(o(4, 8), 2, ids=ids, weights=o(4, 2, dtype=BF16)),
                 lambda: bsq.route_backward(o(4, 8), o(3, 2, dtype=I32), w), lambda: bsq.route_backward(o(4, 8), ids, o(4, 3)),
                 lambda: bsq.sort_experts(o(4, 2, dtype=torch.int64), 8), lambda: bsq.sort_experts(o(8, dtype=I32), 8),
                 lambda: bsq.sort_experts(ids, 8, offsets=o(9, dtype=I32)),
                 lambda: bsq.dispatch(o(4, 256), ids), lambda: bsq.dispatch(x, o(5, 2, dtype=I32)), lambda: bsq.dispatch(x, ids, o(4, 3)),
                 lambda: bsq.dispatch(x, ids, bf16=False), lambda: bsq.dispatch(x, ids, S=9, out=o(8, 256, dtype=BF16)),
                 lambda: bsq.combine(o(8, 256), ids), lambda: bsq.combine(y, ids, o(2, 4)), lambda: bsq.combine(y, ids, out=o(8, 256, dtype=BF16)),
                 lambda: bsq.combine_backward(x, None, ids), lambda: bsq.combine_backward(x, o(8, 128, dtype=BF16), ids),
                 lambda: bsq.combine_backward(x, y, ids, S=9), lambda: bsq.combine_backward(x, y, o(5, 2, dtype=I32)),
                 lambda: bsq.fp4_forward(o(4, 128, dtype=BF16), p), lambda: bsq.fp4_forward(x, weight(0, 2)), lambda: bsq.fp4_forward(o(4, 256), p),
                 lambda: bsq.fp4_forward(x, synth.Packed(p.fmt, p.data, None, p.tensor_scale, 1, 64, 256)),
                 lambda: bsq.fp4_forward(x, synth.Packed(p.fmt, None, p.scale, p.tensor_scale, 1, 64, 256)),
                 lambda: bsq.fp4_forward(x, synth.Packed(p.fmt, p.data, p.scale, None, 1, 64, 256)),
                 lambda: bsq.fp4_forward(x, synth.Packed(synth.FMT_MXFP4, p.data, p.scale, None, 1, 64, 256)),
                 lambda: bsq.fp4_grouped_forward(x, weight(0, 3), o(2, dtype=I32)),
                 lambda: bsq.fp4_grouped_forward(x, weight(0, 3), o(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    assert not library.calls


def test_what_is_not_wanted_is_not_made(library):
    o = lambda *s, dtype=F32: operand(0, *s, dtype=dtype)  # noqa: E731
    x, ids, out = o(4, 256, dtype=BF16), o(4, 2, dtype=I32), o(8, 256, dtype=BF16)
    assert [t is None for t in bsq.dispatch(x, ids, out=out)] == [False, True, True]
    assert [t is None for t in bsq.combine_backward(x, None, ids, want_weights=False, grad_y=out)] == [False, True, True, True]
    assert bsq.sort_experts(ids, 8, want_slots=False, offsets=o(8, dtype=I32), rows=o(4, 2, dtype=I32))[2] is None


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_the_launching_streams(monkeypatch, name):
    now, seen = ["current"], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream.name)
        yield
        now.pop()

    class Tensor:
        def __init__(self):
            self.recorded = []
            seen.append((now[-1], self.recorded))

        def record_stream(self, stream):
            self.recorded.append(stream.name)

        def data_ptr(self):
            return 0x10000

    monkeypatch.setattr(torch, "empty", lambda shape, **kw: Tensor())
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(name=now[-1], cuda_stream=0))
    monkeypatch.setattr(bsq, "_lib", Library())
    monkeypatch.setattr(bsq, "_raw_stream", lambda stream, like: 0)
    monkeypatch.setattr(bsq, "_current_device", lambda: 0)
    calls(0, stream=SimpleNamespace(name="side", cuda_stream=1), outs=False)[name]()
    assert seen and all(s == ("side", ["current"]) for s in seen), seen
    del seen[:]
    calls(0, outs=False)[name]()
    assert seen and all(s == ("current", []) for s in seen), seen
