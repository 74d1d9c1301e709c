"""Tensors on a device that is not the current one are refused, and so are given outputs and a
grad_scale on another device than the operands: the library launches on the current device.
On the CPU, with tensors that say which device they are on; no call reaches the library."""

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth


class Operand(torch.Tensor):
    """A CPU tensor that calls itself one of CUDA device `index`."""
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


def operand(index, *shape, dtype=torch.float32):
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
    monkeypatch.setattr(bsq, "_current_device", lambda: 0, raising=False)
    return L


def calls(d, given=None):
    """Every entry point with operands on device d and outputs (adamw: grad_scale) on device `given`."""
    given = d if given is None else given
    out = lambda *shape, dtype=torch.bfloat16: operand(given, *shape, dtype=dtype)  # noqa: E731
    x = operand(d, 4, 256, dtype=torch.bfloat16)
    codes, scale = operand(d, 4, 256, dtype=torch.uint8), operand(d, 4, 2)
    w = synth.Packed(synth.FMT_FP8, operand(d, 1, 256, 256, dtype=torch.uint8), operand(d, 1, 2, 2), None, 1, 256, 256)
    offs = operand(d, 1, dtype=torch.int32)
    table = bsq.adamw_table(*([operand(d, 128)] for _ in range(4)))
    return {
        "quantize_e4m3": lambda: bsq.quantize_e4m3(x, codes=out(4, 256, dtype=torch.uint8), scale=operand(d, 4, 2)),
        "quantize_e4m3 scale": lambda: bsq.quantize_e4m3(x, codes=operand(d, 4, 256, dtype=torch.uint8), scale=out(4, 2, dtype=torch.float32)),
        "fp8_forward": lambda: bsq.fp8_forward(codes, scale, w, out=out(4, 256)),
        "fp8_dgrad": lambda: bsq.fp8_dgrad(codes, scale, w, out=out(4, 256)),
        "fp8_grouped_forward": lambda: bsq.fp8_grouped_forward(codes, scale, w, offs, out=out(4, 256)),
        "fp8_grouped_dgrad": lambda: bsq.fp8_grouped_dgrad(codes, scale, w, offs, out=out(4, 256)),
        "adamw": lambda: bsq.adamw(table, 1, 1e-3, grad_scale=out(1, dtype=torch.float32)),
    }


NAMES = ["quantize_e4m3", "quantize_e4m3 scale", "fp8_forward", "fp8_dgrad", "fp8_grouped_forward", "fp8_grouped_dgrad", "adamw"]


@pytest.mark.parametrize("name", NAMES)
def test_the_current_device_is_taken(library, name):
    calls(0)[name]()
    assert len(library.calls) == 1


@pytest.mark.parametrize("name", NAMES)
def test_another_device_is_refused(library, name):
    with pytest.raises(ValueError, match="cuda:1"):
        calls(1)[name]()
    assert not library.calls


@pytest.mark.parametrize("name", NAMES)
def test_outputs_elsewhere_are_refused(library, name):
    with pytest.raises(ValueError, match="cuda:1"):
        calls(0, given=1)[name]()
    assert not library.calls
