"""A call on another stream than the current one, while the current stream still uses blocks that were
freed on it: the outputs come from the other stream's memory, and hold what they should."""

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth

pytestmark = pytest.mark.gpu

N = 1024


def operands():
    x = synth.randn((N, N), 1.0, 1, "cuda", torch.bfloat16)
    c, s = bsq.quantize_e4m3(synth.randn((1, N, N), 0.5, 2, "cuda"), 128)
    return x, synth.Packed(synth.FMT_FP8, c, s, None, 1, N, N)


def calls():
    x, w = operands()
    codes, scale = bsq.quantize_e4m3(x)
    offs = torch.tensor([N], dtype=torch.int32, device="cuda")
    return {
        "quantize_e4m3": lambda s=None: bsq.quantize_e4m3(x, stream=s)[0],
        "fp8_forward": lambda s=None: bsq.fp8_forward(codes, scale, w, stream=s),
        "fp8_dgrad": lambda s=None: bsq.fp8_dgrad(codes, scale, w, stream=s),
        "fp8_grouped_forward": lambda s=None: bsq.fp8_grouped_forward(codes, scale, w, offs, stream=s),
        "fp8_grouped_dgrad": lambda s=None: bsq.fp8_grouped_dgrad(codes, scale, w, offs, stream=s),
    }


NAMES = ["quantize_e4m3", "fp8_forward", "fp8_dgrad", "fp8_grouped_forward", "fp8_grouped_dgrad"]


@pytest.mark.parametrize("name", NAMES)
def test_freed_blocks_of_the_current_stream_are_left_alone(name):
    call = calls()[name]
    want = call().clone()
    torch.cuda.synchronize()
    side, ready = torch.cuda.Stream(), torch.cuda.Event()
    ready.record()
    side.wait_event(ready)
    busy = torch.ones((4096, 4096), device="cuda")
    freed = set()
    for _ in range(20):
        busy = busy @ busy * 1e-4
        block = torch.empty_like(want)
        block.fill_(3)                      # queued behind the products
        freed.add(block.data_ptr())
        del block
    got = call(side)
    assert got.data_ptr() not in freed
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)
