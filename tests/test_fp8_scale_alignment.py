"""W's block scales of the E4M3 products need their elements' alignment alone: the slice of one expert
out of a stacked weight starts at a multiple of its block count, whatever that is."""

import os

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth

FAKE = 0x10000   # never read: calls without rows end after the checks


@pytest.mark.parametrize("name", ["bsq_fp8_forward", "bsq_fp8_dgrad", "bsq_fp8_grouped_forward", "bsq_fp8_grouped_dgrad"])
def test_checks(name):
    if not os.path.exists(bsq.LIB_PATH):
        from block_scaled_gemm_fp8_gb300 import build
        build.build()

    def call(ws):
        many = ("grouped" in name) * 1
        return getattr(bsq.lib(), name)(None, None, 0, 1, FAKE, ws, *[3][:many], 128, 256, *[FAKE][:many], None, None)
    for ws in (FAKE, FAKE + 4, FAKE + 8, FAKE + 12):
        assert call(ws) == bsq.BSQ_OK, ws
    for ws in (FAKE + 1, FAKE + 2, FAKE + 6, None):
        assert call(ws) == bsq.BSQ_ERR_INVALID_ARG, ws


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 24, 300])
@pytest.mark.parametrize("N,K", [(144, 400), (384, 128), (264, 2064)])
def test_an_experts_slice(M, N, K):
    """The slice's product is that of the same weight on its own, bit for bit."""
    E = 4
    codes, scale = bsq.quantize_e4m3(synth.randn((E, N, K), 0.02, 1, "cuda"), 128)
    x = bsq.quantize_e4m3(synth.randn((M, K), 1.0, 2, "cuda", torch.bfloat16))
    pad = lambda n: -(-n // 16) * 16  # noqa: E731
    g = bsq.quantize_e4m3(synth.randn((M, pad(N)), 1.0, 3, "cuda", torch.bfloat16)) if N % 16 == 0 else None
    offs = torch.tensor([M // 2, M], dtype=torch.int32, device="cuda")
    seen = set()
    for e in range(E):
        part = synth.Packed(synth.FMT_FP8, codes[e:e + 1], scale[e:e + 1], None, 1, N, K)
        own = synth.Packed(synth.FMT_FP8, codes[e:e + 1].clone(), scale[e:e + 1].clone(), None, 1, N, K)
        seen.add(part.scale.data_ptr() % 16)
        assert torch.equal(bsq.fp8_forward(*x, part), bsq.fp8_forward(*x, own))
        if g is not None:
            assert torch.equal(bsq.fp8_dgrad(*g, part), bsq.fp8_dgrad(*g, own))
        if e + 2 <= E:
            two = synth.Packed(synth.FMT_FP8, codes[e:e + 2], scale[e:e + 2], None, 2, N, K)
            ref = synth.Packed(synth.FMT_FP8, codes[e:e + 2].clone(), scale[e:e + 2].clone(), None, 2, N, K)
            assert torch.equal(bsq.fp8_grouped_forward(*x, two, offs), bsq.fp8_grouped_forward(*x, ref, offs))
            if g is not None:
                assert torch.equal(bsq.fp8_grouped_dgrad(*g, two, offs), bsq.fp8_grouped_dgrad(*g, ref, offs))
    assert (scale[0].numel() % 4 == 0) or len(seen) > 1
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)
