"""Products of few rows with 4-bit weights around the contraction's length at which the scales of a tile no longer fit the shared
memory beside the rings, for every launch: the longest that fits, and the next two.

One-hot tokens leave a single product, whose result has one value bit for bit: the weight as the oracle dequantizes it.
"""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth
from tests._util import bf16_vals, oracle_deq

pytestmark = pytest.mark.gpu

GROUP = {synth.FMT_MXFP4: 32, synth.FMT_NVFP4: 16}
# (experts or 0 for a dense product, rows, wide, K of NVFP4); MXFP4 has half as many scales
LAUNCHES = [(0, 8, False, 50176), (0, 9, False, 17408), (0, 17, False, 33792), (0, 8, True, 82944), (0, 13, True, 11008),
            (0, 33, True, 47104), (2, 10, False, 63488), (2, 12, False, 41216), (2, 20, False, 57856), (2, 40, False, 47104)]
FITS = {(synth.FMT_NVFP4, i): case[3] for i, case in enumerate(LAUNCHES)}
FITS.update({(synth.FMT_MXFP4, i): k for i, k in enumerate([100608, 35072, 67840, 166144, 22272, 94208, 126976, 82688, 115968, 94208])})


def weights(fmt, E, N, K, seed):
    """Every code under ordinary scales, drawn on the device."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    draw = lambda low, high, cols: torch.randint(low, high, (E, N, cols), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    scale = draw(120, 132, K // 32) if fmt == synth.FMT_MXFP4 else draw(40, 72, K // 16)
    ts = None if fmt == synth.FMT_MXFP4 else torch.full((E,), 2.0 ** -9, device="cuda")
    return synth.Packed(fmt, draw(0, 256, K // 2), scale, ts, E, N, K)


def columns(w, e, ks):
    """float64 [len(ks), N]: the oracle's values of expert e's columns ks."""
    g = GROUP[w.fmt]
    data = torch.stack([w.data[e, :, k // g * (g // 2):(k // g + 1) * (g // 2)] for k in ks]).cpu()
    scale = torch.stack([w.scale[e, :, k // g, None] for k in ks]).cpu()
    ts = None if w.tensor_scale is None else w.tensor_scale[e].cpu().repeat(len(ks))
    v = oracle_deq(synth.Packed(w.fmt, data, scale, ts, len(ks), w.rows, g))
    return np.stack([v[i, :, k % g] for i, k in enumerate(ks)])


@pytest.mark.parametrize("more", [0, 256, 512])
@pytest.mark.parametrize("fmt", [synth.FMT_MXFP4, synth.FMT_NVFP4])
@pytest.mark.parametrize("launch", range(len(LAUNCHES)))
def test_scales_that_just_fit_and_just_do_not(launch, fmt, more):
    E, rows, wide, _ = LAUNCHES[launch]
    K = FITS[fmt, launch] + more
    N = 32 * torch.cuda.get_device_properties(0).multi_processor_count + 8 if wide else 72
    W = weights(fmt, max(E, 1), N, K, K + rows)
    ks = [K - 1 - i * ((K - 1) // (rows - 1)) for i in range(rows)]
    X = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    X[torch.arange(rows), torch.tensor(ks)] = 1
    if E == 0:
        got, want = bsq.fp4_forward(X, W), columns(W, 0, ks)
    else:
        half = rows // 2 - 1
        got = bsq.fp4_grouped_forward(X, W, torch.tensor([half, rows], dtype=torch.int32, device="cuda"))
        want = np.concatenate([columns(W, 0, ks[:half]), columns(W, 1, ks[half:])])
    assert np.array_equal(bf16_vals(got), want)
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)
