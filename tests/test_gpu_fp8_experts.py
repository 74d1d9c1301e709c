"""The example's layer of FP8 experts: one step against float64 on the dequantized operands, training
that learns, and decode-sized batches that agree with prompt-sized ones.

Tolerances.  The products: as in test_gpu_fp8.py.  The masters' update is at most lr (1 + lr
wd |w|) per element in AdamW's first step (m / sqrt(v) = g / |g|), and equals lr sign(g) up to
eps / |g| and rounding: checked where |g| is above 1e-3 of its mean, to 1 %.
"""

import os
import sys

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def dequantized(codes, scale, block):
    v = codes.view(torch.float8_e4m3fn).double()
    s = scale.double().repeat_interleave(block, -2)[..., :v.shape[-2], :].repeat_interleave(128, -1)[..., :v.shape[-1]]
    return v * s


def near(got, ref):
    got, ref = got.double(), ref
    assert ((got - ref).norm() <= 2.5e-3 * ref.norm()).item(), ((got - ref).norm() / ref.norm()).item()


def test_one_step():
    from fp8_experts import Fp8Experts
    layer = Fp8Experts(4, 272, 400, seed=3)
    counts = [70, 0, 1, 129]
    offsets = torch.from_numpy(synth.offsets_from_counts(counts)).cuda()
    x = synth.randn((200, 400), 1.0, 4, "cuda", torch.bfloat16)
    g = synth.randn((200, 272), 1.0, 5, "cuda", torch.bfloat16)
    w = dequantized(layer.w.data, layer.w.scale, 128)
    xq, gq = (dequantized(*bsq.quantize_e4m3(t), 1) for t in (x, g))
    y, before = layer.forward(x, offsets), layer.master.clone()
    gx = layer.backward(g, x, offsets)
    r0 = 0
    for e, c in enumerate(counts):
        r1 = r0 + c
        if c:
            near(y[r0:r1], xq[r0:r1] @ w[e].T)
            near(gx[r0:r1], gq[r0:r1] @ w[e])
            near(layer.grad[e], g[r0:r1].double().T @ x[r0:r1].double())
        else:
            assert (layer.grad[e] == 0).all()
        r0 = r1
    layer.update(1e-3)
    moved = (layer.master.double() - before.double() * (1 - 1e-3 * 0.01)) / 1e-3
    big = layer.grad.abs() > 1e-3 * layer.grad.abs().float().mean()
    assert (moved[big] + torch.sign(layer.grad[big].double())).abs().max() < 1e-2
    assert (moved[1].abs() < 1e-6 / 1e-3).all()                       # the expert without rows: decay alone
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


def test_training_learns():
    from fp8_experts import Fp8Experts, train
    losses = train(Fp8Experts(4, 256, 512, seed=6), 60)
    assert np.isfinite(losses).all() and np.mean(losses[-5:]) < 0.25 * np.mean(losses[:5]), losses


def test_decode_agrees_with_prompt():
    """Row by row through the few-rows kernel, all at once through the tensor-core one."""
    from fp8_experts import Fp8Experts
    layer = Fp8Experts(2, 256, 640, seed=8)
    x = synth.randn((300, 640), 1.0, 9, "cuda", torch.bfloat16)
    all_rows = layer.forward(x, torch.tensor([150, 300], dtype=torch.int32, device="cuda"))
    for r in (0, 149, 150, 299):
        offs = torch.tensor([1, 1] if r < 150 else [0, 1], dtype=torch.int32, device="cuda")
        near(layer.forward(x[r:r + 1].contiguous(), offs), all_rows[r:r + 1].double())


def test_example_runs(capsys):
    import fp8_experts
    fp8_experts.main()
    assert "loss" in capsys.readouterr().out
