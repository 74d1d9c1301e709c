"""Dense products of few rows with a 4-bit weight of more than 32 rows an SM: tiles of their own, warps beside one another that share the
tokens, a last tile that is not full.  Tolerance as for the narrower ones (tests/test_gpu_fp4.py); one-hot tokens leave one product, bit for bit."""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth
from oracle import gemm as Gm
from tests._util import bf16_vals, oracle_deq

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
FMTS = [synth.FMT_MXFP4, synth.FMT_NVFP4]


def columns(more):
    """N above the limit; no multiple of a tile's 32, 48 or 96 rows."""
    n = 32 * torch.cuda.get_device_properties(0).multi_processor_count + more
    assert n % 8 == 0 and n % 32 and n % 48 and n % 96
    return n


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("more", [8, 9480])
@pytest.mark.parametrize("K", [512, 288, 2080])
def test_forward(fmt, more, K):
    N = columns(more)
    W = synth.make_packed(fmt, 1, N, K, 0.5, seed=K, device="cuda")
    w = oracle_deq(W)[0]
    for M in (1, 8, 9, 13, 16, 17, 33, 64):
        X = synth.randn((M, K), 1.0, M, "cpu", BF16)
        out = torch.full((M + 1, N), 7.0, dtype=BF16, device="cuda")
        bsq.fp4_forward(X.cuda(), W, out=out[:M])
        got, x = bf16_vals(out[:M]), bf16_vals(X)
        ref = x @ w.T
        ok, err, _ = Gm.check(got, ref, Gm.tolerance(K, x, w))
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert ok and rel <= 2.5e-3, f"M{M}: max|err|={err} relF={rel}"
        assert (out[M] == 7).all()
        again = [bsq.fp4_forward(X.cuda(), W) for _ in range(5)]
        assert all(torch.equal(a, out[:M]) for a in again)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 8, 9, 13, 16, 17, 33, 64])
@pytest.mark.parametrize("K", [512, 288, 2080])
def test_one_hot_rows_pick_the_weights_bits(fmt, M, K):
    N = columns(8)
    W = synth.random_codes(fmt, 1, N, K, seed=M, device="cpu", scale_kind="finite")
    want = oracle_deq(W)[0]
    assert np.isfinite(want).all()
    W = W.to("cuda")
    for k0 in sorted({0, K // 2 - M // 2, max(0, K - M)}):
        X = torch.zeros((M, K), dtype=BF16)
        X[torch.arange(M), k0 + torch.arange(M)] = 1
        assert np.array_equal(bf16_vals(bsq.fp4_forward(X.cuda(), W)), want[:, k0:k0 + M].T)
