"""Products of a few BF16 token rows with 4-bit weights (bsq_fp4_forward, bsq_fp4_grouped_forward) against the
oracle's dequantization and 64-bit sums.

Tolerance.  A BF16 product is exact in float32, the sums run in float32; the result is rounded to BF16 once, at most
2^-8 of it (an eighth of the bits less on average).  Elementwise the bound is that of every product of the library (2e-2
sqrt(K) rms rms, plus 2^-8 |ref|); over the matrix the relative error is the BF16 rounding's alone, which is at most
2^-9 rms, so 2.5e-3 leaves 28 % for float32 accumulation.  One-hot rows leave a single product, whose result has one
value bit for bit: the weight's column as bsq_dequant's rule gives it.
"""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth
from oracle import gemm as Gm
from tests._util import bf16_vals, oracle_deq

pytestmark = pytest.mark.gpu

REL = 2.5e-3
FMTS = [synth.FMT_MXFP4, synth.FMT_NVFP4]
BF16 = torch.bfloat16


def close(out, ref, x, w, what):
    ok, err, _ = Gm.check(out, ref, Gm.tolerance(w.shape[-1], x, w))
    norm = np.linalg.norm(ref)
    rel = np.linalg.norm(out - ref) / norm if norm else np.linalg.norm(out)
    assert ok and rel <= REL, f"{what}: max|err|={err} relF={rel}"


def activations(M, K, seed):
    return synth.randn((M, K), 1.0, seed, "cpu", BF16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 4096, 4096), (2, 40, 96), (3, 136, 1056), (7, 264, 160), (8, 64, 2048), (9, 1000, 512),
                                   (16, 512, 3104), (17, 48, 288), (31, 200, 128), (32, 96, 4096), (33, 72, 64), (63, 264, 1120), (64, 1024, 7168),
                                   (65, 256, 512), (200, 264, 1056)])
def test_forward(fmt, M, N, K):
    W = synth.make_packed(fmt, 1, N, K, 0.5, seed=M + N, device="cpu")
    X = activations(M, K, M + K)
    out = bsq.fp4_forward(X.cuda(), W.to("cuda"))
    x, w = bf16_vals(X), oracle_deq(W)[0]
    close(bf16_vals(out), x @ w.T, x, w, f"M{M} N{N} K{K}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [5, 16, 40])
def test_one_hot_rows_pick_the_weights_bits(fmt, M):
    """Every code under ordinary, subnormal and large scales; no NaN (it would reach every row) and no infinity."""
    N, K = 72, 416
    W = synth.random_codes(fmt, 1, N, K, seed=M, device="cpu")
    rng = np.random.default_rng(M)
    if fmt == synth.FMT_MXFP4:
        b = rng.integers(100, 150, W.scale.shape)
        b[:, ::5], b[:, 1::7], b[:, 2::9] = rng.integers(0, 4), 251, rng.integers(128, 132)
        W.scale = torch.from_numpy(b.astype(np.uint8))
    else:
        c = rng.integers(0, 256, W.scale.shape).astype(np.uint8)
        c[(c & 0x7F) == 0x7F] ^= 1
        W.scale, W.tensor_scale = torch.from_numpy(c), torch.tensor([3.3e3 if M == 16 else 1e-3 if M == 5 else 2.0 ** -135])
    want = bf16_vals(bsq.dequant(W.to("cuda")))[0]
    assert np.array_equal(want, oracle_deq(W)[0]) and np.isfinite(want).all()
    for k0 in range(0, K, M):
        n = min(M, K - k0)
        X = torch.zeros((M, K), dtype=BF16)
        X[torch.arange(n), k0 + torch.arange(n)] = 1
        got = bf16_vals(bsq.fp4_forward(X.cuda(), W.to("cuda")))
        assert np.array_equal(got[:n], want[:, k0:k0 + n].T) and not got[n:].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_scales_stay_in_their_rows(fmt):
    N, K = 48, 256
    W = synth.make_packed(fmt, 1, N, K, 0.5, seed=1, device="cpu")
    W.scale[0, 5, 2] = 255 if fmt == synth.FMT_MXFP4 else 0x7F
    X = activations(3, K, 2)
    got = bf16_vals(bsq.fp4_forward(X.cuda(), W.to("cuda")))
    assert np.isnan(got[:, 5]).all() and np.isfinite(np.delete(got, 5, axis=1)).all()
    X[1, 7] = float("inf")
    got = bf16_vals(bsq.fp4_forward(X.cuda(), W.to("cuda")))
    assert not np.isfinite(got[1]).any() and np.isfinite(np.delete(got[[0, 2]], 5, axis=1)).all()


@pytest.mark.parametrize("ts", [2.0 ** -7, -(2.0 ** -7), 2.0 ** -7 * (1 + 2.0 ** -23), 2.0 ** -110, 2.0 ** -110 * (1 - 2.0 ** -24), 0.0, -3e-5, 2.0 ** 116])
@pytest.mark.parametrize("K", [512, 288])
def test_tensor_scales_at_which_the_decoding_changes(ts, K):
    """Every code under every block scale, bit for bit, on both sides of each limit."""
    N = 72
    W = synth.random_codes(synth.FMT_NVFP4, 1, N, K, seed=K, device="cpu")
    c = torch.arange(W.scale.numel(), dtype=torch.int64) * 7 % 256
    c[(c & 0x7F) == 0x7F] = 1
    W.scale, W.tensor_scale = c.to(torch.uint8).view(W.scale.shape), torch.tensor([ts], dtype=torch.float32)
    want = oracle_deq(W)[0]
    assert np.array_equal(bf16_vals(bsq.dequant(W.to("cuda")))[0], want) and np.isfinite(want).all()
    for k0 in range(0, K, 32):
        X = torch.zeros((32, K), dtype=BF16)
        X[torch.arange(32), k0 + torch.arange(32)] = 1
        assert np.array_equal(bf16_vals(bsq.fp4_forward(X.cuda(), W.to("cuda"))), want[:, k0:k0 + 32].T)


@pytest.mark.parametrize("byte", [0, 1, 2, 126, 127, 128, 129, 200, 251])
@pytest.mark.parametrize("K", [512, 288])
def test_block_scales_at_which_the_decoding_changes(byte, K):
    N = 72
    W = synth.random_codes(synth.FMT_MXFP4, 1, N, K, seed=K, device="cpu")
    b = torch.full(W.scale.shape, 120, dtype=torch.uint8)
    b.view(-1)[::5] = byte
    W.scale = b
    want = oracle_deq(W)[0]
    assert np.isfinite(want).all()
    for k0 in range(0, K, 32):
        X = torch.zeros((32, K), dtype=BF16)
        X[torch.arange(32), k0 + torch.arange(32)] = 1
        assert np.array_equal(bf16_vals(bsq.fp4_forward(X.cuda(), W.to("cuda"))), want[:, k0:k0 + 32].T)


@pytest.mark.parametrize("fmt,shift", [(synth.FMT_MXFP4, 1), (synth.FMT_MXFP4, 2), (synth.FMT_MXFP4, 8), (synth.FMT_NVFP4, 2), (synth.FMT_NVFP4, 8)])
@pytest.mark.parametrize("K", [512, 288])
def test_scales_of_any_alignment(fmt, shift, K):
    W, X = synth.make_packed(fmt, 1, 72, K, 0.5, seed=K, device="cpu").to("cuda"), activations(9, K, 3).cuda()
    want = bsq.fp4_forward(X, W)
    buffer = torch.zeros(W.scale.numel() + 32, dtype=torch.uint8, device="cuda")
    moved = buffer[shift:shift + W.scale.numel()].view(W.scale.shape)
    moved.copy_(W.scale.view(torch.uint8))
    W.scale = moved
    assert moved.data_ptr() % 16 == shift and torch.equal(bsq.fp4_forward(X, W), want)
    offsets = torch.tensor([9], dtype=torch.int32, device="cuda")
    assert torch.equal(bsq.fp4_grouped_forward(X, W, offsets), bsq.fp4_grouped_forward(X, W.__class__(fmt, W.data, moved.clone(), W.tensor_scale, 1, 72, K), offsets))


@pytest.mark.parametrize("M", [1, 16, 40])
@pytest.mark.parametrize("K", [32, 96, 256, 288, 2080])
def test_infinite_tensor_scale(M, K):
    """Positive codes, scales and tokens: every sum is infinite, whatever lies behind the last column."""
    W = synth.make_packed(synth.FMT_NVFP4, 1, 72, K, 0.5, seed=K, device="cpu")
    W.data = (W.data & 0x77) | 0x11
    W.scale = torch.full_like(W.scale.view(torch.uint8), 0x38)
    W.tensor_scale = torch.tensor([float("inf")])
    out = bsq.fp4_forward(torch.ones((M, K), dtype=BF16).cuda(), W.to("cuda"))
    assert (out.float() == float("inf")).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K,counts", [(64, 64, [1]), (72, 160, [0, 3, 0, 1]), (136, 1056, [8, 0, 9, 1, 17, 0, 0, 5]), (40, 2048, [0, 0, 64]),
                                        (264, 512, [33, 100, 0, 7]), (48, 96, [1] * 40), (512, 3104, [2, 1, 0, 1, 4, 1]), (64, 256, [0, 0, 0])])
def test_grouped(fmt, N, K, counts):
    E, used = len(counts), sum(counts)
    S = used + 3
    W = synth.make_packed(fmt, E, N, K, 0.5, seed=N, device="cpu")
    X = activations(S, K, K)
    X[used:] = float("nan")                     # rows behind the last expert: never read, never written
    offs = synth.offsets_from_counts(counts)
    out = torch.full((S, N), 7.0, dtype=BF16, device="cuda")
    bsq.fp4_grouped_forward(X.cuda(), W.to("cuda"), torch.from_numpy(offs).cuda(), out=out)
    got, x, w, r0 = bf16_vals(out), bf16_vals(X), oracle_deq(W), 0
    assert (got[used:] == 7).all()
    for e, c in enumerate(counts):
        if c:
            close(got[r0:r0 + c], x[r0:r0 + c] @ w[e].T, x[r0:r0 + c], w[e], f"expert {e}")
        r0 += c
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("offs", [[3, 2, 5], [-1, 2, 5], [1, 2, 9]])
def test_bad_offsets_are_reported_and_nothing_is_written(offs):
    W = synth.make_packed(synth.FMT_MXFP4, 3, 64, 128, 0.5, seed=1, device="cuda")
    out = torch.full((8, 64), 7.0, dtype=BF16, device="cuda")
    bsq.fp4_grouped_forward(activations(8, 128, 1).cuda(), W, torch.tensor(offs, dtype=torch.int32, device="cuda"), out=out)
    st, code = bsq.get_device_error()
    assert st == bsq.BSQ_ERR_INVALID_ARG and code == 2 and (out == 7).all()
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


def test_results_repeat_and_do_not_depend_on_the_other_rows():
    """A row's sum has one order: the same bits again, and beside other rows of the same pass."""
    W = synth.make_packed(synth.FMT_NVFP4, 1, 4096, 4096, 0.5, seed=2, device="cuda")
    X = activations(8, 4096, 3).cuda()
    a = bsq.fp4_forward(X, W)
    assert all(torch.equal(a, bsq.fp4_forward(X, W)) for _ in range(10))
    assert torch.equal(a[2:3], bsq.fp4_forward(X[2:3].contiguous(), W))


def test_far_experts():
    """Weights beyond 2^31 bytes."""
    E, N, K = 300, 2048, 7168
    one = synth.make_packed(synth.FMT_MXFP4, 1, N, K, 0.5, seed=3, device="cuda")
    data = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((E, N, K // 32), dtype=torch.uint8, device="cuda")
    data[-1], scale[-1] = one.data[0], one.scale[0]
    W = synth.Packed(synth.FMT_MXFP4, data, scale, None, E, N, K)
    X = activations(2, K, 4).cuda()
    offs = torch.ones(E, dtype=torch.int32, device="cuda")
    offs[-1] = 2
    out = bsq.fp4_grouped_forward(X, W, offs)
    assert not out[0].any() and torch.equal(out[1:], bsq.fp4_forward(X[1:].contiguous(), one))


def test_empty():
    W = synth.make_packed(synth.FMT_MXFP4, 1, 64, 128, 0.5, seed=1, device="cuda")
    assert bsq.fp4_forward(torch.zeros((0, 128), dtype=BF16, device="cuda"), W).shape == (0, 64)
    Z = synth.Packed(synth.FMT_MXFP4, W.data[:, :, :0].contiguous(), W.scale[:, :, :0].contiguous(), None, 1, 64, 0)
    assert not bsq.fp4_forward(torch.zeros((3, 0), dtype=BF16, device="cuda"), Z).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,at", [(40, {0: 1, 31: 2, 32: 1, 39: 3}), (1024, {1023: 1}), (1024, {5: 9, 700: 1, 701: 1}), (300, {})])
def test_few_rows_on_many_experts(fmt, E, at):
    """Fewer rows than experts: only those that have any take part."""
    N, K, used = 72, 288, sum(at.values())
    W = synth.make_packed(fmt, E, N, K, 0.5, seed=E, device="cuda")
    X = activations(max(used, 2), K, 3)
    offs = synth.offsets_from_counts([at.get(e, 0) for e in range(E)])
    out = torch.full((len(X), N), 7.0, dtype=BF16, device="cuda")
    bsq.fp4_grouped_forward(X.cuda(), W, torch.from_numpy(offs).cuda(), out=out)
    got, x, r0 = bf16_vals(out), bf16_vals(X), 0
    assert (got[used:] == 7).all()
    for e, c in at.items():
        one = synth.Packed(fmt, W.data[e:e + 1].cpu(), W.scale[e:e + 1].cpu(), None if W.tensor_scale is None else W.tensor_scale[e:e + 1].cpu(), 1, N, K)
        w = oracle_deq(one)[0]
        close(got[r0:r0 + c], x[r0:r0 + c] @ w.T, x[r0:r0 + c], w, f"expert {e}")
        r0 += c


@pytest.mark.parametrize("offs", [[0, 1, 0, 1, 2], [0, 0, -1, 0, 0], [0, 0, 0, 0, 3], [5, 5, 5, 5, 5]])
def test_bad_offsets_of_many_experts(offs):
    W = synth.make_packed(synth.FMT_NVFP4, 5, 64, 256, 0.5, seed=1, device="cuda")
    out = torch.full((2, 64), 7.0, dtype=BF16, device="cuda")
    bsq.fp4_grouped_forward(activations(2, 256, 1).cuda(), W, torch.tensor(offs, dtype=torch.int32, device="cuda"), out=out)
    assert bsq.get_device_error() == (bsq.BSQ_ERR_INVALID_ARG, 2) and (out == 7).all()
