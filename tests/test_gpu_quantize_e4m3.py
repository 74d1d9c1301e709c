"""bsq_quantize_e4m3 against its definition: a = max |x| of a block, scale = a / 448, code =
E4M3(x * (448 / a)), each step rounded to float32.  numpy's float32 division and product are
IEEE, so scales and codes are compared bit for bit; against x / scale in 64 bits the codes
are the nearest E4M3 values up to the two float32 roundings of x * (448 / a), 2^-23 of it."""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu


def reference(x, block_rows):
    """(codes, scale) of float32 x [b, r, c]."""
    b, r, c = x.shape
    rb, cb = -(-r // block_rows), -(-c // 128)
    pad = np.zeros((b, rb * block_rows, cb * 128), np.float32)
    pad[:, :r, :c] = x
    t = pad.reshape(b, rb, block_rows, cb, 128)
    a = np.abs(t).max(axis=(2, 4))
    a = np.where(a == 0, np.float32(448), np.maximum(a, np.float32(2.0 ** -100))).astype(np.float32)
    scale = a / np.float32(448)
    with np.errstate(invalid="ignore"):
        q = t * (np.float32(448) / a)[:, :, None, :, None]
    q = np.clip(q, np.float32(-448), np.float32(448)).reshape(b, rb * block_rows, cb * 128)[:, :r, :c]
    codes = torch.from_numpy(np.ascontiguousarray(q)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, scale


def draw(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=g))
    return x.to(dtype)


def same(codes, ref):
    codes, nan = codes.cpu().numpy(), (ref & 0x7F) == 0x7F
    np.testing.assert_array_equal((codes & 0x7F) == 0x7F, nan)
    np.testing.assert_array_equal(codes[~nan], ref[~nan])


SHAPES = [(1, 1, 16), (1, 1, 128), (2, 3, 144), (1, 127, 1040), (3, 130, 272), (1, 300, 4096), (2, 129, 1008)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_bit_exact(shape, block_rows, dtype):
    x = draw(shape, 1, dtype)
    x[0, 0, :16] = 0
    codes, scale = bsq.quantize_e4m3(x.cuda(), block_rows)
    rc, rs = reference(x.float().numpy(), block_rows)
    np.testing.assert_array_equal(scale.cpu().numpy(), rs)
    same(codes, rc)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_nearest_in_64_bits(block_rows):
    x = draw((1, 256, 512), 2, torch.float32)
    codes, scale = bsq.quantize_e4m3(x.cuda(), block_rows)
    v = codes.view(torch.float8_e4m3fn).double().cpu()
    s = scale.double().cpu().repeat_interleave(block_rows, 1).repeat_interleave(128, 2)
    q = x.double() / s
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    assert ((v - q).abs() <= 0.5 * step + 2.0 ** -22 * q.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_special_blocks(block_rows, dtype):
    """Zero blocks (scale 1), tiny ones (the floor of 2^-100), subnormals, -0, infinities, NaN; each in
    a block of its own, the neighbours untouched."""
    x = draw((1, 256, 128 * 8), 3, dtype)
    x[0, :128, :128] = 0
    x[0, :128, 128:256] *= 1e-38
    x[0, :128, 256:384] = -0.0
    x[0, 5, 400] = float("inf")
    x[0, 6, 530] = float("nan")
    x[0, 7, 650] = -float("inf")
    x[0, :128, 768:896] = 3.0e38 * torch.sign(x[0, :128, 768:896])
    codes, scale = bsq.quantize_e4m3(x.cuda(), block_rows)
    rc, rs = reference(x.float().numpy(), block_rows)
    np.testing.assert_array_equal(scale.cpu().numpy(), rs)
    same(codes, rc)
    assert scale[0, 0, 0] == 1 and (codes[0, :128, :128] == 0).all()


def test_two_dimensions_given_outputs_and_stream():
    x = draw((1, 64, 256), 4, torch.bfloat16)[0].cuda()
    codes, scale = torch.empty((64, 256), dtype=torch.uint8, device="cuda"), torch.empty((64, 2), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bsq.quantize_e4m3(x, 1, codes=codes, scale=scale, stream=side)
    torch.cuda.synchronize()
    rc, rs = reference(x.float().cpu().numpy()[None], 1)
    same(codes, rc[0])
    np.testing.assert_array_equal(scale.cpu().numpy(), rs[0])


def test_refusals():
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: bsq.quantize_e4m3(x.half()), lambda: bsq.quantize_e4m3(x.t()), lambda: bsq.quantize_e4m3(x.cpu()),
                lambda: bsq.quantize_e4m3(x[0]), lambda: bsq.quantize_e4m3(x, codes=torch.empty((4, 128), dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bsq.BsqError):
        bsq.quantize_e4m3(x[:, :24].contiguous())       # columns not a multiple of 16
    with pytest.raises(bsq.BsqError):
        bsq.quantize_e4m3(x, block_rows=64)
    assert bsq.quantize_e4m3(x[:0])[0].shape == (0, 256)
