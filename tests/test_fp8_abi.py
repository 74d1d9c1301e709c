"""Host-side validation of the FP8 operators and AdamW on the CPU: bad arguments are refused before
a GPU is touched, empty problems return without one."""

import ctypes
import os

import pytest

from block_scaled_gemm_fp8_gb300 import bsq

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced by host validation
INVALID, UNSUPPORTED, OK = bsq.BSQ_ERR_INVALID_ARG, bsq.BSQ_ERR_UNSUPPORTED, bsq.BSQ_OK


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bsq.LIB_PATH):
        from block_scaled_gemm_fp8_gb300 import build
        build.build()
    return bsq.lib()


def test_binding_has_every_new_entry_point(L):
    for n in ("bsq_quantize_e4m3", "bsq_fp8_forward", "bsq_fp8_dgrad", "bsq_fp8_grouped_forward", "bsq_fp8_grouped_dgrad", "bsq_adamw"):
        assert hasattr(L, n) and n in bsq.SIGNATURES
        assert n + "(" in open(bsq.HEADER_PATH).read()


def test_quantize(L):
    def q(dtype=0, x=FAKE, batch=1, rows=4, cols=256, block=1, codes=FAKE, scale=FAKE):
        return L.bsq_quantize_e4m3(dtype, x, batch, rows, cols, block, codes, scale, None)
    assert q(dtype=2) == INVALID and q(rows=-1) == INVALID and q(block=64) == INVALID
    assert q(cols=24) == UNSUPPORTED and q(rows=1 << 31) == UNSUPPORTED
    assert q(x=None) == INVALID and q(x=FAKE + 8) == INVALID
    assert q(codes=None) == INVALID and q(codes=FAKE + 8) == INVALID
    assert q(scale=None) == INVALID and q(scale=FAKE + 2) == INVALID
    assert q(rows=0, x=None, codes=None, scale=None) == OK and q(batch=0) == OK
    assert "bsq_quantize_e4m3" in (q(block=2), bsq.last_error())[1]


@pytest.mark.parametrize("name", ["bsq_fp8_forward", "bsq_fp8_dgrad"])
@pytest.mark.parametrize("grouped", [False, True])
def test_products(L, name, grouped):
    dgrad = name.endswith("dgrad")

    def call(x=FAKE, xs=FAKE, M=64, fmt=1, w=FAKE, ws=FAKE, N=128, K=256, y=FAKE, E=3, offs=FAKE):
        if grouped:
            return getattr(L, name.replace("fp8_", "fp8_grouped_"))(x, xs, M, fmt, w, ws, E, N, K, offs, y, None)
        return getattr(L, name)(x, xs, M, fmt, w, ws, N, K, y, None)
    assert call(M=-1) == INVALID and call(N=-8) == INVALID and call(M=1 << 31) == UNSUPPORTED
    assert call(fmt=9) == INVALID and call(fmt=-1) == INVALID
    for fmt in (0, 2, 3, 4, 5):
        assert call(fmt=fmt) == UNSUPPORTED
    assert call(x=None) == INVALID and call(x=FAKE + 8) == INVALID
    assert call(xs=None) == INVALID and call(xs=FAKE + 2) == INVALID
    assert call(w=None) == INVALID and call(w=FAKE + 4) == INVALID and call(ws=None) == INVALID
    assert call(y=None) == INVALID and call(y=FAKE + 8) == INVALID
    assert call(K=264) == UNSUPPORTED                       # W's row pitch
    assert call(N=132) == UNSUPPORTED
    assert call(N=136) == UNSUPPORTED if dgrad else True    # the gradient codes' row pitch
    assert call(M=0, x=None, xs=None, y=None) == OK
    if grouped:
        assert call(E=0) == INVALID and call(E=1025) == UNSUPPORTED and call(offs=None) == INVALID
        assert call(offs=FAKE + 2) == INVALID
        assert call(**({"N": 0} if dgrad else {"K": 0}), x=None) == UNSUPPORTED
    assert call(**({"K": 0} if dgrad else {"N": 0}), y=None, w=None, ws=None) == OK


def test_adamw(L):
    def step(count=1, gd=0, bits=32, step=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, gs=None, tensors=True, **t):
        d = dict(param=FAKE, grad=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, copy=None, n=100, weight_decay=0.0, counter=0)
        items = (bsq._AdamwTensor * 1)(bsq._AdamwTensor(*{**d, **t}.values()))
        return L.bsq_adamw(ctypes.addressof(items) if tensors else None, count, gd, bits, step, lr, b1, b2, eps, gs, 0, None)
    assert step(count=-1) == INVALID and step(tensors=False) == INVALID
    assert step(count=0, tensors=False) == OK and step(n=0, param=None) == OK
    assert step(gd=2) == INVALID and step(bits=16) == INVALID and step(step=0) == INVALID
    assert step(b1=1.0) == INVALID and step(b2=-0.1) == INVALID and step(b1=float("nan")) == INVALID
    assert step(lr=float("inf")) == INVALID and step(eps=-1e-8) == INVALID and step(gs=FAKE + 1) == INVALID
    assert step(n=-1) == INVALID and step(n=(1 << 40) + 1) == UNSUPPORTED
    for name in ("param", "grad", "m", "v"):
        assert step(**{name: None}) == INVALID
    assert step(param=FAKE + 2) == INVALID and step(grad=FAKE + 1) == INVALID and step(gd=1, grad=FAKE + 2) == INVALID
    assert step(m=FAKE + 1) == INVALID and step(copy=FAKE + 1) == INVALID and step(weight_decay=float("nan")) == INVALID
    assert step(bits=8, m_scale=None) == INVALID and step(bits=8, v_scale=FAKE + 2) == INVALID
    assert "bsq_adamw" in bsq.last_error()


def test_struct_layout_matches_the_header():
    """Seven pointers, a length, a float and a counter: 72 bytes on every 64-bit ABI."""
    assert ctypes.sizeof(bsq._AdamwTensor) == 72 and bsq._AdamwTensor.n.offset == 56 and bsq._AdamwTensor.counter.offset == 68
