"""Host-side validation of the router, the operators between tokens and rows and the 4-bit products on the
CPU: bad arguments are refused before a GPU is touched, empty problems return without one."""

import os

import pytest

from block_scaled_gemm_fp8_gb300 import bsq

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced by host validation
INVALID, UNSUPPORTED, OK = bsq.BSQ_ERR_INVALID_ARG, bsq.BSQ_ERR_UNSUPPORTED, bsq.BSQ_OK
NAMES = ("bsq_route", "bsq_route_backward", "bsq_sort_experts", "bsq_dispatch", "bsq_combine", "bsq_combine_backward",
         "bsq_fp4_forward", "bsq_fp4_grouped_forward")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bsq.LIB_PATH):
        from block_scaled_gemm_fp8_gb300 import build
        build.build()
    return bsq.lib()


def test_binding_has_every_new_entry_point(L):
    header = open(bsq.HEADER_PATH).read()
    for n in NAMES:
        assert hasattr(L, n) and n in bsq.SIGNATURES and n + "(" in header


def test_route(L):
    def call(dtype=0, x=FAKE, T=4, E=8, k=2, gate=0, renorm=1, bias=None, factor=1.0, ids=FAKE, w=FAKE):
        return L.bsq_route(dtype, x, T, E, k, gate, renorm, bias, factor, ids, w, None)
    assert call(dtype=2) == INVALID and call(gate=2) == INVALID and call(gate=-1) == INVALID and call(T=-1) == INVALID
    assert call(k=0) == INVALID and call(k=9) == INVALID and call(E=0) == INVALID
    assert call(E=1025) == UNSUPPORTED and call(E=64, k=33) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED
    assert call(factor=float("nan")) == INVALID and call(factor=float("inf")) == INVALID
    assert call(x=None) == INVALID and call(x=FAKE + 1) == INVALID and call(dtype=1, x=FAKE + 2) == INVALID
    assert call(ids=None) == INVALID and call(w=None) == INVALID and call(ids=FAKE + 2) == INVALID and call(w=FAKE + 1) == INVALID
    assert call(bias=FAKE + 2) == INVALID
    assert "bsq_route" in bsq.last_error()
    assert call(T=0, x=None, ids=None, w=None) == OK


def test_route_backward(L):
    def call(dtype=0, x=FAKE, T=4, E=8, k=2, gate=0, ids=FAKE, gw=FAKE, out=FAKE):
        return L.bsq_route_backward(dtype, x, T, E, k, gate, 1, 1.0, ids, gw, out, None)
    assert call(dtype=2) == INVALID and call(gate=7) == INVALID and call(k=9) == INVALID and call(E=1025) == UNSUPPORTED
    assert call(ids=None) == INVALID and call(gw=None) == INVALID and call(out=None) == INVALID
    assert call(gw=FAKE + 2) == INVALID and call(out=FAKE + 1) == INVALID and call(dtype=1, out=FAKE + 2) == INVALID
    assert call(T=0, x=None, ids=None, gw=None, out=None) == OK


def test_sort(L):
    def call(ids=FAKE, T=4, k=2, E=8, offs=FAKE, rows=FAKE, slots=None):
        return L.bsq_sort_experts(ids, T, k, E, offs, rows, slots, None)
    assert call(T=-1) == INVALID and call(k=0) == INVALID and call(E=0) == INVALID
    assert call(k=33) == UNSUPPORTED and call(E=1025) == UNSUPPORTED and call(T=1 << 30) == UNSUPPORTED
    assert call(ids=None) == INVALID and call(offs=None) == INVALID and call(rows=None) == INVALID
    for name in ("ids", "offs", "rows", "slots"):
        assert call(**{name: FAKE + 2}) == INVALID


def test_dispatch(L):
    def call(x=FAKE, T=4, K=256, rows=FAKE, k=2, w=None, S=8, out=FAKE, codes=FAKE, scale=FAKE):
        return L.bsq_dispatch(x, T, K, rows, k, w, S, out, codes, scale, None)
    assert call(T=-1) == INVALID and call(S=-1) == INVALID and call(K=-8) == INVALID and call(S=1 << 31) == UNSUPPORTED
    assert call(k=0) == INVALID and call(k=33) == UNSUPPORTED and call(K=252) == UNSUPPORTED
    assert call(K=264) == UNSUPPORTED and call(K=264, T=0, codes=None, scale=None) == OK   # codes want whole sixteens
    assert call(x=None) == INVALID and call(x=FAKE + 8) == INVALID and call(rows=None) == INVALID and call(rows=FAKE + 2) == INVALID
    assert call(w=FAKE + 2) == INVALID and call(out=FAKE + 8) == INVALID and call(codes=FAKE + 8) == INVALID
    assert call(codes=None) == INVALID and call(scale=None) == INVALID and call(scale=FAKE + 2) == INVALID
    assert call(out=None, codes=None, scale=None) == INVALID
    assert call(T=0, x=None, rows=None) == OK and call(K=0) == OK and call(S=0, out=None, codes=None, scale=None) == OK


def test_combine(L):
    def call(y=FAKE, S=8, N=256, rows=FAKE, k=2, w=None, T=4, out=FAKE):
        return L.bsq_combine(y, S, N, rows, k, w, T, out, None)
    assert call(T=-1) == INVALID and call(N=260) == UNSUPPORTED and call(k=33) == UNSUPPORTED and call(k=0) == INVALID
    assert call(y=None) == INVALID and call(y=FAKE + 8) == INVALID and call(out=None) == INVALID and call(out=FAKE + 8) == INVALID
    assert call(rows=None) == INVALID and call(w=FAKE + 1) == INVALID
    assert call(T=0, rows=None, out=None) == OK and call(N=0, y=None, out=None) == OK


def test_combine_backward(L):
    def call(g=FAKE, y=FAKE, S=8, N=256, rows=FAKE, k=2, w=None, T=4, gy=FAKE, codes=None, scale=None, gw=FAKE):
        return L.bsq_combine_backward(g, y, S, N, rows, k, w, T, gy, codes, scale, gw, None)
    assert call(T=-1) == INVALID and call(N=260) == UNSUPPORTED and call(N=264, codes=FAKE, scale=FAKE) == UNSUPPORTED
    assert call(g=None) == INVALID and call(g=FAKE + 8) == INVALID and call(y=None) == INVALID and call(y=FAKE + 8) == INVALID
    assert call(codes=FAKE) == INVALID and call(scale=FAKE) == INVALID and call(gy=FAKE + 8) == INVALID and call(gw=FAKE + 2) == INVALID
    assert call(y=None, gy=None, gw=None) == OK and call(T=0, g=None, y=None, rows=None) == OK
    assert call(N=0, g=None, y=None, gw=None) == OK


@pytest.mark.parametrize("grouped", [False, True])
def test_fp4(L, grouped):
    def call(x=FAKE, M=4, fmt=2, w=FAKE, ws=FAKE, ts=FAKE, N=128, K=256, y=FAKE, E=3, offs=FAKE):
        if grouped:
            return L.bsq_fp4_grouped_forward(x, M, fmt, w, ws, ts, E, N, K, offs, y, None)
        return L.bsq_fp4_forward(x, M, fmt, w, ws, ts, N, K, y, None)
    assert call(M=-1) == INVALID and call(N=-8) == INVALID and call(K=-32) == INVALID and call(fmt=9) == INVALID and call(fmt=-1) == INVALID
    assert call(M=(1 << 31) - 100) == UNSUPPORTED and call(N=(1 << 31) - 100) == UNSUPPORTED and call(K=(1 << 24) + 32) == UNSUPPORTED
    for fmt in (0, 1, 4, 5):
        assert call(fmt=fmt) == UNSUPPORTED
    assert call(fmt=3, K=48) == UNSUPPORTED and call(fmt=2, K=48) == INVALID and call(N=132) == UNSUPPORTED
    assert call(x=None) == INVALID and call(x=FAKE + 8) == INVALID and call(w=None) == INVALID and call(w=FAKE + 8) == INVALID
    assert call(ws=None) == INVALID and call(fmt=3, ts=None) == INVALID and call(fmt=3, ts=FAKE + 2) == INVALID and call(fmt=3, ws=FAKE + 1) == INVALID
    assert call(y=None) == INVALID and call(y=FAKE + 8) == INVALID
    assert call(M=0, ws=FAKE + 1) == OK and call(M=0, x=None, y=None) == OK and call(N=0, y=None, w=None, ws=None) == OK
    if not grouped:
        assert call(M=65, ws=FAKE + 8) == INVALID              # the tile kernel's alignment
    if grouped:
        assert call(E=0) == INVALID and call(E=1025) == UNSUPPORTED and call(offs=None) == INVALID and call(offs=FAKE + 2) == INVALID
        assert call(K=0, x=None) == UNSUPPORTED
