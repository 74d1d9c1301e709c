"""Grouped products refuse sizes whose last tile or block would end past 2^31: rows of an expert's last
tile are counted in 32 bits.  Calls that end in the checks, with addresses that nothing reads."""

import os

import pytest

from block_scaled_gemm_fp8_gb300 import bsq

FAKE, TOP = 0x10000, 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bsq.LIB_PATH):
        from block_scaled_gemm_fp8_gb300 import build
        build.build()
    return bsq.lib()


@pytest.mark.parametrize("name", ["bsq_fp8_grouped_forward", "bsq_fp8_grouped_dgrad"])
def test_grouped(L, name):
    # y is null: a call whose sizes are taken is refused for that, before a GPU is looked for
    def call(S=64, N=128):
        return getattr(L, name)(FAKE, FAKE, S, 1, FAKE, FAKE, 3, N, 256, FAKE, None, None)
    for S in (TOP - 126, TOP - 50, TOP):
        assert call(S=S) == bsq.BSQ_ERR_UNSUPPORTED and "2^31-128" in bsq.last_error(), S
    assert call(N=TOP - 119) == bsq.BSQ_ERR_UNSUPPORTED and "2^31-128" in bsq.last_error()   # a multiple of 8
    assert call(S=TOP - 127) == bsq.BSQ_ERR_INVALID_ARG and "null" in bsq.last_error()
    assert call(N=TOP - 127) == bsq.BSQ_ERR_INVALID_ARG and "null" in bsq.last_error()
