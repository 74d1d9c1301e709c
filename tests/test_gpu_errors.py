"""A CUDA error that a call has reported does not also meet the caller's next CUDA call."""

import ctypes

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu


def test_a_reported_error_is_not_left_behind():
    """Reading the error word waits for its stream, which a stream that is being captured refuses."""
    torch.zeros(1, device="cuda")
    lib, runtime = bsq.lib(), ctypes.CDLL("libcudart.so.13")       # the runtime that the library and torch share
    side, code, graph = torch.cuda.Stream(), ctypes.c_int32(), ctypes.c_void_p()
    handle = ctypes.c_void_p(side.cuda_stream)
    torch.cuda.synchronize()
    assert runtime.cudaPeekAtLastError() == 0
    assert runtime.cudaStreamBeginCapture(handle, 2) == 0          # relaxed: other streams are not concerned
    status, left = lib.bsq_get_device_error(ctypes.byref(code), handle), runtime.cudaPeekAtLastError()
    runtime.cudaStreamEndCapture(handle, ctypes.byref(graph))      # the capture has become invalid
    runtime.cudaGetLastError()
    assert status == bsq.BSQ_ERR_CUDA and bsq.last_error()
    assert left == 0
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)
