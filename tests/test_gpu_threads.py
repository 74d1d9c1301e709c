"""Calls from several host threads at once whose launches of one kernel differ in their shared memory: none is refused, and each gets
what it gets alone.

The threads call the C entry points with arguments that are made before, on streams of their own: the interpreter's lock is held so
shortly between two calls that the calls meet.
"""

import ctypes
import sys
import threading

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth

pytestmark = pytest.mark.gpu

THREADS, CALLS = 8, 3000
BF16, I32 = torch.bfloat16, torch.int32


def ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def at_once(calls):
    """calls: (entry point, arguments) of each thread, CALLS times each; what the refused ones said."""
    refused, start = [], threading.Barrier(len(calls))

    def loop(entry, args):
        start.wait()
        for i in range(CALLS):
            if entry(*args):
                refused.append((i, bsq.lib().bsq_last_error()))
                return

    threads = [threading.Thread(target=loop, args=c) for c in calls]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert refused == []
    torch.cuda.synchronize()
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("fmt", [synth.FMT_MXFP4, synth.FMT_NVFP4])
@pytest.mark.parametrize("E,rows,Ks", [(2, 4, (7168, 5120)), (0, 1, (4096, 512)), (0, 16, (4096, 512)), (3, 40, (2048, 1024))])
def test_products_of_two_lengths(fmt, E, rows, Ks):
    calls, results, held = [], [], []
    for i in range(THREADS):
        K, side = Ks[i % 2], torch.cuda.Stream()
        w = synth.make_packed(fmt, max(E, 1), 72, K, 0.5, seed=K, device="cuda")
        x = synth.randn((rows, K), 1.0, K, "cuda", BF16)
        out = torch.zeros((rows, 72), dtype=BF16, device="cuda")
        held.append((w, x, side))
        packed = (fmt, ptr(w.data), ptr(w.scale), ptr(w.tensor_scale))
        if E:
            offsets = (torch.arange(1, E + 1, device="cuda") * rows // E).to(I32)
            held.append(offsets)
            results.append((out, bsq.fp4_grouped_forward(x, w, offsets)))
            calls.append((bsq.lib().bsq_fp4_grouped_forward, (ptr(x), rows, *packed, E, 72, K, ptr(offsets), ptr(out), ctypes.c_void_p(side.cuda_stream))))
        else:
            results.append((out, bsq.fp4_forward(x, w)))
            calls.append((bsq.lib().bsq_fp4_forward, (ptr(x), rows, *packed, 72, K, ptr(out), ctypes.c_void_p(side.cuda_stream))))
    torch.cuda.synchronize()
    at_once(calls)
    assert all(torch.equal(got, want) for got, want in results)


@pytest.mark.parametrize("T", [64, 512, 3000])
def test_sorts_for_two_numbers_of_experts(T):
    """One CTA, a cluster of eight and one of sixteen."""
    calls, results, held = [], [], []
    for i in range(THREADS):
        E, side = (1024, 400)[i % 2], torch.cuda.Stream()
        ids = torch.randint(0, E, (T, 8), generator=torch.Generator().manual_seed(i)).to(I32).cuda()
        got = [torch.zeros(n, dtype=I32, device="cuda") for n in (E, 8 * T, 8 * T)]
        held.append((ids, side))
        results.append((got, bsq.sort_experts(ids, E)))
        calls.append((bsq.lib().bsq_sort_experts, (ptr(ids), T, 8, E, *map(ptr, got), ctypes.c_void_p(side.cuda_stream))))
    torch.cuda.synchronize()
    at_once(calls)
    assert all(torch.equal(a, b.view(-1)) for got, want in results for a, b in zip(got, want))
