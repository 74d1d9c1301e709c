"""Failure detection of the FP8 product kernel when the wait runs out at the end of a CTA's work:
with BSQ_TEST_DROP_ANNOUNCE=2 its producer requests every k-block but the last and ends, so that
the MMA warp's wait runs out after the producer has left, with the promotion warps in the middle
of a tile.  Every role leaves, the copies that were requested have landed, the call records
BSQ_DEVERR_TIMEOUT, and the next call is right.  A child process, as in test_gpu_fp8_timeout.py."""

import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = textwrap.dedent("""
    import os, sys
    sys.path.insert(0, {root!r})
    import torch
    from block_scaled_gemm_fp8_gb300 import bsq, synth

    def operands(M, N, K, E):
        x = synth.randn((M, K), 1.0, 1, "cuda", torch.bfloat16)
        c, s = bsq.quantize_e4m3(synth.randn((E, N, K), 0.5, 2, "cuda"), 128)
        return (*bsq.quantize_e4m3(x), synth.Packed(synth.FMT_FP8, c, s, None, E, N, K))

    one = operands(3000, 2048, 640, 1)      # 192 tiles of 5 k-blocks: one CTA each, some take a second
    single = operands(300, 256, 128, 1)     # one k-block: nothing is ever requested
    split = operands(100, 512, 2048, 1)     # 2 tiles: clusters of 4, four k-blocks a CTA
    many = operands(700, 512, 640, 3)
    offs = torch.tensor([100, 100, 700], dtype=torch.int32, device="cuda")
    calls = {{
        "one": lambda: bsq.fp8_forward(*one),
        "single": lambda: bsq.fp8_forward(*single),
        "split": lambda: bsq.fp8_forward(*split),
        "grouped": lambda: bsq.fp8_grouped_forward(*many, offs),
    }}
    for name, call in calls.items():
        want = call()
        torch.cuda.synchronize()
        os.environ["BSQ_WAIT_LIMIT_MS"] = "50"
        os.environ["BSQ_TEST_DROP_ANNOUNCE"] = "2"
        call()
        st, code = bsq.get_device_error()
        assert st == bsq.BSQ_ERR_TIMEOUT and code == 1, (name, st, code)
        del os.environ["BSQ_WAIT_LIMIT_MS"], os.environ["BSQ_TEST_DROP_ANNOUNCE"]
        got = call()
        assert bsq.get_device_error() == (bsq.BSQ_OK, 0)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), name
        print("ok", name)
""")


def test_wait_runs_out_after_the_producer_has_ended():
    env = {k: v for k, v in os.environ.items() if not k.startswith("BSQ_")}
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("ok ") == 4, r.stdout
