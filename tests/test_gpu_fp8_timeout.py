"""Failure detection of the FP8 product kernel without a GPU fault: with BSQ_TEST_DROP_ANNOUNCE=1 its
producer never requests an operand, so the MMA warp's wait runs out after 50 ms; every role
leaves, the call records BSQ_DEVERR_TIMEOUT, and the next call is right.  Covers a tile per
CTA, tiles split over a cluster, and the grouped form, in a child process whose environment
touches no other test."""

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

    one = operands(3000, 2048, 512, 1)      # 192 tiles: one CTA each, some take a second
    split = operands(100, 512, 2048, 1)     # 2 tiles: clusters of 4
    many = operands(700, 512, 640, 3)
    offs = torch.tensor([100, 100, 700], dtype=torch.int32, device="cuda")
    calls = {{
        "one": lambda: bsq.fp8_forward(*one),
        "split": lambda: bsq.fp8_forward(*split),
        "grouped": lambda: bsq.fp8_grouped_forward(*many, offs),
    }}
    for name, call in calls.items():
        want = call()
        torch.cuda.synchronize()
        os.environ["BSQ_WAIT_LIMIT_MS"] = "50"
        os.environ["BSQ_TEST_DROP_ANNOUNCE"] = "1"
        call()
        st, code = bsq.get_device_error()
        assert st == bsq.BSQ_ERR_TIMEOUT and code == 1, (name, st, code)
        del os.environ["BSQ_WAIT_LIMIT_MS"], os.environ["BSQ_TEST_DROP_ANNOUNCE"]
        got = call()
        assert bsq.get_device_error() == (bsq.BSQ_OK, 0)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), name
        print("ok", name)
""")


def test_wait_runs_out_then_next_call_is_correct():
    env = {k: v for k, v in os.environ.items() if not k.startswith("BSQ_")}
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("ok ") == 3, r.stdout
