"""bsq_adamw's 8-bit states in blocks whose scales are infinite or NaN, of both states or of one alone.

The codes are compared with the float32 formula over whole blocks (the tensor operations of
test_gpu_adamw.py, each rounded by itself): equal where the formula gives a number, and the NaN
code where it gives NaN, whichever element of the block it is.  Conversion keeps NaN as NaN and
no other operation is in question, so the comparison is exact."""

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq
from tests.test_gpu_adamw import B, BETAS, EPS, LR, in_float32, make, table

pytestmark = pytest.mark.gpu

N = 8 * B + 40


def draw():
    t = make(N, torch.float32, 8, 120)
    g = t["g"]
    g[:B] = 1e25 * torch.sign(g[:B])             # g^2 is infinite in every element, m is not
    g[B:2 * B] = 1e20                            # the same, with every m on one side
    g[2 * B + 5] = 3e19                          # g^2 infinite in one element
    t["ms"][3] = float("nan")                    # m alone
    t["vs"][4] = float("nan")                    # sqrt(v) alone
    t["ms"][5] = float("inf")
    t["vs"][6] = float("inf")
    g[7 * B + 100] = float("nan")
    g[8 * B:] = 1e25                             # the part block at the end
    return t


@pytest.mark.parametrize("offset", [0, 1])
def test_codes_follow_the_formula(offset):
    t = draw()
    if offset:   # the same values in buffers without alignment
        for k in ("p", "g", "m", "v", "copy"):
            t[k] = torch.empty(N + 1, dtype=t[k].dtype, device="cuda")[1:].copy_(t[k])
    m, ms, v, vs = in_float32(t, 5, 1.0, 11)
    bsq.adamw(table([t]), 5, LR, BETAS, EPS, seed=11)
    for name, codes, scale, want, wanted in (("m", t["m"], t["ms"], m, ms), ("v", t["v"], t["vs"], v, vs)):
        got = codes.view(torch.float8_e4m3fn).float()
        assert torch.equal(torch.isnan(scale), torch.isnan(wanted)), name
        assert torch.equal(torch.nan_to_num(scale), torch.nan_to_num(wanted)), name
        wrong = torch.nonzero(torch.isnan(got) != torch.isnan(want)).flatten().tolist()
        assert not wrong, (name, wrong)
        ok = ~torch.isnan(want)
        assert torch.equal(got[ok] + 0.0, want[ok] + 0.0), name
