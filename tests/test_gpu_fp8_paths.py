"""E4M3 products on the paths that test_gpu_fp8.py's shapes do not reach: grouped calls whose tiles are
split over a cluster (12 k-blocks or more and few tiles), and dense calls of few rows with CTAs
enough for the small ones.  References, tolerances and helpers are that file's."""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth
from oracle import gemm as Gm
from tests.test_gpu_fp8 import check, draw_rows, draw_weight, packed, row_values, weight_values

pytestmark = pytest.mark.gpu

SPLIT = [[64, 0, 8, 15, 2, 33], [0, 0, 129, 1, 0, 127], [70], [0, 90, 0], [31, 33, 64, 128, 5, 0, 0, 6]]


@pytest.mark.parametrize("counts", SPLIT)
@pytest.mark.parametrize("inner,outer", [(2064, 272), (4112, 528), (1536, 16)])
@pytest.mark.parametrize("direction", ["forward", "dgrad"])
def test_grouped_over_a_cluster(direction, inner, outer, counts):
    """Uneven parts of the contraction, ragged experts and empty ones, clusters without a tile, and rows
    past the last offset, whose codes are NaN and whose outputs stay."""
    E, used, S = len(counts), sum(counts), sum(counts) + 5
    assert S > 64 and E <= S                                   # the tensor-core kernel
    assert (-(-S // 128) + E) * -(-outer // 256) * 2 <= bsq.num_sms() and -(-inner // 128) >= 12   # ... split
    offs = synth.offsets_from_counts(counts)
    xc, xs = draw_rows(S, inner, 30)
    xc[used:] = 0x7F
    xs[used:] = np.nan
    wc, ws = draw_weight(E, *((outer, inner) if direction == "forward" else (inner, outer)), 31)
    call = bsq.fp8_grouped_forward if direction == "forward" else bsq.fp8_grouped_dgrad
    args = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws), torch.from_numpy(offs).cuda()
    y = torch.full((S, outer), 7.0, dtype=torch.bfloat16, device="cuda")
    call(*args, out=y)
    assert (y[used:] == 7.0).all()
    x, w = row_values(xc[:used], xs[:used]), weight_values(wc, ws)
    for e in range(E):
        r0, r1 = Gm.expert_rows(offs, e)
        if r1 > r0:
            we = w[e].T if direction == "forward" else w[e]
            check(y[r0:r1], x[r0:r1] @ we, x[r0:r1], w[e], inner, f"{direction} expert {e}")
    again = torch.full_like(y, 7.0)
    call(*args, out=again)
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("direction", ["forward", "dgrad"])
@pytest.mark.parametrize("offs", [[40, 20, 70], [10, 30, 71], [-1, 20, 30]])
def test_bad_offsets_over_a_cluster_write_nothing(direction, offs):
    S, inner, outer = 70, 2064, 272
    xc, xs = draw_rows(S, inner, 32)
    wc, ws = draw_weight(3, *((outer, inner) if direction == "forward" else (inner, outer)), 33)
    y = torch.full((S, outer), 3.0, dtype=torch.bfloat16, device="cuda")
    call = bsq.fp8_grouped_forward if direction == "forward" else bsq.fp8_grouped_dgrad
    call(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws),
         torch.tensor(offs, dtype=torch.int32, device="cuda"), out=y)
    assert bsq.get_device_error() == (bsq.BSQ_ERR_INVALID_ARG, 2)
    assert (y == 3.0).all()


# rows, N, K: CTAs of 8 warps, of 4 (five an SM), of 8 for 9 to 16 rows, and two passes over W
WIDE = [(1, 9992, 400), (8, 9992, 400), (8, 24328, 144), (5, 24840, 2576), (9, 9992, 400), (13, 9992, 400), (16, 24328, 144),
        (17, 9736, 272), (31, 9736, 272), (32, 24328, 144)]


@pytest.mark.parametrize("M,N,K", WIDE)
def test_few_rows_of_a_wide_weight(M, N, K):
    assert -(-N // 32) >= 2 * bsq.num_sms()
    xc, xs = draw_rows(M, K, 34)
    wc, ws = draw_weight(1, N, K, 35)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bsq.fp8_forward(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws), out=y)
    x, w = row_values(xc, xs), weight_values(wc, ws)[0]
    check(y, x @ w.T, x, w, K, "forward")
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)
