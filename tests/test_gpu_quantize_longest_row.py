"""bsq_quantize_e4m3 of rows as long as they may be, 2^31 - 16 columns: the last piece that a warp takes
of a row ends past 2^31.  Zeros but for a few values whose codes and scales are known: a block
whose largest magnitude is 448 has scale 1 and its values for codes."""

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu

COLS = 2 ** 31 - 16


@pytest.mark.parametrize("block_rows", [1, 128])
def test_longest_row(block_rows):
    places = {0: 448.0, 5: -2.0, 127: 1.0, 2 ** 30 + 64: 448.0, 2 ** 31 - 1024: 448.0, 2 ** 31 - 513: -448.0, 2 ** 31 - 512: 448.0,
              2 ** 31 - 128: 448.0, 2 ** 31 - 17: -0.5}
    x = torch.zeros((1, COLS), dtype=torch.bfloat16, device="cuda")
    for i, v in places.items():
        x[0, i] = v
    codes, scale = bsq.quantize_e4m3(x, block_rows)
    del x
    assert scale.shape == (1, 2 ** 24)
    for i, v in places.items():
        assert codes[0, i].view(torch.float8_e4m3fn).float().item() == v, i
    assert int(torch.count_nonzero(codes)) == len(places)
    assert (scale == 1).all()
