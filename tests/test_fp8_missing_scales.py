"""A weight without block scales (BF16, or a packed one whose scale is missing) is refused with
ValueError by the E4M3 products, as every other wrong operand is.  On the CPU, with tensors
that call themselves CUDA ones."""

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth
from tests.test_binding_devices import library, operand  # noqa: F401


@pytest.mark.parametrize("name", ["fp8_forward", "fp8_dgrad", "fp8_grouped_forward", "fp8_grouped_dgrad"])
@pytest.mark.parametrize("fmt,missing", [(synth.FMT_BF16, "scale"), (synth.FMT_FP8, "scale"), (synth.FMT_FP8, "data")])
def test_refused(library, name, fmt, missing):  # noqa: F811
    codes, scale = operand(0, 4, 256, dtype=torch.uint8), operand(0, 4, 2)
    data = operand(0, 1, 256, 256, dtype=torch.bfloat16 if fmt == synth.FMT_BF16 else torch.uint8)
    w = synth.Packed(fmt, data, operand(0, 1, 2, 2), None, 1, 256, 256)
    setattr(w, missing, None)
    offs = [operand(0, 1, dtype=torch.int32)] if "grouped" in name else []
    with pytest.raises(ValueError, match=name):
        getattr(bsq, name)(codes, scale, w, *offs)
    assert not library.calls
