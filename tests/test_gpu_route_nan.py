"""Where a NaN among a token's logits reaches their gradient: everywhere under the softmax over all, else only where a chosen logit is one."""

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("E", [20, 96, 600])
def test_nan_reaches_the_gradient_where_it_is_read(gate, renorm, E):
    x = torch.randn((4, E), generator=torch.Generator().manual_seed(E))
    clean = x.clone()
    x[0, 7] = x[1, 7] = x[2, 7] = float("nan")
    ids = torch.tensor([[1, 2, 3], [1, 7, 3], [-1, -1, -1], [1, 7, 3]], dtype=torch.int32, device="cuda")
    g = torch.randn((4, 3), generator=torch.Generator().manual_seed(1)).cuda()
    got, ref = (bsq.route_backward(t.cuda(), ids, g, gate=gate, renormalize=renorm).cpu() for t in (x, clean))
    every = gate == "softmax" and not renorm
    if every:
        assert got[0].isnan().all() and got[1].isnan().all()
    else:
        assert torch.equal(got[0], ref[0])                           # chosen: 1, 2 and 3
        assert got[1, 7].isnan()
        others = [e for e in range(E) if e not in (1, 3, 7)]
        assert not got[1, others].any()
        assert got[1, [1, 3]].isnan().all() if renorm else torch.equal(got[1, [1, 3]], ref[1, [1, 3]])
    assert not got[2].any() and torch.equal(got[3], ref[3])
