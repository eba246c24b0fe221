"""The experts on MXFP4 weights for one row of 128 values of h, the smallest there
is: its scales are read by every workgroup of a wide y, many more than run at once,
while others store y.  The sums of a row do not depend on the rows beside it, so the
same token twice gives the same bits.
"""
import dataclasses

import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests import test_gpu_mx4 as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("d", [128, 4096, 1 << 16])
def test_one_row_of_h(d, a):
    desc, x, w, route, packed = M.make(2, d, 1, 0, 128, 1, a, seed=d)
    x[1] = x[0]
    two = torch.full((2, d), float("nan"), dtype=M.BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, two)
    one = dataclasses.replace(desc, T=1)
    r = zcmoe.RouteBuffers(one)
    r.logits.copy_(route.logits[:1])
    zcmoe.zc_moe_route(one, None, None, torch.zeros(1, device="cuda"), r)
    for _ in range(4):
        out = M.check(one, x[:1], w, r, packed, a)
        assert torch.equal(out[0], two[0]) and torch.equal(two[0], two[1])
