"""The join of the norm backward's partial rows into dgamma.

r, rstd and gamma are 1, so dgamma is the column sum of dy, whole numbers below
2^20.  A partial row adds at most 4 rows a wavefront and 4 wavefronts: below 2^24,
exact in fp32.  Up to 2048 rows the sum is below 2^31: exact in binary64, and
rounded once to fp32 it has one right value.  (A join in fp32 rounds on the way.)
"""
import pytest
import torch

from moe_layer_zero_amd import zcmoe

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.mark.parametrize("d", [8, 64, 260, 1024, 1028, 1544, 4104])
@pytest.mark.parametrize("T", [1, 31, 512, 1003, 2048])
def test_partial_rows_are_joined_exactly(T, d):
    print(f"[norm sums] T={T} d={d}", flush=True)
    dy = torch.randint(-(1 << 20), 1 << 20, (T, d), generator=torch.Generator().manual_seed(T + d)).float()
    one = torch.ones((T, d), device="cuda")
    gamma, rstd = torch.ones(d, device="cuda"), torch.ones(T, device="cuda")
    dr, dg = torch.empty_like(one), torch.full((d,), float("nan"), device="cuda")
    zcmoe.zc_rmsnorm_backward(zcmoe.NormDesc(T, d, F32), dy.cuda(), one, gamma, rstd, dr, dg)
    torch.cuda.synchronize()
    assert torch.equal(dg.cpu(), dy.double().sum(0).float())
