"""The norm and the balance loss at the sizes where another kernel shape or
split takes over.  Counts and rows are compared bit for bit; the balance values
with the tolerances derived in test_gpu_balance, the norm's with those of
test_gpu_norm.
"""
import numpy as np
import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests import test_gpu_balance as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.mark.parametrize("S", [128, 129, 256, 257, 1023, 1024, 1025])
def test_balance_at_the_splits_in_the_number_of_sequences(S):
    T, N, Z, K = 2 * S + 5, 12, 4, 3
    print(f"[balance] S={S}", flush=True)
    l = B.scores(T, N + Z, S)
    cu = np.linspace(0, T - 1, S + 1).round().astype(int).tolist()
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(S)) < 0.6).to(torch.uint8)
    B.check(l, B.topk(l, K), N, K, 4, 1.8, 0.3, cu, mask)


@pytest.mark.parametrize("picks", [8191, 8192, 16384, 32768, 32769, 65536, 65537, 140000])
@pytest.mark.parametrize("S", [1, 40])
def test_balance_of_one_sequence_that_holds_the_batch(picks, S):
    # the others are empty; parts end inside the sequence
    N, Z, K = 12, 4, 8
    T = -(-picks // K)
    print(f"[balance] picks={picks} S={S}", flush=True)
    l = B.scores(T, N + Z, picks)
    cu = [0] * (S // 2 + 1) + [T] * (S - S // 2)
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.9).to(torch.uint8)
    B.check(l, B.topk(l, K), N, K, 12, 4.0, 0.3, cu, mask)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vecs", [64, 65, 128, 129, 193, 256, 257, 512, 513, 768, 769, 1025])
def test_a_norms_row_does_not_depend_on_the_others(vecs, dtype):
    d = vecs * (8 if dtype == BF else 4)
    T = 9
    g = torch.Generator().manual_seed(vecs)
    x, res = [torch.randn((T, d), generator=g).to(dtype) for _ in range(2)]
    gamma = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    print(f"[norm] d={d} {dtype}", flush=True)

    def run(lo, hi):
        a, b, w = x[lo:hi].cuda(), res[lo:hi].cuda(), gamma.cuda()
        y, r = torch.full_like(a, float("nan")), torch.full_like(a, float("nan"))
        rs = torch.full((hi - lo,), float("nan"), device="cuda")
        zcmoe.zc_rmsnorm_forward(zcmoe.NormDesc(hi - lo, d, dtype), a, w, y, res=b, r=r, rstd=rs)
        torch.cuda.synchronize()
        return y.cpu(), r.cpu(), rs.cpu()

    y, r, rs = run(0, T)
    assert torch.equal(r, (x.float() + res.float()).to(dtype))
    rd = r.double()
    rstd = 1 / torch.sqrt((rd * rd).mean(1, keepdim=True) + float(np.float32(1e-6)))
    want = rd * rstd * gamma.double()
    # rstd within 48 u, two products and one rounding
    half = torch.finfo(dtype).eps / 2
    assert ((rs.double()[:, None] - rstd).abs() <= 48 * U * rstd).all()
    assert ((y.double() - want).abs() <= (half + 50 * U) * want.abs()).all()
    for i in range(T):
        for a, b in zip(run(i, i + 1), (y, r, rs)):
            assert torch.equal(a[0], b[i])
