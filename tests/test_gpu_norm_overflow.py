"""RMS norm where r * gamma, or y itself, is beyond fp32.

An infinite gamma gives infinities of r's sign (NaN where r is 0), as 0 and
infinity multiply; a finite product beyond fp32 gives y where y fits its type.
Tolerance of a finite y there: rstd's error (48 u, derived in test_gpu_norm), two
products and one rounding, h + 51 u with u = 2^-24 and h half a step of the type.
"""
import numpy as np
import pytest
import torch

from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32

# each number of threads a row
WIDTHS = [8, 512, 640, 1664, 2048, 4096, 6144, 16384, 32768]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_infinite_gamma(d, dtype):
    print(f"[norm inf] d={d} {dtype}", flush=True)
    T = 40
    x, res, gamma = N.inputs(T, d, dtype, d)
    want = N.forward(x, res, gamma)[1].cpu()
    x[:, 1], res[:, 1] = 0, 0          # r = 0 under an infinite gamma
    gamma[0], gamma[1], gamma[d - 1] = float("inf"), float("inf"), float("-inf")
    r, y, rstd, _, _ = N.forward(x, res, gamma)
    r, y = r.cpu().float(), y.cpu().float()
    assert torch.isnan(y[:, 1]).all()
    nonzero = r[:, [0, d - 1]] != 0
    sign = torch.sign(r[:, [0, d - 1]]) * torch.tensor([1.0, -1.0])
    assert (y[:, [0, d - 1]] == sign * float("inf"))[nonzero].all()
    assert nonzero.any() and torch.isfinite(rstd).all()
    assert torch.isfinite(y[:, 2:d - 1]).all() and torch.isfinite(want.float()).all()


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_products_beyond_fp32_with_y_inside(d, dtype):
    print(f"[norm large] d={d} {dtype}", flush=True)
    T = 40
    x, _, gamma = N.inputs(T, d, dtype, d + 1)
    x, gamma = (x.float() * 1e15).to(dtype), (gamma.float() * 1e28).to(dtype)
    assert torch.isinf(x.float().abs().amax() * gamma.float().abs().amax())
    ro, yo, so = N.reference(x, None, gamma)
    _, y, rstd, _, _ = N.forward(x, None, gamma)
    assert ((rstd.cpu().double() - so).abs() <= 48 * U * so).all()
    half = torch.finfo(dtype).eps / 2
    assert ((y.cpu().double() - yo).abs() <= (half + 51 * U) * yo.abs()).all()


def test_y_beyond_fp32_is_an_infinity():
    T, d = 7, 264
    x, _, gamma = N.inputs(T, d, F32, 5)
    x = x * 1e-20
    gamma[3], gamma[4] = 3e37, -3e37
    x[:, 3:5] = 1e-10                       # about 16 times the row's mean
    _, y, _, _, _ = N.forward(x, None, gamma, eps=1e-30)
    yo = N.reference(x, None, gamma, float(np.float32(1e-30)))[1]
    assert (yo[:, 3] > 3.5e38 * 0.9).all()
    y = y.cpu()
    assert (y[:, 3] == float("inf")).all() and (y[:, 4] == float("-inf")).all()
    assert torch.isfinite(y[:, 5:]).all()


def test_codes_of_infinities_saturate():
    T, d = 33, 1024
    x, res, gamma = N.inputs(T, d, BF, 9)
    gamma[32], gamma[40] = float("inf"), float("-inf")
    r, y, _, codes, scales = N.forward(x, res, gamma, mx=True)
    r, codes = r.cpu().float(), codes.cpu()
    for c, s in ((32, 1.0), (40, -1.0)):
        keep = r[:, c] != 0
        want = torch.where(r[:, c] * s > 0, 0x7e, 0xfe).to(torch.uint8)   # +-448
        assert torch.equal(codes[:, c][keep], want[keep])
    assert ((codes & 0x7f) != 0x7f).all()
    # the other blocks are those of finite rows
    q, S = N.mx_reference(y.cpu()[:, 64:])
    got = codes.view(torch.float8_e4m3fn).double().numpy()[:, 64:].reshape(-1, 32)
    np.testing.assert_array_equal(got, q)
