"""Gradients that are not finite, whatever bits their NaNs carry, show in what an AdamW
step writes, and in nothing else: weights of 32 and of 16 bits, rounded to nearest
and stochastically, states of 32 and of 8 bits.
"""
import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests.test_gpu_optim import BF, F32, KINDS, Case

pytestmark = pytest.mark.gpu

# a NaN of all ones is what memory filled with 0xff holds
NANS = [0x7fffffff, -1, 0x7fc00000, -0x400000, 0x7fffff01, 0x7f800001, 0x7fc0ffff]
N = 3 * 128 + 5


def steps(dtype, gdtype, master, bits, rounding, seed, bad):
    c = Case([N], dtype, gdtype, master, bits)
    for i, word in bad.items():
        g = c.dev["g"][0]
        if gdtype == F32:
            g.view(torch.int32)[i] = word
        else:
            g.view(torch.int16)[i] = word >> 16
    zcmoe.zc_adamw_step(zcmoe.AdamW(rounding=rounding, seed=seed), c.t, 2)
    return {k: t[0].float().cpu() for k, t in c.dev.items()}


@pytest.mark.parametrize("rounding", [0, 1])
@pytest.mark.parametrize("dtype,gdtype,master,bits", KINDS)
def test_nan_gradients_show(dtype, gdtype, master, bits, rounding):
    # in whole vectors, and among the last elements
    at = [0, 3, 130, 131, N - 5, N - 2, N - 1]
    words = [w for w in NANS if gdtype == F32 or w >> 16 & 0x7f]
    for seed in range(12):
        bad = {i: words[(k + seed) % len(words)] for k, i in enumerate(at)}
        got = steps(dtype, gdtype, master, bits, rounding, seed, bad)
        want = steps(dtype, gdtype, master, bits, rounding, seed, {})
        hit = torch.zeros(N, dtype=torch.bool)
        hit[at] = True
        for k in ("p", "m", "v", "master"):
            if k in got:
                assert torch.equal(torch.isnan(got[k]), hit), k
        for k in ("p", "master"):
            if k in got:
                assert torch.equal(got[k][~hit], want[k][~hit]), k


@pytest.mark.parametrize("rounding", [0, 1])
@pytest.mark.parametrize("dtype,gdtype,master,bits", KINDS)
def test_infinite_gradients_show(dtype, gdtype, master, bits, rounding):
    bad = {140: 0x7f800000, N - 1: -0x800000}
    got = steps(dtype, gdtype, master, bits, rounding, 3, bad)
    want = steps(dtype, gdtype, master, bits, rounding, 3, {})
    hit = torch.zeros(N, dtype=torch.bool)
    hit[list(bad)] = True
    for k in ("p", "master"):
        if k in got:
            assert torch.equal(torch.isnan(got[k]), hit) and torch.equal(got[k][~hit], want[k][~hit])
    # 8-bit states share a scale: the block's are lost with it
    lost = hit if bits == 32 else torch.arange(N) // 128 % 2 == 1
    for k in ("m", "v"):
        assert torch.equal(~torch.isfinite(got[k]), lost), k


def test_infinite_weights_stay():
    p = [torch.tensor([float("inf"), -float("inf"), 1.0, 3.3895e38] * 9, device="cuda").to(BF)]
    before = p[0].clone()
    t = zcmoe.adamw_tensors(p, [torch.zeros(36, device="cuda")])
    for k in range(1, 6):
        zcmoe.zc_adamw_step(zcmoe.AdamW(lr=0.0, rounding=1, seed=k), t, k)
    assert torch.equal(p[0], before)
