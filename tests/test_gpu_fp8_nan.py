"""NaN and infinities through the MXFP8 quantizers of x, h and the weights: a NaN
is not made a number, neither in a token's x nor in a weight, and rows that the
norm quantized give what the layer's own quantization of the same rows gives.
Comparisons are of equal bits (NaN for NaN).
"""
import dataclasses

import pytest
import torch

from moe_layer_zero_amd import synth, zcmoe
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def layer(T):
    sh = dataclasses.replace(synth.CONFIGS["small_bf16"], T=T)
    L = H.to_dev(synth.make_layer(sh, "cpu"))
    desc = dataclasses.replace(H.desc_of(sh), weight_layout=zcmoe.ZC_WEIGHTS_MXFP8)
    route = zcmoe.RouteBuffers(desc)
    route.logits.copy_(torch.randn((T, sh.E), generator=torch.Generator().manual_seed(T)))
    zcmoe.zc_moe_route(desc, None, None, torch.zeros(sh.E, device="cuda"), route)
    return sh, L, desc, route


def experts(desc, x, route, w, xq=None):
    out = torch.full_like(x, 7.0)
    zcmoe.zc_moe_experts(desc, x, route, *w, out, xq=xq)
    torch.cuda.synchronize()
    return out.cpu()


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


# row tiles of 32, 64, 128 and 256
@pytest.mark.parametrize("T", [5, 300, 600, 1300, 2800])
def test_a_tokens_nan_reaches_its_output_and_no_other(T):
    print(f"[fp8 nan] T={T}", flush=True)
    sh, L, desc, route = layer(T)
    w = zcmoe.quantize_expert_weights(desc, L["wg"], L["wu"], L["wd"])
    want = experts(desc, L["x"], route, w)
    x = L["x"].clone()
    rows = sorted({1, T // 2, T - 1})
    for i, t in enumerate(rows):
        x[t, (37 * i + 5) % sh.d] = float("nan")
    got = experts(desc, x, route, w)
    keep = torch.ones(T, dtype=torch.bool)
    keep[rows] = False
    assert torch.equal(got[keep], want[keep])
    ffn = (route.topk_idx.cpu() < sh.N).any(1)
    for t in rows:
        assert ffn[t] and torch.isnan(got[t]).all(), t


def test_a_weights_nan_reaches_the_outputs_it_feeds():
    T, e = 300, 9
    sh, L, desc, route = layer(T)
    want = experts(desc, L["x"], route, zcmoe.quantize_expert_weights(desc, L["wg"], L["wu"], L["wd"]))
    hit = (route.topk_idx.cpu() == e).any(1)
    assert hit.any() and not hit.all()
    wd = L["wd"].clone()
    wd[e, 70, 33] = float("nan")      # output column 70 of that expert
    got = experts(desc, L["x"], route, zcmoe.quantize_expert_weights(desc, L["wg"], L["wu"], wd))
    assert torch.isnan(got[hit, 70]).all()
    other = torch.ones(sh.d, dtype=torch.bool)
    other[70] = False
    assert torch.equal(got[:, other], want[:, other]) and torch.equal(got[~hit], want[~hit])
    wu = L["wu"].clone()
    wu[e, 5, 100] = float("nan")      # a column of h, so every output of its tokens
    got = experts(desc, L["x"], route, zcmoe.quantize_expert_weights(desc, L["wg"], wu, L["wd"]))
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("T", [5, 300])
def test_rows_quantized_by_the_norm_are_those_the_layer_makes(T):
    sh, L, desc, route = layer(T)
    w = zcmoe.quantize_expert_weights(desc, L["wg"], L["wu"], L["wd"])
    x = L["x"].clone()
    gamma = torch.ones(sh.d, dtype=BF, device="cuda")
    gamma[40] = float("inf")          # infinities in every row, of either sign
    x[2, 40] = 0                      # 0 * inf: one NaN in a row
    x[T - 1, 7] = float("nan")        # a row of NaN
    x[0, 8] = float("inf")
    y, xq = torch.empty_like(x), zcmoe.mx_buffers(T, sh.d)
    zcmoe.zc_rmsnorm_forward(zcmoe.NormDesc(T, sh.d, BF), x, gamma, y, codes=xq[0], scales=xq[1])
    torch.cuda.synchronize()
    assert torch.isinf(y[1, 40]) and torch.isnan(y[2, 40]) and torch.isnan(y[T - 1]).all()
    a, b = experts(desc, y, route, w), experts(desc, y, route, w, xq)
    assert same(a, b)
    assert torch.isnan(a[2]).all() and torch.isnan(a[T - 1]).all()
    # and the whole forward, on its own routing
    out, r2 = torch.empty_like(y), zcmoe.RouteBuffers(desc)
    zcmoe.zc_moe_forward(desc, y, L["wr"], L["bias"], *w, out, r2)
    assert same(out.cpu(), experts(desc, y, r2, w, xq))
