"""The caller's score gradient (dlogits) in the backward of bf16 layers.

With dout = 0 the layer's own gradient of the scores is 0, so dw_router =
dlogits^T x and dx = dlogits w_router.  Tolerance (u = 2^-24): dlogits enters as
a pair of bf16 values, off by 2^-18 relative; n terms, two products each, are
added in fp32 (exact products, at most 2 n + 8 roundings, the partial sums of a
split among them): c = 2^-18 + (2 n + 8) u of the sum of absolute products; and
one rounding to bf16, 2^-8 relative.
"""
import dataclasses

import pytest
import torch

from moe_layer_zero_amd import synth, zcmoe
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

U, HB = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def setup(T, d, N, Z, K, gate_norm):
    sh = dataclasses.replace(synth.CONFIGS["small_bf16"], T=T, d=d, N=N, Z=Z, K=K)
    L = H.to_dev(synth.make_layer(sh, "cpu"))
    desc = H.desc_of(sh, gate_norm)
    route, out, saved = H.run_forward(desc, L, saved=True)
    g = torch.Generator().manual_seed(T + d)
    # of very different sizes from token to token
    dl = (torch.randn((T, N + Z), generator=g) * torch.exp2(torch.randint(-20, 10, (T, 1), generator=g))).cuda()
    return sh, L, desc, route, saved, dl


def backward(desc, L, route, saved, dout, dl, lb=None):
    g = [torch.full_like(L[k], float("nan")) for k in ("x", "wr", "wg", "wu", "wd")]
    zcmoe.zc_moe_backward(desc, L["x"], L["wr"], L["wg"], L["wu"], L["wd"], route, saved, dout, *g, lb=lb,
                          dlogits=dl)
    torch.cuda.synchronize()
    return [t.cpu() for t in g]


@pytest.mark.parametrize("gate_norm", [0, 1])
@pytest.mark.parametrize("T,d,N,Z,K", [(1, 1024, 64, 32, 6), (333, 1024, 64, 32, 6), (77, 192, 5, 2, 3),
                                       (2048, 256, 64, 0, 4)])
def test_router_gradients_are_those_of_dlogits(T, d, N, Z, K, gate_norm):
    print(f"[scores bf16] T={T} d={d} N={N} Z={Z} gate_norm={gate_norm}", flush=True)
    sh, L, desc, route, saved, dl = setup(T, d, N, Z, K, gate_norm)
    dx, dwr, dwg, dwu, dwd = backward(desc, L, route, saved, torch.zeros_like(L["x"]), dl)
    x, wr, g = L["x"].cpu().double(), L["wr"].cpu().double(), dl.cpu().double()
    for got, want, terms, n in ((dwr, g.T @ x, g.abs().T @ x.abs(), T),
                                (dx, g @ wr, g.abs() @ wr.abs(), N + Z)):
        tol = (2.0 ** -18 + (2 * n + 8) * U) * terms
        assert ((got.double() - want).abs() <= tol * (1 + HB) + HB * want.abs() + 2.0 ** -133).all()
    assert all((t == 0).all() for t in (dwg, dwu, dwd))


@pytest.mark.parametrize("gate_norm", [0, 1])
@pytest.mark.parametrize("with_lb", [False, True])
def test_zero_dlogits_change_nothing_and_experts_do_not_see_them(gate_norm, with_lb):
    sh, L, desc, route, saved, dl = setup(333, 1024, 64, 32, 6, gate_norm)
    dout = synth.make_dy(sh).cuda()
    lb = zcmoe.LoadBalance(8, 4.5, 0.1) if with_lb else None
    plain = backward(desc, L, route, saved, dout, None, lb)
    for a, b in zip(plain, backward(desc, L, route, saved, dout, torch.zeros_like(dl), lb)):
        assert torch.equal(a, b)
    for a, b in list(zip(plain, backward(desc, L, route, saved, dout, dl, lb)))[2:]:
        assert torch.equal(a, b)
