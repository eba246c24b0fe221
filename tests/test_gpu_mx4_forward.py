"""The forward on MXFP4 weights, eager and without allocations, gives what routing and
zc_moe_experts give on the same x, bit for bit, quantized by the call or before it;
and y is kept in the bits that the header names.
"""
import dataclasses

import pytest
import torch

from moe_layer_zero_amd import synth, zcmoe
from tests import gpu_harness as H
from tests import test_gpu_mx4 as M

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("T", [1, 3, 40, 48, 500])
def test_every_way_gives_the_same_bits(T, a):
    sh = dataclasses.replace(synth.CONFIGS["small_bf16"], T=T, d=512, N=8, Z=4, K=3)
    L = H.to_dev(synth.make_layer(sh, "cpu"))
    desc = dataclasses.replace(H.desc_of(sh, 1, 0.5), weight_layout=zcmoe.mxfp4_layout(a))
    packed = zcmoe.mxfp4_expert_weights(desc, L["wg"], L["wu"], L["wd"])
    # the layer's input: normalized rows, as bf16 and as the norm quantizes them
    x, one = torch.empty_like(L["x"]), torch.ones(512, dtype=BF, device="cuda")
    xq = zcmoe.mx_buffers(T, 512)
    zcmoe.zc_rmsnorm_forward(zcmoe.NormDesc(T, 512, BF), L["x"], one, x, codes=xq[0], scales=xq[1])
    if a == 4:
        xq = zcmoe.zc_mxfp4_quantize(x)
    outs = [torch.full((T, 512), float("nan"), dtype=BF, device="cuda") for _ in range(4)]
    r1, r2, r3 = (zcmoe.RouteBuffers(desc) for _ in range(3))
    zcmoe.zc_moe_forward(desc, x, L["wr"], L["bias"], *packed, outs[0], r1)
    zcmoe.zc_moe_forward_noalloc(desc, x, L["wr"], L["bias"], *packed, outs[1], r2)
    zcmoe.zc_moe_route(desc, x, L["wr"], L["bias"], r3)
    zcmoe.zc_moe_experts(desc, x, r3, *packed, outs[2])
    zcmoe.zc_moe_experts(desc, x, r3, *packed, outs[3], xq=xq)
    torch.cuda.synchronize()
    for r in (r2, r3):
        assert torch.equal(r.topk_idx, r1.topk_idx) and torch.equal(r.topk_gate, r1.topk_gate)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    w = [tuple(t.cpu() for t in zcmoe.zc_mxfp4_quantize(L[n])) for n in ("wg", "wu", "wd")]
    ref, tol = M.reference(desc, x.cpu(), w, r1, a)
    err = abs(outs[0].cpu().double().numpy() - ref)
    assert (err <= tol * (1 + M.HB) + M.HB * abs(ref) + 2.0 ** -133).all()


# T, N, Z, d, I, and whether y is fp32; K = 2
LAYERS = [
    (10, 2, 0, 512, 512, True),        # 10 picks an expert
    (11, 2, 0, 512, 512, False),       # 11
    (21, 2, 2, 512, 512, True),        # 10.5
    (22, 2, 2, 512, 512, False),
    (300, 2, 0, 1024, 512, False),
    (300, 2, 0, 640, 512, True),       # d and I have to be multiples of 512 both
    (300, 2, 0, 512, 384, True),
    (11, 2, 0, 512, 1 << 22, True),    # a matrix of 2^31 values
]


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("T,N,Z,d,I,fp32", LAYERS)
def test_bits_of_y(T, N, Z, d, I, fp32, a):
    """Everything before y is exact: x = (1, 0, ...), gate 64 and up 1, so h = 64
    (silu(64) = 64 in fp32), and y = 64 * 128.5 = 8224 from one expert, 64 * -128 =
    -8192 from the other.  8224 takes 9 bits: in bf16 it is 8192 (a tie, to even), and
    the half of both, 16 in fp32, is gone."""
    desc = zcmoe.LayerDesc(T, d, N, Z, I, 2, BF, weight_layout=zcmoe.mxfp4_layout(a))
    u8 = dict(dtype=torch.uint8, device="cuda")

    def matrix(R, Cc):
        return torch.zeros((N, R, Cc // 2), **u8), torch.full((N, R, Cc // 32), 127, **u8)

    gate, up, down = matrix(I, d), matrix(I, d), matrix(d, I)
    gate[0][..., 0] = 6                # 4 ...
    gate[1][..., 0] = 127 + 4          # ... times 16
    up[0][..., 0] = 2                  # 1
    down[0][0, :, :10] = 0x77          # twenty times 6,
    down[0][0, :, 10] = 0x47           # 6 and 2,
    down[0][0, :, 11] = 0x01           # and 0.5
    down[0][1, :, :10] = 0xff
    down[0][1, :, 10] = 0xcf
    packed = zcmoe.pack_mxfp4_expert_weights(desc, gate, up, down)
    x = torch.zeros((T, d), dtype=BF, device="cuda")
    x[:, 0] = 1.0
    route = zcmoe.RouteBuffers(desc)
    route.logits.fill_(-1e4)
    route.logits[:, :2] = 0.0
    zcmoe.zc_moe_route(desc, None, None, torch.zeros(N + Z, device="cuda"), route)
    assert bool((route.topk_idx < 2).all()) and bool((route.topk_gate == 0.5).all())
    out = torch.full((T, d), float("nan"), dtype=BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x, route, *packed, out)
    assert bool((out == (16.0 if fp32 else 0.0)).all())
