"""The sequence balance loss with offsets and masks that are slices of larger
tensors, at any byte: equal bits with tensors of their own.
"""
import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests import test_gpu_balance as B

pytestmark = pytest.mark.gpu

T, N, Z, K, S = 333, 12, 4, 3, 3


def setup():
    l = B.scores(T, N + Z, 5)
    desc = zcmoe.LayerDesc(T, 64, N, Z, 64, K, torch.bfloat16)
    route = zcmoe.RouteBuffers(desc)
    route.logits, route.topk_idx = l.cuda(), B.topk(l, K).cuda()
    cu = torch.tensor([0, 100, 101, 330], dtype=torch.int32, device="cuda")
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(2)) < 0.7).cuda()
    return desc, route, cu, mask


def outputs():
    return [torch.full((1 + S,), float("nan"), device="cuda"),
            torch.full((S, N + Z), -1, dtype=torch.int32, device="cuda"),
            torch.full((T, N + Z), float("nan"), device="cuda")]


def run(desc, route, cu, mask, stream=None):
    out = outputs()
    torch.cuda.synchronize()
    zcmoe.zc_moe_seq_balance(desc, zcmoe.LoadBalance(4, 2.0, 0.1), route, *out, cu_seqlens=cu, mask=mask,
                             stream=stream)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("off", [1, 2, 4, 8, 13, 16])
@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
@pytest.mark.parametrize("side", [False, True])
def test_slices(off, dtype, side):
    desc, route, cu, mask = setup()
    mask = mask.to(dtype)
    want = run(desc, route, cu, mask)
    cu_all = torch.cat([torch.full((off,), 7, dtype=torch.int32, device="cuda"), cu])
    mask_all = torch.cat([torch.ones(off, dtype=dtype, device="cuda"), mask])
    got = run(desc, route, cu_all[off:], mask_all[off:], torch.cuda.Stream() if side else None)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_slices_in_a_graph_follow_their_tensor():
    desc, route, cu, mask = setup()
    mask_all = torch.cat([mask.new_ones(5), mask])
    out, ws = outputs(), zcmoe.seq_balance_workspace(desc, S)
    lb = zcmoe.LoadBalance(4, 2.0, 0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zcmoe.zc_moe_seq_balance(desc, lb, route, *out, cu_seqlens=cu, mask=mask_all[5:], ws=ws)
    for k in range(3):
        mask_all[5:] = (torch.rand(T, generator=torch.Generator().manual_seed(10 + k)) < 0.5).cuda()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, run(desc, route, cu, mask_all[5:].clone())):
            assert torch.equal(a, b)
