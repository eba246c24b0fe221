"""Memory that the binding allocates for a call on a given stream: it belongs to
that stream, so it is neither taken from under the current stream's queued work
nor given back to it while the call still runs.  All comparisons are of equal
bits: the same kernels on the same inputs.
"""
import pytest
import torch

from moe_layer_zero_amd import zcmoe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def busy(n=40):
    """Some milliseconds of copies on the current stream."""
    a = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    for _ in range(n):
        b.copy_(a)


def test_scratch_is_not_taken_from_the_current_streams_work():
    T, d = 2048, 2048
    desc = zcmoe.NormDesc(T, d, BF)
    dy, r = torch.randn(T, d, device="cuda").to(BF), torch.randn(T, d, device="cuda").to(BF)
    gamma, rstd = torch.ones(d, device="cuda", dtype=BF), torch.ones(T, device="cuda")
    dr, dg = torch.empty_like(r), torch.empty_like(gamma)
    want = [torch.empty_like(t) for t in (dr, dg)]
    zcmoe.zc_rmsnorm_backward(desc, dy, r, gamma, rstd, *want)
    side = torch.cuda.Stream()
    n = zcmoe.norm_workspace(desc).numel()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = torch.empty(n, dtype=torch.uint8, device="cuda")
    # a block of the workspace's size, still to be read when it is dropped
    block = torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    busy()
    kept.copy_(block)
    del block
    zcmoe.zc_rmsnorm_backward(desc, dy, r, gamma, rstd, dr, dg, stream=side)
    torch.cuda.synchronize()
    assert bool((kept == 7).all())
    assert torch.equal(dr, want[0]) and torch.equal(dg, want[1])


def test_quantized_weights_between_two_calls_of_another_stream():
    N, I, d = 16, 512, 1024
    desc = zcmoe.LayerDesc(1, d, N, 8, I, 4, BF, weight_layout=zcmoe.int4_layout(64))
    w = [torch.randn(N, R, C, device="cuda").to(BF) for R, C in ((I, d), (I, d), (d, I))]
    want = zcmoe.int4_expert_weights(desc, *w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        busy()
    got = zcmoe.int4_expert_weights(desc, *w, stream=side)
    # what the call dropped must not come back here while it is still queued
    junk = [torch.full(s, 0xff, dtype=torch.uint8, device="cuda")
            for s in [(N * I * d // 2,), (N * I * d // 64 * 2,)] * 3]
    torch.cuda.synchronize()
    assert all(bool((j == 0xff).all()) for j in junk)
    for g, h in zip(got, want):
        assert torch.equal(g, h)


def test_balance_and_experts_without_a_workspace_on_another_stream():
    T, d, N, Z, I, K = 96, 256, 8, 4, 128, 2
    desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF, weight_layout=zcmoe.int4_layout(32))
    packed = zcmoe.int4_expert_weights(
        desc, *[torch.randn(N, R, C, device="cuda").to(BF) for R, C in ((I, d), (I, d), (d, I))])
    x = torch.randn(T, d, device="cuda").to(BF)
    route = zcmoe.RouteBuffers(desc)
    route.logits.copy_(torch.randn(T, N + Z, device="cuda"))
    zcmoe.zc_moe_route(desc, None, None, torch.zeros(N + Z, device="cuda"), route)
    lb = zcmoe.LoadBalance(D=N, K_e=1.5, alpha=0.1)

    def run(stream=None):
        out = torch.empty_like(x)
        loss = torch.empty(2, device="cuda")
        counts = torch.empty((1, N + Z), dtype=torch.int32, device="cuda")
        dl = torch.empty((T, N + Z), device="cuda")
        torch.cuda.synchronize()
        zcmoe.zc_moe_experts(desc, x, route, *packed, out, stream=stream)
        zcmoe.zc_moe_seq_balance(desc, lb, route, loss, counts, dl, stream=stream)
        torch.cuda.synchronize()
        return out, loss, counts, dl

    want, side = run(), torch.cuda.Stream()
    for _ in range(3):
        for g, h in zip(run(side), want):
            assert torch.equal(g, h)
