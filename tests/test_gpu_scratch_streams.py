"""Scratch that a call on a given stream allocates by itself, while the other
stream is busy: the call neither writes a block that queued work of the current
stream has still to read, nor loses its own to the current stream's next tensor
while it is still queued.  Comparisons are of equal bits with the same call alone.
"""
import dataclasses

import pytest
import torch

from moe_layer_zero_amd import synth, zcmoe
from tests import gpu_harness as H
from tests.test_gpu_operator_streams import busy

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def cases():
    """name -> function that gives (bytes of scratch, call(stream) -> outputs)."""
    sh = dataclasses.replace(synth.CONFIGS["small_bf16"], T=200, forward_only=False)

    def layer(layout=0):
        L = H.to_dev(synth.make_layer(sh, "cpu"))
        desc = dataclasses.replace(H.desc_of(sh), weight_layout=layout)
        w = (L["wg"], L["wu"], L["wd"])
        if zcmoe.int4_group(desc):
            w = zcmoe.int4_expert_weights(desc, *w)
        route = zcmoe.RouteBuffers(desc)
        zcmoe.zc_moe_route(desc, L["x"], L["wr"], L["bias"], route)
        return L, desc, w, route

    def forward(layout):
        L, desc, w, route = layer(layout)

        def call(s):
            out = torch.empty_like(L["x"])
            torch.cuda.synchronize()
            return [out], lambda: zcmoe.zc_moe_forward(desc, L["x"], L["wr"], L["bias"], *w, out, route,
                                                       stream=s)
        return zcmoe.zc_moe_workspace_size(desc, zcmoe.ZC_OP_FORWARD), call

    def experts():
        L, desc, w, route = layer(zcmoe.int4_layout(32))

        def call(s):
            out = torch.empty_like(L["x"])
            return [out], lambda: zcmoe.zc_moe_experts(desc, L["x"], route, *w, out, stream=s)
        return zcmoe.zc_moe_workspace_size(desc, zcmoe.ZC_OP_EXPERTS), call

    def backward(scores):
        L, desc, w, route = layer()
        out, saved = torch.empty_like(L["x"]), zcmoe.saved_buffer(desc)
        zcmoe.zc_moe_forward(desc, L["x"], L["wr"], L["bias"], *w, out, route, saved)
        dout = torch.randn(out.shape, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
        dl = torch.randn(route.logits.shape, generator=torch.Generator().manual_seed(2)).cuda()

        def call(s):
            g = [torch.empty_like(t) for t in (L["x"], L["wr"], *w)]
            return g, lambda: zcmoe.zc_moe_backward(desc, L["x"], L["wr"], *w, route, saved, dout, *g,
                                                    stream=s, dlogits=dl if scores else None)
        return zcmoe.zc_moe_workspace_size(desc, zcmoe.ZC_OP_BACKWARD), call

    def balance():
        T, N, Z, K, S = 5000, 64, 32, 6, 3
        desc = zcmoe.LayerDesc(T, 64, N, Z, 64, K, BF)
        route = zcmoe.RouteBuffers(desc)
        route.logits.copy_(torch.randn((T, N + Z), generator=torch.Generator().manual_seed(3)))
        zcmoe.zc_moe_route(desc, None, None, torch.zeros(N + Z, device="cuda"), route)
        cu = torch.tensor([0, 100, 2000, 5000], dtype=torch.int32, device="cuda")
        lb = zcmoe.LoadBalance(8, 4.5, 0.1)

        def call(s):
            o = [torch.empty(1 + S, device="cuda"), torch.empty((S, N + Z), dtype=torch.int32, device="cuda"),
                 torch.empty((T, N + Z), device="cuda")]
            return o, lambda: zcmoe.zc_moe_seq_balance(desc, lb, route, *o, cu_seqlens=cu, stream=s)
        return zcmoe.seq_balance_workspace(desc, S).numel(), call

    def route():
        L, desc, w, _ = layer()

        def call(s):
            r = zcmoe.RouteBuffers(desc)
            r.perm.zero_()   # (entries past the FFN picks are left as they are)
            return [r.logits, r.topk_idx, r.topk_gate, r.counts, r.offsets, r.perm, r.inv], \
                lambda: zcmoe.zc_moe_route(desc, L["x"], L["wr"], L["bias"], r, stream=s)
        return zcmoe.zc_moe_workspace_size(desc, zcmoe.ZC_OP_ROUTE), call

    def lb_loss():
        L, desc, w, r = layer()
        lb = zcmoe.LoadBalance(8, 4.5, 0.1)

        def call(s):
            o = torch.empty(1 + 2 * 9, dtype=torch.float64, device="cuda")
            return [o], lambda: zcmoe.zc_moe_lb_loss(desc, lb, r, out=o, stream=s)
        return zcmoe.zc_moe_workspace_size(desc, zcmoe.ZC_OP_LB_LOSS), call

    return {"forward": lambda: forward(0), "forward_int4": lambda: forward(zcmoe.int4_layout(64)),
            "experts_int4": experts, "backward": lambda: backward(False),
            "backward_scores": lambda: backward(True), "seq_balance": balance, "route": route,
            "lb_loss": lb_loss}


@pytest.mark.parametrize("name", sorted(cases()))
def test_scratch_of_a_call_on_another_stream(name):
    print(f"[scratch] {name}", flush=True)
    n, call = cases()[name]()
    n = max(n, 256)
    want, go = call(None)
    torch.cuda.synchronize()
    go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # a block of the scratch's size, dropped while the current stream has still to read it
    got, go = call(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = torch.empty(n, dtype=torch.uint8, device="cuda")
    block = torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    busy()
    kept.copy_(block)
    del block
    go()
    torch.cuda.synchronize()
    assert bool((kept == 7).all())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # the side stream is busy: what the call dropped must not come back here before it ran
    del kept
    got, go = call(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        busy()
    go()
    junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((j == 0xff).all()) for j in junk)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_weight_sets_made_on_a_busy_stream_are_not_those_of_dropped_blocks():
    sh = synth.CONFIGS["small_bf16"]
    L = H.to_dev(synth.make_layer(dataclasses.replace(sh, T=1), "cpu"))
    desc, w = H.desc_of(sh), (L["wg"], L["wu"], L["wd"])
    side = torch.cuda.Stream()
    for make in (zcmoe.pack_expert_weights, zcmoe.quantize_expert_weights):
        want = [t.clone() for t in make(desc, *w)]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        kept = [torch.empty_like(t) for t in want]
        blocks = [torch.full_like(t, 7) for t in want]
        torch.cuda.synchronize()
        busy()
        for k, b in zip(kept, blocks):
            k.copy_(b)
        del blocks, b
        got = make(desc, *w, stream=side)
        torch.cuda.synchronize()
        assert all(bool((k == 7).all()) for k in kept)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del kept, k, got, a, b
