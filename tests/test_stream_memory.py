"""Every tensor that the binding allocates for a call on a given stream is taken
from that stream: scratch that is dropped on return goes back to the stream that
still uses it, and an output does not come from a block that queued work of
another stream may still read.  Checked on the host, with a library that does nothing
and a stream context that is only noted down.
"""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from moe_layer_zero_amd import zcmoe

BF, F32 = torch.bfloat16, torch.float32
T, d, N, Z, I, K = 6, 512, 8, 4, 512, 2


class NoLibrary:
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith(("_size", "_bytes")) else zcmoe.ZC_OK


@pytest.fixture
def taken(monkeypatch):
    """Notes the stream current at each allocation that the binding makes."""
    current, got = [None], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def noting(make):
        def f(*a, **kw):
            got.append(current[-1])
            return make(*a, **kw)
        return f

    monkeypatch.setattr(zcmoe, "_LIB", NoLibrary())
    monkeypatch.setattr(zcmoe, "_ptr", lambda t: None)
    monkeypatch.setattr(zcmoe._Args, "__call__", lambda self, t, *a: None)
    monkeypatch.setattr(zcmoe._Args, "run", lambda self, *a, **kw: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for n in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, n, noting(getattr(torch, n)))
    return got


def calls():
    desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF)
    q4 = zcmoe.LayerDesc(T, d, N, Z, I, K, BF, weight_layout=zcmoe.int4_layout(64))
    x, w = torch.zeros((T, d), dtype=BF), torch.zeros((N, I, d), dtype=BF)
    wd, wr = torch.zeros((N, d, I), dtype=BF), torch.zeros((N + Z, d), dtype=BF)
    bias, lb = torch.zeros(N + Z), zcmoe.LoadBalance(4, 1.5, 0.1)
    r = zcmoe.RouteBuffers(desc, "cpu")
    saved = torch.zeros(16, dtype=torch.uint8)
    set4 = torch.zeros(4096, dtype=torch.uint8)
    norm = zcmoe.NormDesc(T, d, BF)
    # the call, and how many tensors it allocates
    return {
        "route": (1, lambda s: zcmoe.zc_moe_route(desc, x, wr, bias, r, stream=s)),
        "forward": (1, lambda s: zcmoe.zc_moe_forward(desc, x, wr, bias, w, w, wd, x, r, stream=s)),
        "forward_int4": (1, lambda s: zcmoe.zc_moe_forward(q4, x, wr, bias, set4, set4, set4, x, r, stream=s)),
        "backward": (1, lambda s: zcmoe.zc_moe_backward(desc, x, wr, w, w, wd, r, saved, x, x, wr, w,
                                                        w, wd, stream=s)),
        "backward_scores": (1, lambda s: zcmoe.zc_moe_backward(desc, x, wr, w, w, wd, r, saved, x, x, wr,
                                                               w, w, wd, stream=s, dlogits=r.logits)),
        "lb_loss": (2, lambda s: zcmoe.zc_moe_lb_loss(desc, lb, r, stream=s)),
        "route_stats": (3, lambda s: zcmoe.zc_moe_route_stats(desc, r, stream=s)),
        "pack": (3, lambda s: zcmoe.pack_expert_weights(desc, w, w, wd, stream=s)),
        "quantize": (3, lambda s: zcmoe.quantize_expert_weights(desc, w, w, wd, stream=s)),
        "int4": (9, lambda s: zcmoe.int4_expert_weights(q4, w, w, wd, stream=s)),
        "experts": (1, lambda s: zcmoe.zc_moe_experts(q4, x, r, set4, set4, set4, x, stream=s)),
        "seq_balance": (1, lambda s: zcmoe.zc_moe_seq_balance(desc, lb, r, bias, r.topk_idx, stream=s)),
        "norm_backward": (1, lambda s: zcmoe.zc_rmsnorm_backward(norm, x, x, x[0], bias, x, x[0], stream=s)),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_allocations_belong_to_the_calls_stream(taken, name):
    n, call = calls()[name]
    side = SimpleNamespace(cuda_stream=1)
    del taken[:]
    call(side)
    assert taken == [side] * n
    del taken[:]
    call(None)
    assert taken == [None] * n
