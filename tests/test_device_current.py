"""A call on tensors of another GPU than the current one: it runs with their
device current, on that device's stream, and a stream of a third one is refused.
Checked on the host, on tensors that only say where they are, with a library that
notes the stream and the device it is called with.
"""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from moe_layer_zero_amd import zcmoe

BF = torch.bfloat16
T, d, N, Z, I, K = 6, 512, 8, 4, 512, 2


class On1(torch.Tensor):
    """Says that it lives on GPU 1."""
    is_cuda = True

    def get_device(self):
        return 1


def on1(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(On1)


class Library:
    def __init__(self):
        self.device, self.calls = 0, []

    def __getattr__(self, name):
        if name.endswith(("_size", "_bytes")):
            return lambda *a: 4096

        def call(*a):
            self.calls.append((name, self.device, a[-1]))
            return zcmoe.ZC_OK
        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()

    @contextlib.contextmanager
    def device(i):
        old, L.device = L.device, i
        yield
        L.device = old

    monkeypatch.setattr(zcmoe, "_LIB", L)
    monkeypatch.setattr(zcmoe, "_alloc", lambda stream, make, *a, **kw: on1(4096, dtype=torch.uint8))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: L.device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda dev=None: SimpleNamespace(cuda_stream=100 + (L.device if dev is None else dev)))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    return L


def calls():
    desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF)
    x, w, wd, wr = on1(T, d), on1(N, I, d), on1(N, d, I), on1(N + Z, d)
    f32, i32 = torch.float32, torch.int32
    bias, lb = on1(N + Z, dtype=f32), zcmoe.LoadBalance(4, 1.5, 0.1)
    r = zcmoe.RouteBuffers(desc, "cpu")
    for n, t in list(vars(r).items()):
        setattr(r, n, t.as_subclass(On1))
    saved, hist, moments = on1(16, dtype=torch.uint8), on1(K + 1, dtype=i32), on1(2, dtype=torch.float64)
    lbo, dst = on1(11, dtype=torch.float64), on1(4096, dtype=torch.uint8)
    grads = (x, wr, w, w, wd)
    return {
        "zc_moe_route": lambda **k: zcmoe.zc_moe_route(desc, x, wr, bias, r, **k),
        "zc_moe_forward": lambda **k: zcmoe.zc_moe_forward(desc, x, wr, bias, w, w, wd, x, r, **k),
        "zc_moe_forward_noalloc": lambda **k: zcmoe.zc_moe_forward_noalloc(desc, x, wr, bias, w, w, wd, x, r, **k),
        "zc_moe_backward": lambda **k: zcmoe.zc_moe_backward(desc, x, wr, w, w, wd, r, saved, x, *grads, **k),
        "zc_moe_backward_scores": lambda **k: zcmoe.zc_moe_backward(desc, x, wr, w, w, wd, r, saved, x, *grads,
                                                                    dlogits=r.logits, **k),
        "zc_moe_lb_loss": lambda **k: zcmoe.zc_moe_lb_loss(desc, lb, r, lbo, **k),
        "zc_moe_route_stats": lambda **k: zcmoe.zc_moe_route_stats(desc, r, hist, moments, **k),
        "zc_moe_accumulate_counts": lambda **k: zcmoe.zc_moe_accumulate_counts(r.counts, r.counts, **k),
        "zc_moe_pid_update": lambda **k: zcmoe.zc_moe_pid_update(N, Z, K, r.counts, 5, 0.1, 1.5, bias, **k),
        "zc_moe_pack_weights": lambda **k: zcmoe.zc_moe_pack_weights(desc, 0, w, w, **k),
        "zc_moe_quantize_weights": lambda **k: zcmoe.zc_moe_quantize_weights(desc, 0, w, dst, **k),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_the_tensors_device_is_current(library, name):
    call = calls()[name]
    call()
    assert library.calls == [(name, 1, 101)] and library.device == 0
    call(stream=SimpleNamespace(cuda_stream=77, device_index=1))
    assert library.calls[1:] == [(name, 1, 77)]
    with pytest.raises(ValueError):
        call(stream=SimpleNamespace(cuda_stream=78, device_index=0))
    assert len(library.calls) == 2
