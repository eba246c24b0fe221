"""The calls on a layer's weights (gradient norm, AdamW, MXFP4) run with their
tensors' GPU current, on its stream, refuse a stream of another one, and take what
they allocate from the call's stream.  Checked on the host, as for the other calls.
"""
import dataclasses
from types import SimpleNamespace

import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests.test_device_current import On1, library, on1  # noqa: F401
from tests.test_stream_memory import taken  # noqa: F401

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
T, d, N, Z, I, K = 6, 512, 8, 4, 512, 2


def calls(t):
    """t(*shape, dtype=): makes a tensor."""
    desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF, weight_layout=zcmoe.mxfp4_layout(8))
    d4 = dataclasses.replace(desc, weight_layout=zcmoe.mxfp4_layout(4))
    x, codes, scales = t(T, d), t(T, d // 2, dtype=U8), t(T, d // 32, dtype=U8)
    sets = [t(4096, dtype=U8) for _ in range(3)]
    wc, ws = t(N, I, d // 2, dtype=U8), t(N, I, d // 32, dtype=U8)
    r = zcmoe.RouteBuffers(desc, "cpu")
    for n, v in list(vars(r).items()):
        setattr(r, n, v.as_subclass(On1))
    grads = zcmoe.TensorList([t(7), t(3000)])
    f = lambda n=7: [t(n, dtype=F32)]  # noqa: E731
    adam = zcmoe.AdamWTensors(f(), f(), f(), f())
    step, out = t(1, dtype=torch.int64), t(2, dtype=F32)
    return {
        "zc_grad_norm": lambda **k: zcmoe.zc_grad_norm(grads, 1.0, out, step=step, **k),
        "zc_adamw_step": lambda **k: zcmoe.zc_adamw_step(zcmoe.AdamW(), adam, step, factor=out[1:], **k),
        "zc_adamw_step_host": lambda **k: zcmoe.zc_adamw_step(zcmoe.AdamW(), adam, 3, **k),
        "zc_mxfp4_quantize": lambda **k: zcmoe.zc_mxfp4_quantize(x, codes, scales, **k),
        "zc_moe_mxfp4_pack": lambda **k: zcmoe.zc_moe_mxfp4_pack(desc, 0, wc, ws, sets[0], **k),
        "zc_moe_experts": lambda **k: zcmoe.zc_moe_experts(desc, x, r, *sets, x, **k),
        "zc_moe_experts_rows": lambda **k: zcmoe.zc_moe_experts(d4, x, r, *sets, x, xq=(codes, scales), **k),
        "zc_moe_forward": lambda **k: zcmoe.zc_moe_forward(d4, x, t(N + Z, d), t(N + Z, dtype=F32), *sets, x, r, **k),
    }


NAMES = ["zc_adamw_step", "zc_adamw_step_host", "zc_grad_norm", "zc_moe_experts", "zc_moe_experts_rows",
         "zc_moe_forward", "zc_moe_mxfp4_pack", "zc_mxfp4_quantize"]


@pytest.mark.parametrize("name", NAMES)
def test_the_tensors_device_is_current(library, name):  # noqa: F811
    call = calls(on1)[name]
    fn = name.replace("_host", "").replace("_rows", "")
    call()
    assert library.calls == [(fn, 1, 101)] and library.device == 0
    call(stream=SimpleNamespace(cuda_stream=77, device_index=1))
    assert library.calls[1:] == [(fn, 1, 77)]
    with pytest.raises(ValueError):
        call(stream=SimpleNamespace(cuda_stream=78, device_index=0))
    assert len(library.calls) == 2


def test_tensors_on_two_gpus(library, monkeypatch):  # noqa: F811
    class On2(On1):
        def get_device(self):
            return 2

    a, b = on1(7, dtype=F32), torch.zeros(7).as_subclass(On2)
    with pytest.raises(ValueError):
        zcmoe.TensorList([a, b])
    with pytest.raises(ValueError):
        zcmoe.AdamWTensors([a], [b], [a], [a])
    one = zcmoe.AdamWTensors([a], [a], [a], [a])
    with pytest.raises(ValueError):
        zcmoe.zc_adamw_step(zcmoe.AdamW(), one, 1, factor=b[:1])
    with pytest.raises(ValueError):
        zcmoe.zc_grad_norm(zcmoe.TensorList([a]), 1.0, b[:2])
    assert library.calls == []


def allocating():
    desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF, weight_layout=zcmoe.mxfp4_layout(8))
    x, w, wd = torch.zeros((T, d), dtype=BF), torch.zeros((N, I, d), dtype=BF), torch.zeros((N, d, I), dtype=BF)
    sets = torch.zeros(4096, dtype=U8)
    r = zcmoe.RouteBuffers(desc, "cpu")
    p = [on1(7), on1(300)]
    return {
        "grad_norm": (1, lambda s: zcmoe.zc_grad_norm(zcmoe.TensorList(p), 1.0, torch.zeros(2), stream=s)),
        "adamw_tensors": (4, lambda s: zcmoe.adamw_tensors(p, p, master=True, stream=s)),
        "adamw_tensors_8": (8, lambda s: zcmoe.adamw_tensors(p, p, bits=8, stream=s)),
        "quantize": (2, lambda s: zcmoe.zc_mxfp4_quantize(x, stream=s)),
        "pack": (9, lambda s: zcmoe.mxfp4_expert_weights(desc, w, w, wd, stream=s)),
        "experts": (1, lambda s: zcmoe.zc_moe_experts(desc, x, r, sets, sets, sets, x, stream=s)),
    }


@pytest.mark.parametrize("name", ["adamw_tensors", "adamw_tensors_8", "experts", "grad_norm", "pack", "quantize"])
def test_allocations_belong_to_the_calls_stream(taken, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(zcmoe, "_list_of", lambda tensors, *a: list(tensors))
    monkeypatch.setattr(zcmoe, "_one_gpu", lambda *a: None)
    n, call = allocating()[name]
    side = SimpleNamespace(cuda_stream=1)
    del taken[:]
    call(side)
    # (the gradient norm's own output is the test's)
    own = [s for s in taken if s is not None]
    assert own == [side] * n and len(taken) - n == (name == "grad_norm")
    del taken[:]
    call(None)
    assert taken == [None] * (n + (name == "grad_norm"))
