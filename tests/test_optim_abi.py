"""Host-side checks of the gradient norm and the AdamW step, before any work is
queued."""
import ctypes as C

import pytest
import torch

from moe_layer_zero_amd import zcmoe

BAD, UNS, WS = zcmoe.ZC_ERR_INVALID, zcmoe.ZC_ERR_UNSUPPORTED, zcmoe.ZC_ERR_WORKSPACE
BF, F32 = zcmoe.ZC_BF16, zcmoe.ZC_F32
NONE = C.POINTER(zcmoe.zc_adamw_tensor)()


def ptr(i):
    return (i + 1) << 30  # distinct, aligned, never dereferenced


def grads(*sizes):
    return (zcmoe.zc_grad_tensor * len(sizes))(*(zcmoe.zc_grad_tensor(ptr(i), n) for i, n in enumerate(sizes)))


def norm(t, count=None, dtype=BF, max_norm=1.0, out=ptr(40), step=ptr(41), ws=ptr(42), ws_bytes=1 << 24):
    return zcmoe.lib().zc_grad_norm(t, len(t) if count is None else count, dtype, max_norm, out, step, ws,
                                    ws_bytes, None)


def test_grad_norm_refusals():
    L = zcmoe.lib()
    assert norm(grads(5), count=-1) == BAD and L.zc_last_error().decode() != ""
    assert norm(grads(5), count=1 << 21) == BAD
    assert norm(grads(5), dtype=7) == BAD
    assert norm(grads(-1)) == BAD
    assert norm(grads(1 << 36)) == UNS
    assert norm(None, count=1) == BAD
    for m in (0.0, -1.0, float("nan")):
        assert norm(grads(5), max_norm=m) == BAD
    assert norm(grads(5), out=None) == BAD
    assert norm(grads(5), out=ptr(40) + 2) == BAD
    assert norm(grads(5), step=ptr(41) + 4) == BAD
    assert norm(grads(5), ws=None) == WS
    assert norm(grads(5), ws_bytes=8) == WS
    assert norm(grads(5), ws=ptr(42) + 16) == BAD
    t = grads(5)
    t[0].g = None
    assert norm(t) == BAD
    t[0].g = ptr(0) + 8
    assert norm(t) == BAD
    # an output over a gradient, or over another output
    assert norm(grads(5), out=ptr(0) + 8) == BAD
    assert norm(grads(5), step=ptr(40)) == BAD
    assert norm(grads(1 << 20), ws=ptr(0) + 256) == BAD


def test_grad_norm_workspace():
    L = zcmoe.lib()
    assert L.zc_grad_norm_workspace_size(grads(1), 1, BF) == 256
    assert L.zc_grad_norm_workspace_size(grads(1), 1, 9) == 0
    assert L.zc_grad_norm_workspace_size(grads(-1), 1, BF) == 0
    assert L.zc_grad_norm_workspace_size(grads(1 << 36), 1, BF) == 0
    # a layer of 19 billion weights: some hundred thousand partial sums
    n = 512 * 2048 * 6144
    assert 0 < L.zc_grad_norm_workspace_size(grads(n, n, n), 3, BF) < 1 << 21


def tensors(count=1, n=1000, bits=32, master=False, **over):
    t = (zcmoe.zc_adamw_tensor * count)()
    for i in range(count):
        a = [ptr(8 * i + k) for k in range(7)]
        t[i] = zcmoe.zc_adamw_tensor(a[0], a[1], a[2] if master else None, a[3], a[4],
                                     a[5] if bits == 8 else None, a[6] if bits == 8 else None, n, 0.1)
        for k, v in over.items():
            setattr(t[i], k, v)
    return t


def adamw(t, count=None, factor=None, dev_lr=None, dev_step=None, **over):
    kw = dict(p_dtype=BF, g_dtype=BF, state=0, rounding=0, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1,
              seed=0)
    kw.update(over)
    c = zcmoe.zc_adamw_cfg(*kw.values())
    return zcmoe.lib().zc_adamw_step(C.byref(c), t, len(t) if count is None else count, factor, dev_lr, dev_step,
                                     None)


@pytest.mark.parametrize("kw,code", [
    (dict(p_dtype=2), BAD), (dict(g_dtype=-1), BAD), (dict(p_dtype=F32), UNS),
    (dict(state=2), BAD), (dict(rounding=2), BAD),
    (dict(lr=-1e-3), BAD), (dict(lr=float("nan")), BAD), (dict(lr=float("inf")), BAD),
    (dict(beta1=1.0), BAD), (dict(beta1=-0.1), BAD), (dict(beta2=1.0), BAD), (dict(beta2=float("nan")), BAD),
    (dict(eps=0.0), BAD), (dict(eps=-1e-8), BAD), (dict(eps=1e-60), BAD), (dict(eps=float("inf")), BAD),
    (dict(step=0), BAD), (dict(step=-3), BAD),
])
def test_adamw_bad_settings(kw, code):
    assert adamw(tensors(), **kw) == code and zcmoe.lib().zc_last_error().decode() != ""


def test_adamw_refusals():
    L = zcmoe.lib()
    assert L.zc_adamw_step(None, tensors(), 1, None, None, None, None) == BAD
    assert adamw(NONE, count=1) == BAD
    assert adamw(tensors(), count=-1) == BAD
    assert adamw(tensors(n=-1)) == BAD
    assert adamw(tensors(n=1 << 36)) == UNS
    assert adamw(tensors(weight_decay=float("nan"))) == BAD
    for k in ("p", "g", "m", "v"):
        assert adamw(tensors(**{k: None})) == BAD
        assert adamw(tensors(**{k: ptr(30) + 4})) == BAD
    assert adamw(tensors(bits=8), state=1, dev_step=ptr(90) + 4) == BAD
    for k in ("m_scale", "v_scale"):
        assert adamw(tensors(bits=8, **{k: None}), state=1) == BAD
        assert adamw(tensors(**{k: ptr(30)})) == BAD  # scales of 32-bit states
    assert adamw(tensors(), factor=ptr(90) + 2) == BAD
    assert adamw(tensors(), dev_lr=ptr(90) + 2) == BAD
    # fp32 copies: of bf16 weights, for all tensors or none
    assert adamw(tensors(master=True), p_dtype=F32, g_dtype=F32) == BAD
    t = tensors(2, master=True)
    t[1].master = None
    assert adamw(t) == BAD
    t = tensors(2)
    t[1].master = ptr(60)
    assert adamw(t) == BAD
    t = tensors(3, master=True)
    t[0].n, t[0].master, t[2].master = 0, None, None  # (the first counts for neither)
    assert adamw(t) == BAD


def test_adamw_overlaps():
    assert adamw(tensors(m=ptr(0))) == BAD            # m over p
    assert adamw(tensors(g=ptr(0))) == BAD            # g over p
    assert adamw(tensors(v=ptr(3) + 3984)) == BAD     # v begins inside m
    assert adamw(tensors(), factor=ptr(0) + 4) == BAD  # the factor inside p
    assert adamw(tensors(), dev_lr=ptr(4) + 4) == BAD
    assert adamw(tensors(), dev_step=ptr(3) + 8) == BAD
    # the same tensor twice, and a gradient that is another tensor's weights
    t = tensors(2)
    t[1] = t[0]
    assert adamw(t) == BAD
    t = tensors(70)
    t[69].g = t[3].p
    assert adamw(t) == BAD
    t = tensors(3, bits=8)
    t[2].v_scale = t[0].m_scale
    assert adamw(t, state=1) == BAD


def test_binding_checks():
    f = torch.zeros(4)
    with pytest.raises(ValueError):
        zcmoe.TensorList([f])  # not on the GPU
    with pytest.raises(TypeError):
        zcmoe.TensorList([1.0])
    with pytest.raises(ValueError):
        zcmoe.TensorList([f.double()])
    with pytest.raises(ValueError):
        zcmoe.adamw_tensors([], [], bits=16)
    empty = zcmoe.adamw_tensors([], [])
    zcmoe.zc_adamw_step(zcmoe.AdamW(), empty, 1)  # nothing to do
