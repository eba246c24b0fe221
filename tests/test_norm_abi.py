"""Host-side checks of the RMS norm calls, before any work is queued."""
import ctypes as C

import pytest
import torch

from moe_layer_zero_amd import zcmoe

A = [C.c_void_p((i + 1) << 30) for i in range(10)]  # distinct, aligned, never dereferenced
BF, F32 = torch.bfloat16, torch.float32


def fwd(L, desc, **over):
    a = dict(x=A[0], res=A[1], gamma=A[2], r=A[3], y=A[4], rstd=A[5], codes=None, scales=None)
    a.update(over)
    d = desc.c() if desc is not None else None
    return L.zc_rmsnorm_forward(C.byref(d) if d is not None else None, a["x"], a["res"], a["gamma"],
                                a["r"], a["y"], a["rstd"], a["codes"], a["scales"], None)


def bwd(L, desc, ws_bytes=1 << 29, **over):
    a = dict(dy=A[0], r=A[1], gamma=A[2], rstd=A[3], dres=A[4], dr=A[5], dgamma=A[6], ws=A[7])
    a.update(over)
    d = desc.c()
    return L.zc_rmsnorm_backward(C.byref(d), a["dy"], a["r"], a["gamma"], a["rstd"], a["dres"],
                                 a["dr"], a["dgamma"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), zcmoe.ZC_ERR_INVALID),
    (dict(d=0), zcmoe.ZC_ERR_INVALID),
    (dict(eps=0.0), zcmoe.ZC_ERR_INVALID),
    (dict(eps=float("nan")), zcmoe.ZC_ERR_INVALID),
    (dict(eps=float("inf")), zcmoe.ZC_ERR_INVALID),
    (dict(d=12), zcmoe.ZC_ERR_UNSUPPORTED),
    (dict(d=10, dtype=F32), zcmoe.ZC_ERR_UNSUPPORTED),
    (dict(d=32776), zcmoe.ZC_ERR_UNSUPPORTED),
    (dict(T=1 << 31), zcmoe.ZC_ERR_UNSUPPORTED),
])
def test_bad_norm_descriptions(kw, code):
    L = zcmoe.lib()
    base = dict(T=4, d=256, dtype=BF)
    base.update(kw)
    desc = zcmoe.NormDesc(**base)
    assert fwd(L, desc) == code and L.zc_last_error().decode() != ""
    assert bwd(L, desc) == code
    d = desc.c()
    assert L.zc_rmsnorm_workspace_size(C.byref(d)) == 0


def test_norm_pointer_checks():
    L = zcmoe.lib()
    desc = zcmoe.NormDesc(4, 256, BF)
    assert fwd(L, None) == zcmoe.ZC_ERR_INVALID
    for k in ("x", "gamma", "y"):
        assert fwd(L, desc, **{k: None}) == zcmoe.ZC_ERR_INVALID
    assert fwd(L, desc, x=C.c_void_p((1 << 30) + 8)) == zcmoe.ZC_ERR_INVALID
    for k in ("dy", "r", "gamma", "rstd", "dr", "dgamma"):
        assert bwd(L, desc, **{k: None}) == zcmoe.ZC_ERR_INVALID
    # codes and scales come together, on bf16 rows of whole groups of 128
    assert fwd(L, desc, codes=A[6]) == zcmoe.ZC_ERR_INVALID
    assert fwd(L, zcmoe.NormDesc(4, 256, F32), codes=A[6], scales=A[7]) == zcmoe.ZC_ERR_UNSUPPORTED
    assert fwd(L, zcmoe.NormDesc(4, 192, BF), codes=A[6], scales=A[7]) == zcmoe.ZC_ERR_UNSUPPORTED
    d = desc.c()
    need = L.zc_rmsnorm_workspace_size(C.byref(d))
    assert need >= 256 * 4  # one row of partial sums at least
    assert bwd(L, desc, ws_bytes=need - 1) == zcmoe.ZC_ERR_WORKSPACE
    assert bwd(L, desc, ws=None) == zcmoe.ZC_ERR_WORKSPACE


def test_norm_overlap_checks():
    L = zcmoe.lib()
    desc = zcmoe.NormDesc(4, 256, BF)
    near = C.c_void_p((1 << 30) + 512)  # one row further: not the very same buffer
    assert fwd(L, desc, r=A[4], y=A[4]) == zcmoe.ZC_ERR_INVALID       # two outputs
    assert fwd(L, desc, y=near) == zcmoe.ZC_ERR_INVALID
    assert fwd(L, desc, r=near) == zcmoe.ZC_ERR_INVALID
    assert fwd(L, desc, rstd=A[0]) == zcmoe.ZC_ERR_INVALID
    assert fwd(L, desc, y=A[2]) == zcmoe.ZC_ERR_INVALID               # gamma is not in place
    assert fwd(L, desc, codes=A[0], scales=A[7]) == zcmoe.ZC_ERR_INVALID
    assert bwd(L, desc, dr=near) == zcmoe.ZC_ERR_INVALID
    assert bwd(L, desc, ws=A[1]) == zcmoe.ZC_ERR_INVALID
    assert bwd(L, desc, dgamma=A[5]) == zcmoe.ZC_ERR_INVALID
    assert "overlaps" in L.zc_last_error().decode()


def test_norm_binding_rejects():
    desc = zcmoe.NormDesc(4, 256, BF)
    x, g = torch.zeros(4, 256, dtype=BF), torch.ones(256, dtype=BF)
    with pytest.raises(ValueError):
        zcmoe.zc_rmsnorm_forward(desc, x, g, torch.empty_like(x))      # host tensors
    with pytest.raises(ValueError):
        zcmoe.zc_rmsnorm_forward(desc, x[:3], g, torch.empty_like(x))  # shape
    with pytest.raises(ValueError):
        zcmoe.zc_rmsnorm_forward(desc, x.float(), g, torch.empty_like(x))
    with pytest.raises(ValueError):
        zcmoe.zc_rmsnorm_forward(zcmoe.NormDesc(4, 256, torch.float16), x, g, x)
