"""Host-side checks of the sequence balance loss and of the backward's score
gradient, before any work is queued."""
import ctypes as C

import pytest
import torch

from moe_layer_zero_amd import zcmoe

A = [C.c_void_p((i + 1) << 32) for i in range(20)]  # distinct, aligned, never dereferenced


def call(desc=None, cfg=(4, 1.5, 0.1), S=3, ws_bytes=1 << 31, **over):
    L = zcmoe.lib()
    desc = desc or zcmoe.LayerDesc(64, 128, 8, 4, 64, 2, torch.float32)
    a = dict(logits=A[0], idx=A[1], cu=A[2], mask=A[3], loss=A[4], counts=A[5], dl=A[6], ws=A[7],
             r=True)
    a.update(over)
    r = zcmoe.zc_route_buf(logits=a["logits"], topk_idx=a["idx"])
    d, c = desc.c(), zcmoe.zc_lb_cfg(*cfg)
    return L.zc_moe_seq_balance(C.byref(d), C.byref(c), C.byref(r) if a["r"] else None, S, a["cu"],
                                a["mask"], a["loss"], a["counts"], a["dl"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("cfg", [(3, 1.5, 0.1), (0, 1.5, 0.1), (4, 2.0, 0.1), (4, 0.0, 0.1),
                                 (4, float("nan"), 0.1), (4, 1.5, float("inf"))])
def test_bad_settings(cfg):
    assert call(cfg=cfg) == zcmoe.ZC_ERR_INVALID


def test_pointers_sequences_and_workspace():
    for k in ("r", "logits", "idx", "loss", "counts"):
        assert call(**{k: None}) == zcmoe.ZC_ERR_INVALID, k
    assert call(S=0) == zcmoe.ZC_ERR_INVALID
    assert call(S=(1 << 20) + 1) == zcmoe.ZC_ERR_INVALID
    assert call(S=3, cu=None) == zcmoe.ZC_ERR_INVALID      # several sequences need offsets
    assert call(ws=None) == zcmoe.ZC_ERR_WORKSPACE
    desc = zcmoe.LayerDesc(64, 128, 8, 4, 64, 2, torch.float32)
    d = desc.c()
    need = zcmoe.lib().zc_moe_seq_balance_workspace_size(C.byref(d), 3)
    assert need > 0 and call(ws_bytes=need - 1) == zcmoe.ZC_ERR_WORKSPACE
    assert zcmoe.lib().zc_moe_seq_balance_workspace_size(C.byref(d), 0) == 0
    big = zcmoe.LayerDesc((1 << 25) + 1, 128, 8, 4, 64, 2, torch.float32)
    assert call(big, ws_bytes=1 << 40) == zcmoe.ZC_ERR_UNSUPPORTED
    assert call(mask=C.c_void_p((1 << 32) + 4)) == zcmoe.ZC_ERR_INVALID
    # no output over an input or another output
    for k, at in (("loss", 0), ("counts", 1), ("dl", 0), ("ws", 2), ("dl", 5), ("counts", 4)):
        assert call(**{k: A[at]}) == zcmoe.ZC_ERR_INVALID, k
        assert "overlaps" in zcmoe.lib().zc_last_error().decode()


def test_backward_with_scores_checks_its_gradient():
    L = zcmoe.lib()
    d = zcmoe.LayerDesc(64, 128, 8, 4, 64, 2, torch.float32).c()
    r = zcmoe.zc_route_buf(*A[:7])
    st = L.zc_moe_backward_scores(C.byref(d), *A[:5], C.byref(r), *A[5:12], None,
                                  C.c_void_p((1 << 32) + 4), A[12], 1 << 40, None)
    assert st == zcmoe.ZC_ERR_INVALID and "dlogits" in L.zc_last_error().decode()


def test_binding_rejects():
    desc = zcmoe.LayerDesc(6, 64, 8, 4, 64, 2)
    r = zcmoe.RouteBuffers(desc, device="cpu")
    lb = zcmoe.LoadBalance(4, 1.5, 0.1)
    with pytest.raises(ValueError):   # host tensors
        zcmoe.zc_moe_seq_balance(desc, lb, r, torch.empty(2), torch.empty((1, 12), dtype=torch.int32))
    with pytest.raises(ValueError):   # counts of the wrong type
        zcmoe.zc_moe_seq_balance(desc, lb, r, torch.empty(2), torch.empty((1, 12)))
