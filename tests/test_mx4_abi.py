"""Host-side checks of the MXFP4 calls, before any work is queued."""
import ctypes as C

import pytest
import torch

from moe_layer_zero_amd import zcmoe

A = [C.c_void_p((i + 1) << 40) for i in range(20)]  # distinct, aligned, never dereferenced
BF = torch.bfloat16
BAD, UNS, WS = zcmoe.ZC_ERR_INVALID, zcmoe.ZC_ERR_UNSUPPORTED, zcmoe.ZC_ERR_WORKSPACE


def desc(a=8, **kw):
    base = dict(T=64, d=256, N=8, Z=4, I=128, K=2, dtype=BF, weight_layout=zcmoe.mxfp4_layout(a))
    base.update(kw)
    return zcmoe.LayerDesc(**base)


def test_layouts_and_sizes():
    L = zcmoe.lib()
    for a in (8, 4):
        d = desc(a).c()
        # scales of 256 steps take the room of 512
        assert L.zc_moe_mxfp4_weight_bytes(C.byref(d), 0) == 8 * 128 * 256 // 2 + 8 * 8 * 256
        assert L.zc_moe_mxfp4_weight_bytes(C.byref(d), 1) == 8 * 128 * 256 // 2 + 8 * 16 * 256
        assert L.zc_moe_mxfp4_weight_bytes(C.byref(d), 2) == 0
        big = desc(a, d=6144, I=2048, N=512, Z=256, K=12, T=1).c()
        n = 512 * 6144 * 2048
        assert L.zc_moe_mxfp4_weight_bytes(C.byref(big), 0) == n // 2 + n // 32
        for op in (zcmoe.ZC_OP_FORWARD, zcmoe.ZC_OP_EXPERTS):
            assert L.zc_moe_workspace_size(C.byref(d), op) > 0
    assert L.zc_moe_mxfp4_weight_bytes(C.byref(desc(weight_layout=0).c()), 0) == 0
    for bad in (16, 0, 6):
        with pytest.raises(ValueError):
            zcmoe.mxfp4_layout(bad)


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("kw", [dict(dtype=torch.float32), dict(d=192), dict(I=64)])
def test_unsupported_layers(a, kw):
    L = zcmoe.lib()
    d = desc(a, **kw).c()
    assert L.zc_moe_mxfp4_weight_bytes(C.byref(d), 0) == 0
    assert L.zc_moe_mxfp4_pack(C.byref(d), 0, A[0], A[1], A[2], None) == UNS
    assert L.zc_moe_workspace_size(C.byref(d), zcmoe.ZC_OP_FORWARD) == 0


def test_pack_arguments():
    L = zcmoe.lib()
    f, d = L.zc_moe_mxfp4_pack, desc().c()
    assert f(C.byref(d), 2, A[0], A[1], A[2], None) == BAD
    assert f(None, 0, A[0], A[1], A[2], None) == BAD
    for k in range(3):
        a = [A[0], A[1], A[2]]
        a[k] = None
        assert f(C.byref(d), 0, *a, None) == BAD
        a[k] = C.c_void_p(A[k].value + 8)
        assert f(C.byref(d), 0, *a, None) == BAD
    assert f(C.byref(d), 0, A[0], A[1], A[0], None) == BAD
    assert "overlap" in L.zc_last_error().decode()
    assert f(C.byref(desc(weight_layout=0).c()), 0, A[0], A[1], A[2], None) == BAD


def test_quantize_arguments():
    q = lambda R=4, Cc=64, dt=1, src=A[0], co=A[1], sc=A[2], va=None: \
        zcmoe.lib().zc_mxfp4_quantize(R, Cc, dt, src, co, sc, va, None)  # noqa: E731
    assert q(R=-1) == BAD and q(Cc=0) == BAD and q(dt=2) == BAD
    assert q(Cc=48) == UNS and q(Cc=16) == UNS
    assert q(R=1 << 36, Cc=32) == UNS and q(R=1, Cc=1 << 31) == UNS
    for k in ("src", "co", "sc"):
        assert q(**{k: None}) == BAD
        assert q(**{k: C.c_void_p((1 << 30) + 4)}) == BAD
    assert q(va=C.c_void_p((1 << 30) + 4)) == BAD
    assert q(co=A[0]) == BAD and q(sc=A[1]) == BAD and q(va=A[1]) == BAD
    assert q(va=C.c_void_p(A[0].value + 16)) == BAD  # in place is the very buffer


def test_serves_inference_only():
    L = zcmoe.lib()
    for a in (8, 4):
        d = desc(a).c()
        r = zcmoe.zc_route_buf(*A[:7])
        st = L.zc_moe_forward(C.byref(d), *A[7:14], C.byref(r), A[14], A[15], 1 << 39, None)
        assert st == UNS and "row-major" in L.zc_last_error().decode()
        st = L.zc_moe_backward(C.byref(d), *A[7:12], C.byref(r), *A[12:19], None, A[19], 1 << 39, None)
        assert st == UNS


@pytest.mark.parametrize("a", [8, 4])
def test_experts_arguments(a):
    d = desc(a)
    ok = dict(x=A[7], wg=A[8], wu=A[9], wd=A[10], xc=None, xs=None, out=A[11], ws=A[12])

    def experts(ws_bytes=1 << 30, **over):
        v = {**ok, **over}
        c, r = d.c(), zcmoe.zc_route_buf(None, A[0], A[1], None, A[2], A[3], A[4])
        return zcmoe.lib().zc_moe_experts(C.byref(c), v["x"], C.byref(r), v["wg"], v["wu"], v["wd"], v["xc"],
                                          v["xs"], v["out"], v["ws"], ws_bytes, None)

    for k in ("x", "wg", "wu", "wd", "out"):
        assert experts(**{k: None}) == BAD, k
    need = zcmoe.zc_moe_workspace_size(d, zcmoe.ZC_OP_EXPERTS)
    assert experts(ws_bytes=need - 1) == WS
    assert experts(xc=A[13]) == BAD and experts(xs=A[13]) == BAD
    rows = 64 * 256 // (2 if a == 4 else 1)  # bytes of x's codes
    assert experts(xc=A[13], xs=A[14], out=C.c_void_p(A[13].value + rows - 16)) == BAD
    gu = zcmoe.lib().zc_moe_mxfp4_weight_bytes(C.byref(d.c()), 0)
    assert experts(out=C.c_void_p(A[8].value + gu - 16)) == BAD
    assert experts(ws=C.c_void_p(A[10].value + gu)) == BAD  # w_down's set is larger here: inside it


def test_bindings_reject():
    d = desc()
    w = torch.zeros((8, 128, 256), dtype=BF)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for bad in (lambda: zcmoe.zc_mxfp4_quantize(w.double()), lambda: zcmoe.zc_mxfp4_quantize(w[..., :48]),
                lambda: zcmoe.zc_mxfp4_quantize(torch.zeros((), dtype=BF)),
                lambda: zcmoe.zc_mxfp4_quantize(w, codes=u8(8, 128, 128), scales=u8(8, 128, 8)),  # host tensors
                lambda: zcmoe.mxfp4_expert_weights(desc(weight_layout=0), w, w, w),
                lambda: zcmoe.mxfp4_expert_weights(d, w.transpose(1, 2), w, w),
                lambda: zcmoe.zc_moe_mxfp4_pack(d, 0, u8(8, 128, 128), u8(8, 128, 8), u8(16)),
                lambda: zcmoe.zc_moe_mxfp4_pack(d, 1, u8(8, 128, 128), u8(8, 128, 8)),
                lambda: zcmoe.zc_moe_experts(d, torch.zeros((64, 256), dtype=BF), zcmoe.RouteBuffers(d, "cpu"),
                                             w, w, w, torch.zeros((64, 256), dtype=BF))):
        with pytest.raises(ValueError):
            bad()
