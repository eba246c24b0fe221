"""Python binding of libzcmoe (include/zc_moe.h): argument marshalling only.

Every step of the layer runs in the HIP library; this module turns torch
tensors into the device pointers, sizes and the stream handle the C ABI
takes, checks dtypes, shapes and devices before the call, and raises
ZcError on any non-OK status.  PyTorch supplies device memory and streams.
There is no fallback: if the library is not built, loading it raises.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libzcmoe.so")

ZC_OK, ZC_ERR_INVALID, ZC_ERR_UNSUPPORTED, ZC_ERR_WORKSPACE, ZC_ERR_HIP = range(5)
ZC_F32, ZC_BF16 = 0, 1
ZC_OP_ROUTE, ZC_OP_FORWARD, ZC_OP_BACKWARD, ZC_OP_LB_LOSS, ZC_OP_ROUTE_STATS = 0, 1, 2, 3, 4
ZC_OP_EXPERTS = 5
ZC_WEIGHTS_ROWMAJOR, ZC_WEIGHTS_PACKED, ZC_WEIGHTS_MXFP8 = 0, 1, 2
ZC_WEIGHTS_INT4_G32, ZC_WEIGHTS_INT4_G64, ZC_WEIGHTS_INT4_G128 = 4, 5, 6
ZC_WEIGHTS_MXFP4_A8, ZC_WEIGHTS_MXFP4_A4 = 8, 9
ZC_PACK_GATE_UP, ZC_PACK_DOWN = 0, 1
ZC_STATE_F32, ZC_STATE_8BIT = 0, 1
ZC_ROUND_NEAREST, ZC_ROUND_STOCHASTIC = 0, 1
STATE_BLOCK = 128  # values that share a scale of the 8-bit states

# Every symbol include/zc_moe.h declares.
EXPORTS = ("zc_moe_workspace_size", "zc_moe_saved_size", "zc_moe_route", "zc_moe_forward",
           "zc_moe_forward_noalloc", "zc_moe_backward", "zc_moe_lb_loss", "zc_moe_route_stats", "zc_moe_accumulate_counts",
           "zc_moe_pid_update", "zc_moe_pack_weights", "zc_moe_quantized_weight_bytes",
           "zc_moe_quantize_weights",
           "zc_moe_backward_scores", "zc_moe_seq_balance_workspace_size", "zc_moe_seq_balance",
           "zc_moe_experts", "zc_moe_int4_weight_bytes", "zc_moe_int4_quantize",
           "zc_moe_int4_pack",
           "zc_mxfp4_quantize", "zc_moe_mxfp4_weight_bytes", "zc_moe_mxfp4_pack",
           "zc_rmsnorm_forward", "zc_rmsnorm_workspace_size", "zc_rmsnorm_backward",
           "zc_grad_norm_workspace_size", "zc_grad_norm", "zc_adamw_step",
           "zc_moe_profile",
           "zc_moe_profile_read",
           "zc_moe_phase_name", "zc_status_string", "zc_last_error")
ZC_NUM_PHASES = 27


class ZcError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status}: {detail}")
        self.status = status


class zc_moe_desc(C.Structure):
    _fields_ = [("T", C.c_int64), ("d", C.c_int64), ("N", C.c_int64), ("Z", C.c_int64),
                ("I", C.c_int64), ("K", C.c_int64), ("dtype", C.c_int32),
                ("gate_norm", C.c_int32), ("out_scale", C.c_float),
                ("weight_layout", C.c_int32), ("cu_limit", C.c_int32)]


class zc_lb_cfg(C.Structure):
    _fields_ = [("D", C.c_int64), ("K_e", C.c_double), ("alpha", C.c_double)]


class zc_route_buf(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("topk_idx", C.c_void_p), ("topk_gate", C.c_void_p),
                ("counts", C.c_void_p), ("offsets", C.c_void_p), ("perm", C.c_void_p),
                ("inv", C.c_void_p)]


class zc_norm_desc(C.Structure):
    _fields_ = [("T", C.c_int64), ("d", C.c_int64), ("dtype", C.c_int32), ("eps", C.c_float)]


class zc_grad_tensor(C.Structure):
    _fields_ = [("g", C.c_void_p), ("n", C.c_int64)]


class zc_adamw_tensor(C.Structure):
    _fields_ = [("p", C.c_void_p), ("g", C.c_void_p), ("master", C.c_void_p), ("m", C.c_void_p),
                ("v", C.c_void_p), ("m_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("n", C.c_int64), ("weight_decay", C.c_double)]


class zc_adamw_cfg(C.Structure):
    _fields_ = [("p_dtype", C.c_int32), ("g_dtype", C.c_int32), ("state", C.c_int32),
                ("rounding", C.c_int32), ("lr", C.c_double), ("beta1", C.c_double),
                ("beta2", C.c_double), ("eps", C.c_double), ("step", C.c_int64),
                ("seed", C.c_uint32)]


_LIB = None


def lib() -> C.CDLL:
    """Load libzcmoe.so; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m moe_layer_zero_amd.build` (no fallback path exists)")
        L = C.CDLL(LIB_PATH)
        P, D = C.POINTER(zc_moe_desc), C.POINTER(zc_route_buf)
        v, i64, sz = C.c_void_p, C.c_int64, C.c_size_t
        L.zc_moe_workspace_size.argtypes = [P, C.c_int]
        L.zc_moe_workspace_size.restype = sz
        L.zc_moe_saved_size.argtypes = [P]
        L.zc_moe_saved_size.restype = sz
        L.zc_moe_route.argtypes = [P, v, v, v, D, v, sz, v]
        L.zc_moe_forward.argtypes = [P, v, v, v, v, v, v, v, D, v, v, sz, v]
        L.zc_moe_forward_noalloc.argtypes = [P, v, v, v, v, v, v, v, D, v]
        LB = C.POINTER(zc_lb_cfg)
        L.zc_moe_backward.argtypes = [P, v, v, v, v, v, D, v, v, v, v, v, v, v, LB, v, sz, v]
        L.zc_moe_lb_loss.argtypes = [P, LB, D, v, v, sz, v]
        L.zc_moe_route_stats.argtypes = [P, D, v, v, v, sz, v]
        L.zc_moe_accumulate_counts.argtypes = [i64, v, v, v]
        L.zc_moe_pid_update.argtypes = [i64, i64, i64, v, i64, C.c_double, C.c_double, v, v]
        L.zc_moe_pack_weights.argtypes = [P, C.c_int, v, v, v]
        L.zc_moe_quantized_weight_bytes.argtypes = [P]
        L.zc_moe_quantized_weight_bytes.restype = sz
        L.zc_moe_quantize_weights.argtypes = [P, C.c_int, v, v, v]
        L.zc_moe_backward_scores.argtypes = [P, v, v, v, v, v, D, v, v, v, v, v, v, v, LB, v, v, sz,
                                             v]
        L.zc_moe_seq_balance_workspace_size.argtypes = [P, i64]
        L.zc_moe_seq_balance_workspace_size.restype = sz
        L.zc_moe_seq_balance.argtypes = [P, LB, D, i64, v, v, v, v, v, v, sz, v]
        L.zc_moe_experts.argtypes = [P, v, D, v, v, v, v, v, v, v, sz, v]
        L.zc_moe_int4_weight_bytes.argtypes = [P]
        L.zc_moe_int4_weight_bytes.restype = sz
        L.zc_moe_int4_quantize.argtypes = [P, C.c_int, v, v, v, v]
        L.zc_moe_int4_pack.argtypes = [P, C.c_int, v, v, v, v]
        L.zc_mxfp4_quantize.argtypes = [i64, i64, C.c_int, v, v, v, v, v]
        L.zc_moe_mxfp4_weight_bytes.argtypes = [P, C.c_int]
        L.zc_moe_mxfp4_weight_bytes.restype = sz
        L.zc_moe_mxfp4_pack.argtypes = [P, C.c_int, v, v, v, v]
        NP = C.POINTER(zc_norm_desc)
        L.zc_rmsnorm_forward.argtypes = [NP, v, v, v, v, v, v, v, v, v]
        L.zc_rmsnorm_workspace_size.argtypes = [NP]
        L.zc_rmsnorm_workspace_size.restype = sz
        L.zc_rmsnorm_backward.argtypes = [NP, v, v, v, v, v, v, v, v, sz, v]
        GT = C.POINTER(zc_grad_tensor)
        L.zc_grad_norm_workspace_size.argtypes = [GT, i64, C.c_int]
        L.zc_grad_norm_workspace_size.restype = sz
        L.zc_grad_norm.argtypes = [GT, i64, C.c_int, C.c_double, v, v, v, sz, v]
        L.zc_adamw_step.argtypes = [C.POINTER(zc_adamw_cfg), C.POINTER(zc_adamw_tensor), i64, v, v, v,
                                    v]
        for f in ("zc_grad_norm", "zc_adamw_step", "zc_mxfp4_quantize", "zc_moe_mxfp4_pack", "zc_moe_experts", "zc_moe_int4_quantize", "zc_moe_int4_pack",
                  "zc_moe_backward_scores", "zc_moe_seq_balance", "zc_rmsnorm_forward", "zc_rmsnorm_backward",
                  "zc_moe_route", "zc_moe_forward", "zc_moe_forward_noalloc",
                  "zc_moe_backward", "zc_moe_lb_loss",
                  "zc_moe_route_stats", "zc_moe_accumulate_counts", "zc_moe_pid_update",
                  "zc_moe_pack_weights", "zc_moe_quantize_weights"):
            getattr(L, f).restype = C.c_int
        L.zc_moe_profile.argtypes = [C.c_int]
        L.zc_moe_profile.restype = C.c_int
        L.zc_moe_profile_read.argtypes = [C.POINTER(C.c_double), C.POINTER(C.c_int32)]
        L.zc_moe_profile_read.restype = C.c_int
        L.zc_moe_phase_name.argtypes = [C.c_int]
        L.zc_moe_phase_name.restype = C.c_char_p
        L.zc_status_string.argtypes = [C.c_int]
        L.zc_status_string.restype = C.c_char_p
        L.zc_last_error.argtypes = []
        L.zc_last_error.restype = C.c_char_p
        _LIB = L
    return _LIB


def _check(status: int, where: str) -> None:
    if status != ZC_OK:
        raise ZcError(status, where, lib().zc_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensors passed to the HIP library must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the HIP library must be contiguous")
    return C.c_void_p(t.data_ptr())


class _Args:
    """Device addresses of one call's tensors, checked: shape, dtype, contiguity,
    and that all of them live on one GPU.  (Calls of a few microseconds go
    through here, so it touches each tensor as little as it can.)"""
    __slots__ = ("where", "dev")

    def __init__(self, where):
        self.where, self.dev = where, None

    def __call__(self, t, shape, dtype, name):
        if t is None:
            return None
        if t.shape != shape or t.dtype != dtype:
            _check_layer_tensor(t, shape, dtype, name)
        dev = t.get_device()
        if dev != self.dev:
            if dev < 0:
                raise ValueError("tensors passed to the HIP library must live on the GPU")
            if self.dev is not None:
                raise ValueError(f"{self.where}: {name} is on GPU {dev}, other tensors on GPU {self.dev}")
            self.dev = dev
        if not t.is_contiguous():
            raise ValueError("tensors passed to the HIP library must be contiguous")
        return t.data_ptr()

    def run(self, fn, *args, stream=None):
        """fn(*args, stream) with the tensors' device current.  The default
        stream is that device's current one."""
        if stream is None:
            handle = torch._C._cuda_getCurrentRawStream(self.dev)  # the handle alone
        elif stream.device_index != self.dev:
            raise ValueError(f"{self.where}: stream of GPU {stream.device_index}, tensors on GPU {self.dev}")
        else:
            handle = stream.cuda_stream
        if torch.cuda.current_device() == self.dev:
            st = fn(*args, handle)
        else:
            with torch.cuda.device(self.dev):
                st = fn(*args, handle)
        if st != ZC_OK:
            _check(st, self.where)


def _call(where, t, stream, fn, *args):
    """fn(*args, stream), as _Args.run, for the GPU of tensor t (the library
    refuses the call if there is none)."""
    a = _Args(where)
    a.dev = torch.cuda.current_device() if t is None else t.get_device()
    a.run(fn, *args, stream=stream)


def _alloc(stream, make, *args, **kw):
    """make(*args, **kw), its memory taken from the stream that will use it: a
    block of another stream's may still be in use there, and goes back to that
    stream, not to this one, when it is dropped.  (So it is with everything that
    a call here allocates, outputs too.)"""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _aligned(stream, t):
    """t, or a copy of it (made on the call's stream) where it does not start at a
    multiple of 16 bytes, as the library wants it: a slice of a larger batch."""
    return t if t is None or t.data_ptr() % 16 == 0 else _alloc(stream, torch.clone, t)


@dataclass
class LayerDesc:
    T: int
    d: int
    N: int
    Z: int
    I: int
    K: int
    dtype: torch.dtype = torch.bfloat16
    gate_norm: int = 1
    out_scale: float = 1.0
    weight_layout: int = ZC_WEIGHTS_ROWMAJOR
    cu_limit: int = 0

    @property
    def E(self) -> int:
        return self.N + self.Z

    def c(self) -> zc_moe_desc:
        if self.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("layer dtype must be float32 or bfloat16")
        return zc_moe_desc(self.T, self.d, self.N, self.Z, self.I, self.K,
                           ZC_F32 if self.dtype == torch.float32 else ZC_BF16,
                           self.gate_norm, self.out_scale, self.weight_layout,
                           self.cu_limit)


class RouteBuffers:
    """Device buffers of zc_route_buf, allocated with torch."""

    def __init__(self, desc: LayerDesc, device="cuda"):
        T, E, N, K = desc.T, desc.E, desc.N, desc.K
        i32 = torch.int32
        self.logits = torch.empty((T, E), dtype=torch.float32, device=device)
        self.topk_idx = torch.empty((T, K), dtype=i32, device=device)
        self.topk_gate = torch.empty((T, K), dtype=torch.float32, device=device)
        self.counts = torch.empty(E, dtype=i32, device=device)
        self.offsets = torch.empty(N + 1, dtype=i32, device=device)
        self.perm = torch.empty(max(T * K, 1), dtype=i32, device=device)
        self.inv = torch.empty(max(T * K, 1), dtype=i32, device=device)

    def c(self) -> zc_route_buf:
        return zc_route_buf(*(_ptr(getattr(self, f)) for f, _ in zc_route_buf._fields_))


def zc_moe_workspace_size(desc: LayerDesc, op: int) -> int:
    d = desc.c()
    return int(lib().zc_moe_workspace_size(C.byref(d), op))


def zc_moe_saved_size(desc: LayerDesc) -> int:
    d = desc.c()
    return int(lib().zc_moe_saved_size(C.byref(d)))


def workspace(desc: LayerDesc, op: int, device="cuda") -> torch.Tensor:
    n = zc_moe_workspace_size(desc, op)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def saved_buffer(desc: LayerDesc, device="cuda") -> torch.Tensor:
    return torch.empty(max(zc_moe_saved_size(desc), 256), dtype=torch.uint8, device=device)


def saved_views(desc: LayerDesc, saved: torch.Tensor) -> dict:
    """Views of a filled saved buffer (its layout is the one zc_moe_saved_size
    documents): a, u, h fp32 [T*K][I] and y [T*K][d] in the layer dtype,
    rows in dispatch order."""
    rows, I, d = desc.T * desc.K, desc.I, desc.d
    a256 = lambda n: (n + 255) // 256 * 256  # noqa: E731
    piece = a256(rows * I * 4)
    out = {}
    for i, k in enumerate(("a", "u", "h")):
        out[k] = saved[i * piece:i * piece + rows * I * 4].view(torch.float32).view(rows, I)
    es = 4 if desc.dtype == torch.float32 else 2
    out["y"] = saved[3 * piece:3 * piece + rows * d * es].view(desc.dtype).view(rows, d)
    return out


def _check_layer_tensor(t, shape, dtype, name):
    if t is None:
        return
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")


def int4_layout(G: int) -> int:
    """Weight layout of 4-bit weights with groups of G (32, 64 or 128)."""
    try:
        return {32: ZC_WEIGHTS_INT4_G32, 64: ZC_WEIGHTS_INT4_G64, 128: ZC_WEIGHTS_INT4_G128}[G]
    except KeyError:
        raise ValueError(f"groups of {G}: 32, 64 or 128 are supported") from None


def int4_group(desc: LayerDesc) -> int:
    """Group size of desc's 4-bit weight layout, 0 for the other layouts."""
    return {ZC_WEIGHTS_INT4_G32: 32, ZC_WEIGHTS_INT4_G64: 64,
            ZC_WEIGHTS_INT4_G128: 128}.get(desc.weight_layout, 0)


def mxfp4_layout(row_bits: int) -> int:
    """Weight layout of MXFP4 weights whose rows are MXFP8 (8) or MXFP4 (4)."""
    try:
        return {8: ZC_WEIGHTS_MXFP4_A8, 4: ZC_WEIGHTS_MXFP4_A4}[row_bits]
    except KeyError:
        raise ValueError(f"rows of {row_bits} bits: 8 or 4 are supported") from None


def _is_mxfp4(desc: LayerDesc) -> bool:
    return desc.weight_layout in (ZC_WEIGHTS_MXFP4_A8, ZC_WEIGHTS_MXFP4_A4)


def _check_weights(desc, w_router, w_gate, w_up, w_down):
    dt = desc.dtype
    _check_layer_tensor(w_router, (desc.E, desc.d), dt, "w_router")
    if desc.weight_layout == ZC_WEIGHTS_MXFP8 or int4_group(desc) or _is_mxfp4(desc):
        d = desc.c()
        if _is_mxfp4(desc):
            sizes = [int(lib().zc_moe_mxfp4_weight_bytes(C.byref(d), w))
                     for w in (ZC_PACK_GATE_UP, ZC_PACK_GATE_UP, ZC_PACK_DOWN)]
        else:
            size = lib().zc_moe_int4_weight_bytes if int4_group(desc) else lib().zc_moe_quantized_weight_bytes
            sizes = [int(size(C.byref(d)))] * 3
        for t, name, n in zip((w_gate, w_up, w_down), ("w_gate", "w_up", "w_down"), sizes):
            if t is not None and (t.dtype != torch.uint8 or t.numel() < n):
                raise ValueError(f"{name}: expected a quantized weight set of {n} uint8")
        return
    _check_layer_tensor(w_gate, (desc.N, desc.I, desc.d), dt, "w_gate")
    _check_layer_tensor(w_up, (desc.N, desc.I, desc.d), dt, "w_up")
    _check_layer_tensor(w_down, (desc.N, desc.d, desc.I), dt, "w_down")


def zc_moe_route(desc: LayerDesc, x, w_router, bias, route: RouteBuffers, ws=None, stream=None):
    """Router + dispatch.  x = w_router = None routes the scores already in
    route.logits."""
    if x is not None:
        _check_layer_tensor(x, (desc.T, desc.d), desc.dtype, "x")
        _check_weights(desc, w_router, None, None, None)
    _check_layer_tensor(bias, (desc.E,), torch.float32, "bias")
    if ws is None:
        ws = _alloc(stream, workspace, desc, ZC_OP_ROUTE, bias.device)
    d, r = desc.c(), route.c()
    _call("zc_moe_route", bias, stream, lib().zc_moe_route, C.byref(d), _ptr(x), _ptr(w_router),
          _ptr(bias), C.byref(r), _ptr(ws), ws.numel())


def zc_moe_forward(desc: LayerDesc, x, w_router, bias, w_gate, w_up, w_down, out,
                   route: RouteBuffers, saved=None, ws=None, stream=None):
    _check_layer_tensor(x, (desc.T, desc.d), desc.dtype, "x")
    _check_layer_tensor(out, (desc.T, desc.d), desc.dtype, "out")
    _check_layer_tensor(bias, (desc.E,), torch.float32, "bias")
    _check_weights(desc, w_router, w_gate, w_up, w_down)
    if ws is None:
        ws = _alloc(stream, workspace, desc, ZC_OP_FORWARD, x.device)
    d, r = desc.c(), route.c()
    _call("zc_moe_forward", bias, stream, lib().zc_moe_forward, C.byref(d), _ptr(x), _ptr(w_router),
          _ptr(bias), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(out), C.byref(r), _ptr(saved),
          _ptr(ws), ws.numel())


def zc_moe_experts(desc: LayerDesc, x, route: RouteBuffers, w_gate, w_up, w_down, out, xq=None,
                   ws=None, stream=None):
    """The experts and the combine on routing that zc_moe_route left in route.
    xq: (codes, scales) of x, from zc_rmsnorm_forward for MXFP8 and MXFP4_A8 weights,
    from zc_mxfp4_quantize for MXFP4_A4 weights."""
    T, K, N, dt = desc.T, desc.K, desc.N, desc.dtype
    a, sh, i32, u8 = _Args("zc_moe_experts"), (desc.T, desc.d), torch.int32, torch.uint8
    px, po = a(x, sh, dt, "x"), a(out, sh, dt, "out")
    r = zc_route_buf(topk_idx=a(route.topk_idx, (T, K), i32, "route.topk_idx"),
                     topk_gate=a(route.topk_gate, (T, K), torch.float32, "route.topk_gate"),
                     offsets=a(route.offsets, (N + 1,), i32, "route.offsets"),
                     perm=a(route.perm, (max(T * K, 1),), i32, "route.perm"),
                     inv=a(route.inv, (max(T * K, 1),), i32, "route.inv"))
    _check_weights(desc, None, w_gate, w_up, w_down)
    w = [None if t is None else a(t, t.shape, t.dtype, n)
         for t, n in ((w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down"))]
    cols = desc.d // 2 if desc.weight_layout == ZC_WEIGHTS_MXFP4_A4 else desc.d
    codes, scales = (None, None) if xq is None else (
        a(xq[0], (T, cols), u8, "xq codes"), a(xq[1], (T, desc.d // 32), u8, "xq scales"))
    if ws is None:
        ws = _alloc(stream, workspace, desc, ZC_OP_EXPERTS, x.device)
    n = ws.numel() * ws.element_size()
    a.run(lib().zc_moe_experts, C.byref(desc.c()), px, C.byref(r), *w, codes, scales, po,
          a(ws, ws.shape, ws.dtype, "ws"), n, stream=stream)


NOALLOC_SCRATCH_BYTES = 64 << 20  # ZC_NOALLOC_SCRATCH_BYTES


def zc_moe_forward_noalloc(desc: LayerDesc, x, w_router, bias, w_gate, w_up, w_down, out,
                           route: RouteBuffers, stream=None):
    """The inference forward on the library's own per-device scratch (no
    workspace argument, nothing allocated); rejects layers whose forward
    workspace exceeds NOALLOC_SCRATCH_BYTES."""
    _check_layer_tensor(x, (desc.T, desc.d), desc.dtype, "x")
    _check_layer_tensor(out, (desc.T, desc.d), desc.dtype, "out")
    _check_layer_tensor(bias, (desc.E,), torch.float32, "bias")
    _check_weights(desc, w_router, w_gate, w_up, w_down)
    d, r = desc.c(), route.c()
    _call("zc_moe_forward_noalloc", bias, stream, lib().zc_moe_forward_noalloc, C.byref(d), _ptr(x),
          _ptr(w_router), _ptr(bias), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(out), C.byref(r))


@dataclass
class LoadBalance:
    """Device-level load-balance loss settings: D groups of N/D consecutive
    FFN experts, expected FFN experts per token K_e, balance factor alpha."""
    D: int
    K_e: float
    alpha: float

    def c(self) -> zc_lb_cfg:
        return zc_lb_cfg(int(self.D), float(self.K_e), float(self.alpha))


def zc_moe_backward(desc: LayerDesc, x, w_router, w_gate, w_up, w_down, route: RouteBuffers,
                    saved, dout, dx, dw_router, dw_gate, dw_up, dw_down, ws=None, stream=None,
                    lb: "LoadBalance | None" = None, dlogits=None):
    """All gradients of the layer.  lb adds the device-level load-balance
    loss; dlogits (fp32 [T][E], from zc_moe_seq_balance or the caller's own
    loss) is added to the gradient of the router scores."""
    for t, n in ((x, "x"), (dout, "dout"), (dx, "dx")):
        _check_layer_tensor(t, (desc.T, desc.d), desc.dtype, n)
    _check_weights(desc, w_router, w_gate, w_up, w_down)
    _check_weights(desc, dw_router, dw_gate, dw_up, dw_down)
    if ws is None:
        ws = _alloc(stream, workspace, desc, ZC_OP_BACKWARD, x.device)
    d, r = desc.c(), route.c()
    lbc = None if lb is None else C.byref(lb.c())
    a = (C.byref(d), _ptr(x), _ptr(w_router), _ptr(w_gate), _ptr(w_up), _ptr(w_down), C.byref(r),
         _ptr(saved), _ptr(dout), _ptr(dx), _ptr(dw_router), _ptr(dw_gate), _ptr(dw_up),
         _ptr(dw_down), lbc)
    if dlogits is None:
        _call("zc_moe_backward", w_router, stream, lib().zc_moe_backward, *a, _ptr(ws), ws.numel())
    else:
        _check_layer_tensor(dlogits, (desc.T, desc.E), torch.float32, "dlogits")
        _call("zc_moe_backward_scores", w_router, stream, lib().zc_moe_backward_scores, *a,
              _ptr(dlogits), _ptr(ws), ws.numel())


def zc_moe_lb_loss(desc: LayerDesc, lb: LoadBalance, route: RouteBuffers, out=None, ws=None,
                   stream=None):
    """Queues the device-level load-balance loss of the routed batch; returns
    out, a float64 GPU tensor [1 + 2(D+1)]: L, f_1..f_{D+1}, P_1..P_{D+1}."""
    if out is None:
        out = _alloc(stream, torch.empty, 1 + 2 * (lb.D + 1), dtype=torch.float64,
                     device=route.counts.device)
    _check_layer_tensor(out, (1 + 2 * (lb.D + 1),), torch.float64, "out")
    if ws is None:
        ws = _alloc(stream, workspace, desc, ZC_OP_LB_LOSS, route.counts.device)
    d, r, c = desc.c(), route.c(), lb.c()
    _call("zc_moe_lb_loss", out, stream, lib().zc_moe_lb_loss, C.byref(d), C.byref(c), C.byref(r),
          _ptr(out), _ptr(ws), ws.numel())
    return out


def seq_balance_workspace(desc: LayerDesc, S: int, device="cuda") -> torch.Tensor:
    d = desc.c()
    n = int(lib().zc_moe_seq_balance_workspace_size(C.byref(d), S))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def zc_moe_seq_balance(desc: LayerDesc, lb: LoadBalance, route: RouteBuffers, loss, counts,
                       dlogits=None, cu_seqlens=None, mask=None, ws=None, stream=None):
    """Balance loss of the packed sequences of a routed batch: loss fp32 [1+S]
    (L, then each sequence's), counts int32 [S][E] and, where given, the
    gradient of the router scores dlogits fp32 [T][E].  cu_seqlens int32
    [S+1]; mask uint8 or bool [T], nonzero for valid tokens; both may be slices
    that start anywhere (one not at a multiple of 16 bytes is copied first)."""
    cu_seqlens, mask = _aligned(stream, cu_seqlens), _aligned(stream, mask)
    S = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    T, E, i32, f32 = desc.T, desc.E, torch.int32, torch.float32
    a = _Args("zc_moe_seq_balance")
    lg = a(route.logits, (T, E), f32, "route.logits")
    ti = a(route.topk_idx, (T, desc.K), i32, "route.topk_idx")
    p = (a(cu_seqlens, (S + 1,), i32, "cu_seqlens"),
         a(mask, (T,), torch.bool if mask is not None and mask.dtype == torch.bool else torch.uint8,
           "mask"),
         a(loss, (1 + S,), f32, "loss"), a(counts, (S, E), i32, "counts"),
         a(dlogits, (T, E), f32, "dlogits"))
    if ws is None:
        ws = _alloc(stream, seq_balance_workspace, desc, S, loss.device)
    n = ws.numel() * ws.element_size()
    r = zc_route_buf(logits=lg, topk_idx=ti)
    a.run(lib().zc_moe_seq_balance, C.byref(desc.c()), C.byref(lb.c()), C.byref(r), S, *p,
          a(ws, ws.shape, ws.dtype, "ws"), n, stream=stream)


def zc_moe_route_stats(desc: LayerDesc, route: RouteBuffers, hist=None, moments=None, ws=None,
                       stream=None):
    """Queues the FFN-experts-per-token statistics of a routed batch; returns
    (hist [K+1] int32, moments [2] float64 = mean, std), both on the GPU."""
    dev = route.counts.device
    if hist is None:
        hist = _alloc(stream, torch.empty, desc.K + 1, dtype=torch.int32, device=dev)
    if moments is None:
        moments = _alloc(stream, torch.empty, 2, dtype=torch.float64, device=dev)
    _check_layer_tensor(hist, (desc.K + 1,), torch.int32, "hist")
    _check_layer_tensor(moments, (2,), torch.float64, "moments")
    if ws is None:
        ws = _alloc(stream, workspace, desc, ZC_OP_ROUTE_STATS, dev)
    d, r = desc.c(), route.c()
    _call("zc_moe_route_stats", hist, stream, lib().zc_moe_route_stats, C.byref(d), C.byref(r),
          _ptr(hist), _ptr(moments), _ptr(ws), ws.numel())
    return hist, moments


def zc_moe_accumulate_counts(counts, acc, stream=None):
    """acc += counts (int32 [E] GPU tensors): per-expert token counts over
    several micro-batches, for one Eq.(2) update with T_all = their tokens."""
    E = counts.numel()
    _check_layer_tensor(counts, (E,), torch.int32, "counts")
    _check_layer_tensor(acc, (E,), torch.int32, "acc")
    _call("zc_moe_accumulate_counts", acc, stream, lib().zc_moe_accumulate_counts, E, _ptr(counts),
          _ptr(acc))


def zc_moe_pid_update(N: int, Z: int, K: int, counts, T_all: int, mu: float, K_e: float, bias,
                      stream=None):
    _check_layer_tensor(counts, (N + Z,), torch.int32, "counts")
    _check_layer_tensor(bias, (N + Z,), torch.float32, "bias")
    _call("zc_moe_pid_update", bias, stream, lib().zc_moe_pid_update, N, Z, K, _ptr(counts), T_all,
          float(mu), float(K_e), _ptr(bias))


def zc_moe_pack_weights(desc: LayerDesc, which: int, src, dst, stream=None):
    """Packs w_gate or w_up (which = ZC_PACK_GATE_UP, [N][I][d]) or w_down
    (ZC_PACK_DOWN, [N][d][I]) into dst, a tensor of the same shape and dtype
    whose bytes then hold the packed layout."""
    shape = (desc.N, desc.I, desc.d) if which == ZC_PACK_GATE_UP else (desc.N, desc.d, desc.I)
    _check_layer_tensor(src, shape, desc.dtype, "src")
    _check_layer_tensor(dst, shape, desc.dtype, "dst")
    d = desc.c()
    _call("zc_moe_pack_weights", dst, stream, lib().zc_moe_pack_weights, C.byref(d), which, _ptr(src),
          _ptr(dst))


def pack_expert_weights(desc: LayerDesc, w_gate, w_up, w_down, stream=None):
    """Packed copies (new tensors) of the three expert weight tensors."""
    out = []
    for w, which in ((w_gate, ZC_PACK_GATE_UP), (w_up, ZC_PACK_GATE_UP), (w_down, ZC_PACK_DOWN)):
        p = _alloc(stream, torch.empty_like, w)
        zc_moe_pack_weights(desc, which, w, p, stream)
        out.append(p)
    return tuple(out)


def zc_moe_profile(on: bool) -> None:
    _check(lib().zc_moe_profile(1 if on else 0), "zc_moe_profile")


def zc_moe_profile_read() -> dict:
    """{phase name: (total ms, launches)} of the events recorded since the
    last read (waits for them)."""
    tot = (C.c_double * ZC_NUM_PHASES)()
    cnt = (C.c_int32 * ZC_NUM_PHASES)()
    _check(lib().zc_moe_profile_read(tot, cnt), "zc_moe_profile_read")
    return {lib().zc_moe_phase_name(i).decode(): (tot[i], cnt[i])
            for i in range(ZC_NUM_PHASES) if cnt[i]}


def zc_moe_quantize_weights(desc: LayerDesc, which: int, src, dst=None, stream=None):
    """FP8 blockwise (MXFP8) quantization of w_gate or w_up (which =
    ZC_PACK_GATE_UP, [N][I][d]) or w_down (ZC_PACK_DOWN, [N][d][I]) into dst,
    a uint8 GPU tensor of zc_moe_quantized_weight_bytes(desc) bytes (allocated
    when None).  Returns dst."""
    shape = (desc.N, desc.I, desc.d) if which == ZC_PACK_GATE_UP else (desc.N, desc.d, desc.I)
    _check_layer_tensor(src, shape, desc.dtype, "src")
    d = desc.c()
    n = int(lib().zc_moe_quantized_weight_bytes(C.byref(d)))
    if dst is None:
        dst = _alloc(stream, torch.empty, max(n, 16), dtype=torch.uint8, device=src.device)
    if dst.dtype != torch.uint8 or dst.numel() < n:
        raise ValueError(f"dst: expected at least {n} uint8, got {dst.numel()} {dst.dtype}")
    _call("zc_moe_quantize_weights", dst, stream, lib().zc_moe_quantize_weights, C.byref(d), which,
          _ptr(src), _ptr(dst))
    return dst


def quantize_expert_weights(desc: LayerDesc, w_gate, w_up, w_down, stream=None):
    """The three MXFP8 weight sets a ZC_WEIGHTS_MXFP8 forward takes."""
    return (zc_moe_quantize_weights(desc, ZC_PACK_GATE_UP, w_gate, stream=stream),
            zc_moe_quantize_weights(desc, ZC_PACK_GATE_UP, w_up, stream=stream),
            zc_moe_quantize_weights(desc, ZC_PACK_DOWN, w_down, stream=stream))


def _int4_shapes(desc: LayerDesc, which: int):
    G = int4_group(desc)
    if not G:
        raise ValueError("desc.weight_layout is no 4-bit layout (see int4_layout)")
    N, R, Cc = (desc.N, desc.I, desc.d) if which == ZC_PACK_GATE_UP else (desc.N, desc.d, desc.I)
    return (N, R, Cc), (N, R, Cc // 2), (N, R, Cc // G)


def zc_moe_int4_quantize(desc: LayerDesc, which: int, src, codes=None, scales=None, stream=None):
    """w_gate or w_up (ZC_PACK_GATE_UP, [N][I][d]) or w_down (ZC_PACK_DOWN,
    [N][d][I]) as 4-bit codes (uint8 [N][R][C/2]) and group scales (bf16
    [N][R][C/G]); both are allocated when None and returned.  (What a call on
    a given stream allocates belongs to that stream.)"""
    full, cs, ss = _int4_shapes(desc, which)
    if codes is None:
        codes = _alloc(stream, torch.empty, cs, dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = _alloc(stream, torch.empty, ss, dtype=torch.bfloat16, device=src.device)
    a = _Args("zc_moe_int4_quantize")
    a.run(lib().zc_moe_int4_quantize, C.byref(desc.c()), which, a(src, full, torch.bfloat16, "src"),
          a(codes, cs, torch.uint8, "codes"), a(scales, ss, torch.bfloat16, "scales"), stream=stream)
    return codes, scales


def zc_moe_int4_pack(desc: LayerDesc, which: int, codes, scales, dst=None, stream=None):
    """4-bit codes and scales in their natural layout (zc_moe_int4_quantize, or
    made elsewhere) -> the weight set a forward with desc's layout takes, a
    uint8 tensor (allocated when None).  Returns it."""
    _, cs, ss = _int4_shapes(desc, which)
    d = desc.c()
    n = int(lib().zc_moe_int4_weight_bytes(C.byref(d)))
    if dst is None:
        dst = _alloc(stream, torch.empty, max(n, 16), dtype=torch.uint8, device=codes.device)
    if dst.dtype != torch.uint8 or dst.numel() < n:
        raise ValueError(f"dst: expected at least {n} uint8, got {dst.numel()} {dst.dtype}")
    a = _Args("zc_moe_int4_pack")
    a.run(lib().zc_moe_int4_pack, C.byref(d), which, a(codes, cs, torch.uint8, "codes"),
          a(scales, ss, torch.bfloat16, "scales"), a(dst, dst.shape, dst.dtype, "dst"),
          stream=stream)
    return dst


def pack_int4_expert_weights(desc: LayerDesc, gate, up, down, stream=None):
    """The three weight sets of a 4-bit forward, from (codes, scales) pairs in
    the natural layout."""
    return (zc_moe_int4_pack(desc, ZC_PACK_GATE_UP, *gate, stream=stream),
            zc_moe_int4_pack(desc, ZC_PACK_GATE_UP, *up, stream=stream),
            zc_moe_int4_pack(desc, ZC_PACK_DOWN, *down, stream=stream))


def int4_expert_weights(desc: LayerDesc, w_gate, w_up, w_down, stream=None):
    """The three weight sets of a 4-bit forward, quantized from bf16 weights."""
    return tuple(zc_moe_int4_pack(desc, which, *zc_moe_int4_quantize(desc, which, w, stream=stream),
                                  stream=stream)
                 for w, which in ((w_gate, ZC_PACK_GATE_UP), (w_up, ZC_PACK_GATE_UP),
                                  (w_down, ZC_PACK_DOWN)))


def mxfp4_buffers(R: int, C: int, device="cuda"):
    """(codes [R][C/2], scales [R][C/32]) uint8: the rows zc_mxfp4_quantize writes."""
    return (torch.empty((R, C // 2), dtype=torch.uint8, device=device),
            torch.empty((R, C // 32), dtype=torch.uint8, device=device))


def zc_mxfp4_quantize(src, codes=None, scales=None, values=None, stream=None):
    """Rows [..., C] (bf16 or fp32, C a multiple of 32) as MXFP4: codes uint8 [..., C/2]
    (two a byte, the even column in the low half) and scales uint8 [..., C/32] (E8M0);
    both are allocated when None and returned.  values (as src; may be src): what
    they stand for."""
    if src.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"src: expected float32 or bfloat16, got {src.dtype}")
    if src.dim() < 1 or src.shape[-1] < 32 or src.shape[-1] % 32:
        raise ValueError(f"src: rows of {tuple(src.shape)[-1:]} values, a multiple of 32 is needed")
    Cc, lead = src.shape[-1], tuple(src.shape[:-1])
    R = src.numel() // Cc
    if codes is None:
        codes = _alloc(stream, torch.empty, lead + (Cc // 2,), dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = _alloc(stream, torch.empty, lead + (Cc // 32,), dtype=torch.uint8, device=src.device)
    a, u8 = _Args("zc_mxfp4_quantize"), torch.uint8
    p = (a(src, src.shape, src.dtype, "src"), a(codes, lead + (Cc // 2,), u8, "codes"),
         a(scales, lead + (Cc // 32,), u8, "scales"), a(values, src.shape, src.dtype, "values"))
    a.run(lib().zc_mxfp4_quantize, R, Cc, ZC_BF16 if src.dtype == torch.bfloat16 else ZC_F32, *p,
          stream=stream)
    return codes, scales


def _mxfp4_shape(desc: LayerDesc, which: int):
    if not _is_mxfp4(desc):
        raise ValueError("desc.weight_layout is no MXFP4 layout (see mxfp4_layout)")
    return (desc.N, desc.I, desc.d) if which == ZC_PACK_GATE_UP else (desc.N, desc.d, desc.I)


def zc_moe_mxfp4_pack(desc: LayerDesc, which: int, codes, scales, dst=None, stream=None):
    """MXFP4 codes [N][R][C/2] and scales [N][R][C/32] of w_gate or w_up
    (ZC_PACK_GATE_UP, [N][I][d]) or w_down (ZC_PACK_DOWN, [N][d][I]), from
    zc_mxfp4_quantize or made elsewhere -> the weight set a forward with desc's
    layout takes, a uint8 tensor (allocated when None).  Returns it."""
    N, R, Cc = _mxfp4_shape(desc, which)
    d = desc.c()
    n = int(lib().zc_moe_mxfp4_weight_bytes(C.byref(d), which))
    if dst is None:
        dst = _alloc(stream, torch.empty, max(n, 16), dtype=torch.uint8, device=codes.device)
    if dst.dtype != torch.uint8 or dst.numel() < n:
        raise ValueError(f"dst: expected at least {n} uint8, got {dst.numel()} {dst.dtype}")
    a, u8 = _Args("zc_moe_mxfp4_pack"), torch.uint8
    a.run(lib().zc_moe_mxfp4_pack, C.byref(d), which, a(codes, (N, R, Cc // 2), u8, "codes"),
          a(scales, (N, R, Cc // 32), u8, "scales"), a(dst, dst.shape, dst.dtype, "dst"), stream=stream)
    return dst


def pack_mxfp4_expert_weights(desc: LayerDesc, gate, up, down, stream=None):
    """The three weight sets of an MXFP4 forward, from (codes, scales) pairs."""
    return (zc_moe_mxfp4_pack(desc, ZC_PACK_GATE_UP, *gate, stream=stream),
            zc_moe_mxfp4_pack(desc, ZC_PACK_GATE_UP, *up, stream=stream),
            zc_moe_mxfp4_pack(desc, ZC_PACK_DOWN, *down, stream=stream))


def mxfp4_expert_weights(desc: LayerDesc, w_gate, w_up, w_down, stream=None):
    """The three weight sets of an MXFP4 forward, quantized from bf16 weights."""
    out = []
    for w, which, name in ((w_gate, ZC_PACK_GATE_UP, "w_gate"), (w_up, ZC_PACK_GATE_UP, "w_up"),
                           (w_down, ZC_PACK_DOWN, "w_down")):
        _check_layer_tensor(w, _mxfp4_shape(desc, which), desc.dtype, name)
        out.append(zc_moe_mxfp4_pack(desc, which, *zc_mxfp4_quantize(w, stream=stream), stream=stream))
    return tuple(out)


@dataclass
class NormDesc:
    """Rows of an RMS norm: T rows of d values, eps under the root."""
    T: int
    d: int
    dtype: torch.dtype = torch.bfloat16
    eps: float = 1e-6

    def c(self) -> zc_norm_desc:
        if self.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("norm dtype must be float32 or bfloat16")
        return zc_norm_desc(self.T, self.d, ZC_F32 if self.dtype == torch.float32 else ZC_BF16,
                            self.eps)


def mx_buffers(T: int, d: int, device="cuda"):
    """(codes [T][d], scales [T][d/32]) uint8: the MXFP8 rows zc_rmsnorm_forward
    writes and zc_moe_experts reads."""
    return (torch.empty((T, d), dtype=torch.uint8, device=device),
            torch.empty((T, d // 32), dtype=torch.uint8, device=device))


def norm_workspace(desc: NormDesc, device="cuda") -> torch.Tensor:
    d = desc.c()
    n = int(lib().zc_rmsnorm_workspace_size(C.byref(d)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def zc_rmsnorm_forward(desc: NormDesc, x, gamma, y, res=None, r=None, rstd=None, codes=None,
                       scales=None, stream=None):
    """r = x + res; y = r / sqrt(mean(r^2) + eps) * gamma, and y as MXFP8 in
    codes and scales (mx_buffers) where given.  r and y may be x or res in
    place."""
    T, d, dt = desc.T, desc.d, desc.dtype
    a, sh, u8 = _Args("zc_rmsnorm_forward"), (desc.T, desc.d), torch.uint8
    p = (a(x, sh, dt, "x"), a(res, sh, dt, "res"), a(gamma, (d,), dt, "gamma"), a(r, sh, dt, "r"),
         a(y, sh, dt, "y"), a(rstd, (T,), torch.float32, "rstd"), a(codes, sh, u8, "codes"),
         a(scales, (T, d // 32), u8, "scales"))
    a.run(lib().zc_rmsnorm_forward, C.byref(desc.c()), *p, stream=stream)


def zc_rmsnorm_backward(desc: NormDesc, dy, r, gamma, rstd, dr, dgamma, dres=None, ws=None,
                        stream=None):
    """Gradients of zc_rmsnorm_forward: dr (of x and res alike, with dres, the
    residual stream's own gradient, added) and dgamma."""
    T, d, dt = desc.T, desc.d, desc.dtype
    a, sh = _Args("zc_rmsnorm_backward"), (desc.T, desc.d)
    p = (a(dy, sh, dt, "dy"), a(r, sh, dt, "r"), a(gamma, (d,), dt, "gamma"),
         a(rstd, (T,), torch.float32, "rstd"), a(dres, sh, dt, "dres"), a(dr, sh, dt, "dr"),
         a(dgamma, (d,), dt, "dgamma"))
    if ws is None:
        ws = _alloc(stream, norm_workspace, desc, gamma.device)
    n = ws.numel() * ws.element_size()
    a.run(lib().zc_rmsnorm_backward, C.byref(desc.c()), *p, a(ws, ws.shape, ws.dtype, "ws"), n,
          stream=stream)


# ------------------------------------------------------- the weights' step
def _list_of(tensors, name, dtypes, like=None):
    """tensors as a list of contiguous GPU tensors of one dtype (among dtypes);
    like: the sizes they have."""
    out = list(tensors)
    if like is not None and len(out) != len(like):
        raise ValueError(f"{name}: {len(out)} tensors, expected {len(like)}")
    for i, t in enumerate(out):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{i}]: expected a torch.Tensor")
        if t.dtype not in dtypes or t.dtype != out[0].dtype:
            raise ValueError(f"{name}[{i}]: dtype {t.dtype}, expected one of {dtypes} and the same for all")
        if not t.is_cuda:
            raise ValueError("tensors passed to the HIP library must live on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensors passed to the HIP library must be contiguous")
        if like is not None and t.numel() != like[i]:
            raise ValueError(f"{name}[{i}]: {t.numel()} elements, expected {like[i]}")
    # (of their own: a tensor that is given other memory later would take this from us)
    return [t.detach() for t in out]


def _one_gpu(where, tensors):
    dev = None
    for t in tensors:
        if dev is not None and t.get_device() != dev:
            raise ValueError(f"{where}: tensors on GPU {dev} and on GPU {t.get_device()}")
        dev = t.get_device()
    return dev


class TensorList:
    """The gradients that zc_grad_norm takes: contiguous GPU tensors of one dtype
    (bf16 or fp32).  Holds the tensors' memory, whose contents may change between calls;
    a tensor that is given other memory (t.data = ...) needs a new list."""

    def __init__(self, tensors):
        self.tensors = _list_of(tensors, "tensors", (torch.float32, torch.bfloat16))
        self.device_index = _one_gpu("TensorList", self.tensors)
        self.sizes = [t.numel() for t in self.tensors]
        self.dtype = ZC_BF16 if self.tensors and self.tensors[0].dtype == torch.bfloat16 else ZC_F32
        self._c = (zc_grad_tensor * len(self.tensors))(
            *(zc_grad_tensor(t.data_ptr() or None, t.numel()) for t in self.tensors))

    def __len__(self):
        return len(self.tensors)


def grad_norm_workspace(grads: TensorList, device=None) -> torch.Tensor:
    n = int(lib().zc_grad_norm_workspace_size(grads._c, len(grads), grads.dtype))
    if device is None:
        device = "cuda" if grads.device_index is None else f"cuda:{grads.device_index}"
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def zc_grad_norm(grads: TensorList, max_norm: float, out, step=None, ws=None, stream=None):
    """Norm of all gradients and the factor that clips it to max_norm (inf: no
    clipping) into out, fp32 [2]; the factor is 0 where the norm is not finite.
    step (int64 [1]): one more unless it is.  out[1:] is what zc_adamw_step takes."""
    a = _Args("zc_grad_norm")
    a.dev = grads.device_index
    p = a(out, (2,), torch.float32, "out"), a(step, (1,), torch.int64, "step")
    if ws is None:
        ws = _alloc(stream, grad_norm_workspace, grads, out.device)
    n = ws.numel() * ws.element_size()
    a.run(lib().zc_grad_norm, grads._c, len(grads), grads.dtype, float(max_norm), *p,
          a(ws, ws.shape, ws.dtype, "ws"), n, stream=stream)


@dataclass
class AdamW:
    """Settings of zc_adamw_step.  rounding: of 8-bit states, and of bf16 weights
    without a copy in fp32."""
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.95
    eps: float = 1e-8
    rounding: int = ZC_ROUND_NEAREST
    seed: int = 0


class AdamWTensors:
    """The tensors of an AdamW step: weights (bf16 or fp32), gradients (the same
    or fp32), states m and v, for bf16 weights where wanted their fp32 copies
    master, and a weight decay for all or for each.  States: fp32, or
    torch.float8_e4m3fn with m_scale and v_scale, fp32 [ceil(n / 128)] (v's codes
    are of its square root); see adamw_tensors for a set that starts at zero.
    Holds the tensors' memory; gradients may be written anew between steps, and a
    tensor that is given other memory (t.data = ...) needs a new set."""

    def __init__(self, params, grads, m, v, master=None, m_scale=None, v_scale=None,
                 weight_decay=0.0):
        f32, bf, f8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
        self.params = _list_of(params, "params", (f32, bf))
        n = [t.numel() for t in self.params]
        bf16 = bool(n) and self.params[0].dtype == bf
        self.grads = TensorList(_list_of(grads, "grads", (bf, f32) if bf16 else (f32,), n))
        self.m, self.v = _list_of(m, "m", (f32, f8), n), _list_of(v, "v", (f32, f8), n)
        self.bits = 8 if n and self.m[0].dtype == f8 else 32
        if n and self.v[0].dtype != self.m[0].dtype:
            raise ValueError("m and v: both fp32 or both float8_e4m3fn")
        blocks = [-(-k // STATE_BLOCK) for k in n]
        if n and (self.bits == 8) != (m_scale is not None and v_scale is not None):
            raise ValueError("m_scale and v_scale go with float8_e4m3fn states")
        self.m_scale = None if m_scale is None else _list_of(m_scale, "m_scale", (f32,), blocks)
        self.v_scale = None if v_scale is None else _list_of(v_scale, "v_scale", (f32,), blocks)
        if master is not None and n and not bf16:
            raise ValueError("master goes with bf16 weights")
        self.master = None if master is None else _list_of(master, "master", (f32,), n)
        decay = [float(weight_decay)] * len(n) if isinstance(weight_decay, (int, float)) \
            else [float(w) for w in weight_decay]
        if len(decay) != len(n):
            raise ValueError(f"weight_decay: {len(decay)} values, expected {len(n)}")
        every = [self.params, self.grads.tensors, self.master, self.m, self.v, self.m_scale, self.v_scale]
        self.device_index = _one_gpu("AdamWTensors", [t for ts in every if ts is not None for t in ts])
        none = [None] * len(n)
        self._c = (zc_adamw_tensor * len(n))(
            *(zc_adamw_tensor(*(None if t is None else t.data_ptr() or None for t in ts), k, w)
              for *ts, k, w in zip(*(none if ts is None else ts for ts in every), n, decay)))
        self._cfg = (ZC_BF16 if bf16 else ZC_F32, self.grads.dtype,
                     ZC_STATE_8BIT if self.bits == 8 else ZC_STATE_F32)

    def __len__(self):
        return len(self.params)


def adamw_tensors(params, grads, bits: int = 32, master: bool = False, weight_decay=0.0, stream=None):
    """AdamWTensors with states of zeros in `bits` (32 or 8); master: with fp32
    copies of the bf16 weights, made here."""
    if bits not in (8, 32):
        raise ValueError(f"states of {bits} bits: 8 or 32 are supported")
    params = list(params)

    def make():
        f32 = torch.float32
        zeros = lambda dt: [torch.zeros(p.shape, dtype=dt, device=p.device) for p in params]  # noqa: E731
        kw = {}
        if bits == 8:
            # zeros of float8: bytes of zero
            m, v = ([t.view(torch.float8_e4m3fn) for t in zeros(torch.uint8)] for _ in range(2))
            for k in ("m_scale", "v_scale"):
                kw[k] = [torch.zeros(-(-p.numel() // STATE_BLOCK), dtype=f32, device=p.device)
                         for p in params]
        else:
            m, v = zeros(f32), zeros(f32)
        if master:
            kw["master"] = [p.to(f32) for p in params]
        return AdamWTensors(params, grads, m, v, weight_decay=weight_decay, **kw)

    return _alloc(stream, make)


def zc_adamw_step(cfg: AdamW, tensors: AdamWTensors, step, factor=None, lr=None, stream=None):
    """One AdamW step, in place.  step: an int, counted from 1, or int64 [1] on the
    GPU; factor, lr (fp32 [1] on the GPU, or None): the gradients' factor, and a
    learning rate in place of cfg's."""
    a = _Args("zc_adamw_step")
    a.dev = tensors.device_index
    if not len(tensors):
        return
    on_gpu = isinstance(step, torch.Tensor)
    p = (a(factor, (1,), torch.float32, "factor"), a(lr, (1,), torch.float32, "lr"),
         a(step, (1,), torch.int64, "step") if on_gpu else None)
    c = zc_adamw_cfg(*tensors._cfg, cfg.rounding, cfg.lr, cfg.beta1, cfg.beta2, cfg.eps,
                     0 if on_gpu else int(step), cfg.seed & 0xFFFFFFFF)
    a.run(lib().zc_adamw_step, C.byref(c), tensors._c, len(tensors), *p, stream=stream)
