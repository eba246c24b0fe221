"""GPU parity of the experts on 4-bit weights with group scales, of
zc_moe_experts against zc_moe_forward, and of the quantizer.

Reference: the layer's formulas in binary64 on the weights the codes and scales
stand for and on the GPU's own picks and gates.  Tolerance, by parts, with
u = 2^-24 and h = 2^-8 (half a step of bf16):
  a product z = sum_c v_c W_c: a group's sum runs in fp32 over G products
    v (128 + q) and G products -136 v, its partial sums at most 279 sum|v|
    in size; G/32 matrix steps each, of at most 33 roundings: 2 (G/32) 33 u
    of that.  Scaled by |s|; the scaled groups (C/G of them, then 3 joins)
    are added in fp32: (C/G + 4) u of the sum of their absolute values, that
    in turn at most |v| |W| + the error.  So
    E(z) = 2 (G/32) 33 u * 279 * sum_g |s_g| sum|v| + (C/G + 4) u |v| |W|.
  silu(a) u: silu's slope is at most 1.1; exp, reciprocal and two products
    cost (|a| + 12) u relative; rounding to bf16 costs h.
  y: E(y) on the rounded h, plus |W| times h's own error.
  out: K + 2 fp32 roundings of the sum of absolute terms, then h.
"""
import dataclasses

import numpy as np
import pytest
import torch

from moe_layer_zero_amd import synth, zcmoe
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

U, HB = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(N, R, C, G, seed):
    codes = torch.randint(0, 256, (N, R, C // 2), generator=gen(seed), dtype=torch.uint8)
    scales = ((torch.rand((N, R, C // G), generator=gen(seed + 1)) + 0.5) * 0.2 / C ** 0.5).to(BF)
    scales[torch.rand(scales.shape, generator=gen(seed + 2)) < 0.2] *= -1  # of either sign
    return codes, scales


def values(codes, scales, G):
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double() - 8
    return (q.view(*q.shape[:-1], -1, G) * scales.double()[..., None]).view(q.shape).numpy()


def make(T, d, N, Z, I, K, G, seed=0, skew=None):
    desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF, weight_layout=zcmoe.int4_layout(G))
    x = torch.randn((T, d), generator=gen(seed + 1)).to(BF)
    w = [weights(N, R, C, G, seed + 10 * i) for i, (R, C) in enumerate(((I, d), (I, d), (d, I)))]
    logits = torch.randn((T, N + Z), generator=gen(seed + 2))
    if skew is not None:
        logits[:, skew] += 20.0     # everybody's pick
    route = zcmoe.RouteBuffers(desc)
    route.logits.copy_(logits)
    zcmoe.zc_moe_route(desc, None, None, torch.zeros(N + Z, device="cuda"), route)
    packed = zcmoe.pack_int4_expert_weights(desc, *[(c.cuda(), s.cuda()) for c, s in w])
    return desc, x, w, route, packed


def product(v, W, s, G):
    """v W^T, |v| |W|^T and the fp32 error bound of the kernels' product."""
    C = W.shape[1]
    z, za = v @ W.T, np.abs(v) @ np.abs(W).T
    groups = np.abs(v).reshape(len(v), -1, G).sum(-1) @ np.abs(s).T
    return z, za, 2 * (G / 32) * 33 * U * 279 * groups + (C / G + 4) * U * za


def reference(desc, x, w, route, G, pick=slice(None)):
    T, N, K, I = desc.T, desc.N, desc.K, desc.I
    xd = x[pick].double().numpy()
    idx, gate = route.topk_idx[pick].cpu().numpy(), route.topk_gate[pick].cpu().double().numpy()
    ident = np.where(idx >= N, gate, 0).sum(1, keepdims=True)
    out, tol, terms = ident * xd, np.zeros_like(xd), np.abs(ident * xd)
    W = [values(c, s, G) for c, s in w]
    S = [s.double().numpy() for _, s in w]
    for e in range(N):
        t, r = np.nonzero(idx == e)
        if len(t) == 0:
            continue
        v = xd[t]
        a, _, ea = product(v, W[0][e], S[0][e], G)
        b, _, eb = product(v, W[1][e], S[1][e], G)
        si = a / (1 + np.exp(-a))
        hh = si * b
        eh = 1.1 * ea * (np.abs(b) + eb) + np.abs(si) * eb + (np.abs(a) + ea + 12) * U * np.abs(hh)
        eh = eh * (1 + HB) + HB * np.abs(hh) + 2.0 ** -133
        y, ya, ey = product(hh, W[2][e], S[2][e], G)
        ey = ey * (1 + HB) + eh @ np.abs(W[2][e]).T
        g = gate[t, r][:, None]
        out[t] += g * y
        tol[t] += g * ey
        terms[t] += np.abs(g * y)
    sc = abs(desc.out_scale)
    return out * desc.out_scale, sc * (tol + (K + 3) * U * (terms + tol))


def check(desc, x, w, route, packed, G):
    out = torch.full((desc.T, desc.d), float("nan"), dtype=BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, out)
    torch.cuda.synchronize()
    ref, tol = reference(desc, x, w, route, G)
    err = np.abs(out.cpu().double().numpy() - ref)
    bound = tol * (1 + HB) + HB * np.abs(ref) + 2.0 ** -133
    assert (err <= bound).all(), (err / bound).max()
    # errors are far from all alike: in the norm, three roundings to bf16 (h
    # twice over, out) and nothing more
    assert np.linalg.norm(err) <= 3 * HB * np.linalg.norm(ref)
    return out


CASES = [
    # T, d, N, Z, I, K: rows an expert from one to hundreds, every tile height
    (1, 128, 1, 0, 128, 1),       # one code block: three of four wavefronts have none
    (1, 256, 8, 4, 128, 3),
    (3, 384, 5, 0, 256, 5),       # every token through every expert
    (16, 640, 16, 7, 384, 4),
    (17, 1280, 3, 1, 128, 2),
    (40, 128, 2, 0, 512, 1),
    (65, 512, 4, 2, 256, 2),      # 32 rows a tile
    (200, 256, 9, 3, 128, 2),     # 64 rows a tile
    (700, 128, 7, 3, 256, 3),
]


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c)) for c in CASES])
def test_parity(case, G):
    print(f"[int4] {case} G={G}", flush=True)
    check(*make(*case, G, seed=100 + case[0]), G)


@pytest.mark.parametrize("T", [15, 16, 33, 129])
def test_one_expert_takes_every_token(T):
    """Row tiles of one height over an expert with many more rows than the
    average, the rest nearly empty."""
    print(f"[int4 skew] T={T}", flush=True)
    check(*make(T, 256, 32, 8, 128, 2, 64, seed=7, skew=5), 64)


def test_offsets_beyond_32_bits():
    """Rows of h past the 2^32nd element, more tiles than one grid has
    workgroups, and more rows than the 64-row kernel takes: tokens all over the
    batch against the reference."""
    T, d, N, Z, I, K, G = 600_000, 128, 8, 4, 2048, 8, 64
    desc, x, w, route, packed = make(T, d, N, Z, I, K, G, seed=11)
    assert int(route.offsets[-1]) * I > 1 << 32
    out = torch.full((T, d), float("nan"), dtype=BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, out)
    pick = torch.tensor([0, 1, 77_777, 299_999, 450_001, T - 2, T - 1])
    ref, tol = reference(desc, x, w, route, G, pick)
    err = np.abs(out[pick].cpu().double().numpy() - ref)
    assert (err <= tol * (1 + HB) + HB * np.abs(ref) + 2.0 ** -133).all()
    assert torch.isfinite(out[::997].float()).all()


def test_all_picks_on_zero_computation_experts():
    desc, x, w, route, packed = make(9, 256, 4, 4, 128, 1, 128, seed=3, skew=6)
    assert (route.topk_idx >= 4).all()
    out = check(desc, x, w, route, packed, 128)
    assert torch.equal(out.cpu(), x)


def test_no_tokens_and_no_ffn_experts():
    d0 = zcmoe.LayerDesc(0, 256, 4, 2, 128, 2, BF, weight_layout=zcmoe.int4_layout(32))
    r = zcmoe.RouteBuffers(d0)
    e = torch.empty((0, 256), dtype=BF, device="cuda")
    zcmoe.zc_moe_route(d0, None, None, torch.zeros(6, device="cuda"), r)
    n = zcmoe.lib().zc_moe_int4_weight_bytes(__import__("ctypes").byref(d0.c()))
    w = torch.zeros(n, dtype=torch.uint8, device="cuda")
    zcmoe.zc_moe_experts(d0, e, r, w, w, w, e.clone())
    dz = zcmoe.LayerDesc(5, 256, 0, 4, 128, 2, BF, weight_layout=zcmoe.int4_layout(32))
    rz = zcmoe.RouteBuffers(dz)
    rz.logits.copy_(torch.randn((5, 4), generator=gen(1)))
    zcmoe.zc_moe_route(dz, None, None, torch.zeros(4, device="cuda"), rz)
    x = torch.randn((5, 256), generator=gen(2)).to(BF).cuda()
    out = torch.empty_like(x)
    zcmoe.zc_moe_experts(dz, x, rz, None, None, None, out)
    # two gates that sum to 1 within a rounding each
    assert ((out.double() - x.double()).abs() <= (HB + 4 * U) * x.double().abs()).all()


def test_a_rows_infinity_and_nan_stay_in_its_row():
    desc, x, w, route, packed = make(20, 256, 8, 0, 128, 2, 128, seed=5)
    want = torch.empty((20, 256), dtype=BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, want)
    x[3, 7], x[11, 9] = float("nan"), float("inf")
    out = torch.empty_like(want)
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, out)
    keep = [t for t in range(20) if t not in (3, 11)]
    assert torch.equal(out[keep], want[keep])
    assert torch.isnan(out[[3, 11]]).all()


@pytest.mark.parametrize("G", [32, 64, 128])
def test_quantizer(G):
    N, R, C = 3, 128, 256
    desc = zcmoe.LayerDesc(1, C, N, 0, R, 1, BF, weight_layout=zcmoe.int4_layout(G))
    w = torch.randn((N, R, C), generator=gen(9)).to(BF)
    w[0, 0, :G] = 0
    w[0, 1, 3] = float("nan")
    w[0, 2, C - 1] = float("inf")
    w[0, 3, :G] = 2.0 ** -133                 # the scale rounds to a subnormal or to 0
    w[1] *= 2.0 ** 100
    w[2] *= 2.0 ** -100
    codes, scales = zcmoe.zc_moe_int4_quantize(desc, zcmoe.ZC_PACK_GATE_UP, w.cuda())
    g = w.float().view(N, R, -1, G)
    bad = ~torch.isfinite(g).all(-1)
    s = torch.where(bad, torch.zeros(()), g.abs().amax(-1) / 7.0).to(BF)
    q = torch.where((s.float() > 0)[..., None], torch.round(g / s.float()[..., None]), torch.zeros(()))
    q = torch.where(bad[..., None], torch.zeros(()), q.nan_to_num()).clamp(-8, 7).to(torch.int64) + 8
    q = q.view(N, R, C)
    assert torch.equal(torch.isnan(scales.cpu()), bad)
    assert torch.equal(scales.cpu()[~bad], s[~bad])
    assert torch.equal(codes.cpu().long(), q[..., 0::2] | q[..., 1::2] << 4)
    # the values they stand for are within half a step of the weights (plus
    # bf16's rounding of the step, taken seven times at most)
    v = torch.from_numpy(values(codes.cpu(), scales.cpu(), G))
    okay = ~bad.repeat_interleave(G, -1) & (s.float() > 2.0 ** -100).repeat_interleave(G, -1)
    step = s.double().repeat_interleave(G, -1)
    assert ((v - w.double()).abs() <= (0.5 + 7 * HB) * step)[okay].all()


@pytest.mark.parametrize("T", [5, 300])
def test_forward_quantized_from_bf16(T):
    """The whole forward, weights quantized by the library: router, experts and
    combine against zc_moe_experts on the forward's own routing, bit for bit,
    with and without a workspace of the caller's."""
    sh = dataclasses.replace(synth.CONFIGS["small_bf16"], T=T)
    L = H.to_dev(synth.make_layer(sh, "cpu"))
    desc = dataclasses.replace(H.desc_of(sh, 1, 0.5), weight_layout=zcmoe.int4_layout(64))
    packed = zcmoe.int4_expert_weights(desc, L["wg"], L["wu"], L["wd"])
    outs = []
    route = zcmoe.RouteBuffers(desc)
    out = torch.empty((T, sh.d), dtype=BF, device="cuda")
    zcmoe.zc_moe_forward(desc, L["x"], L["wr"], L["bias"], *packed, out, route)
    again = torch.empty_like(out)
    zcmoe.zc_moe_experts(desc, L["x"], route, *packed, again)
    assert torch.equal(out, again)
    if T == 5:
        zcmoe.zc_moe_forward_noalloc(desc, L["x"], L["wr"], L["bias"], *packed, again,
                                     zcmoe.RouteBuffers(desc))
        assert torch.equal(out, again)
        w = [tuple(t.cpu() for t in zcmoe.zc_moe_int4_quantize(desc, k, L[n])) for n, k in
             (("wg", 0), ("wu", 0), ("wd", 1))]
        ref, tol = reference(desc, L["x"].cpu(), w, route, 64)
        err = np.abs(out.cpu().double().numpy() - ref)
        assert (err <= tol * (1 + HB) + HB * np.abs(ref) + 2.0 ** -133).all()


@pytest.mark.parametrize("layout", ["fp32", "rowmajor", "packed", "mxfp8", "mxfp8_rows", "small"])
def test_experts_equal_the_forward(layout):
    """zc_moe_experts on the routing of a forward gives its output bit for bit;
    with MXFP8 weights also from rows the norm quantized."""
    sh = synth.CONFIGS["tiny_fp32"] if layout == "fp32" else \
        dataclasses.replace(synth.CONFIGS["small_bf16"], T=333)
    if layout == "small":
        sh = dataclasses.replace(sh, d=192, I=64)   # the generic bf16 kernels
    L = H.to_dev(synth.make_layer(sh, "cpu"))
    desc = H.desc_of(sh)
    w, xq = (L["wg"], L["wu"], L["wd"]), None
    if layout == "packed":
        w = zcmoe.pack_expert_weights(desc, *w)
        desc = dataclasses.replace(desc, weight_layout=zcmoe.ZC_WEIGHTS_PACKED)
    elif layout.startswith("mxfp8"):
        w = zcmoe.quantize_expert_weights(desc, *w)
        desc = dataclasses.replace(desc, weight_layout=zcmoe.ZC_WEIGHTS_MXFP8)
    if layout == "mxfp8_rows":
        nd = zcmoe.NormDesc(sh.T, sh.d, BF)
        y, xq = torch.empty_like(L["x"]), zcmoe.mx_buffers(sh.T, sh.d)
        g = (1 + 0.2 * torch.randn(sh.d, generator=gen(4))).to(BF).cuda()
        zcmoe.zc_rmsnorm_forward(nd, L["x"], g, y, codes=xq[0], scales=xq[1])
        L["x"] = y
    route = zcmoe.RouteBuffers(desc)
    out, again = torch.empty_like(L["x"]), torch.empty_like(L["x"])
    zcmoe.zc_moe_forward(desc, L["x"], L["wr"], L["bias"], *w, out, route)
    zcmoe.zc_moe_experts(desc, L["x"], route, *w, again, xq=xq)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


def test_norm_then_forward_in_a_graph_on_another_stream():
    """A decode step as it is served: norm with residual, router, 4-bit experts,
    captured once and replayed on new inputs."""
    T, d, N, Z, I, K, G = 24, 512, 16, 8, 256, 4, 64
    desc, x, w, route, packed = make(T, d, N, Z, I, K, G, seed=30)
    nd = zcmoe.NormDesc(T, d, BF)
    wr = (torch.randn((N + Z, d), generator=gen(31)) * 0.05).to(BF).cuda()
    bias = torch.zeros(N + Z, device="cuda")
    gamma = torch.ones(d, dtype=BF, device="cuda")
    xg, res = x.cuda(), torch.zeros((T, d), dtype=BF, device="cuda")
    r, y, out = (torch.empty_like(xg) for _ in range(3))
    ws = zcmoe.workspace(desc, zcmoe.ZC_OP_FORWARD)

    def step():
        zcmoe.zc_rmsnorm_forward(nd, xg, gamma, y, res=res, r=r)
        zcmoe.zc_moe_forward(desc, y, wr, bias, *packed, out, route, ws=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        xg.copy_(torch.randn((T, d), generator=gen(40 + k)).to(BF))
        res.copy_(torch.randn((T, d), generator=gen(50 + k)).to(BF))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        # the same experts by the routed call, on a stream of their own
        other = torch.cuda.Stream()
        zcmoe.zc_moe_experts(desc, y, route, *packed, out, stream=other)
        other.synchronize()
        assert torch.equal(got, out)
