"""MXFP4 rows and the experts on MXFP4 weights against their definition in 64 bits.

Quantization is exact arithmetic, so codes and scales are compared bit for bit.
Products: operands are exact, a sum of n products in fp32 is off by at most (n + 8)
u sum |x w| (u = 2^-24), whatever the order (n additions, and 8 for the joining of
partial sums).  a and u of gate/up carry that error; silu adds 12 roundings' worth
(hardware exp and reciprocal, and |a| u for the exponent's argument).  h is then
rounded to a code: a value known to +-e may go to any code that one of that
interval goes to, at the scale of the block's largest value, known to its +-e.
"""
import dataclasses

import numpy as np
import pytest
import torch

from moe_layer_zero_amd import synth, zcmoe
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HB = 2.0 ** -8  # half a step of bf16
BF, F32 = torch.bfloat16, torch.float32
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def gen(seed):
    return torch.Generator().manual_seed(seed)


def unpack(codes):
    return E2M1[np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)]


def exponents(top, bits):
    """E8M0 of blocks whose largest magnitude is top (finite)."""
    e = np.floor(np.log2(np.maximum(top, 2.0 ** -150))) - (2 if bits == 4 else 8) + 127
    return np.maximum(np.where(top > 0, e, 0), 0)


def rounded(b, S, bits):
    """Blocks b [..., 32] to 4-bit or 8-bit codes' values at the scales S."""
    low, digits, most = (0, 1, 6.0) if bits == 4 else (-6, 3, 448.0)
    s = 2.0 ** (S[..., None] - 127)
    t = b / s
    unit = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** low))) - digits)
    return np.clip(np.round(t / unit) * unit, -most, most) * s


def blocks(v):
    return v.reshape(*v.shape[:-1], -1, 32)


def quantized(v, bits):
    b = blocks(v)
    return rounded(b, exponents(np.abs(b).max(-1), bits), bits).reshape(v.shape)


def quantized_range(v, err, bits):
    """Smallest and largest value that v known to +-err is rounded to."""
    b, e = blocks(v), blocks(err)
    ends = []
    for top in ((np.abs(b) - e).max(-1), (np.abs(b) + e).max(-1)):
        S = exponents(np.maximum(top, 0), bits)
        ends += [rounded(b - e, S, bits), rounded(b + e, S, bits)]
    return np.minimum.reduce(ends).reshape(v.shape), np.maximum.reduce(ends).reshape(v.shape)


# -------------------------------------------------------------- quantizer
def run_rows(x, values=True, **kw):
    v = torch.empty_like(x) if values else None
    codes, scales = zcmoe.zc_mxfp4_quantize(x, values=v, **kw)
    return codes.cpu().numpy(), scales.cpu().numpy(), v


def check_rows(x):
    codes, scales, v = run_rows(x.cuda())
    d = x.double().numpy()
    b = blocks(d)
    S = exponents(np.abs(b).max(-1), 4)
    q = rounded(b, S, 4)
    assert (scales.reshape(S.shape) == S).all()
    got = blocks(unpack(codes)) * 2.0 ** (scales[..., None].astype(np.float64) - 127)
    assert (got == q).all() and (np.signbit(got) == np.signbit(b)).all()
    assert torch.equal(v.cpu(), torch.from_numpy(q.reshape(d.shape)).to(x.dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (7, 96), (257, 1024), (2, 5, 160), (1000, 6144)])
def test_rows(shape, dtype):
    g = gen(shape[-1])
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape[:-1] + (1,), generator=g))
    x[..., ::32] = 0.0
    check_rows(x.to(dtype))


def test_rows_every_bf16_value():
    # beside a 1, beside a large value, and in blocks of their own
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    v = v[torch.isfinite(v)]
    v = v[: v.numel() // 31 * 31].view(-1, 31)
    for beside in (1.0, 1e30, 1e-30, 0.0):
        check_rows(torch.cat([torch.full((v.shape[0], 1), beside, dtype=BF), v], 1))


def test_rows_at_the_borders():
    # ties, and the next numbers on both sides of them
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9999995, 4.0, 0.5])
    up, down = torch.nextafter(t, torch.tensor(9.0)), torch.nextafter(t, torch.tensor(0.0))
    x = torch.cat([torch.tensor([4.0]), t, up.clamp(max=7.9999995), down])[:32]
    x = torch.cat([x, torch.zeros(32 - x.numel())])
    for k in (-130, -126, -20, 0, 60, 124):
        check_rows(torch.ldexp(x, torch.tensor(k))[None])
        check_rows(-torch.ldexp(x, torch.tensor(k))[None])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_not_finite(dtype):
    x = torch.ones((4, 96), dtype=dtype)
    x[0, 40] = float("inf")
    x[1, 40] = -float("inf")
    x[2, 40] = float("nan")
    codes, scales, v = run_rows(x.cuda())
    assert scales[0].tolist() == scales[1].tolist() == [125, 253, 125] and scales[2].tolist() == [125, 255, 125]
    assert codes[0, 20] & 15 == 7 and codes[1, 20] & 15 == 15 and not codes[2, 16:32].any()
    assert (codes[:, :16] == 0x66).all() and (codes[:, 32:] == 0x66).all()  # 1 = 4 / 4
    v = v.cpu()
    assert v[0, 40] == float("inf") and v[1, 40] == -float("inf")
    assert bool(torch.isnan(v[2, 32:64]).all()) and bool((v[:, :32] == 1).all()) and bool((v[3] == 1).all())


def test_rows_in_place_and_without_values():
    x = torch.randn((33, 128), generator=gen(3)).to(BF).cuda()
    codes, scales, v = run_rows(x)
    c2, s2, _ = run_rows(x, values=False)
    assert (codes == c2).all() and (scales == s2).all()
    zcmoe.zc_mxfp4_quantize(x, values=x)
    assert torch.equal(x, v)
    # what has been rounded stays, but for a block whose largest was clamped to 6
    c3, s3, v3 = run_rows(x)
    assert torch.equal(v3, v)
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    assert zcmoe.zc_mxfp4_quantize(e)[0].shape == (0, 32)


def test_rows_past_32_bits():
    R, Cc = (1 << 32) // 2048 + 3, 2048
    x = torch.zeros((R, Cc), dtype=BF, device="cuda")
    tail = torch.randn((3, Cc), generator=gen(9)).to(BF)
    x[-3:] = tail.cuda()
    codes, scales = zcmoe.zc_mxfp4_quantize(x)
    c, s, _ = run_rows(tail.cuda())
    assert (codes[-3:].cpu().numpy() == c).all() and (scales[-3:].cpu().numpy() == s).all()
    assert not bool(codes[:-3].any()) and not bool(scales[:-3].any())


# ---------------------------------------------------------------- experts
def weights(N, R, C, seed):
    codes = torch.randint(0, 256, (N, R, C // 2), generator=gen(seed), dtype=torch.uint8)
    e = 127 + round(np.log2(1 / (2.93 * C ** 0.5)))
    scales = torch.randint(e - 3, e + 3, (N, R, C // 32), generator=gen(seed + 1), dtype=torch.uint8)
    return codes, scales


def matrix(codes, scales):
    w = unpack(codes.numpy())
    return (blocks(w) * 2.0 ** (scales.double().numpy()[..., None] - 127)).reshape(w.shape)


def make(T, d, N, Z, I, K, a, seed=0, skew=None, **kw):
    desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF, weight_layout=zcmoe.mxfp4_layout(a), **kw)
    x = torch.randn((T, d), generator=gen(seed + 1)).to(BF)
    w = [weights(N, R, C, seed + 10 * i) for i, (R, C) in enumerate(((I, d), (I, d), (d, I)))]
    logits = torch.randn((T, N + Z), generator=gen(seed + 2))
    if skew is not None:
        logits[:, skew] += 20.0     # everybody's pick
    route = zcmoe.RouteBuffers(desc)
    route.logits.copy_(logits)
    zcmoe.zc_moe_route(desc, None, None, torch.zeros(N + Z, device="cuda"), route)
    packed = zcmoe.pack_mxfp4_expert_weights(desc, *[(c.cuda(), s.cuda()) for c, s in w])
    return desc, x, w, route, packed


def product(v, W):
    z, za = v @ W.T, np.abs(v) @ np.abs(W).T
    return z, (W.shape[1] + 8) * U * za


def reference(desc, x, w, route, a):
    N, K = desc.N, desc.K
    xd = x.double().numpy()
    xq = quantized(xd, a) if len(xd) else xd
    idx, gate = route.topk_idx.cpu().numpy(), route.topk_gate.cpu().double().numpy()
    ident = np.where(idx >= N, gate, 0).sum(1, keepdims=True)
    out, tol, terms = ident * xd, np.zeros_like(xd), np.abs(ident * xd)
    for e in range(N):
        t, r = np.nonzero(idx == e)
        if len(t) == 0:
            continue
        Wg, Wu, Wd = (matrix(c[e], s[e]) for c, s in w)
        g1, e1 = product(xq[t], Wg)
        u1, e2 = product(xq[t], Wu)
        si = g1 / (1 + np.exp(-g1))
        h = si * u1
        eh = 1.1 * e1 * (np.abs(u1) + e2) + np.abs(si) * e2 + (np.abs(g1) + e1 + 12) * U * np.abs(h)
        hq = quantized(h, a)
        lo, hi = quantized_range(h, eh, a)
        off = np.maximum(hi - hq, hq - lo)
        y, ey = product(hq, Wd)
        ey = ey + (1 + (Wd.shape[1] + 8) * U) * off @ np.abs(Wd).T + y_round(desc) * (np.abs(y) + off @ np.abs(Wd).T)
        g = gate[t, r][:, None]
        out[t] += g * y
        tol[t] += g * ey
        terms[t] += np.abs(g * y)
    sc = abs(desc.out_scale)
    return out * desc.out_scale, sc * (tol + (K + 3) * U * (terms + tol))


def y_round(desc):
    """y is kept in fp32, but in bf16 by the kernel of many rows."""
    many = desc.T * desc.K // desc.E > 10 and desc.d % 512 == 0 and desc.I % 512 == 0
    return HB if many else 0.0


def check(desc, x, w, route, packed, a):
    out = torch.full((desc.T, desc.d), float("nan"), dtype=BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, out)
    torch.cuda.synchronize()
    ref, tol = reference(desc, x, w, route, a)
    err = np.abs(out.cpu().double().numpy() - ref)
    bound = tol * (1 + HB) + HB * np.abs(ref) + 2.0 ** -133
    assert (err <= bound).all(), (err / bound).max()
    # in the norm the roundings of y and out are most of it
    assert np.linalg.norm(err) <= 2 * HB * np.linalg.norm(ref)
    return out


CASES = [
    # T, d, N, Z, I, K: rows an expert from one to hundreds
    (1, 128, 1, 0, 128, 1),       # one code block: three of four wavefronts have none
    (1, 256, 8, 4, 128, 3),
    (3, 384, 5, 0, 256, 5),       # every token through every expert
    (16, 640, 16, 7, 384, 4),     # five and three code blocks: part of a scale word unused
    (17, 1280, 3, 1, 128, 2),
    (40, 128, 2, 0, 512, 1),
    (65, 512, 4, 2, 256, 2),
    (200, 256, 9, 3, 128, 2),
    (700, 128, 7, 3, 256, 3),
    (333, 512, 3, 1, 1024, 2),    # hundreds of rows an expert, whole groups of 512 steps
    (520, 1024, 2, 1, 512, 2),
    (1100, 512, 2, 0, 512, 1),
    (150, 2560, 2, 1, 512, 2),    # rows' scales in parts of 2048 steps, the last one short
    (90, 512, 1, 1, 4608, 1),
    (130, 2048, 2, 0, 3584, 1),
    (340, 2560, 2, 1, 512, 2),    # tiles of 160 MXFP4 rows
    (230, 512, 1, 1, 4608, 1),
]


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c)) for c in CASES])
def test_experts(case, a):
    check(*make(*case, a), a)


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_experts_ragged_tiles(rows, a):
    # one expert takes everything: tiles that end inside a block of rows
    check(*make(rows, 512, 3, 1, 512, 1, a, seed=rows, skew=1), a)


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("rows", [109, 110, 127, 129, 144, 145, 159, 160, 161, 177, 319, 320, 321, 500])
def test_experts_ragged_tiles_of_many_rows(rows, a):
    check(*make(rows, 512, 1, 0, 1024, 1, a, seed=rows), a)


@pytest.mark.parametrize("a", [8, 4])
def test_experts_past_31_bits(a):
    # h of more than 2^31 bytes in 8 bits: the last tokens' rows lie behind that
    T, n = 70000, 24
    desc, x, w, route, packed = make(T, 512, 2, 0, 32768, 1, a)
    assert T * 32768 > 1 << 31
    out = torch.full((T, 512), float("nan"), dtype=BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, out)
    torch.cuda.synchronize()
    assert not bool(torch.isnan(out).any())
    tail = dataclasses.replace(desc, T=n)
    for part in (slice(0, n), slice(T - n, T)):
        r = zcmoe.RouteBuffers(tail, "cpu")
        r.topk_idx, r.topk_gate = route.topk_idx[part], route.topk_gate[part]
        ref, tol = reference(tail, x[part], w, r, a)
        err = np.abs(out[part].cpu().double().numpy() - ref)
        assert (err <= tol * (1 + HB) + HB * np.abs(ref) + 2.0 ** -133).all()


def test_no_rows_to_quantize():
    codes, scales = zcmoe.zc_mxfp4_quantize(torch.empty((0, 64), dtype=BF, device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (0, 2)


@pytest.mark.parametrize("a", [8, 4])
def test_experts_left_without_rows(a):
    T, N = 600, 24
    desc, x, w, route, packed = make(T, 512, N, 4, 512, 3, a)
    route.logits[:, 5:20] -= 1e4    # nobody's pick
    zcmoe.zc_moe_route(desc, None, None, torch.zeros(desc.E, device="cuda"), route)
    assert int((route.counts[:N] == 0).sum()) == 15
    check(desc, x, w, route, packed, a)


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("kw", [dict(gate_norm=0), dict(out_scale=-1.75), dict(cu_limit=8)])
def test_experts_settings(kw, a):
    for T in (5, 400):
        check(*make(T, 512, 4, 2, 512, 3, a, **kw), a)


@pytest.mark.parametrize("a", [8, 4])
def test_no_tokens_and_no_experts(a):
    desc, x, w, route, packed = make(0, 256, 4, 2, 128, 2, a)
    out = torch.empty((0, 256), dtype=BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, out)
    desc = zcmoe.LayerDesc(5, 256, 0, 4, 128, 2, BF, weight_layout=zcmoe.mxfp4_layout(a))
    x = torch.randn((5, 256)).to(BF).cuda()
    route, out = zcmoe.RouteBuffers(desc), torch.empty_like(x)
    zcmoe.zc_moe_forward(desc, x, torch.zeros((4, 256), dtype=BF, device="cuda"),
                         torch.zeros(4, device="cuda"), None, None, None, out, route)
    assert torch.equal(out, x)


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("T", [3, 500])
def test_forward_is_route_and_experts(T, a):
    sh = dataclasses.replace(synth.CONFIGS["small_bf16"], T=T, d=512, N=8, Z=4, K=3)
    L = H.to_dev(synth.make_layer(sh, "cpu"))
    desc = dataclasses.replace(H.desc_of(sh, 1, 0.5), weight_layout=zcmoe.mxfp4_layout(a))
    packed = zcmoe.mxfp4_expert_weights(desc, L["wg"], L["wu"], L["wd"])
    outs = [torch.full((T, 512), float("nan"), dtype=BF, device="cuda") for _ in range(4)]
    r1, r2 = zcmoe.RouteBuffers(desc), zcmoe.RouteBuffers(desc)
    zcmoe.zc_moe_forward(desc, L["x"], L["wr"], L["bias"], *packed, outs[0], r1)
    zcmoe.zc_moe_forward_noalloc(desc, L["x"], L["wr"], L["bias"], *packed, outs[1], r2)
    zcmoe.zc_moe_experts(desc, L["x"], r1, *packed, outs[2])
    # rows that were quantized before
    if a == 4:
        xq = zcmoe.zc_mxfp4_quantize(L["x"])
    else:
        xq = zcmoe.mx_buffers(T, 512)
        nd, one = zcmoe.NormDesc(T, 512, BF), torch.ones(512, dtype=BF, device="cuda")
        y = torch.empty_like(L["x"])
        zcmoe.zc_rmsnorm_forward(nd, L["x"], one, y, codes=xq[0], scales=xq[1])
        zcmoe.zc_moe_experts(desc, y, r1, *packed, outs[2])
        outs[0] = outs[1] = torch.empty_like(y)
        zcmoe.zc_moe_experts(desc, y, r1, *packed, outs[0])
        L["x"] = y
    zcmoe.zc_moe_experts(desc, L["x"], r1, *packed, outs[3], xq=xq)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    # the weights' own values
    ws = []
    for n in ("wg", "wu", "wd"):
        c, s = zcmoe.zc_mxfp4_quantize(L[n])
        ws.append((c.cpu(), s.cpu()))
    check(desc, L["x"].cpu(), ws, r1, packed, a)


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("T", [40, 600])
def test_not_finite_stays_where_it_belongs(T, a):
    desc, x, w, route, packed = make(T, 512, 4, 0, 512, 2, a)
    good = check(desc, x, w, route, packed, a)
    bad = x.clone()
    bad[7, 130] = float("nan")
    out = torch.empty_like(good)
    zcmoe.zc_moe_experts(desc, bad.cuda(), route, *packed, out)
    nan = torch.isnan(out).all(1).cpu()
    assert nan.tolist() == [t == 7 for t in range(T)]
    rest = torch.arange(T) != 7
    assert torch.equal(out.cpu()[rest], good.cpu()[rest])
    # a scale of a weight that is NaN reaches the tokens of its expert
    c, s = w[2]
    s = s.clone()
    s[2, 100, 3] = 255
    wd = zcmoe.zc_moe_mxfp4_pack(desc, zcmoe.ZC_PACK_DOWN, c.cuda(), s.cuda())
    zcmoe.zc_moe_experts(desc, x.cuda(), route, packed[0], packed[1], wd, out)
    hit = (route.topk_idx == 2).any(1).cpu()
    nan = torch.isnan(out).cpu()
    assert torch.equal(nan[:, 100], hit) and not bool(nan[:, :100].any()) and not bool(nan[:, 101:].any())


@pytest.mark.parametrize("a", [8, 4])
@pytest.mark.parametrize("T", [9, 700])
def test_captured_replayed_and_on_another_stream(T, a):
    desc, x, w, route, packed = make(T, 512, 6, 2, 512, 2, a)
    x = x.cuda()
    ws = zcmoe.workspace(desc, zcmoe.ZC_OP_EXPERTS)
    out, want = torch.empty_like(x), torch.empty_like(x)
    run = lambda o, **kw: zcmoe.zc_moe_experts(desc, x, route, *packed, o, ws=ws, **kw)  # noqa: E731
    run(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for k in range(4):
        x.copy_(torch.randn(x.shape, generator=gen(k)).to(BF))
        run(want)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("a", [8, 4])
def test_calls_at_once_on_two_streams(a):
    sets = [make(T, 512, 5, 1, 512, 2, a, seed=T) for T in (30, 450)]
    want = [check(*s, a) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    xs = [s[1].cuda() for s in sets]
    torch.cuda.synchronize()
    outs = [torch.empty_like(x) for x in xs]
    for _ in range(5):
        for (desc, _, _, route, packed), x, o, st in zip(sets, xs, outs, streams):
            zcmoe.zc_moe_experts(desc, x, route, *packed, o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, v) for o, v in zip(outs, want))
