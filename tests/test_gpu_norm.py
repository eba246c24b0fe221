"""GPU parity of the RMS norm (with the residual's addition and the MXFP8
output) and of its backward against the formulas in binary64.

Tolerances.  u = 2^-24 (fp32 half step), h = half a step of the output type
(2^-8 bf16, 2^-24 fp32), relative.
  r:     one fp32 addition and one rounding of exact inputs: equal bits.
  rstd:  the sum of d squares in fp32 along a tree at most 64 terms deep per
         thread plus 16 levels: relative error (64 + 16) u of a sum of
         positive terms, halved by the root, plus the mean's division, eps'
         addition, the root and the reciprocal: at most 48 u.
  y:     rstd's error and two products, then the rounding: h + 50 u, relative.
  dr:    rstd (a - n c) + dres: with A = |a| + |n| |c| the inner error is at
         most A * 8 u plus |n| * |error of c|; c is a mean of products whose
         absolute sum is C = mean|a n|: error at most 90 u C.  So
         rstd (8 u A + 90 u C |n|) + 2 u |dr - dres| + h |dr| .
  dgamma: a sum of T products in fp32 along at most (rows per partial + 64 +
         16) terms: that many u times the sum of absolute products, plus h.
"""
import numpy as np
import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, seed, dtype, std=1.0):
    return (torch.randn(shape, generator=gen(seed)) * std).to(dtype)


def inputs(T, d, dtype, seed=0):
    gamma = (1.0 + 0.3 * torch.randn(d, generator=gen(seed + 3))).to(dtype)
    return randn((T, d), seed + 1, dtype), randn((T, d), seed + 2, dtype, 3.0), gamma


def forward(x, res, gamma, eps=1e-6, mx=False, keep_r=True):
    T, d = x.shape
    desc = zcmoe.NormDesc(T, d, x.dtype, eps)
    xg, gg = x.cuda(), gamma.cuda()
    rg = None if res is None else res.cuda()
    r = torch.full_like(xg, float("nan")) if keep_r else None
    y = torch.full_like(xg, float("nan"))
    rstd = torch.full((T,), float("nan"), device="cuda")
    codes, scales = zcmoe.mx_buffers(T, d) if mx else (None, None)
    zcmoe.zc_rmsnorm_forward(desc, xg, gg, y, res=rg, r=r, rstd=rstd, codes=codes, scales=scales)
    torch.cuda.synchronize()
    return r, y, rstd, codes, scales


def reference(x, res, gamma, eps=1e-6):
    r = x if res is None else (x.float() + res.float()).to(x.dtype)
    rd = r.double()
    rstd = 1.0 / torch.sqrt((rd * rd).mean(-1) + eps)
    return r, rd * rstd[:, None] * gamma.double(), rstd


def check_forward(x, res, gamma, eps=1e-6, mx=False):
    r, y, rstd, codes, scales = forward(x, res, gamma, eps, mx)
    ro, yo, so = reference(x, res, gamma, eps)
    assert torch.equal(r.cpu(), ro)
    assert ((rstd.cpu().double() - so).abs() <= 48 * U * so).all()
    err = (y.cpu().double() - yo).abs()
    # below the smallest normal a step is absolute
    assert (err <= (HALF[x.dtype] + 50 * U) * yo.abs() + 2.0 ** -133).all()
    return r, y, rstd, codes, scales


# widths: one vector, ragged over 64 lanes, each threads-per-row variant and
# its border, the largest
SHAPES = [(1, 8), (3, 24), (5, 512), (7, 520), (1, 1032), (130, 2048), (9, 2056), (4, 4096),
          (6, 6144), (2, 8192), (3, 8200), (2, 16392), (2, 32768)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_forward(T, d, dtype):
    print(f"[norm] T={T} d={d} {dtype}", flush=True)
    x, res, gamma = inputs(T, d, dtype)
    check_forward(x, res, gamma)
    check_forward(x, None, gamma)


def test_forward_fp32_width_of_one_vector():
    x, res, gamma = inputs(5, 4, F32)
    check_forward(x, res, gamma)


def mx_reference(y):
    """MXFP8 of bf16 rows: codes as values, biased scales in block order."""
    v = y.double().numpy().reshape(-1, 32)
    top = np.abs(v).max(1)
    S = np.zeros(len(top))
    nz = top >= 2.0 ** -126
    S[nz] = np.maximum(np.floor(np.log2(top[nz])) - 8 + 127, 0)
    w = np.clip(v * 2.0 ** (127 - S)[:, None], -448, 448)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(w), 2.0 ** -6))) - 3)
    return np.rint(w / step) * step, S


@pytest.mark.parametrize("T,d", [(1, 128), (5, 640), (3, 2048), (257, 6144), (2, 8320), (2, 32768)])
def test_mxfp8_output(T, d):
    print(f"[norm mx] T={T} d={d}", flush=True)
    x, res, gamma = inputs(T, d, BF)
    # blocks of zeros, of subnormals, and of far apart magnitudes
    x[0, :32] = 0
    res[0, :32] = 0
    gamma[-32:] = gamma[-32:] * 2.0 ** -120
    _, y, _, codes, scales = check_forward(x, res, gamma, mx=True)
    q, S = mx_reference(y.cpu())
    got = codes.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(-1, 32)
    np.testing.assert_array_equal(got, q)
    order = scales.cpu().numpy().reshape(T, d // 128, 4)[..., [0, 2, 1, 3]].reshape(-1)
    np.testing.assert_array_equal(order, S)


def test_non_finite_rows_stay_in_their_row():
    x, res, gamma = inputs(6, 640, BF)
    ref = forward(x, res, gamma, mx=True)
    x[1, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4, :] = 0
    res[4, :] = 0
    r, y, rstd, codes, scales = forward(x, res, gamma, mx=True)
    for row in (0, 2, 5):
        for a, b in zip((r, y, rstd, codes, scales), ref):
            assert torch.equal(a[row], b[row])
    assert torch.isnan(y[1]).all() and torch.isnan(rstd[1])
    assert (codes[1] & 0x7f == 0x7f).all()  # the NaN code
    assert rstd[3] == 0 and torch.isnan(y[3, 7])  # 0 * inf; the others are 0
    assert (y[3].float().nan_to_num() == 0).all()
    assert (y[4] == 0).all() and torch.isfinite(rstd[4]) and (scales[4] == 0).all()


@pytest.mark.parametrize("eps", [1e-45, 1e-38, 1e-20, 4.0])
def test_rows_next_to_nothing_and_their_eps(eps):
    x, res, gamma = inputs(4, 264, F32)
    x[0], res[0] = 0, 0
    x[1] *= 1e-22   # squares of the order of the smallest fp32 numbers vanish
    res[1] = 0
    r, y, rstd, _, _ = forward(x, res, gamma, eps)
    ro, yo, so = reference(x, res, gamma, float(np.float32(eps)))
    assert torch.equal(r.cpu(), ro)
    for t in (0, 2, 3):
        assert abs(rstd[t].item() - so[t].item()) <= 48 * U * so[t].item()
    assert (y[0] == 0).all() and torch.isfinite(y).all()


def test_many_narrow_rows():
    """More rows than one grid's workgroups: the grid goes round again."""
    T, d = (1 << 22) + 4099, 8
    x = torch.randn((T, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    gamma = torch.ones(d, dtype=BF, device="cuda")
    y, rstd = torch.full_like(x, float("nan")), torch.empty(T, device="cuda")
    zcmoe.zc_rmsnorm_forward(zcmoe.NormDesc(T, d, BF), x, gamma, y, rstd=rstd)
    xd = x.double()
    s = 1.0 / torch.sqrt((xd * xd).mean(-1) + 1e-6)
    assert ((rstd.double() - s).abs() <= 48 * U * s).all()
    yo = xd * s[:, None]
    assert ((y.double() - yo).abs() <= (HALF[BF] + 50 * U) * yo.abs()).all()


def test_offsets_beyond_32_bits():
    """Rows whose elements lie past 2^31: the last ones against the formula,
    forward (with codes) and backward."""
    T, d, n = 360_000, 6144, 5
    assert T * d > 1 << 31
    x = torch.zeros((T, d), dtype=BF, device="cuda")
    tail, res, gamma = inputs(n, d, BF, 120)
    x[-n:] = tail.cuda()
    desc = zcmoe.NormDesc(T, d, BF)
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    codes, scales = zcmoe.mx_buffers(T, d)
    zcmoe.zc_rmsnorm_forward(desc, x, gamma.cuda(), y, rstd=rstd, codes=codes, scales=scales)
    want = forward(tail, None, gamma, mx=True)
    for a, b in zip((y, rstd, codes, scales), want[1:]):
        assert torch.equal(a[-n:], b)
    assert (y[:-n:1000] == 0).all()
    # backward: the rows in front give nothing but rstd * 0 * gamma = 0
    dy = torch.zeros_like(x)
    dyt = randn((n, d), 121, BF)
    dy[-n:] = dyt.cuda()
    dr, dg = y, torch.empty_like(gamma.cuda())
    zcmoe.zc_rmsnorm_backward(desc, dy, x, gamma.cuda(), rstd, dr, dg)
    ro, tol, go, ga = backward_reference(dyt, tail, gamma, rstd[-n:].cpu(), None)
    assert ((dr[-n:].cpu().double() - ro).abs() <= tol + (HALF[BF] + 2 * U) * ro.abs()).all()
    assert ((dg.cpu().double() - go).abs() <= 90 * U * ga + HALF[BF] * go.abs()).all()
    assert (dr[:-n:1000] == 0).all()


def test_in_place_and_no_kept_sum():
    x, res, gamma = inputs(33, 2056, BF)
    r0, y0, s0, _, _ = forward(x, res, gamma)
    desc = zcmoe.NormDesc(33, 2056, BF)
    xg, rg, gg = x.cuda(), res.cuda(), gamma.cuda()
    zcmoe.zc_rmsnorm_forward(desc, xg, gg, xg, res=rg, r=rg)  # y over x, r over res
    assert torch.equal(xg, y0) and torch.equal(rg, r0)
    y1 = torch.empty_like(y0)
    zcmoe.zc_rmsnorm_forward(desc, x.cuda(), gg, y1, res=res.cuda())
    assert torch.equal(y1, y0)
    dy, dres = randn((33, 2056), 8, BF).cuda(), randn((33, 2056), 9, BF).cuda()
    dr, dg = torch.empty_like(dy), torch.empty_like(gg)
    zcmoe.zc_rmsnorm_backward(desc, dy, r0, gg, s0, dr, dg, dres=dres)
    for target in ("dy", "r", "dres"):
        t = dict(dy=dy.clone(), r=r0.clone(), dres=dres.clone())
        dg2 = torch.empty_like(gg)
        zcmoe.zc_rmsnorm_backward(desc, t["dy"], t["r"], gg, s0, t[target], dg2, dres=t["dres"])
        assert torch.equal(t[target], dr) and torch.equal(dg2, dg), target


def backward_reference(dy, r, gamma, rstd, dres):
    dy, r, g, s = dy.double(), r.double(), gamma.double(), rstd.double()[:, None]
    a, n = dy * g, r * s
    c, C = (a * n).mean(-1, keepdim=True), (a * n).abs().mean(-1, keepdim=True)
    core = s * (a - n * c)
    dr = core + (0 if dres is None else dres.double())
    tol = s * (8 * U * (a.abs() + (n * c).abs()) + 90 * U * C * n.abs()) + 2 * U * core.abs()
    return dr, tol, (dy * n).sum(0), (dy * n).abs().sum(0)


def check_backward(T, d, dtype, with_res=True):
    r, dy, gamma = inputs(T, d, dtype, 40)
    dres = randn((T, d), 50, dtype) if with_res else None
    rstd = (1.0 / torch.sqrt((r.double() ** 2).mean(-1) + 1e-6)).float()
    desc = zcmoe.NormDesc(T, d, dtype)
    dr = torch.full((T, d), float("nan"), dtype=dtype, device="cuda")
    dg = torch.full((d,), float("nan"), dtype=dtype, device="cuda")
    zcmoe.zc_rmsnorm_backward(desc, dy.cuda(), r.cuda(), gamma.cuda(), rstd.cuda(), dr, dg,
                              dres=None if dres is None else dres.cuda())
    torch.cuda.synchronize()
    ro, tol, go, ga = backward_reference(dy, r, gamma, rstd, dres)
    h = HALF[dtype]
    assert ((dr.cpu().double() - ro).abs() <= tol + (h + 2 * U) * ro.abs() + 2.0 ** -133).all()
    depth = T // 512 + 1 + 64 + 16 + 4
    assert ((dg.cpu().double() - go).abs() <= depth * U * ga + h * go.abs() + 2.0 ** -133).all()


@pytest.mark.parametrize("T,d", SHAPES + [(1003, 1544), (2100, 64)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_backward(T, d, dtype):
    print(f"[norm bwd] T={T} d={d} {dtype}", flush=True)
    check_backward(T, d, dtype)
    check_backward(T, d, dtype, with_res=False)


def test_backward_against_differences():
    """The forward's own change along a direction, in fp32 at a step e: the
    difference quotient is off by the third derivative times e^2 and by the
    rounding of y, 2^-24 |y| / e an element."""
    T, d, e = 4, 64, 2.0 ** -7
    x, v, gamma = inputs(T, d, F32, 60)
    w = randn((T, d), 70, F32)
    _, _, s, _, _ = forward(x, None, gamma)
    desc = zcmoe.NormDesc(T, d, F32)
    dr, dg = torch.empty((T, d), device="cuda"), torch.empty(d, device="cuda")
    zcmoe.zc_rmsnorm_backward(desc, w.cuda(), x.cuda(), gamma.cuda(), s, dr, dg)
    dv = v / v.norm()  # direction of length one
    yp = forward(x + e * dv, None, gamma)[1].cpu().double()
    ym = forward(x - e * dv, None, gamma)[1].cpu().double()
    quotient = ((yp - ym) / (2 * e) * w.double()).sum()
    slope = (dr.cpu().double() * dv.double()).sum()
    # with |x| about 1 a value, third derivatives are of order |w| |gamma| / d
    scale = (w.abs() * yp.abs()).sum().item()
    assert abs(quotient - slope) <= e * e * scale + 4 * U * scale / e
    # gamma enters linearly
    t = randn((d,), 71, F32)
    yg = forward(x, None, gamma + t)[1].cpu().double() - forward(x, None, gamma)[1].cpu().double()
    lin = (dg.cpu().double() * t.double()).sum()
    big = (w.double().abs() * (yp.abs() + yg.abs())).sum().item()
    assert abs((yg * w.double()).sum() - lin) <= 200 * U * big


def test_no_rows():
    desc = zcmoe.NormDesc(0, 256, BF)
    e = torch.empty((0, 256), dtype=BF, device="cuda")
    g = torch.ones(256, dtype=BF, device="cuda")
    zcmoe.zc_rmsnorm_forward(desc, e, g, e.clone())
    dg = torch.full_like(g, 5.0)
    zcmoe.zc_rmsnorm_backward(desc, e, e, g, torch.empty(0, device="cuda"), e.clone(), dg)
    assert (dg == 0).all()


def test_runs_on_a_given_stream_and_in_a_graph():
    T, d = 300, 2048
    x, res, gamma = (t.cuda() for t in inputs(T, d, BF, 80))
    desc = zcmoe.NormDesc(T, d, BF)
    r, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(T, device="cuda")
    dr, dg = torch.empty_like(x), torch.empty_like(gamma)
    ws = zcmoe.norm_workspace(desc)

    def step():
        zcmoe.zc_rmsnorm_forward(desc, x, gamma, y, res=res, r=r, rstd=rstd)
        zcmoe.zc_rmsnorm_backward(desc, y, r, gamma, rstd, dr, dg, dres=res, ws=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        x.copy_(inputs(T, d, BF, 90 + k)[0])
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (r, y, rstd, dr, dg)]
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        zcmoe.zc_rmsnorm_forward(desc, x, gamma, y, res=res, r=r, rstd=rstd, stream=other)
        zcmoe.zc_rmsnorm_backward(desc, y, r, gamma, rstd, dr, dg, dres=res, stream=other)
        other.synchronize()
        for a, b in zip(got, (r, y, rstd, dr, dg)):
            assert torch.equal(a, b)


def test_layer_reads_the_normed_rows():
    """Norm, layer and both backward passes in a row: the layer's dx feeds the
    norm's backward, whose residual gradient is the layer output's own."""
    sh = H.synth.CONFIGS["tiny_fp32"]
    L = H.to_dev(H.synth.make_layer(sh, "cpu"))
    desc, nd = H.desc_of(sh), zcmoe.NormDesc(sh.T, sh.d, F32)
    _, res, gamma = (t.cuda() for t in inputs(sh.T, sh.d, F32, 100))
    r, y = torch.empty_like(L["x"]), torch.empty_like(L["x"])
    rstd = torch.empty(sh.T, device="cuda")
    zcmoe.zc_rmsnorm_forward(nd, L["x"], gamma, y, res=res, r=r, rstd=rstd)
    route, out, saved = H.run_forward(desc, dict(L, x=y), saved=True)
    dout = H.synth.make_dy(sh).cuda()
    g = H.run_backward(desc, dict(L, x=y), route, saved, dout)
    dr, dg = torch.empty_like(r), torch.empty_like(gamma)
    zcmoe.zc_rmsnorm_backward(nd, g["dx"], r, gamma, rstd, dr, dg, dres=dout)
    ro, tol, go, ga = backward_reference(g["dx"].cpu(), r.cpu(), gamma.cpu(), rstd.cpu(), dout.cpu())
    assert ((dr.cpu().double() - ro).abs() <= tol + 3 * U * ro.abs()).all()
    assert ((dg.cpu().double() - go).abs() <= 90 * U * ga + U * go.abs()).all()
