"""The gradient norm and the AdamW step against their formulas in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32.  Counting each rounding of the
formula once, constants among them (b1, 1 - b1, ... are rounded to fp32):
  g' = factor g: u;  m = b1 m0 + c1 g': at most 5 u (|b1 m0| + |c1 g'|);
  v = b2 v0 + c2 g'^2, all terms positive: at most 7 u v;
  8-bit states are decoded with one rounding (m0) or three (v0): 6 u and 10 u;
  the step s = rate m / (sqrt(v) root + eps): m's error, half of v's, and 17 u: 1 -
  b^t to 3 u (its argument, and 1 ulp of expm1), so rate to 5 (lr, quotient) and root to
  3.5 (half of 3, sqrt, quotient); sqrt, eps, the two products and the sum one each (5);
  the hardware's reciprocal (1 ulp) two, and the product with it one;
  p = p keep - s: two for the product, one for the difference.
Weights in bf16 add half a step of theirs, 2^-8 |p| (a whole one where they are
rounded stochastically); 8-bit codes half a step or a whole one likewise.
"""
import ctypes as C

import numpy as np
import pytest
import torch

from moe_layer_zero_amd import zcmoe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SIZES = [1, 7, 8, 0, 127, 128, 129, 1000, 4097, 70001]


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ norm
def norm_of(tensors, max_norm=1.0, step=None):
    out = torch.full((2,), -7.0, device="cuda")
    zcmoe.zc_grad_norm(zcmoe.TensorList(tensors), max_norm, out, step=step)
    return out.cpu().double()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [[1], [5], [0, 3, 0], SIZES, [8191, 8192, 8193], [3] * 500 + [40000] * 3,
                                   [3_000_001]])
def test_norm(dtype, sizes):
    g = gen(len(sizes) + sizes[-1])
    ts = [torch.randn(n, generator=g).to(dtype) for n in sizes]
    ref = float(torch.cat([t.double() for t in ts]).square().sum().sqrt())
    dev = [t.cuda() for t in ts]
    step = torch.tensor([41], device="cuda")
    out = norm_of(dev, 0.25 * ref, step)
    # sums in 64 bits: the rounding to fp32 is what is left
    assert abs(float(out[0]) - ref) <= 1.01 * U * ref
    assert abs(float(out[1]) - 0.25) <= 1.01 * U * 0.25
    assert int(step) == 42
    assert float(norm_of(dev, 4.0 * ref)[1]) == 1.0 == float(norm_of(dev, float("inf"))[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_large_and_small_values(dtype):
    # squares beyond fp32, and below it
    for v in (1e30, 1e-30):
        t = torch.full((1000,), v, device="cuda").to(dtype)
        ref = float(t.double().square().sum().sqrt())
        assert abs(float(norm_of([t], ref)[0]) - ref) <= 1.01 * U * ref


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norm_not_finite(bad):
    ts = [torch.ones(n, device="cuda") for n in (5, 3000, 40000)]
    ts[2][39999] = bad
    step = torch.tensor([3], device="cuda")
    out = norm_of(ts, 1.0, step)
    assert not np.isfinite(float(out[0])) and float(out[1]) == 0.0 and int(step) == 3


def test_norm_of_nothing():
    step = torch.tensor([0], device="cuda")
    for ts in ([torch.empty(0, device="cuda")], [torch.zeros(5, device="cuda")]):
        out = norm_of(ts, 1.0, step)
        assert out.tolist() == [0.0, 1.0]
    assert int(step) == 2


def test_norm_beyond_fp32():
    # factor 0 is for norms that are not finite: this one is, in 64 bits
    step = torch.tensor([0], device="cuda")
    out = norm_of([torch.full((4,), 3e38, device="cuda")], 1e-9, step)
    assert out[0] == float("inf") and 0 < float(out[1]) <= 2.0 ** -148 and int(step) == 1


def test_norm_of_an_empty_list():
    step = torch.tensor([0], device="cuda")
    assert norm_of([], 1.0, step).tolist() == [0.0, 1.0] and int(step) == 1


def test_norm_is_the_same_each_time():
    ts = [torch.randn(n, device="cuda") for n in (100, 5_000_011, 77)]
    first = norm_of(ts, 1.0)
    for _ in range(5):
        assert torch.equal(norm_of(ts, 1.0), first)


# ----------------------------------------------------------------- AdamW
def mix(x):
    M = np.uint64(0xFFFFFFFF)
    x = x * np.uint64(0x9E3779B1) & M
    x = x ^ x >> np.uint64(15)
    x = x * np.uint64(0x85EBCA77) & M
    return x ^ x >> np.uint64(13)


def noise(n, seed, t, place, first=0):
    """The 32 random bits of elements first .. first + n - 1 of a tensor."""
    M = 0xFFFFFFFF
    i = np.arange(first, first + n, dtype=np.uint64)
    key = (seed + 0x9E3779B9 * place & M) ^ (t * 0x85EBCA77 & M)
    k = np.uint64(key) + (i >> np.uint64(32)) * np.uint64(0xC2B2AE3D) & np.uint64(M)
    return mix((i & np.uint64(M)) ^ k)


def unit_of(a):
    """Distance of the E4M3 values around a >= 0."""
    return 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)


def check_codes(x, tol, codes, scale, r, root):
    """codes * scale stand for x (64 bits, each known to tol): nearest, or down
    after r of a distance."""
    n = x.size
    c = codes.astype(np.float64)
    s = np.repeat(scale.astype(np.float64), 128)[:n]
    pad = -n % 128
    top = np.pad(np.abs(x), (0, pad)).reshape(-1, 128).max(1)
    slack = np.pad(tol, (0, pad)).reshape(-1, 128).max(1)
    want = np.maximum(top / 448, 2.0 ** -120)
    assert (np.abs(scale - want) <= slack / 448 + 3 * U * want).all()
    a = np.abs(x) / s
    unit = unit_of(a)
    off = tol / s + 4 * U * a  # in units of the scale: x's error, and the quotient's roundings
    got = np.abs(c)
    if r is None:
        fine = np.abs(got - a) <= unit / 2 + off
    else:
        # between the neighbours that a - off and a + off go to, 448 at most
        lo, hi = (np.floor(np.maximum(v, 0) / unit_of(np.maximum(v, 0)) + r) * unit_of(np.maximum(v, 0))
                  for v in (a - off, a + off))
        fine = (got >= np.minimum(lo, 448)) & (got <= np.minimum(hi, 448))
    if root:
        fine |= (got == 2.0 ** -9) & (a <= 2.0 ** -9 + off)
        assert ((got > 0) | (x == 0)).all()
    assert fine.all(), np.flatnonzero(~fine)[:5]
    assert (np.sign(c) * np.sign(x) >= 0).all()


class Case:
    """Tensors of an AdamW step in larger buffers, whose ends stay as they were."""

    def __init__(self, sizes, dtype, gdtype, master, bits, seed=1, spread=1.0):
        g = gen(seed)
        self.bits, self.sizes, self.buf = bits, sizes, {}
        rnd = lambda n: torch.randn(n, generator=g)  # noqa: E731
        p = [rnd(n) * 0.02 for n in sizes]
        gr = [rnd(n) * 1e-3 * torch.exp(spread * rnd(n)) for n in sizes]
        m = [0.3e-3 * rnd(n) for n in sizes]
        r = [(0.5e-3 * rnd(n)).abs() + 1e-5 for n in sizes]
        self.decay = [0.1 * (i % 3) for i in range(len(sizes))]
        self.lists = dict(p=[t.to(dtype) for t in p], g=[t.to(gdtype) for t in gr])
        if master:
            self.lists["master"] = p
        if bits == 8:
            for k, ts in (("m", m), ("v", r)):
                sc, co = [], []
                for t in ts:
                    b = torch.nn.functional.pad(t, (0, -t.numel() % 128)).view(-1, 128)
                    s = b.abs().amax(1) / 448
                    sc.append(s)
                    co.append((b / s[:, None]).to(F8).view(-1)[:t.numel()].clone())
                self.lists[k], self.lists[k + "_scale"] = co, sc
        else:
            self.lists["m"], self.lists["v"] = m, [t * t for t in r]
        self.dev = {k: [self.inside(k, i, t) for i, t in enumerate(ts)] for k, ts in self.lists.items()}
        d = self.dev
        self.t = zcmoe.AdamWTensors(d["p"], d["g"], d["m"], d["v"], master=d.get("master"),
                                    m_scale=d.get("m_scale"), v_scale=d.get("v_scale"),
                                    weight_decay=self.decay)

    def inside(self, k, i, t):
        b = torch.full((t.numel() * t.element_size() + 64,), 0x5a, dtype=torch.uint8, device="cuda")
        self.buf[k, i] = b
        v = b[:t.numel() * t.element_size()].view(t.dtype)
        v.view(torch.uint8).copy_(t.contiguous().view(torch.uint8))
        return v

    def get(self, k, i):
        t = self.dev[k][i].cpu()
        return t.float().double().numpy() if t.dtype in (BF, F8) else t.double().numpy()

    def bytes(self):
        return {k: b.cpu() for k, b in self.buf.items()}

    def check(self, cfg, t, factor=1.0, lr=None):
        """The step that was made against the formula on what was there before."""
        for b in self.buf.values():
            assert bool((b[-64:] == 0x5a).all())
        f = lambda x: np.float64(np.float32(x))  # noqa: E731  as it is held on the device
        lr, factor = cfg.lr if lr is None else f(lr), f(factor)
        sr = cfg.rounding == zcmoe.ZC_ROUND_STOCHASTIC
        for i, n in enumerate(self.sizes):
            if n == 0:
                continue
            L = {k: (ts[i].float() if ts[i].dtype in (BF, F8) else ts[i]).double().numpy()
                 for k, ts in self.lists.items()}
            g = factor * L["g"]
            m0, v0, e8 = L["m"], L["v"], self.bits == 8
            if e8:
                m0 = m0 * np.repeat(L["m_scale"], 128)[:n]
                v0 = (v0 * np.repeat(L["v_scale"], 128)[:n]) ** 2
            m = cfg.beta1 * m0 + (1 - cfg.beta1) * g
            tm = (6 if e8 else 5) * U * (np.abs(cfg.beta1 * m0) + np.abs((1 - cfg.beta1) * g))
            v = cfg.beta2 * v0 + (1 - cfg.beta2) * g * g
            rv = (10 if e8 else 7) * U
            p0 = L["master"] if "master" in L else L["p"]
            den = np.sqrt(v / (1 - cfg.beta2 ** t)) + cfg.eps
            rate = lr / (1 - cfg.beta1 ** t)
            step = rate * m / den
            p = p0 * (1 - lr * self.decay[i]) - step
            tp = 3 * U * np.abs(p0) + rate / den * tm + np.abs(step) * (rv / 2 + 17 * U) + U * np.abs(p)
            if "master" in L:
                got = self.get("master", i)
                assert (np.abs(got - p) <= tp).all()
                assert torch.equal(self.dev["p"][i], self.dev["master"][i].to(BF))
            elif self.lists["p"][i].dtype == F32:
                assert (np.abs(self.get("p", i) - p) <= tp).all()
            elif not sr:
                assert (np.abs(self.get("p", i) - p) <= tp + 2.0 ** -8 * np.abs(p)).all()
            else:
                r = (noise(n, cfg.seed, t, i) * np.uint64(0xC2B2AE3D) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)
                got, d = np.abs(self.get("p", i)), []
                for a in (np.abs(p) - tp, np.abs(p) + tp):
                    a = np.maximum(a, 2.0 ** -126)
                    un = 2.0 ** (np.floor(np.log2(a)) - 7)
                    d.append(np.floor(a / un + r.astype(np.float64) / 65536) * un)
                assert ((got >= d[0]) & (got <= d[1])).all()
            if not e8:
                assert (np.abs(self.get("m", i) - m) <= tm).all()
                assert (np.abs(self.get("v", i) - v) <= rv * v).all()
            else:
                z = noise(n, cfg.seed, t, i)
                lo = (z & np.uint64(0xFFFF)).astype(np.float64) / 65536 if sr else None
                hi = (z >> np.uint64(16)).astype(np.float64) / 65536 if sr else None
                root = np.sqrt(v)
                check_codes(m, tm, self.get("m", i), self.get("m_scale", i), lo, False)
                check_codes(root, (rv / 2 + U) * root, self.get("v", i), self.get("v_scale", i), hi, True)


KINDS = [(dt, gd, ma, bits) for dt, gd, ma in ((BF, BF, False), (BF, BF, True), (BF, F32, False),
                                               (BF, F32, True), (F32, F32, False)) for bits in (32, 8)]


@pytest.mark.parametrize("sr", [False, True])
@pytest.mark.parametrize("dtype,gdtype,master,bits", KINDS)
def test_adamw(dtype, gdtype, master, bits, sr):
    c = Case(SIZES, dtype, gdtype, master, bits)
    cfg = zcmoe.AdamW(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, rounding=int(sr), seed=99)
    zcmoe.zc_adamw_step(cfg, c.t, 5)
    c.check(cfg, 5)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("t,kw", [(1, {}), (1, dict(eps=1e-16)), (1000, dict(beta2=0.999)),
                                  (3, dict(beta1=0.0, beta2=0.0)), (2_000_000_000, {}), (7, dict(lr=0.0))])
def test_adamw_settings(bits, t, kw):
    c = Case([300, 5000], F32, F32, False, bits, seed=3)
    cfg = zcmoe.AdamW(**{**dict(lr=1e-2), **kw})
    zcmoe.zc_adamw_step(cfg, c.t, t)
    c.check(cfg, t)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [8, 9, 63, 84, 150])
def test_adamw_many_tensors(bits, count):
    # more than one launch's list, with empty tensors in it: a tensor's place in the
    # list counts for its random bits
    sizes = [(i * 37) % 301 for i in range(count)]
    sizes[0] = sizes[-1] = 0
    c = Case(sizes, BF, BF, False, bits, seed=count)
    cfg = zcmoe.AdamW(rounding=zcmoe.ZC_ROUND_STOCHASTIC, seed=4000000000)
    zcmoe.zc_adamw_step(cfg, c.t, 9)
    c.check(cfg, 9)


@pytest.mark.parametrize("dtype,gdtype,master,bits", KINDS)
def test_adamw_long_tensors(dtype, gdtype, master, bits):
    # several rounds in a workgroup
    c = Case([9_000_001, 3], dtype, gdtype, master, bits, seed=8)
    cfg = zcmoe.AdamW(rounding=zcmoe.ZC_ROUND_STOCHASTIC, seed=5)
    zcmoe.zc_adamw_step(cfg, c.t, 2)
    c.check(cfg, 2)


def test_adamw_scalars_on_the_device():
    c = Case([1000, 50], BF, BF, True, 32)
    cfg = zcmoe.AdamW(lr=123.0)
    one = lambda v, dt=F32: torch.tensor([v], dtype=dt, device="cuda")  # noqa: E731
    zcmoe.zc_adamw_step(cfg, c.t, one(6, torch.int64), factor=one(0.37), lr=one(2e-3))
    c.check(cfg, 6, factor=0.37, lr=2e-3)


@pytest.mark.parametrize("dtype,gdtype,master,bits", KINDS)
def test_factor_zero_leaves_everything(dtype, gdtype, master, bits):
    c = Case(SIZES, dtype, gdtype, master, bits)
    before = c.bytes()
    zcmoe.zc_adamw_step(zcmoe.AdamW(rounding=1), c.t, 2, factor=torch.zeros(1, device="cuda"))
    after = c.bytes()
    assert all(torch.equal(before[k], after[k]) for k in before)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_first_tensor_empty(bits):
    c = Case([0, 300, 0, 7], BF, BF, True, bits, seed=6)
    cfg = zcmoe.AdamW(lr=1e-3)
    zcmoe.zc_adamw_step(cfg, c.t, 2)
    torch.cuda.synchronize()
    c.check(cfg, 2)


def test_lists_keep_their_memory():
    # a tensor that is given other memory leaves the list with what it was made of
    g, p = torch.full((1000,), 2.0, device="cuda"), torch.ones(1000, device="cuda")
    grads, opt = zcmoe.TensorList([g]), zcmoe.adamw_tensors([p], [g])
    before = p.detach()
    g.data, p.data = torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda")
    torch.full((1000,), 7.0, device="cuda")  # takes no block that the lists still use
    out = torch.zeros(2, device="cuda")
    zcmoe.zc_grad_norm(grads, 1.0, out)
    zcmoe.zc_adamw_step(zcmoe.AdamW(lr=0.5, eps=1e-12), opt, 1)
    assert abs(float(out[0]) - 4000 ** 0.5) < 1e-4 and not bool(p.any())
    assert bool((before - 0.5).abs().max() < 1e-5)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_from_zeros(bits):
    # the first step from zero states moves every weight by about lr against its gradient
    p = [torch.zeros(n, device="cuda") for n in (1, 300)]
    g = [torch.randn(n, device="cuda") + 3 for n in (1, 300)]
    t = zcmoe.adamw_tensors(p, g, bits=bits)
    zcmoe.zc_adamw_step(zcmoe.AdamW(lr=0.5, eps=1e-16), t, 1)
    for q, h in zip(p, g):
        # m / sqrt(v) = +-1 up to the roundings counted above: 5 + 7 / 2 + 17, and 1 for p
        assert bool(((q + 0.5 * torch.sign(h)).abs() <= 0.5 * 27 * U).all())
    if bits == 8:
        assert all(bool((v.float() > 0).all()) for v in t.v)


def test_master_copies():
    p = [torch.randn(33, device="cuda").to(BF)]
    t = zcmoe.adamw_tensors(p, [torch.randn(33, device="cuda").to(BF)], master=True)
    assert torch.equal(t.master[0], p[0].float())


def test_stochastic_rounding_keeps_the_mean():
    # a weight whose step is a tenth of its distance moves that far on average;
    # rounded to nearest it stays
    n = 1 << 20
    p = [torch.ones(n, dtype=BF, device="cuda")]
    g = [torch.full((n,), -1.0, dtype=BF, device="cuda")]
    lr = 0.1 * 2.0 ** -7
    for rounding in (0, 1):
        t = zcmoe.adamw_tensors(p, g)
        for k in range(1, 5):
            zcmoe.zc_adamw_step(zcmoe.AdamW(lr=lr, rounding=rounding, seed=7), t, k)
        moved = float((p[0].double() - 1).mean()) / (4 * lr)
        if rounding == 0:
            assert moved == 0.0
        else:
            # 4 n draws of variance below 0.25 distances squared: six deviations of the mean
            assert abs(moved - 1) <= 6 * 0.5 * (4 * n) ** -0.5 * 2.0 ** -7 / lr


def test_second_moment_follows_smaller_gradients():
    # v of a block whose one large gradient stays and whose others shrink: rounded
    # stochastically its states follow on average, to nearest they stand still
    n, steps = 128 * 64, 200
    got = []
    for rounding in (0, 1):
        p = [torch.zeros(n, device="cuda")]
        g = [torch.full((n,), 0.02, device="cuda")]
        g[0][::128] = 1.0
        t = zcmoe.adamw_tensors(p, g, bits=8)
        cfg = zcmoe.AdamW(lr=0.0, beta2=0.99, rounding=rounding, seed=1)
        t.v[0].copy_(torch.full((n,), 44.8, device="cuda").to(F8))
        t.v[0].view(-1, 128)[:, 0] = torch.tensor(448.0).to(F8)
        t.v_scale[0].fill_(1 / 448)
        for k in range(1, steps + 1):
            zcmoe.zc_adamw_step(cfg, t, k)
        r = (t.v[0].float().view(-1, 128) * t.v_scale[0][:, None]).double()
        got.append(float((r[:, 1:] ** 2).mean()))
    v0 = (44.0 / 448) ** 2  # 44.8 as E4M3
    want = 0.99 ** steps * v0 + (1 - 0.99 ** steps) * 0.02 ** 2
    assert abs(got[0] - v0) < 0.01 * v0
    # (the draws' variance comes on top of the mean of v; standing still is six times off)
    assert want * 0.9 < got[1] < want * 1.4


def test_adamw_past_32_bits():
    n = (1 << 32) + 133
    p = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-200:] = 1.0
    t = zcmoe.adamw_tensors([p], [g], bits=8)
    cfg = zcmoe.AdamW(lr=0.3, rounding=1, seed=3)
    zcmoe.zc_adamw_step(cfg, t, 1)
    r = (noise(200, 3, 1, 0, n - 200) * np.uint64(0xC2B2AE3D) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)
    un = 2.0 ** (np.floor(np.log2(0.3)) - 7)
    want = np.floor(0.3 / un + r / 65536) * un
    got = -p[-200:].double().cpu().numpy()
    near = np.abs(0.3 / un + r / 65536 - np.round(0.3 / un + r / 65536)) < 1e-3
    assert ((got == want) | near).all() and not bool(p[:-200].any())
    assert bool((t.v[0][-200:].float() > 0).all()) and not bool(t.v[0][-4000:-400].float().any())
    out = torch.empty(2, device="cuda")
    zcmoe.zc_grad_norm(t.grads, 1.0, out)
    assert abs(float(out[0]) - 200 ** 0.5) <= 1e-6 * 200 ** 0.5


def small_step(bits=8, seed=2):
    c = Case([5000, 77, 0, 128 * 9], BF, BF, False, bits, seed=seed)
    out, step = torch.empty(2, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = zcmoe.grad_norm_workspace(c.t.grads)
    cfg = zcmoe.AdamW(rounding=1, seed=11)

    def one(stream=None):
        zcmoe.zc_grad_norm(c.t.grads, 1e-3, out, step=step, ws=ws, stream=stream)
        zcmoe.zc_adamw_step(cfg, c.t, step, factor=out[1:], stream=stream)

    return c, one, out, step


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_go_on(bits):
    a, eager, _, _ = small_step(bits)
    b, other, _, sb = small_step(bits)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other()
    torch.cuda.current_stream().wait_stream(s)
    eager()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other()
    for k in range(4):
        for x in (a, b):
            for i, g in enumerate(x.dev["g"]):
                g.copy_(torch.randn(g.shape, generator=gen(10 * k + i)).to(BF))
        eager()
        graph.replay()
        torch.cuda.synchronize()
        x, y = a.bytes(), b.bytes()
        assert all(torch.equal(x[j], y[j]) for j in x)
    assert int(sb) == 5


def test_nonfinite_gradient_skips_the_step():
    c, one, out, step = small_step()
    c.dev["g"][0][17] = float("nan")
    before = c.bytes()
    one()
    after = c.bytes()
    assert int(step) == 0 and all(torch.equal(before[k], after[k]) for k in before)
    c.dev["g"][0][17] = 0.5
    one()
    assert int(step) == 1 and not torch.equal(c.bytes()["p", 0], before["p", 0])


def test_nan_gradient_is_not_hidden():
    for bits, rounding in ((32, 0), (8, 0), (8, 1)):
        c = Case([300], F32, F32, False, bits)
        c.dev["g"][0][130] = float("nan")
        zcmoe.zc_adamw_step(zcmoe.AdamW(rounding=rounding), c.t, 2)
        bad = torch.isnan(c.dev["p"][0])
        assert bad.tolist() == [i == 130 for i in range(300)]
        assert bool(torch.isnan(c.dev["m"][0].float())[130])
        assert not bool(torch.isnan(c.dev["m"][0].float())[:128].any())


def test_other_stream():
    a, one, _, _ = small_step()
    b, two, _, _ = small_step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one()
    two(stream=s)
    torch.cuda.synchronize()
    x, y = a.bytes(), b.bytes()
    assert all(torch.equal(x[j], y[j]) for j in x)


def test_binding_refusals():
    f = lambda n, dt=F32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    z8 = lambda n: f(n, torch.uint8).view(F8)  # noqa: E731
    A = zcmoe.AdamWTensors
    ok = A([f(5)], [f(5)], [f(5)], [f(5)])
    for bad in (lambda: A([f(5)], [f(4)], [f(5)], [f(5)]), lambda: A([f(5)], [f(5), f(5)], [f(5)], [f(5)]),
                lambda: A([f(5)], [f(5, BF)], [f(5)], [f(5)]), lambda: A([f(5)], [f(5)], [f(5)], [z8(5)]),
                lambda: A([f(5)], [f(5)], [z8(5)], [z8(5)]),
                lambda: A([f(5)], [f(5)], [z8(5)], [z8(5)], m_scale=[f(2)], v_scale=[f(1)]),
                lambda: A([f(5)], [f(5)], [f(5)], [f(5)], master=[f(5)]),
                lambda: A([f(5)], [f(5)], [f(5)], [f(5)], weight_decay=[0.1, 0.2]),
                lambda: A([f(10)[::2]], [f(5)], [f(5)], [f(5)]),
                lambda: A([f(5), f(5, BF)], [f(5), f(5)], [f(5), f(5)], [f(5), f(5)]),
                lambda: zcmoe.zc_adamw_step(zcmoe.AdamW(), ok, torch.zeros(1, dtype=torch.int32, device="cuda")),
                lambda: zcmoe.zc_adamw_step(zcmoe.AdamW(), ok, torch.zeros(1, dtype=torch.int64)),
                lambda: zcmoe.zc_adamw_step(zcmoe.AdamW(), ok, 1, factor=f(2))):
        with pytest.raises(ValueError):
            bad()
    x = f(5)
    with pytest.raises(zcmoe.ZcError):  # the same tensor twice
        zcmoe.zc_adamw_step(zcmoe.AdamW(), A([x, x], [f(5)] * 2, [f(5), f(5)], [f(5), f(5)]), 1)
    with pytest.raises(zcmoe.ZcError):  # not at a multiple of 16 bytes
        zcmoe.zc_adamw_step(zcmoe.AdamW(), A([f(8)[1:6]], [f(5)], [f(5)], [f(5)]), 1)
    with pytest.raises(zcmoe.ZcError):
        zcmoe.zc_adamw_step(zcmoe.AdamW(), ok, 0)


def test_profile_phases():
    c, one, _, _ = small_step()
    zcmoe.zc_moe_profile(True)
    one()
    got = zcmoe.zc_moe_profile_read()
    zcmoe.zc_moe_profile(False)
    assert {"grad_norm", "adamw"} <= set(got)
    assert C.c_char_p(zcmoe.lib().zc_moe_phase_name(26)).value == b"adamw"
