"""Cases and plain forms of the operators that follow a layer's weights from
its gradients to 4-bit serving.

Four calls are measured:
  gnorm      the norm of all gradients, the clip factor and the step count
  adamw      an AdamW step over many tensors, states in 32 or in 8 bits
  mx4_rows   rows to MXFP4: codes, scales and the values they stand for
  experts    the expert products of a routed batch from MXFP4 weights, rows in
             MXFP8 (a=8) or MXFP4 (a=4), and the weighted sum of the picks
The plain forms are elementary torch operations in 32 bits (64 for long
sums); with `own` set, run() makes the framework's calls instead.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128  # values that share a scale of the 8-bit states
HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8)
STEP, SEED, DECAY = 7, 12345, 0.1
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def listed():
    return [
        # the gradients of the smallest layer: latency
        dict(name="gnorm_tiny", op="gnorm", d=128, N=8, Z=4, I=64, dtype="fp32"),
        # one device's share of the training layer (16 of its 128 experts)
        dict(name="gnorm_share", op="gnorm", d=2048, N=16, Z=64, I=1024, dtype="bf16"),
        # the smallest layer's step, everything in fp32: latency
        dict(name="adamw_tiny", op="adamw", d=128, N=8, Z=4, I=64, dtype="fp32", gdtype="fp32",
             master=False, bits=32, stochastic=False),
        # many tensors of odd sizes, bf16 weights without a copy in fp32, gradients summed in fp32
        dict(name="adamw_61_ragged", op="adamw", count=61, most=300007, dtype="bf16", gdtype="fp32",
             master=False, bits=8, stochastic=True),
        # the training layer's share: bf16 weights with their fp32 copy, 32-bit states
        dict(name="adamw_share_32", op="adamw", d=2048, N=16, Z=64, I=1024, dtype="bf16", gdtype="bf16",
             master=True, bits=32, stochastic=False),
        # the same in as little memory as it takes
        dict(name="adamw_share_8", op="adamw", d=2048, N=16, Z=64, I=1024, dtype="bf16", gdtype="bf16",
             master=False, bits=8, stochastic=True),
        # a decode batch's rows of a LongCat-sized layer
        dict(name="mx4_rows_256x6144", op="mx4_rows", R=256, C=6144, dtype="bf16"),
        # a prefill batch's rows
        dict(name="mx4_rows_16384x6144", op="mx4_rows", R=16384, C=6144, dtype="bf16"),
        # one token through a LongCat-sized layer: matrix-vector products
        dict(name="experts_a8_1", op="experts", T=1, d=6144, N=512, Z=256, I=2048, K=12, a=8),
        # the decode batch of that layer
        dict(name="experts_a8_256", op="experts", T=256, d=6144, N=512, Z=256, I=2048, K=12, a=8),
        # a small layer at a ragged batch: hundreds of rows an expert
        dict(name="experts_a8_4093", op="experts", T=4093, d=1024, N=64, Z=32, I=512, K=6, a=8),
        # the prefill batch of the LongCat-sized layer
        dict(name="experts_a4_16384", op="experts", T=16384, d=6144, N=512, Z=256, I=2048, K=12, a=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_tensors(rng):
    if rng.random() < 0.5:
        return dict(count=_log(rng, 1, 200), most=_log(rng, 1, 400000))
    return dict(d=64 * _log(rng, 1, 32), N=_log(rng, 1, 16), Z=rng.randint(0, 64), I=64 * _log(rng, 1, 16))


def draw(rng):
    op = rng.choice(["gnorm", "adamw", "adamw", "mx4_rows", "experts", "experts", "experts"])
    if op == "gnorm":
        return dict(op=op, dtype=rng.choice(["bf16", "fp32"]), **_draw_tensors(rng))
    if op == "adamw":
        dt = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, dtype=dt, gdtype=rng.choice([dt, "fp32"]),
                    master=dt == "bf16" and rng.random() < 0.5, bits=rng.choice([8, 32]),
                    stochastic=rng.random() < 0.5, **_draw_tensors(rng))
    if op == "mx4_rows":
        return dict(op=op, R=_log(rng, 1, 16384), C=32 * _log(rng, 1, 192), dtype=rng.choice(["bf16", "fp32"]))
    return dict(op=op, T=_log(rng, 1, 4096), d=128 * rng.randint(1, 16), N=_log(rng, 8, 64),
                Z=rng.randint(0, 32), I=128 * rng.randint(1, 8), K=rng.randint(1, 8), a=rng.choice([4, 8]))


# ------------------------------------------------------------------ inputs
def _gen(seed, code):
    g = torch.Generator(device="cuda")
    g.manual_seed(1013 * seed + code)
    return g


def _randn(shape, seed, code, dtype=torch.float32, std=1.0):
    return torch.randn(shape, generator=_gen(seed, code), device="cuda").mul_(std).to(dtype)


def _sizes(case):
    """Sizes of the tensors, and whether weight decay takes them: a layer's norm
    weight (not), router and expert weights, or `count` tensors of up to `most`."""
    if "count" in case:
        n = [1 + int((case["most"] - 1) * (0.6180339887 * i % 1.0) ** 3) for i in range(1, case["count"] + 1)]
        n[-1] = case["most"]
        return n, [i % 3 != 0 for i in range(len(n))]
    d, w = case["d"], case["N"] * case["I"] * case["d"]
    return [d, (case["N"] + case["Z"]) * d, w, w, w], [False, True, True, True, True]


def _padded(sizes):
    # every tensor begins at a whole block of one buffer
    return [-(-n // BLOCK) * BLOCK for n in sizes]


def _flat(case, seed, code, std, dtype):
    """One buffer with a tensor at the start of each piece and zeros between."""
    sizes = _sizes(case)[0]
    pad = _padded(sizes)
    t = torch.randn(sum(pad), generator=_gen(seed, code), device="cuda").mul_(std)
    at = 0
    for n, p in zip(sizes, pad):
        t[at + n:at + p] = 0
        at += p
    return t.to(dtype)


def _pieces(case, t, per=1):
    sizes = _sizes(case)[0]
    out, at = [], 0
    for n, p in zip(sizes, _padded(sizes)):
        out.append(t[at // per:at // per + (n if per == 1 else p // per)])
        at += p
    return out


def _adamw_inputs(case, seed):
    # gradients of uneven size, states as some steps of such gradients leave them
    sizes, decays = _sizes(case)
    s = dict(p=_flat(case, seed, 1, 0.02, torch.float32))
    n = s["p"].numel()
    size = torch.exp(_randn((n // BLOCK, 1), seed, 2)).mul_(1e-3)
    g = _flat(case, seed, 3, 1.0, torch.float32).view(-1, BLOCK).mul_(size)
    m = _flat(case, seed, 4, 0.3, torch.float32).view(-1, BLOCK).mul_(size)
    r = _flat(case, seed, 5, 0.5, torch.float32).view(-1, BLOCK).mul_(size).add_(0.5 * g).abs_()
    s["g"] = g.view(-1).to(DTYPES[case["gdtype"]])
    if case["bits"] == 8:
        for name, t in (("m", m), ("v", r)):
            scale = (t.abs().amax(-1) / 448.0).clamp(min=2.0 ** -120)
            q = t / scale[:, None]
            s[name], s[name + "s"] = q.clamp(-448, 448).to(F8).view(-1), scale
    else:
        s["m"], s["v"] = m.view(-1), (r * r).view(-1)
    if case["master"]:
        s["master"] = s["p"]
    s["p"] = s["p"].to(DTYPES[case["dtype"]])
    s["factor"] = torch.rand(1, generator=_gen(seed, 6), device="cuda").mul_(0.5).add_(0.5)
    s["step"] = torch.full((1,), STEP, dtype=torch.int64, device="cuda")
    blocks = torch.tensor([p // BLOCK for p in _padded(sizes)], device="cuda")
    s["decay"] = torch.tensor([DECAY if w else 0.0 for w in decays], device="cuda").repeat_interleave(blocks)[:, None]
    if case["stochastic"]:
        # element number inside its tensor, and the tensor's number
        first = torch.cumsum(blocks, 0) - blocks
        which = torch.arange(len(sizes), device="cuda").repeat_interleave(blocks)
        s["block"] = torch.arange(n // BLOCK, device="cuda") - first[which]
        s["which"] = which
    return s


def _largest(scores, K):
    # ties to the lower index
    val, idx = torch.sort(scores, dim=-1, descending=True, stable=True)
    return val[:, :K], idx[:, :K]


def _experts_inputs(case, seed):
    T, d, N, I, E = case["T"], case["d"], case["N"], case["I"], case["N"] + case["Z"]
    K = min(case["K"], E)
    s = dict(x=_randn((T, d), seed, 1, BF), logits=_randn((T, E), seed, 2))
    for i, (name, R, C) in enumerate((("wg", I, d), ("wu", I, d), ("wd", d, I))):
        # the codes of normal weights in blocks of 32 are spread about evenly
        s[name] = torch.randint(0, 256, (N, R, C // 2), generator=_gen(seed, 10 + i), device="cuda",
                                dtype=torch.uint8)
        e = 127 + round(math.log2(1 / (2.93 * math.sqrt(C))))
        s[name + "_s"] = torch.randint(e - 1, e + 2, (N, R, C // 32), generator=_gen(seed, 20 + i),
                                       device="cuda", dtype=torch.uint8)
    top, idx = _largest(s["logits"], K)
    s["idx"], s["gate"] = idx, torch.softmax(top.double(), -1).float()
    return s


def prepare(case, seed):
    op, st = case["op"], dict(case=case)
    if op == "gnorm":
        st["g"] = _flat(case, seed, 1, 1e-3, DTYPES[case["dtype"]])
        st["step"] = torch.full((1,), STEP, dtype=torch.int64, device="cuda")
        st["max"] = 0.5e-3 * math.sqrt(sum(_sizes(case)[0]))
    elif op == "adamw":
        st.update(_adamw_inputs(case, seed))
    elif op == "mx4_rows":
        st["x"] = _randn((case["R"], case["C"]), seed, 1, DTYPES[case["dtype"]])
    else:
        st.update(_experts_inputs(case, seed))
        N = case["N"]
        # the batch's rows expert by expert, each expert's part as long as the longest
        idx = st["idx"].reshape(-1)
        order = torch.sort(idx, stable=True).indices
        counts = torch.bincount(idx, minlength=N + case["Z"])
        first = torch.cumsum(counts, 0) - counts
        place = torch.empty_like(idx)
        place[order] = torch.arange(idx.numel(), device="cuda") - first[idx[order]]
        st["place"], st["most"] = place, max(1, int(counts[:N].max()))
    if own:
        _prepare_own(case, st)
    return st


def _prepare_own(case, st):
    from moe_layer_zero_amd import zcmoe
    st["z"], op = zcmoe, case["op"]
    if op == "gnorm":
        st["grads"] = zcmoe.TensorList(_pieces(case, st["g"]))
        st["out"] = torch.empty(2, device="cuda")
        st["ws"] = zcmoe.grad_norm_workspace(st["grads"])
    elif op == "adamw":
        cut = {k: _pieces(case, st[k]) for k in ("p", "g", "m", "v", "master") if k in st}
        if case["bits"] == 8:
            cut["ms"], cut["vs"] = (_pieces(case, st[k], BLOCK) for k in ("ms", "vs"))
        st["cfg"] = zcmoe.AdamW(**HYPER, seed=SEED,
                                rounding=zcmoe.ZC_ROUND_STOCHASTIC if case["stochastic"] else zcmoe.ZC_ROUND_NEAREST)
        st["opt"] = zcmoe.AdamWTensors(cut["p"], cut["g"], cut["m"], cut["v"], master=cut.get("master"),
                                       m_scale=cut.get("ms"), v_scale=cut.get("vs"),
                                       weight_decay=[DECAY if w else 0.0 for w in _sizes(case)[1]])
    elif op == "mx4_rows":
        st["out"] = zcmoe.mxfp4_buffers(case["R"], case["C"]) + (torch.empty_like(st["x"]),)
    else:
        desc = zcmoe.LayerDesc(case["T"], case["d"], case["N"], case["Z"], case["I"], st["idx"].shape[1], BF,
                               weight_layout=zcmoe.mxfp4_layout(case["a"]))
        st["desc"] = desc
        st["packed"] = zcmoe.pack_mxfp4_expert_weights(
            desc, *((st.pop(n), st.pop(n + "_s")) for n in ("wg", "wu", "wd")))
        st["route"] = zcmoe.RouteBuffers(desc)
        st["route"].logits = st["logits"]
        zcmoe.zc_moe_route(desc, None, None, torch.zeros(desc.E, device="cuda"), st["route"])
        st["ws"] = zcmoe.workspace(desc, zcmoe.ZC_OP_EXPERTS)
        st["out"] = torch.empty((case["T"], case["d"]), dtype=BF, device="cuda")


def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(op, st)
    return {"gnorm": _gnorm, "adamw": _adamw, "mx4_rows": _mx4_rows, "experts": _experts}[op](st)


def _run_own(op, st):
    z = st["z"]
    if op == "gnorm":
        z.zc_grad_norm(st["grads"], st["max"], st["out"], step=st["step"], ws=st["ws"])
        return [st["out"], st["step"]]
    if op == "adamw":
        z.zc_adamw_step(st["cfg"], st["opt"], st["step"], factor=st["factor"])
        return _adamw_outputs(st)
    if op == "mx4_rows":
        codes, scales, values = st["out"]
        z.zc_mxfp4_quantize(st["x"], codes, scales, values=values)
        return [values, scales.view(torch.float8_e8m0fnu)]
    z.zc_moe_experts(st["desc"], st["x"], st["route"], *st["packed"], st["out"], ws=st["ws"])
    return st["out"]


def _adamw_outputs(st):
    return [st[k] for k in ("p", "master", "m", "v", "ms", "vs") if k in st]


# ------------------------------------------------------------- plain forms
def _gnorm(st):
    norm = st["g"].float().square().sum(dtype=torch.float64).sqrt()
    factor = torch.where(norm > st["max"], st["max"] / norm, torch.ones_like(norm))
    factor = torch.where(torch.isfinite(norm), factor, torch.zeros_like(norm))
    st["step"].add_((factor != 0).long())
    return [torch.stack([norm, factor]).float(), st["step"]]


def _noise(st):
    """The step's random bits, 32 for each element, from its number in its tensor,
    the tensor's and the seed."""
    i = st["block"][:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    key = (SEED + 0x9E3779B9 * st["which"]) & 0xFFFFFFFF
    key = (key ^ (st["step"] * 0x85EBCA77)) & 0xFFFFFFFF
    key = key[:, None] + 0xC2B2AE3D * (i >> 32) & 0xFFFFFFFF
    return _mix(i & 0xFFFFFFFF ^ key)


def _noise_p(noise):
    # the 16 bits that round a weight
    return (noise * 0xC2B2AE3D & 0xFFFFFFFF) >> 16


def _mix(x):
    x = x * 0x9E3779B1 & 0xFFFFFFFF
    x = x ^ x >> 15
    x = x * 0x85EBCA77 & 0xFFFFFFFF
    return x ^ x >> 13


def _eight(t, add, floor):
    """t [blocks][128] as E4M3 values times a scale each: rounded to nearest, or
    down after `add` (in steps) is added; floor: no positive value becomes 0."""
    scale = (t.abs().amax(-1) / 448.0).clamp(min=2.0 ** -120)
    q = t / scale[:, None]
    step = torch.exp2((torch.frexp(q.abs()).exponent - 1).clamp(min=-6).to(q.dtype) - 3)
    n = q.abs() / step
    n = torch.round(n) if add is None else torch.floor(n + add)
    if floor:
        n = torch.where((n == 0) & (t > 0), torch.ones_like(n), n)
    return torch.copysign((n * step).clamp(max=448.0), q).to(F8).view(-1), scale


def _adamw(st):
    c, h = st["case"], HYPER
    f = lambda k: st[k].float().view(-1, BLOCK)  # noqa: E731
    g = f("g") * st["factor"]
    m, v = f("m"), f("v")
    if c["bits"] == 8:
        m, v = m * st["ms"][:, None], (v * st["vs"][:, None]).square()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * (g * g)
    t = st["step"].double()
    rate = (h["lr"] / -torch.expm1(t * math.log(h["beta1"]))).float()
    root = (-torch.expm1(t * math.log(h["beta2"]))).rsqrt().float()
    p = f("master") if c["master"] else f("p")
    p = p * (1 - h["lr"] * st["decay"]) - rate * (m / (v.sqrt() * root + h["eps"]))
    noise = _noise(st) if c["stochastic"] else None
    if c["master"]:
        st["master"].copy_(p.view(-1))
    if noise is not None and c["dtype"] == "bf16" and not c["master"]:
        bits = p.view(torch.int32) + _noise_p(noise).int() & -65536
        p = bits.view(torch.float32)
    st["p"].copy_(p.view(-1))
    if c["bits"] == 8:
        lo = hi = None
        if noise is not None:
            lo, hi = (noise & 0xFFFF).float() * 2.0 ** -16, (noise >> 16).float() * 2.0 ** -16
        q, s = _eight(m, lo, False)
        st["m"].copy_(q)
        st["ms"].copy_(s)
        q, s = _eight(v.sqrt(), hi, True)
        st["v"].copy_(q)
        st["vs"].copy_(s)
    else:
        st["m"].copy_(m.view(-1))
        st["v"].copy_(v.view(-1))
    return _adamw_outputs(st)


def _mx(v, emax, top, mantissa):
    """Rows [R][C] in blocks of 32 with a scale 2^(floor(log2 max) - emax) each: the
    values, nearest with ties to even up to `top`, and the biased exponents."""
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1 - emax + 127
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(min=0)
    t = torch.ldexp(b, (127 - e)[..., None])
    low = 0 if mantissa == 1 else -6  # exponent of the smallest normal value
    k = (torch.frexp(t.abs()).exponent - 1).clamp(min=low) - mantissa
    q = torch.ldexp(torch.round(torch.ldexp(t, -k)), k).clamp(-top, top)
    return torch.ldexp(q, (e - 127)[..., None]).view(v.shape), e


def _mx4(v):
    return _mx(v, 2, 6.0, 1)


def _rows(v, a):
    return _mx4(v)[0] if a == 4 else _mx(v, 8, 448.0, 3)[0]


def _mx4_rows(st):
    q, e = _mx4(st["x"].float())
    return [q.to(st["x"].dtype), e.to(torch.uint8).view(torch.float8_e8m0fnu)]


def _weights(codes, scales):
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    w = torch.stack((e2m1[(codes & 15).int()], e2m1[(codes >> 4).int()]), -1).flatten(-2)
    shape = w.shape
    return w.view(*shape[:-1], -1, 32).mul_(torch.exp2(scales.float() - 127)[..., None]).view(shape)


def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _experts(st):
    c = st["case"]
    T, N, d, a = c["T"], c["N"], c["d"], c["a"]
    x, idx, gate = st["x"].float(), st["idx"], st["gate"]
    K = idx.shape[1]
    ident = torch.where(idx < N, torch.zeros_like(gate), gate).sum(-1, keepdim=True)
    gate = torch.where(idx < N, gate, torch.zeros_like(gate))
    xq = _rows(x, a)
    if T * K <= N:
        # few picks: each pick's own weights
        e, most = idx.clamp(max=N - 1).view(-1), 1
        rows = xq[:, None, :].expand(T, K, d).reshape(T * K, d, 1)
        back = torch.arange(T * K, device="cuda")
    else:
        # many: each expert's rows side by side
        most, e = st["most"], slice(None)
        flat = idx.reshape(-1)
        live = flat < N
        back = torch.where(live, flat * most + st["place"], torch.full_like(flat, N * most))
        rows = torch.zeros((N * most + 1, d), device="cuda")
        rows[back] = torch.where(live[:, None], xq[:, None, :].expand(T, K, d).reshape(T * K, d), 0.0)
        rows = rows[:N * most].view(N, most, d).transpose(1, 2)
    h = _silu(torch.bmm(_weights(st["wg"][e], st["wg_s"][e]), rows))
    h = (h * torch.bmm(_weights(st["wu"][e], st["wu_s"][e]), rows)).transpose(1, 2)
    h = _rows(h.reshape(-1, c["I"]), a).view(-1, most, c["I"]).transpose(1, 2)
    y = torch.bmm(_weights(st["wd"][e], st["wd_s"][e]), h).transpose(1, 2).reshape(-1, d)
    y = y[back.clamp(max=y.shape[0] - 1)].view(T, K, d)
    return (ident * x + (gate[..., None] * y).sum(1)).to(BF)


# ------------------------------------------------------------------- bounds
def work(case):
    op = case["op"]
    if op in ("gnorm", "adamw"):
        n = sum(_sizes(case)[0])
        if op == "gnorm":
            return dict(bytes=n * (2 if case["dtype"] == "bf16" else 4), flops=2 * n)
        ps, gs = ((2 if case[k] == "bf16" else 4) for k in ("dtype", "gdtype"))
        # the weights and their states read and written; with an fp32 copy the weights are only written
        per = gs + (ps + 8 if case["master"] else 2 * ps) + (16 if case["bits"] == 32 else 4 + 16.0 / BLOCK)
        return dict(bytes=int(n * per), flops=16 * n)
    if op == "mx4_rows":
        n, es = case["R"] * case["C"], 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=2 * es * n + n // 2 + n // 32, flops=4 * n)
    T, N, E, d, I = case["T"], case["N"], case["N"] + case["Z"], case["d"], case["I"]
    K = min(case["K"], E)
    hit = N * (1.0 - (1.0 - K / E) ** T)  # experts with at least one row, on average
    return dict(bytes=int(hit * 3 * d * I * (0.5 + 1 / 32)) + 4 * T * d + 8 * T * K,
                flops=int(6 * T * K * N / E * d * I))


# ------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "gnorm":
        g = _flat(case, seed, 1, 1e-3, DTYPES[case["dtype"]]).double()
        norm, most = float(torch.linalg.vector_norm(g)), 0.5e-3 * math.sqrt(sum(_sizes(case)[0]))
        return [torch.tensor([norm, min(1.0, most / norm)], dtype=torch.float64), None]
    if op == "adamw":
        return _exact_adamw(case, _adamw_inputs(case, seed))
    if op == "mx4_rows":
        v, e = _exact_blocks(_randn((case["R"], case["C"]), seed, 1, DTYPES[case["dtype"]]).double(), 4)
        return [v, torch.exp2(e - 127.0)]
    return _exact_experts(case, _experts_inputs(case, seed))


def _exact_codes(t, draw, floor):
    # E4M3: steps of 2^-3 of the value's binade, of 2^-9 below 2^-6
    top = torch.maximum(t.abs().amax(-1) / 448, torch.tensor(2.0 ** -120, dtype=torch.float64, device="cuda"))
    a = (t / top[:, None]).abs()
    unit = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    n = torch.round(a / unit) if draw is None else torch.floor(a / unit + draw)
    if floor:
        n[(n == 0) & (t > 0)] = 1
    return (torch.sign(t) * (n * unit).clamp(max=448)).view(-1), top


def _exact_adamw(case, s):
    shape = (-1, BLOCK)
    g = s["g"].double().view(shape) * s["factor"].double()
    m, r = s["m"].double().view(shape), s["v"].double().view(shape)
    if case["bits"] == 8:
        m, r = m * s["ms"].double()[:, None], (r * s["vs"].double()[:, None]) ** 2
    m = HYPER["beta1"] * m + (1 - HYPER["beta1"]) * g
    r = HYPER["beta2"] * r + (1 - HYPER["beta2"]) * g ** 2
    hat_m, hat_v = m / (1 - HYPER["beta1"] ** STEP), r / (1 - HYPER["beta2"] ** STEP)
    p = s["master" if case["master"] else "p"].double().view(shape)
    p = p - HYPER["lr"] * (s["decay"].double() * p + hat_m / (torch.sqrt(hat_v) + HYPER["eps"]))
    out, bits = [p.view(-1)], _noise(s) if case["stochastic"] else None
    if bits is not None and case["dtype"] == "bf16" and not case["master"]:
        unit = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
        draw = _noise_p(bits).double() / 65536
        out = [(torch.sign(p) * torch.floor(p.abs() / unit + draw) * unit).view(-1)]
    if case["master"]:
        out.append(p.view(-1))
    if case["bits"] == 32:
        return out + [m.view(-1), r.view(-1)]
    lo = None if bits is None else (bits % 65536).double() / 65536
    hi = None if bits is None else (bits // 65536).double() / 65536
    (qm, sm), (qv, sv) = _exact_codes(m, lo, False), _exact_codes(torch.sqrt(r), hi, True)
    return out + [qm, qv, sm, sv]


def _exact_blocks(v, a):
    """MXFP4 (a = 4) or MXFP8 (a = 8) values of rows, and their biased exponents."""
    most, emax, low, digits = (6.0, 2, 0, 1) if a == 4 else (448.0, 8, -6, 3)
    b = v.reshape(-1, 32)
    top = b.abs().max(-1).values
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -126))).sub(emax).clamp(min=-127)
    e = torch.where(top > 0, e, torch.full_like(e, -127.0))
    w = b / torch.exp2(e)[:, None]
    unit = torch.exp2(torch.floor(torch.log2(w.abs().clamp(min=2.0 ** low))) - digits)
    q = (torch.round(w / unit) * unit).clamp(-most, most)
    return (q * torch.exp2(e)[:, None]).view(v.shape), e.view(v.shape[0], -1) + 127


def _exact_experts(case, s):
    N, a = case["N"], case["a"]
    x, idx, g = s["x"].double(), s["idx"], s["gate"].double()
    xq = _exact_blocks(x, a)[0]
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2

    def matrix(name, e):
        c = s[name][e].int()
        w = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.float64, device="cuda")
        for i, n in enumerate((c % 16, c // 16)):
            w[:, i::2] = half[n % 8] * torch.where(n < 8, 1.0, -1.0)
        return w * torch.exp2(s[name + "_s"][e].double() - 127).repeat_interleave(32, dim=1)

    out = x * (g * (idx >= N)).sum(1, keepdim=True)
    for e in range(N):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            gate, up = xq[t] @ matrix("wg", e).T, xq[t] @ matrix("wu", e).T
            h = _exact_blocks(gate * torch.sigmoid(gate) * up, a)[0]
            out[t] += g[t, k][:, None] * (h @ matrix("wd", e).T)
    return out
