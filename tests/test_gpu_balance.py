"""GPU parity of the balance loss of packed sequences, its per-expert counts
and its score gradient against the formulas in binary64.

Tolerances (u = 2^-24).  The fp32 softmax of one token: the exponent's
argument is rounded once (u |l - m|), expf is off by at most 2 u and the sum
of E <= 1024 terms (at most 16 a lane, then 6 levels) by 22 u, the division
by 2 u: relative error of p at most e_p = (R + 32) u with R the largest
|l - m| of a score whose p counts, capped where p underflows.  q = sum p k
(k rounded once): (R + 60) u q, all terms positive.  The gradient p (k - q):
p |k - q| e_p + p (u k + (R + 60) u q) + 4 u |value|.  A loss is a sum of q
in binary64, rounded once more: (R + 62) u L."""
import numpy as np
import pytest
import torch

from moe_layer_zero_amd import synth, zcmoe
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16


def reference(logits, idx, N, K, D, K_e, alpha, cu, mask):
    T, E = logits.shape
    l = logits.double().numpy()
    with np.errstate(all="ignore"):
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    S = len(cu) - 1
    dl, kk, qq = np.zeros((T, E)), np.zeros((T, E)), np.zeros(T)
    counts, losses, rows = np.zeros((S, E), dtype=np.int64), np.zeros(S), []
    for s in range(S):
        t = np.arange(cu[s], cu[s + 1])
        if mask is not None:
            t = t[mask[t] != 0]
        rows.append(t)
        np.add.at(counts[s], idx[t].reshape(-1), 1)
    used = max(1, sum(len(t) > 0 for t in rows))
    for s, t in enumerate(rows):
        if len(t) == 0:
            continue
        f = np.zeros(E)
        f[:N] = np.repeat(counts[s, :N].reshape(D, N // D).sum(1), N // D) * D / (K_e * len(t))
        if E > N:
            f[N:] = counts[s, N:].sum() / ((K - K_e) * len(t))
        k = alpha * f / (used * len(t))
        q = p[t] @ k
        dl[t] = p[t] * (k - q[:, None])
        kk[t], qq[t] = k, q
        losses[s] = alpha * (p[t].mean(0) * f).sum()
    return counts, np.concatenate([[losses.sum() / used], losses]), dl, p, kk, qq


def run(logits, idx, N, K, lb, cu=None, mask=None, grad=True, **kw):
    T, E = logits.shape
    desc = zcmoe.LayerDesc(T, 64, N, E - N, 64, K, BF)
    route = zcmoe.RouteBuffers(desc)
    route.logits, route.topk_idx = logits.cuda(), idx.cuda()
    S = 1 if cu is None else len(cu) - 1
    loss = torch.full((1 + S,), float("nan"), device="cuda")
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    dl = torch.full((T, E), float("nan"), device="cuda") if grad else None
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    mg = None if mask is None else mask.cuda()
    zcmoe.zc_moe_seq_balance(desc, lb, route, loss, counts, dl, cu_seqlens=cug, mask=mg, **kw)
    torch.cuda.synchronize()
    return loss.cpu(), counts.cpu(), None if dl is None else dl.cpu()


def scores(T, E, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, E), generator=g) * std + 0.7 * torch.randn(E, generator=g)


def check(logits, idx, N, K, D, K_e, alpha, cu, mask=None):
    lb = zcmoe.LoadBalance(D, K_e, alpha)
    loss, counts, dl = run(logits, idx, N, K, lb, cu, mask)
    m = None if mask is None else mask.numpy()
    co, lo, do, p, k, q = reference(logits, idx.long().numpy(), N, K, D, K_e, alpha, cu, m)
    np.testing.assert_array_equal(counts.numpy(), co)
    l = logits.double().numpy()
    R = np.minimum((l.max(1) - l.min(1)), 104.0)[:, None] if l.size else np.zeros((0, 1))
    Q = q[:, None]
    tol = p * np.abs(k - Q) * (R + 32) * U + p * (U * np.abs(k) + (R + 60) * U * np.abs(Q)) \
        + 4 * U * np.abs(do) + 2.0 ** -140
    err = np.abs(dl.double().numpy() - do)
    assert (err <= tol).all(), (err / tol).max()
    Rm = R.max() if R.size else 0.0
    assert (np.abs(loss.double().numpy() - lo) <= (Rm + 62) * U * np.abs(lo)).all()


def topk(l, K):
    return torch.topk(l, K, dim=-1).indices.int()


CASES = [
    # T, N, Z, K, D, cu
    (1, 1, 0, 1, 1, [0, 1]),
    (64, 8, 4, 2, 8, [0, 64]),
    (65, 8, 4, 2, 2, [0, 0, 1, 33, 33, 64]),         # empty ones, one token, a token behind
    (300, 96, 0, 6, 4, [0, 150, 300]),
    (257, 130, 63, 7, 130, [0, 17, 256, 257]),
    (1000, 200, 100, 5, 8, [0, 999, 1000]),
    (333, 500, 268, 12, 500, [0, 333]),              # 12 slots a lane
    (400, 1000, 24, 3, 1, [0, 100, 100, 400]),       # 16 slots, one group of all
    (9001, 64, 32, 8, 64, [0, 9001]),                # counted by many workgroups
    (9001, 64, 32, 8, 8, [0, 1, 2, 300, 301, 5000, 5000, 8999]),
]


@pytest.mark.parametrize("case", CASES, ids=[f"T{c[0]}_N{c[1]}_S{len(c[5]) - 1}" for c in CASES])
@pytest.mark.parametrize("masked", [False, True])
def test_parity(case, masked):
    T, N, Z, K, D, cu = case
    print(f"[balance] {case} masked={masked}", flush=True)
    l = scores(T, N + Z, 7 * T + N)
    mask = None
    if masked:
        mask = (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7).to(torch.uint8) * 3
        if len(cu) > 3:
            mask[cu[-2]:cu[-1]] = 0   # a sequence with nothing left
    check(l, topk(l, K), N, K, D, 0.6 * K if Z else float(K), 0.5, cu, mask)


def test_many_short_sequences():
    T, N, Z, K = 3001, 24, 8, 4
    l = scores(T, N + Z, 5)
    cu = list(range(0, T - 1, 3)) + [T - 1]
    check(l, topk(l, K), N, K, 6, 3.0, 1.0, cu)
    # more of them than tokens
    cu = sorted(list(range(T)) + [1500] * 2000)
    check(l, topk(l, K), N, K, 24, 3.0, 1.0, cu)


def test_one_sequence_is_the_whole_batch_loss():
    T, N, Z, K = 777, 64, 32, 6
    l = scores(T, N + Z, 11)
    desc = zcmoe.LayerDesc(T, 64, N, Z, 64, K, BF)
    route = zcmoe.RouteBuffers(desc)
    route.logits.copy_(l)
    zcmoe.zc_moe_route(desc, None, None, torch.zeros(N + Z, device="cuda"), route)
    lb = zcmoe.LoadBalance(8, 4.0, 0.3)
    whole = zcmoe.zc_moe_lb_loss(desc, lb, route)
    loss, counts, _ = run(l, route.topk_idx.cpu(), N, K, lb)
    assert torch.equal(counts[0], route.counts.cpu())
    R = float((l.max(1).values - l.min(1).values).max())
    assert abs(loss[0].item() - whole[0].item()) <= (R + 62) * U * abs(whole[0].item())
    assert loss[0] == loss[1]


def test_extreme_scores():
    T, N, Z, K = 12, 20, 12, 3
    l = scores(T, N + Z, 21)
    l[1, 4] = 1e30                                   # one expert takes all
    l[2, 5:25] = float("-inf")                       # masked experts
    l[3, :] = torch.finfo(torch.float32).min         # all at the lowest value
    l[4, 3] = torch.finfo(torch.float32).min
    check(l, topk(l, K), N, K, 4, 2.0, 1.0, [0, 6, 12])


def test_masked_tokens_and_tokens_behind_hold_anything():
    T, N, Z, K = 40, 12, 4, 2
    l = scores(T, N + Z, 31)
    idx = topk(l, K)
    cu = [0, 20, 30]
    mask = torch.ones(T, dtype=torch.bool)
    mask[[3, 25]] = False
    lb = zcmoe.LoadBalance(4, 1.5, 1.0)
    want = run(l, idx, N, K, lb, cu, mask)
    l2, idx2 = l.clone(), idx.clone()
    l2[3], l2[25], l2[30:] = float("nan"), float("inf"), float("nan")
    idx2[3], idx2[31] = 1 << 30, -5
    got = run(l2, idx2, N, K, lb, cu, mask)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (got[2][3] == 0).all() and (got[2][25] == 0).all() and (got[2][30:] == 0).all()
    # a NaN in a valid token reaches its sequence's loss and its own row only
    l2 = l.clone()
    l2[22, 0] = float("nan")
    loss, counts, dl = run(l2, idx, N, K, lb, cu, mask)
    assert torch.isnan(loss[0]) and torch.isnan(loss[2]) and loss[1] == want[0][1]
    assert torch.isnan(dl[22]).all() and torch.equal(dl[:22], want[2][:22])


def test_everything_masked_and_no_tokens():
    l = scores(10, 12, 41)
    lb = zcmoe.LoadBalance(4, 1.5, 1.0)
    loss, counts, dl = run(l, topk(l, 2), 8, 2, lb, [0, 4, 10], torch.zeros(10, dtype=torch.uint8))
    assert (loss == 0).all() and (counts == 0).all() and (dl == 0).all()
    e = torch.empty((0, 12))
    loss, counts, _ = run(e, torch.empty((0, 2), dtype=torch.int32), 8, 2, lb, [0, 0, 0])
    assert (loss == 0).all() and (counts == 0).all()


def test_bad_offsets_stay_in_their_buffers():
    l = scores(50, 12, 51)
    idx = topk(l, 2)
    lb = zcmoe.LoadBalance(4, 1.5, 1.0)
    want = run(l, idx, 8, 2, lb, [0, 20, 50])
    got = run(l, idx, 8, 2, lb, [-9, 20, 1 << 30])   # clamped
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    loss, counts, dl = run(l, idx, 8, 2, lb, [0, 40, 10, 50, 5])   # descending: bounded only
    assert (counts >= 0).all() and counts.sum() <= 4 * 100


def test_offsets_beyond_32_bits():
    """Scores past the 2^31st: the last sequence's counts, loss and gradient are
    those of the same tokens with as many sequences in front of them."""
    N, Z, K, n = 512, 256, 2, 40
    T = (1 << 31) // (N + Z) + 1000
    g = torch.Generator(device="cuda").manual_seed(5)
    desc = zcmoe.LayerDesc(T, 64, N, Z, 64, K, BF)
    route = zcmoe.RouteBuffers(desc)
    route.logits.normal_(generator=g)
    route.topk_idx.copy_(torch.randint(0, N + Z, (T, 1), generator=g, device="cuda")
                         + torch.tensor([0, 1], device="cuda"))
    route.topk_idx.remainder_(N + Z)
    lb = zcmoe.LoadBalance(8, 1.3, 1.0)
    cu = torch.tensor([0, T // 3, T - n, T], dtype=torch.int32, device="cuda")
    loss = torch.empty(4, device="cuda")
    counts = torch.empty((3, N + Z), dtype=torch.int32, device="cuda")
    dl = torch.empty((T, N + Z), device="cuda")
    zcmoe.zc_moe_seq_balance(desc, lb, route, loss, counts, dl, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert (counts.long().sum(1) == torch.tensor([T // 3, T - n - T // 3, n], device="cuda") * K).all()
    l, idx = route.logits[-n - 2:].cpu(), route.topk_idx[-n - 2:].cpu()
    small = run(l, idx, N, K, lb, [0, 1, 2, n + 2])
    assert torch.equal(counts[2].cpu(), small[1][2]) and torch.equal(dl[-n:].cpu(), small[2][2:])
    assert abs(loss[3].item() - small[0][3].item()) <= 2 * U * abs(small[0][3].item())


def test_loss_without_gradient_and_reproducible():
    T, N, Z, K = 20000, 128, 64, 8
    l = scores(T, N + Z, 61)
    idx = topk(l, K)
    lb = zcmoe.LoadBalance(16, 6.0, 0.1)
    cu = [0, 7000, 7001, 20000]
    a = run(l, idx, N, K, lb, cu)
    b = run(l, idx, N, K, lb, cu)
    c = run(l, idx, N, K, lb, cu, grad=False)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_gradient_against_differences():
    """f held fixed, L is smooth in the scores: the binary64 loss at l +- e v
    (picks kept) against <dlogits, v>, off by e^2 times third derivatives
    (at most |k| each) and by the gradient's own tolerance."""
    T, N, Z, K, D, K_e, alpha, cu = 30, 12, 6, 3, 4, 2.0, 1.0, [0, 11, 30]
    l = scores(T, N + Z, 71)
    idx = topk(l, K)
    _, _, dl = run(l, idx, N, K, zcmoe.LoadBalance(D, K_e, alpha), cu)
    v = torch.randn((T, N + Z), generator=torch.Generator().manual_seed(72)).double()
    e = 1e-4
    lp = reference(l.double() + e * v, idx.long().numpy(), N, K, D, K_e, alpha, cu, None)
    lm = reference(l.double() - e * v, idx.long().numpy(), N, K, D, K_e, alpha, cu, None)
    slope = (lp[1][0] - lm[1][0]) / (2 * e)
    vm = float(v.abs().max())
    third = 8 * np.abs(lp[4]).max(1).sum() * vm ** 3
    grad_tol = 100 * U * (lp[3] * (np.abs(lp[4]) + np.abs(lp[5][:, None])) * v.abs().numpy()).sum()
    assert abs(slope - float((dl.double() * v).sum())) <= e * e * third + grad_tol + 1e-15 / e


def test_graph_replays_and_other_streams():
    T, N, Z, K = 9000, 64, 32, 8
    desc = zcmoe.LayerDesc(T, 64, N, Z, 64, K, BF)
    lb = zcmoe.LoadBalance(8, 6.0, 0.1)
    for tok, cu in ((9000, [0, 4000, 9000]), (500, [0, 20, 500])):
        desc.T = tok
        route = zcmoe.RouteBuffers(desc)
        cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
        outs = [(torch.empty(3, device="cuda"), torch.empty((2, N + Z), dtype=torch.int32, device="cuda"),
                 torch.empty((tok, N + Z), device="cuda")) for _ in range(2)]
        ws = zcmoe.seq_balance_workspace(desc, 2)

        def step(o, **kw):
            zcmoe.zc_moe_seq_balance(desc, lb, route, o[0], o[1], o[2], cu_seqlens=cug, **kw)

        l = scores(tok, N + Z, 80)
        route.logits.copy_(l)
        route.topk_idx.copy_(topk(l, K))
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step(outs[0], ws=ws)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(outs[0], ws=ws)
        for k in range(3):
            l = scores(tok, N + Z, 81 + k)
            route.logits.copy_(l)
            route.topk_idx.copy_(topk(l, K))
            g.replay()
            torch.cuda.synchronize()
            other = torch.cuda.Stream()
            step(outs[1], stream=other)
            other.synchronize()
            for a, b in zip(*outs):
                assert torch.equal(a, b)


@pytest.mark.parametrize("gate_norm", [0, 1])
@pytest.mark.parametrize("with_lb", [False, True])
def test_backward_adds_the_score_gradient(gate_norm, with_lb):
    """Route, forward, balance loss, backward: the layer is linear in its
    score gradient, so dw_router and dx differ from those without it by
    dlogits^T x and dlogits w_router (fp32 layer: 1e-4 of the largest value,
    the tolerance of fp32 layers here)."""
    sh = synth.CONFIGS["tiny_fp32"]
    L = H.to_dev(synth.make_layer(sh, "cpu"))
    desc = H.desc_of(sh, gate_norm)
    route, out, saved = H.run_forward(desc, L, saved=True)
    dout = synth.make_dy(sh).cuda()
    E = sh.N + sh.Z
    loss = torch.empty(3, device="cuda")
    counts = torch.empty((2, E), dtype=torch.int32, device="cuda")
    dl = torch.empty((sh.T, E), device="cuda")
    cu = torch.tensor([0, 20, 60], dtype=torch.int32, device="cuda")
    zcmoe.zc_moe_seq_balance(desc, zcmoe.LoadBalance(4, 1.3, 50.0), route, loss, counts, dl,
                             cu_seqlens=cu)
    lb = zcmoe.LoadBalance(2, 1.3, 1.0) if with_lb else None
    res = []
    for extra in (None, dl):
        g = {k: torch.empty_like(L[w]) for k, w in (("dx", "x"), ("dwr", "wr"), ("dwg", "wg"),
                                                    ("dwu", "wu"), ("dwd", "wd"))}
        zcmoe.zc_moe_backward(desc, L["x"], L["wr"], L["wg"], L["wu"], L["wd"], route, saved, dout,
                              g["dx"], g["dwr"], g["dwg"], g["dwu"], g["dwd"], lb=lb, dlogits=extra)
        torch.cuda.synchronize()
        res.append({k: v.double().cpu() for k, v in g.items()})
    dld, x, wr = dl.double().cpu(), L["x"].double().cpu(), L["wr"].double().cpu()
    for k, add in (("dwr", dld.T @ x), ("dx", dld @ wr)):
        want = res[0][k] + add
        assert add.abs().max() > 0
        assert (res[1][k] - want).abs().max() <= 2e-4 * want.abs().max(), k
    for k in ("dwg", "dwu", "dwd"):
        assert torch.equal(res[0][k], res[1][k])
