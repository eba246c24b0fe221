"""The score gradient of the sequence balance loss at and close to balance,
where k_j - sum_i p_i k_i is a small difference of large numbers.

Picks are dealt out by a rule, so that the counts are known: token t of a
sequence takes the FFN experts (3 t + r) mod N, r = 0..2, and, with
zero-computation experts, one of those.  With T a multiple of N every expert has
the same count and with K_e = 3 every f is 1: the gradient is 0.

Tolerance close to balance (u = 2^-24).  With e_i = exp(l_i - m) (1 + d_i), |d_i|
<= c u, c = R + 4 (the argument is rounded once, R its largest size; expf 2 u and
the reference's own rounding), the weighted mean of k is off by at most
sum_i p_i |d_i| |k_i - q| (1 + 2 c u) <= (c + 1) u M with M = sum_i p_i |k_i - q|
(the same e_i stand in the sum that divides), and p_j by (2 c + 1) u, 1/sum, two
products and one rounding by 4 u more.  The binary64 differences and sums add
2^-48 of the largest |k|.  So
    |error| <= p_j ((2 c + 5) u |k_j - q| + (c + 1) u M + 2^-48 max|k|).
"""
import numpy as np
import pytest
import torch

from tests import test_gpu_balance as B
from moe_layer_zero_amd import zcmoe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def dealt(T, N, Z, t0=0):
    t = torch.arange(t0, t0 + T)[:, None]
    idx = (3 * t + torch.arange(3)) % N
    if Z:
        idx = torch.cat([idx, N + t % Z], 1)
    return idx.int()


# every number of scores a lane, in vectors and one by one
@pytest.mark.parametrize("N", [3, 12, 60, 129, 255, 300, 768, 771, 1023, 1024])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_one_group_and_no_zero_computation_experts_is_exactly_zero(N, T):
    print(f"[balance even] one group N={N} T={T}", flush=True)
    l = B.scores(T, N, N + T, 3.0)
    idx = B.topk(l, min(N, 3))
    K = idx.shape[1]
    for cu in (None, [0, T // 2, T // 2, T]):
        _, _, dl = B.run(l, idx, N, K, zcmoe.LoadBalance(1, float(K), 0.1), cu)
        assert (dl == 0).all(), cu


@pytest.mark.parametrize("N", [2, 5, 32])
def test_every_expert_picked_is_exactly_zero(N):
    T = 50
    l = B.scores(T, N, N, 3.0)
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(N)) < 0.6).to(torch.uint8)
    for D in {1, N}:
        loss, _, dl = B.run(l, B.topk(l, N), N, N, zcmoe.LoadBalance(D, float(N), 0.1), [0, 13, 50], mask)
        assert (dl == 0).all()
        assert abs(loss[0].item() - 0.1) <= 90 * U * 0.1  # f = 1: the softmax's own sum


@pytest.mark.parametrize("N,Z,T", [(12, 4, 12), (12, 0, 48), (12, 4, 24000), (192, 63, 192),
                                   (192, 0, 3840), (768, 256, 1536), (513, 300, 513)])
def test_evenly_filled_sequences_are_exactly_zero(N, Z, T):
    """One batch also holds a sequence that is not even: its own rows only."""
    print(f"[balance even] N={N} Z={Z} T={T}", flush=True)
    K, n = (4, 3) if Z else (3, 3)
    l = B.scores(T + 40, N + Z, T, 3.0)
    idx = torch.cat([dealt(T, N, Z), B.topk(l[T:], K)])
    for D in (1, 3, N):
        _, counts, dl = B.run(l, idx, N, K, zcmoe.LoadBalance(D, float(n), 0.1), [0, T, T + 40])
        assert (counts[0, :N] == counts[0, 0]).all()
        assert (dl[:T] == 0).all()
        if Z or D > 1:
            assert (dl[T:] != 0).any()


@pytest.mark.parametrize("S", [5, 300, 1030])
def test_many_even_sequences_are_exactly_zero(S):
    N, Z, K = 12, 4, 4
    l = B.scores(4 * S, N + Z, S, 3.0)
    idx = torch.cat([dealt(4, N, Z) for _ in range(S)])
    _, _, dl = B.run(l, idx, N, K, zcmoe.LoadBalance(12, 3.0, 0.1), list(range(0, 4 * S + 1, 4)))
    assert (dl == 0).all()


def check_near(l, idx, N, K, D, K_e, alpha=0.1):
    T, E = l.shape
    loss, counts, dl = B.run(l, idx, N, K, zcmoe.LoadBalance(D, K_e, alpha))
    c = np.bincount(idx.reshape(-1).numpy(), minlength=E)
    np.testing.assert_array_equal(counts[0].numpy(), c)
    # k over the common denominator K_e (K - K_e) T^2: whole numbers, K_e = 3
    n = np.zeros(E)
    w = (K - K_e) if E > N else 1.0
    n[:N] = np.repeat(c[:N].reshape(D, -1).sum(1), N // D) * D * w
    n[N:] = c[N:].sum() * K_e
    unit = alpha / (K_e * w * T * T)
    dk = (n - n[0]) * unit
    x = l.double().numpy()
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    diff = dk - (p @ dk)[:, None]
    M = (p * np.abs(diff)).sum(1, keepdims=True)
    e = np.minimum(x.max(1) - x.min(1), 104.0)[:, None] + 4
    tol = p * ((2 * e + 5) * U * np.abs(diff) + (e + 1) * U * M + 2.0 ** -48 * n.max() * unit) + 2.0 ** -140
    err = np.abs(dl.double().numpy() - p * diff)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("N,Z", [(6, 2), (12, 0), (192, 64), (192, 0), (510, 255), (768, 256)])
@pytest.mark.parametrize("rounds", [4, 200])
def test_close_to_balance(N, Z, rounds):
    """All counts alike but for one pick moved."""
    T = N * rounds if N < 100 else N * (rounds // 10 + 1)
    print(f"[balance even] near N={N} Z={Z} T={T}", flush=True)
    l = B.scores(T, N + Z, N + rounds, 1.5)
    idx = dealt(T, N, Z)
    idx[0, 0] = N - 1            # (its own picks are 0, 1, 2)
    for D in (2, N):
        check_near(l, idx, N, idx.shape[1], D, 3.0)


@pytest.mark.parametrize("N,Z", [(9, 0), (192, 64), (765, 0)])
@pytest.mark.parametrize("out", ["first", "last"])
def test_one_expert_without_picks_and_the_others_nearly_even(N, Z, out):
    """k of one expert is far from the others', which differ by one pick in
    hundreds: neither may hide the other."""
    T = 3 * N * (40 if N < 100 else 4)
    print(f"[balance even] outlier N={N} Z={Z} T={T} {out}", flush=True)
    l = B.scores(T, N + Z, N, 1.5)
    l[:, 0 if out == "first" else N - 1] -= 12.0   # it is picked by none: little weight
    idx = dealt(T, N - 1, 0)
    idx[0, 0] = 5
    idx = idx + 1 if out == "first" else idx
    if Z:
        idx = torch.cat([idx, N + torch.arange(T)[:, None] % Z], 1).int()
    check_near(l, idx, N, idx.shape[1], N, 3.0)
