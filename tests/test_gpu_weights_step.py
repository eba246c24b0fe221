"""The calls on a layer's weights as a training run makes them: forward, backward,
the gradients' norm, the AdamW step, the new weights as MXFP4 and the experts on
them, each against its definition in 64 bits; eager, and captured in a graph.
Tolerances are those of the single calls, derived where they are tested.
"""
import dataclasses

import numpy as np
import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests import gpu_harness as H
from tests import test_gpu_mx4 as M
from tests.test_gpu_optim import U, Case, gen

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
N, Z, I, d, K = 4, 2, 512, 1024, 2
SHAPES = [(N + Z, d), (N, I, d), (N, I, d), (N, d, I)]
NAMES = ("wr", "wg", "wu", "wd")


class Layer:
    """A layer whose weights, gradients and states are those of an AdamW case."""

    def __init__(self, T, bits, master, rows):
        self.case = c = Case([int(np.prod(s)) for s in SHAPES], BF, BF, master, bits, seed=T)
        view = lambda k: {n: t.view(s) for n, t, s in zip(NAMES, c.dev[k], SHAPES)}  # noqa: E731
        self.w, self.g = view("p"), view("g")
        self.desc = zcmoe.LayerDesc(T, d, N, Z, I, K, BF)
        self.serve = dataclasses.replace(self.desc, weight_layout=zcmoe.mxfp4_layout(rows))
        self.cfg = zcmoe.AdamW(lr=2e-3, seed=5, rounding=(
            zcmoe.ZC_ROUND_STOCHASTIC if bits == 8 else zcmoe.ZC_ROUND_NEAREST))
        self.grads = zcmoe.TensorList(c.dev["g"])
        self.bias, self.saved = torch.zeros(N + Z, device="cuda"), zcmoe.saved_buffer(self.desc)
        self.route, self.serve_route = zcmoe.RouteBuffers(self.desc), zcmoe.RouteBuffers(self.serve)
        self.norm, self.t = torch.zeros(2, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
        self.q = [[torch.empty((*s[:-1], s[-1] // k), dtype=torch.uint8, device="cuda") for k in (2, 32)]
                  for s in SHAPES[1:]]
        self.sets = zcmoe.pack_mxfp4_expert_weights(self.serve, *self.q)
        self.x = torch.zeros((T, d), dtype=BF, device="cuda")
        self.out, self.served = torch.empty_like(self.x), torch.empty_like(self.x)
        self.dx = torch.empty_like(self.x)

    def batch(self, k):
        self.x.copy_(torch.randn(self.x.shape, generator=gen(100 + k)).to(BF))
        w, g = self.w, self.g
        zcmoe.zc_moe_forward(self.desc, self.x, w["wr"], self.bias, w["wg"], w["wu"], w["wd"], self.out,
                             self.route, self.saved)
        dout = torch.randn(self.x.shape, generator=gen(200 + k)).to(BF).cuda()
        zcmoe.zc_moe_backward(self.desc, self.x, w["wr"], w["wg"], w["wu"], w["wd"], self.route, self.saved,
                              dout, self.dx, g["wr"], g["wg"], g["wu"], g["wd"])

    def step(self):
        zcmoe.zc_grad_norm(self.grads, 0.5, self.norm, step=self.t)
        zcmoe.zc_adamw_step(self.cfg, self.case.t, self.t, factor=self.norm[1:])
        for n, q, s, which in zip(NAMES[1:], self.q, self.sets, (0, 0, 1)):
            zcmoe.zc_mxfp4_quantize(self.w[n], *q)
            zcmoe.zc_moe_mxfp4_pack(self.serve, which, *q, s)
        w = self.w
        zcmoe.zc_moe_forward(self.serve, self.x, w["wr"], self.bias, *self.sets, self.served, self.serve_route)

    def state(self):
        torch.cuda.synchronize()
        return dict(self.case.bytes(), served=self.served.cpu(), norm=self.norm.cpu(), t=self.t.cpu())


@pytest.mark.parametrize("T,bits,master,rows", [(300, 32, True, 8), (9, 8, False, 4), (300, 8, False, 4)])
def test_steps(T, bits, master, rows):
    L = Layer(T, bits, master, rows)
    for k in range(3):
        L.batch(k)
        torch.cuda.synchronize()
        c = L.case
        c.lists = {n: [t.cpu() for t in ts] for n, ts in c.dev.items()}
        L.step()
        torch.cuda.synchronize()
        # the norm, and the factor that it gives
        ref = np.sqrt(sum(float(H.f64(t).__pow__(2).sum()) for t in c.lists["g"]))
        assert ref > 0.5, "the gradients are clipped"
        assert abs(float(L.norm[0]) - ref) <= 1.01 * U * ref
        assert abs(float(L.norm[1]) - 0.5 / ref) <= 2.01 * U * 0.5 / ref
        assert int(L.t) == k + 1
        c.check(L.cfg, k + 1, factor=float(L.norm[1]))
        # the weights' codes, bit for bit
        w = []
        for n, (codes, scales) in zip(NAMES[1:], L.q):
            b = M.blocks(L.w[n].cpu().double().numpy())
            S = M.exponents(np.abs(b).max(-1), 4)
            codes, scales = codes.cpu(), scales.cpu()
            assert (scales.numpy() == S).all()
            assert (M.blocks(M.matrix(codes, scales)) == M.rounded(b, S, 4)).all()
            w.append((codes, scales))
        ref, tol = M.reference(L.serve, L.x.cpu(), w, L.serve_route, rows)
        err = np.abs(L.served.cpu().double().numpy() - ref)
        assert (err <= tol * (1 + M.HB) + M.HB * np.abs(ref) + 2.0 ** -133).all()


@pytest.mark.parametrize("bits,rows", [(32, 8), (8, 4)])
def test_captured_after_the_backward(bits, rows):
    T = 200
    a, b = Layer(T, bits, False, rows), Layer(T, bits, False, rows)
    s = torch.cuda.Stream()
    a.batch(0), b.batch(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b.step()
    torch.cuda.synchronize()
    a.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for k in range(1, 5):
        a.batch(k), b.batch(k)
        a.step()
        graph.replay()
        x, y = a.state(), b.state()
        assert int(x["t"]) == k + 1
        for n in x:
            assert torch.equal(x[n], y[n]), n
