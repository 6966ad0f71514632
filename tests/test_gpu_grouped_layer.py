"""The grouped products and the 4-bit calls run together as they are used: the
experts' forward and backward pass by the router's assignment, then the
trained experts quantized and served to single tokens."""

import numpy as np
import pytest
import torch

from mixture_experts_layer_42_b200 import binding as M
from mixture_experts_layer_42_b200 import inputs
from oracle import moe_oracle as O
from tests.gpu_util import Layer, check_y, host, to_np
from tests.test_gpu_w4 import W4Layer

pytestmark = pytest.mark.gpu


def cfg_of(dtype, **kw):
    base = inputs.MoEConfig("grouped_layer", T=150, dim=256, n_routed=16, n_groups=4, topk_groups=2, topk=4,
                            moe_inter=192, n_shared=0, score="sigmoid", bias="normal", route_scale=2.5,
                            dtype=dtype, seed=41)
    return base.with_(**kw)


class Step:
    """One training step of a layer's routed experts through the C calls: the
    layer's gate, dispatch and combine, and the grouped products between them."""

    def __init__(self, L):
        self.L = L
        c, dev = L.cfg, L.device
        T, R, E = L.T, L.T * c.topk, c.n_routed
        dt = c.torch_dtype
        e = lambda *s, d=dt: torch.empty(*s, dtype=d, device=dev)
        self.wts, self.idx = e(T, c.topk, d=torch.float32), e(T, c.topk, d=torch.int32)
        self.counts, self.offsets = e(E, d=torch.int32), e(E + 1, d=torch.int32)
        self.src, self.pos = e(R, d=torch.int32), e(R, d=torch.int32)
        self.xp, self.a, self.b = e(R, c.dim), e(R, c.moe_inter), e(R, c.moe_inter)
        self.yp, self.y = e(R, c.dim), e(T, c.dim)
        self.dh, self.dxa, self.dxb = e(R, c.moe_inter), e(R, c.dim), e(R, c.dim)
        self.dw = [e(*w.shape, d=torch.float32) for w in L.w[:3]]
        self.ws = M.alloc_workspace(c, T)
        self.wsg = M.alloc_workspace_grouped(R, E, c.moe_inter, c.dim, dt)

    def forward(self):
        L, c = self.L, self.L.cfg
        w1, w3, w2 = L.w[:3]
        M.moe_gate(c, L.x, L.w_r, L.bias, self.wts, self.idx, self.ws)
        M.moe_dispatch(c, self.idx, L.x, self.counts, self.offsets, self.src, self.pos, self.xp, self.ws)
        M.moe_grouped_matmul(self.xp, self.offsets, w1, self.a, self.wsg)
        M.moe_grouped_matmul(self.xp, self.offsets, w3, self.b, self.wsg)
        self.h = (torch.nn.functional.silu(self.a.float()) * self.b.float()).to(c.torch_dtype)
        M.moe_grouped_matmul(self.h, self.offsets, w2, self.yp, self.wsg)
        M.moe_combine(c, self.yp, self.pos, self.wts, None, self.y, self.ws)
        return self.y

    def backward(self, dy):
        """dx and the weights' gradients of sum(dy * y), the routing held."""
        L, c = self.L, self.L.cfg
        w1, w3, w2 = L.w[:3]
        rows = self.src.long()
        wrow = torch.empty(len(rows), device=L.device)
        wrow[self.pos.reshape(-1).long()] = self.wts.reshape(-1)
        dyp = (dy[rows].float() * wrow[:, None]).to(c.torch_dtype)
        M.moe_grouped_matmul_dx(dyp, self.offsets, w2, self.dh, self.wsg)
        M.moe_grouped_matmul_dw(dyp, self.h, self.offsets, self.dw[2], self.wsg)
        a, b, dh = self.a.float(), self.b.float(), self.dh.float()
        s = torch.sigmoid(a)
        da = (dh * b * s * (1 + a * (1 - s))).to(c.torch_dtype)
        db = (dh * a * s).to(c.torch_dtype)
        M.moe_grouped_matmul_dx(da, self.offsets, w1, self.dxa, self.wsg)
        M.moe_grouped_matmul_dx(db, self.offsets, w3, self.dxb, self.wsg)
        M.moe_grouped_matmul_dw(da, self.xp, self.offsets, self.dw[0], self.wsg)
        M.moe_grouped_matmul_dw(db, self.xp, self.offsets, self.dw[1], self.wsg)
        dx = torch.zeros(L.T, c.dim, dtype=torch.float64, device=L.device)
        dx.index_add_(0, rows, self.dxa.double() + self.dxb.double())
        assert M.moe_check_error(self.ws) == M.MOE_OK and M.moe_check_error(self.wsg) == M.MOE_OK
        return dx


def autograd(L, idx, wts, dy):
    """y, dx and the weights' gradients in float64 by torch's autograd."""
    x = L.x.double().requires_grad_()
    w1, w3, w2 = (w.double().requires_grad_() for w in L.w[:3])
    y = torch.zeros(L.T, L.cfg.dim, dtype=torch.float64, device=x.device)
    for e in range(L.cfg.n_routed):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            h = torch.nn.functional.silu(x[t] @ w1[e].T) * (x[t] @ w3[e].T)
            y = y.index_add(0, t, (h @ w2[e].T) * wts[t, j].double()[:, None])
    (y * dy.double()).sum().backward()
    return y.detach(), x.grad, [w1.grad, w3.grad, w2.grad]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step_matches_autograd(dtype):
    # fp32: rounding only, 1e-4 of the largest value as for the layer; bf16:
    # every intermediate is rounded once (2^-8 relative, half a step), eight of
    # them on the longest path (a, b, h, dyp, dh, da, db, dx): 8 * 2^-8 of the
    # largest value
    L = Layer(cfg_of(dtype))
    s = Step(L)
    y = s.forward()
    g = torch.Generator(device="cuda").manual_seed(42)
    dy = torch.randn(L.T, L.cfg.dim, generator=g, device="cuda").to(L.cfg.torch_dtype)
    dx = s.backward(dy)
    ry, rdx, rdw = autograd(L, s.idx, s.wts, dy)
    tol = 1e-4 if dtype == "f32" else 8 * 2.0 ** -8
    for got, ref in [(y, ry), (dx, rdx)] + list(zip(s.dw, rdw)):
        assert (got.double() - ref).abs().max() <= tol * ref.abs().max()


def test_training_step_repeats_bit_for_bit():
    L = Layer(cfg_of("bf16"))
    s = Step(L)
    dy = torch.randn(L.T, L.cfg.dim, generator=torch.Generator("cuda").manual_seed(43), device="cuda").bfloat16()
    first = None
    for _ in range(3):
        y = s.forward().clone()
        dx = s.backward(dy)
        now = [y, dx] + [d.clone() for d in s.dw]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_a_step_lowers_what_it_descends():
    # one small step along the gradient: the change of f = sum(dy * y) is the
    # gradient's prediction (the weights move by 1e-3 of their size, so the
    # second-order term is about 1e-3 of the first; 2 % leaves it room)
    L = Layer(cfg_of("f32", T=60))
    s = Step(L)
    dy = torch.randn(L.T, L.cfg.dim, generator=torch.Generator("cuda").manual_seed(44), device="cuda")
    f0 = (s.forward().double() * dy.double()).sum().item()
    s.backward(dy)
    want = 0.0
    for w, d in zip(L.w[:3], s.dw):
        step = 1e-3 * (w.double().norm() / d.double().norm()).item()
        w.sub_(step * d)
        want -= step * d.double().square().sum().item()
    f1 = (s.forward().double() * dy.double()).sum().item()
    assert abs((f1 - f0) - want) <= 0.02 * abs(want)


@pytest.mark.parametrize("T", [1, 24])
def test_trained_experts_served_in_4_bits(T):
    # the layer's bf16 weights after a step, quantized, serve a decode batch as
    # the oracle does with the same 4-bit weights
    L = Layer(cfg_of("bf16"))
    s = Step(L)
    s.forward()
    s.backward(torch.randn(L.T, L.cfg.dim, generator=torch.Generator("cuda").manual_seed(45),
                           device="cuda").bfloat16())
    for w, d in zip(L.w[:3], s.dw):
        w.sub_((1e-3 * (w.float().norm() / d.norm()) * d).to(w.dtype))
    small = Layer(cfg_of("bf16", T=T), T=T, weights=L.w)
    F = W4Layer(small, 64)
    y, wts, idx = F.forward()
    yref = O.moe_layer(host(small.x), wts.cpu().numpy(), idx.cpu().numpy(), F.experts(), None, act_dtype="bf16")
    check_y(small.cfg, to_np(y), np.asarray(yref))
