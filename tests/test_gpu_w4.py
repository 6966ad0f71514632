"""The 4-bit expert weights on the GPU: the quantizer against its definition
bit for bit, the products against float64, the layer against the oracle.

Tolerance of a product, per element, with S = sum |w_j x_j| over the k inputs:
a code times a bf16 value is exact in fp32, sums within a group and over the
groups err by at most 2^-23 of the partial sums each and a scale's product by
2^-24, so (k + 4) 2^-23 S; the rounding to bf16 adds 2^-8 of the result. The
SwiGLU form carries its two sums' errors through silu (slope at most 1.1), and
the fast exponential errs by (2 + 1.2 |a|) 2^-22, so silu by 2^-21 (4 + |a|)
of itself."""

import time

import numpy as np
import pytest
import torch

from mixture_experts_layer_42_b200 import binding as M
from mixture_experts_layer_42_b200 import inputs
from oracle import moe_oracle as O
from tests.gpu_util import Layer, check_routing, check_y, host, to_np

pytestmark = pytest.mark.gpu

BF = torch.bfloat16

# Below fp32's smallest normal number a sum's rounding is no longer relative:
# half of 2^-149 a step, of sums in units of the scale, so (k + 4) 2^-150 scale
# in all, less than 2^-127 of the magnitudes of the weights summed (a code that
# is not 8 counts one scale at least). A result below bf16's smallest normal
# number is off by half of its step there, 2^-134.
TINY = 2.0 ** -127


def quantize(w, group):
    E, n, k = w.shape
    q = torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, k // group, n, dtype=BF, device="cuda")
    M.moe_quantize_w4(w, group, q, s)
    return q, s


def dequantize(q, s, group):
    """[E, n, k] float64 from codes and scales (exact)."""
    E, n, h = q.shape
    c = torch.stack((q & 15, q >> 4), -1).reshape(E, n, 2 * h // group, group).double() - 8
    return (c * s.double().transpose(1, 2).unsqueeze(-1)).reshape(E, n, 2 * h)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("E,n,k,group", [(1, 8, 32, 32), (3, 40, 96, 32), (2, 24, 320, 64), (2, 136, 640, 128),
                                         (1, 8, 128, 128)])
def test_quantizer_matches_its_definition(E, n, k, group, dtype):
    g = torch.Generator().manual_seed(k)
    w = (torch.randn(E, n, k, generator=g) * torch.exp(3 * torch.randn(E, n, 1, generator=g))).to(dtype)
    w[0, 0, :group] = 0
    q, s = quantize(w.cuda(), group)
    v = w.float().reshape(E, n, k // group, group)
    sc = (v.abs().amax(-1) / 7.0).to(BF)
    sc[sc == 0] = 1.0
    c = (v / sc.float().unsqueeze(-1)).round().clamp(-8, 7).add(8).to(torch.uint8).reshape(E, n, k // 2, 2)
    assert torch.equal(s.cpu(), sc.transpose(1, 2))
    assert torch.equal(q.cpu(), c[..., 0] | (c[..., 1] << 4))


def test_quantizer_on_extreme_groups():
    w = torch.zeros(1, 8, 64)
    w[0, 0, 0] = 3e38
    w[0, 1, 1] = 1e-45                       # its seventh rounds to 0
    w[0, 2, 2] = float("nan")
    w[0, 3, 3] = float("-inf")
    w[0, 4, :32] = torch.linspace(-1, 1, 32)
    w[0, 5, 4] = torch.finfo(torch.float32).max
    q, s = quantize(w.cuda(), 32)
    d = dequantize(q, s, 32).cpu()
    assert abs(d[0, 0, 0] / 3e38 - 1) < 2.0 ** -8 and bool((d[0, 0, 1:] == 0).all())
    assert bool((d[0, 1] == 0).all())
    assert bool(d[0, 2, :32].isnan().all()) and bool((d[0, 2, 32:] == 0).all())
    assert bool(d[0, 3, :32].isnan().all()) and bool((d[0, 3, 32:] == 0).all())
    assert abs(d[0, 5, 4] / w[0, 5, 4].double() - 1) < 2.0 ** -8 and bool((d[0, 5, 5:] == 0).all())
    # nearest code: within half a step, plus the clamped end's scale rounding
    assert bool(((d[0, 4, :32] - w[0, 4, :32]).abs() <= (0.5 + 7 * 2.0 ** -8) / 7).all())


class Problem:
    def __init__(self, counts, n, k, group, gather, mats=1, lead=0, tail=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        E = len(counts)
        self.R = lead + sum(counts) + tail
        off = torch.zeros(E + 1, dtype=torch.int64)
        off[1:] = torch.tensor(counts).cumsum(0)
        self.off = off + lead
        self.offsets = self.off.to(torch.int32).cuda()
        xr = 50 if gather else self.R
        self.x = torch.randn(xr, k, generator=g, device="cuda").to(BF)
        self.src = torch.randint(0, xr, (self.R,), generator=g, device="cuda").to(torch.int32) if gather else None
        self.m = [quantize(torch.randn(E, n, k, generator=g, device="cuda") / k ** 0.5, group) for _ in range(mats)]
        self.E, self.n, self.k, self.group = E, n, k, group
        self.ws = M.alloc_workspace_grouped(self.R, E, n, k, BF)
        self.out = torch.full((self.R, n), 7.0, dtype=BF, device="cuda")

    def run(self, stream=None):
        f = M.moe_grouped_matvec_w4 if len(self.m) == 1 else M.moe_grouped_swiglu_w4
        f(self.x, self.src, self.offsets, *(t for m in self.m for t in m), self.out, self.ws, stream=stream)
        return self.out

    def check(self, out=None, status=M.MOE_OK, skip=()):
        out = self.out if out is None else out
        w = [dequantize(*m, self.group) for m in self.m]
        o = self.off.tolist()
        for e in range(self.E):
            r = slice(o[e], o[e + 1])
            if e in skip or o[e] == o[e + 1]:
                continue
            x = self.x[r].double()
            if self.src is not None:
                ok = (self.src[r] >= 0) & (self.src[r] < self.x.shape[0])
                x = self.x[self.src[r].clamp(0, self.x.shape[0] - 1).long()].double() * ok[:, None]
            a, S = x @ w[0][e].T, x.abs() @ w[0][e].abs().T
            da = (self.k + 4) * 2.0 ** -23 * S + TINY * w[0][e].abs().sum(1)
            ref, tol = a, da
            if len(w) == 2:
                b, Sb = x @ w[1][e].T, x.abs() @ w[1][e].abs().T
                sl = a * torch.sigmoid(a)
                ref = sl * b
                db = (self.k + 4) * 2.0 ** -23 * Sb + TINY * w[1][e].abs().sum(1)
                tol = 1.1 * da * (b.abs() + db) + sl.abs() * db \
                    + 2.0 ** -21 * (4 + a.abs()) * ref.abs() + 1e-30
            tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -134
            bad = ((out[r].double() - ref).abs() > tol)
            assert not bool(bad.any()), (e, int(bad.sum()), bad.nonzero()[0].tolist())
        outside = torch.ones(self.R, dtype=torch.bool)
        outside[o[0]:o[-1]] = False
        assert bool((out[outside.cuda()] == 7.0).all())
        assert M.moe_check_error(self.ws) == status


COUNTS = {
    "one_row": [1],
    "few": [0, 1, 2, 3, 4, 5, 0, 6, 7, 8, 9, 0],
    "edges": [15, 16, 17, 31, 32, 33, 0, 40],
    "mid": [16, 9, 1, 8, 0, 17, 5],
    "many": [65, 0, 130, 1],
    "sparse": [0] * 60 + [1] + [0] * 30 + [2],
}


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k,group", [(8, 32, 32), (40, 96, 32), (136, 320, 64), (72, 128, 128), (264, 2176, 128),
                                       (1000, 1056, 32), (128, 4096, 64)])
@pytest.mark.parametrize("counts", sorted(COUNTS))
def test_products(counts, n, k, group, gather, mats):
    p = Problem(COUNTS[counts], n, k, group, gather, mats, lead=2, tail=3, seed=n + k)
    p.run()
    p.check()


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("n", [640, 1280, 2560])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_few_rows_of_many_tiles(group, n, mats):
    # 60 to 480 tiles of one row: at most one, two and more a multiprocessor
    p = Problem([1] * 6 + [0] + [1] * 6, n, 1152, group, False, mats, lead=1, tail=1, seed=n + group)
    p.run()
    p.check()


def test_layer_sizes():
    counts = [0] * 256
    for e in (3, 17, 40, 99, 120, 200, 222, 255):
        counts[e] = 1
    for mats, n, k in ((2, 2048, 7168), (1, 7168, 2048)):
        p = Problem(counts, n, k, 128, mats == 2, mats, seed=mats)
        p.run()
        p.check()


def test_non_finite_inputs_stay_in_their_rows():
    p = Problem([3, 40], 72, 256, 64, False, seed=3)
    good = p.run().clone()
    p.x[1, 5] = float("inf")
    p.x[20, 9] = float("nan")
    p.x[21] = float("-inf")
    out = p.run()
    hit = torch.zeros(43, dtype=torch.bool)
    hit[[1, 20, 21]] = True
    assert torch.equal(out[~hit], good[~hit])
    assert bool(out[20].isnan().all())
    # an infinity gives what the weights say: +-inf, or NaN where the code stands for 0
    w = dequantize(*p.m[0], 64)[0]
    want = (p.x[1].double()[None, :] * w).sum(1)
    nan = want.isnan()
    assert torch.equal(out[1].isnan(), nan) and torch.equal(out[1][~nan].double(), want[~nan])


@pytest.mark.parametrize("mats", [1, 2])
def test_bad_tokens_and_offsets(mats):
    p = Problem([4, 5, 6], 72, 256, 64, True, mats, seed=4)
    p.src[2] = 50
    p.src[7] = -1
    p.run()
    p.check(status=M.MOE_ERR_DEVICE_CHECK)        # those rows are products of zeros
    p = Problem([4, 5, 6], 72, 256, 64, True, mats, seed=5)
    good = p.run().clone()
    p.check()
    p.offsets.copy_(torch.tensor([0, 4, 9, 16], dtype=torch.int32))
    p.out.fill_(7.0)
    p.run()
    assert M.moe_check_error(p.ws) == M.MOE_ERR_DEVICE_CHECK
    assert torch.equal(p.out[:9], good[:9]) and bool((p.out[9:] == 7.0).all())


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("group", [64, 128])
def test_few_rows_of_any_magnitude(group, mats):
    # magnitudes from 2^-100 to 2^60 within a row, rows of one size, of zeros,
    # of a bf16's smallest and largest
    p = Problem([1, 2, 3, 4, 5, 8], 72, 640, group, False, mats, seed=30)
    g = torch.Generator(device="cuda").manual_seed(31)
    e = torch.randint(-100, 60, (p.R, p.k), generator=g, device="cuda").double()
    x = p.x.double()
    x[0] *= 2.0 ** e[0]
    x[1] = 0
    x[2] *= 2.0 ** -100
    x[3] *= 1e-38 / 8
    x[4] *= 2.0 ** (e[4] / 16)
    x[5, :128] = 0
    x[6] = 1.0
    x[7] *= 2.0 ** 60
    p.x.copy_(x.to(BF))
    for q, s in p.m:                                  # the largest input of every 128 has a weight
        big = p.x.abs().reshape(p.R, -1, 128).argmax(-1) + torch.arange(p.k // 128, device="cuda") * 128
        c = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], q.shape[1], -1)
        c[:, :, big.reshape(-1)] = 15
        q.copy_(c[..., 0::2] | (c[..., 1::2] << 4))
    p.run()
    w = [dequantize(*m, group) for m in p.m]
    if mats == 1:
        p.check()
        return
    p.x[0], p.x[7] = p.x[6], p.x[6]                   # (silu's product of such magnitudes overflows)
    p.run()
    p.check()


@pytest.mark.parametrize("mats", [1, 2])
def test_few_rows_with_non_finite_inputs(mats):
    p = Problem([3, 4, 1, 2], 72, 256, 64, False, mats, seed=32)
    good = p.run().clone()
    p.x[1, 5] = float("inf")
    p.x[4, 9] = float("nan")
    p.x[5, 200] = float("-inf")
    out = p.run()
    hit = torch.zeros(10, dtype=torch.bool)
    hit[[1, 4, 5]] = True
    assert torch.equal(out[~hit], good[~hit])
    assert bool(out[4].isnan().all())
    if mats == 1:
        for r, e in ((1, 0), (5, 1)):
            want = (p.x[r].double()[None, :] * dequantize(*p.m[0], 64)[e]).sum(1)
            nan = want.isnan()
            assert torch.equal(out[r].isnan(), nan) and torch.equal(out[r][~nan].double(), want[~nan])


def test_offsets_that_go_back_and_forth():
    # each second pair is bad, the others all hold every row: more tiles than
    # the launch has, and a sum past 2^31 rows
    E, R = 1024, 1 << 22
    p = Problem([0] * E, 8, 32, 32, False, tail=R, seed=33)
    p.offsets.copy_(torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32))
    p.run()
    assert M.moe_check_error(p.ws) == M.MOE_ERR_DEVICE_CHECK
    assert M.moe_check_error(p.ws) == M.MOE_OK


@pytest.mark.parametrize("mats,rows", [(1, 1), (2, 1), (1, 40), (2, 40)])
def test_a_wait_that_runs_out_is_reported(mats, rows):
    # one CTA's first warp waits on a barrier that nothing completes: the call
    # ends after the limit, and the next one is right
    p = Problem([rows, 0, rows], 520, 2048, 128, True, mats, seed=34)
    M.moe_debug_stall_pipeline(1)
    try:
        t0 = time.time()
        p.run()
        status = M.moe_check_error(p.ws)
        elapsed = time.time() - t0
    finally:
        M.moe_debug_stall_pipeline(0)
    assert status == M.MOE_ERR_TIMEOUT
    assert 0.9 < elapsed < 30
    p.run()
    p.check()


def test_no_rows():
    p = Problem([0, 0], 24, 64, 32, False, seed=6)
    p.run()
    assert M.moe_check_error(p.ws) == M.MOE_OK


@pytest.mark.parametrize("mats", [1, 2])
def test_graph_replays_with_other_rows(mats):
    s = torch.cuda.Stream()
    p = Problem([3, 0, 8, 30], 136, 512, 128, True, mats, seed=7)
    with torch.cuda.stream(s):
        p.run(stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        p.run(stream=s)
    for seed, counts in ((8, [0, 41, 0, 0]), (9, [10, 10, 10, 11]), (10, [40, 0, 1, 0])):
        q = Problem(counts, 136, 512, 128, True, mats, seed=seed)
        for a, b in ((p.x, q.x), (p.src, q.src), (p.offsets, q.offsets)):
            a.copy_(b)
        for a, b in zip(p.m, q.m):
            a[0].copy_(b[0])
            a[1].copy_(b[1])
        p.off = q.off
        p.out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        p.check()


def test_two_streams_give_the_same_bits():
    ps = [Problem([1, 0, 9, 33, 2], 520, 1024, 128, True, m, seed=20 + m) for m in (1, 2)]
    first = [p.run().clone() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                p.out.fill_(7.0)
                p.run()
    torch.cuda.synchronize()
    for p, f in zip(ps, first):
        assert torch.equal(p.out, f)
        p.check()


class W4Layer:
    """A layer's bf16 weights in the 4-bit layout."""

    def __init__(self, L, group):
        self.L, self.group = L, group
        names = ("w1", "w3", "w2", "ws1", "ws3", "ws2")
        self.m = {n: None if t is None else quantize(t if t.dim() == 3 else t.unsqueeze(0), group)
                  for n, t in zip(names, L.w)}
        self.w4 = M.w4_weights(group, *(self.m[n] for n in names))

    def _deq(self, name, e=0):
        q, s = self.m[name]
        return dequantize(q[e:e + 1], s[e:e + 1], self.group)[0].cpu().numpy()

    def experts(self):
        return lambda e: tuple(self._deq(n, e) for n in ("w1", "w3", "w2"))

    def shared(self):
        return None if self.m["ws1"] is None else tuple(self._deq(n) for n in ("ws1", "ws3", "ws2"))

    def forward(self):
        L, cfg = self.L, self.L.cfg
        ws = M.alloc_workspace_w4(cfg, L.T)
        y = torch.empty(L.T, cfg.dim, dtype=BF, device="cuda")
        wts = torch.empty(L.T, cfg.topk, dtype=torch.float32, device="cuda")
        idx = torch.empty(L.T, cfg.topk, dtype=torch.int32, device="cuda")
        M.moe_forward_w4(cfg, L.x, L.w_r, L.bias, self.w4, y, ws, weights_out=wts, idx_out=idx)
        assert M.moe_check_error(ws) == M.MOE_OK
        return y, wts, idx


def small(**kw):
    base = inputs.MoEConfig("w4_small", T=40, dim=384, n_routed=16, n_groups=4, topk_groups=2, topk=4,
                            moe_inter=256, n_shared=1, score="sigmoid", bias="normal", route_scale=2.5,
                            dtype="bf16", seed=31)
    return base.with_(**kw)


@pytest.mark.parametrize("kw,group", [
    ({}, 128), (dict(T=1), 64), (dict(T=3, n_shared=0), 32), (dict(T=300, n_shared=2), 128),
    (dict(dim=352, moe_inter=160, T=33), 32),
    (dict(n_groups=1, topk_groups=1, score="softmax", bias="none", route_scale=1.0), 64),
])
def test_layer_matches_the_oracle(kw, group):
    cfg = small(**kw)
    L = Layer(cfg)
    F = W4Layer(L, group)
    y, wts, idx = F.forward()
    r = L.oracle_route()
    rows = np.nonzero(~check_routing(cfg, idx, wts, r))[0]
    yref = O.moe_layer(host(L.x), r["weights"], r["idx"], F.experts(), F.shared(), act_dtype="bf16",
                       tokens=rows)
    check_y(cfg, to_np(y)[rows], yref)


def test_layer_replays_from_a_graph():
    cfg = small(T=12)
    L = Layer(cfg)
    F = W4Layer(L, 128)
    ws = M.alloc_workspace_w4(cfg, L.T)
    y = torch.empty(L.T, cfg.dim, dtype=BF, device="cuda")
    x = L.x.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def run():
        M.moe_forward_w4(cfg, x, L.w_r, L.bias, F.w4, y, ws, stream=s)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
    gen = torch.Generator().manual_seed(11)
    for _ in range(3):
        x.copy_(torch.randn(L.T, cfg.dim, generator=gen).to(BF).cuda())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, y)
        assert M.moe_check_error(ws) == M.MOE_OK
