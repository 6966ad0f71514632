"""The grouped products moe_grouped_matmul, _dx and _dw on the GPU against the
same products in float64.

Tolerance, per element, for a sum of d products of total magnitude
S = sum |a_i b_i|: every product of two bf16 values is exact in fp32 and one of
two fp32 values is rounded inside an fma; d additions in fp32 err by at most
2^-24 each relative to the partial sums (rounded), or twice that (a tensor
core may truncate), so (d + 2) 2^-23 S in all; the rounding of the result to
its type adds eps / 2 of it (2^-8 of a bf16 result), and an accumulated call
one more fp32 addition."""

import time

import pytest
import torch

from mixture_experts_layer_42_b200 import binding as M

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(params=["auto", "simt"])
def kernel(request):
    M.moe_select_expert_kernel(M.MOE_EXPERT_KERNEL_SIMT if request.param == "simt"
                               else M.MOE_EXPERT_KERNEL_AUTO)
    yield request.param
    M.moe_select_expert_kernel(M.MOE_EXPERT_KERNEL_AUTO)


class Problem:
    """Rows for `counts`, after `lead` rows of no expert and before `tail` of
    none; those rows hold NaN, which no result may read."""

    def __init__(self, counts, n, k, dtype, lead=0, tail=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        E = len(counts)
        R = lead + sum(counts) + tail
        off = torch.zeros(E + 1, dtype=torch.int64)
        off[1:] = torch.tensor(counts).cumsum(0)
        self.off = off + lead
        self.offsets = self.off.to(torch.int32).cuda()
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
        self.x, self.dy, self.w = rnd(R, k), rnd(R, n), rnd(E, n, k)
        for t in (self.x, self.dy):
            t[:lead] = float("nan")
            t[R - tail:] = float("nan")
        self.E, self.R, self.n, self.k, self.dtype, self.lead, self.tail = E, R, n, k, dtype, lead, tail
        self.ws = M.alloc_workspace_grouped(R, E, n, k, dtype)

    def spans(self):
        o = self.off.tolist()
        return [(e, slice(o[e], o[e + 1])) for e in range(self.E)]

    def outside(self):
        m = torch.ones(self.R, dtype=torch.bool)
        m[self.off[0]:self.off[-1]] = False
        return m

    def run(self, op, **kw):
        """The operator's output in a buffer of 7s."""
        full = lambda *s, dtype=self.dtype: torch.full(s, 7.0, dtype=dtype, device="cuda")
        if op == "fwd":
            out = full(self.R, self.n)
            M.moe_grouped_matmul(self.x, self.offsets, self.w, out, self.ws, **kw)
        elif op == "dx":
            out = full(self.R, self.k)
            M.moe_grouped_matmul_dx(self.dy, self.offsets, self.w, out, self.ws, **kw)
        else:
            out = full(self.E, self.n, self.k, dtype=kw.pop("dw_dtype", self.dtype))
            M.moe_grouped_matmul_dw(self.dy, self.x, self.offsets, out, self.ws, **kw)
        return out

    def check(self, op, out, base=None):
        d = torch.float64
        eps = torch.finfo(out.dtype).eps / 2
        for e, r in self.spans():
            x, dy, w = self.x[r].to(d), self.dy[r].to(d), self.w[e].to(d)
            if op == "fwd":
                ref, S, depth, got = x @ w.T, x.abs() @ w.abs().T, self.k, out[r]
            elif op == "dx":
                ref, S, depth, got = dy @ w, dy.abs() @ w.abs(), self.n, out[r]
            else:
                ref, S, depth, got = dy.T @ x, dy.abs().T @ x.abs(), x.shape[0], out[e]
                if base is not None:
                    ref = ref + base[e].to(d)
                    S = S + base[e].to(d).abs()
            tol = (depth + 2) * 2.0 ** -23 * S
            tol = tol + eps * (ref.abs() + tol)
            if not bool(((got.to(d) - ref).abs() <= tol).all()):
                bad = ((got.to(d) - ref).abs() > tol).nonzero()
                raise AssertionError(f"{op} expert {e}: {len(bad)} of {ref.numel()} off, first {bad[0].tolist()} "
                                     f"got {got[tuple(bad[0])].item()} ref {ref[tuple(bad[0])].item()}")
        if op != "dw":
            assert bool((out[self.outside().cuda()] == 7.0).all())
        assert M.moe_check_error(self.ws) == M.MOE_OK


COUNTS = {
    "one_row": [1],
    "edges": [0, 1, 2, 15, 16, 17, 0, 31, 32, 33, 63, 64, 65, 0],
    "tiles": [127, 128, 129, 0, 255, 256, 257],
    "long": [300, 0, 1, 513, 777],
    "hot": [0] * 40 + [1500] + [0] * 20 + [3],
    "none": [0, 0, 0],
}
SIZES = [(8, 8), (64, 128), (72, 40), (136, 264), (256, 512), (520, 1032)]


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("counts", sorted(COUNTS))
def test_products(counts, n, k, dtype, op):
    p = Problem(COUNTS[counts], n, k, dtype, lead=3, tail=5, seed=n + k)
    p.check(op, p.run(op))


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("n,k", [(4, 4), (12, 20), (100, 252)])
def test_fp32_sizes_of_four(n, k, op):
    p = Problem([5, 0, 130, 1], n, k, F32, seed=1)
    p.check(op, p.run(op))


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("counts", ["edges", "tiles", "hot"])
def test_bf16_on_both_kernels(counts, op, kernel):
    p = Problem(COUNTS[counts], 200, 328, BF, lead=1, seed=2)
    p.check(op, p.run(op))


@pytest.mark.parametrize("dtype,dw_dtype", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("n,k", [(72, 40), (264, 520)])
def test_dw_types_and_accumulation(n, k, dtype, dw_dtype, kernel):
    p = Problem([0, 1, 40, 129, 300, 0], n, k, dtype, lead=2, tail=2, seed=3)
    out = p.run("dw", dw_dtype=dw_dtype)
    p.check("dw", out)
    assert bool((out[0] == 0).all()) and bool((out[-1] == 0).all())
    base = torch.randn(out.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).to(dw_dtype)
    acc = base.clone()
    M.moe_grouped_matmul_dw(p.dy, p.x, p.offsets, acc, p.ws, accumulate=True)
    p.check("dw", acc, base)
    assert torch.equal(acc[0], base[0]) and torch.equal(acc[-1], base[-1])


def test_many_experts_and_one_expert():
    for counts in ([3] * 1024, [2000]):
        for op in ("fwd", "dx", "dw"):
            p = Problem(counts, 48, 64, BF, seed=5)
            p.check(op, p.run(op))


def test_layer_sizes():
    # the up-projection of the softmax layer, tall experts and idle ones
    counts = torch.multinomial(torch.arange(1.0, 9.0), 3000, replacement=True,
                               generator=torch.Generator().manual_seed(6)).bincount(minlength=8).tolist() + [0]
    p = Problem(counts, 1408, 2048, BF, seed=6)
    for op in ("fwd", "dx", "dw"):
        p.check(op, p.run(op))


@pytest.mark.parametrize("dtype,on", [(F32, "simt"), (BF, "simt"), (BF, "auto")])
@pytest.mark.parametrize("op,n,k", [("fwd", 2056, 264), ("dx", 264, 2056), ("dw", 520, 1032), ("dw", 1032, 1288)])
def test_calls_of_many_tiles(op, n, k, dtype, on):
    # enough tiles for the large ones of either kernel, and for dw's widths of
    # 128 (520 x 1032) and 256 inputs
    counts = [700, 0, 33, 1300, 65] if op != "dw" else [0, 150, 33] * 20 + [65] * 2 if n == 520 else [320] * 23 + [1]
    M.moe_select_expert_kernel(M.MOE_EXPERT_KERNEL_SIMT if on == "simt" else M.MOE_EXPERT_KERNEL_AUTO)
    try:
        p = Problem(counts, n, k, dtype, lead=1, tail=2, seed=n)
        p.check(op, p.run(op))
        if op == "dw":
            base = torch.randn(p.E, n, k, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).to(dtype)
            out = base.clone()
            M.moe_grouped_matmul_dw(p.dy, p.x, p.offsets, out, p.ws, accumulate=True)
            p.check(op, out, base)
    finally:
        M.moe_select_expert_kernel(M.MOE_EXPERT_KERNEL_AUTO)


def test_rows_past_two_to_the_31_elements():
    # 300k rows of 7168: element offsets pass 2^31; the last rows are right
    k, n, R = 7168, 64, 310_000
    x = torch.zeros(R, k, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    tail = torch.randn(300, k, generator=g, device="cuda").to(BF)
    x[-300:] = tail
    w = torch.randn(2, n, k, generator=g, device="cuda").to(BF)
    off = torch.tensor([0, R - 300, R], dtype=torch.int32, device="cuda")
    ws = M.alloc_workspace_grouped(R, 2, n, k, BF)
    y = torch.full((R, n), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_matmul(x, off, w, y, ws)
    ref = tail.double() @ w[1].double().T
    S = tail.double().abs() @ w[1].double().abs().T
    assert bool(((y[-300:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + (k + 2) * 2.0 ** -23 * S).all())
    assert bool((y[:-300] == 0).all())
    dx = x                                             # dx of R x k, its last rows beyond 2^31
    dy = torch.zeros(R, n, dtype=BF, device="cuda")
    dy[-300:] = torch.randn(300, n, generator=g, device="cuda").to(BF)
    M.moe_grouped_matmul_dx(dy, off, w, dx, ws)
    ref = dy[-300:].double() @ w[1].double()
    S = dy[-300:].double().abs() @ w[1].double().abs()
    assert bool(((dx[-300:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + (n + 2) * 2.0 ** -23 * S).all())
    assert bool((dx[:-300] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_non_finite_rows_stay_with_their_expert(dtype):
    # expert 1's rows hold infinities and NaN: expert 0's and 2's results do not
    counts = [20, 7, 30]
    p = Problem(counts, 64, 72, dtype, seed=8)
    ref = {op: p.run(op) for op in ("fwd", "dx", "dw")}
    p.x[20:27, 3] = float("inf")
    p.dy[20:27, 5] = float("nan")
    for op in ("fwd", "dx", "dw"):
        out = p.run(op)
        if op == "dw":
            assert torch.equal(out[0], ref[op][0]) and torch.equal(out[2], ref[op][2])
            assert bool(out[1].isnan().any())
        else:
            assert torch.equal(out[:20], ref[op][:20]) and torch.equal(out[27:], ref[op][27:])
            assert not bool(out[20:27].isfinite().all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_rows(dtype):
    E, n, k = 3, 16, 24
    ws = M.alloc_workspace_grouped(0, E, n, k, dtype)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    e = lambda c: torch.empty(0, c, dtype=dtype, device="cuda")
    w = torch.randn(E, n, k, device="cuda").to(dtype)
    M.moe_grouped_matmul(e(k), off, w, e(n), ws)
    M.moe_grouped_matmul_dx(e(n), off, w, e(k), ws)
    dw = torch.full_like(w, 5.0)
    M.moe_grouped_matmul_dw(e(n), e(k), off, dw, ws, accumulate=True)
    assert bool((dw == 5.0).all())
    M.moe_grouped_matmul_dw(e(n), e(k), off, dw, ws)
    assert bool((dw == 0).all())
    assert M.moe_check_error(ws) == M.MOE_OK


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_bad_offsets_are_reported_and_skipped(dtype, op):
    # expert 1 ends before it begins and expert 3 past the rows: the others are right
    p = Problem([20, 10, 30, 40], 64, 72, dtype, seed=9)
    good = p.run(op)
    p.offsets.copy_(torch.tensor([0, 20, 15, 60, 101], dtype=torch.int32))
    out = p.run(op)
    assert M.moe_check_error(p.ws) == M.MOE_ERR_DEVICE_CHECK
    assert M.moe_check_error(p.ws) == M.MOE_OK
    if op == "dw":
        assert torch.equal(out[0], good[0]) and bool((out[1] == 0).all()) and bool((out[3] == 0).all())
    else:
        # rows 15-19 lie in the ranges of experts 0 and 2: either's result
        assert torch.equal(out[:15], good[:15]) and bool((out[60:] == 7.0).all())
        rows, w = (p.x if op == "fwd" else p.dy)[20:60].double(), p.w[2].double()
        w = w.T if op == "fwd" else w
        ref, S = rows @ w, rows.abs() @ w.abs()
        eps = torch.finfo(dtype).eps / 2
        assert bool(((out[20:60].double() - ref).abs() <= eps * ref.abs() * 1.01 + 74 * 2.0 ** -23 * S).all())


@pytest.mark.parametrize("op", ["fwd", "dx"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_offsets_that_go_back_and_forth(dtype, op):
    # each second pair is bad, the others all hold every row: more tiles than
    # the launch has, and a sum past 2^31 rows
    E, R = 1024, 1 << 22
    p = Problem([0] * E, 8, 8, dtype, tail=R, seed=12)
    p.offsets.copy_(torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32))
    p.run(op)
    assert M.moe_check_error(p.ws) == M.MOE_ERR_DEVICE_CHECK
    assert M.moe_check_error(p.ws) == M.MOE_OK


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
def test_a_wait_that_runs_out_is_reported(op):
    # the first pair's MMA warp waits on a barrier that nothing completes: the
    # call ends after the limit, and the next one is right
    p = Problem([300, 0, 200], 328, 456, BF, seed=13)
    M.moe_debug_stall_pipeline(1)
    try:
        t0 = time.time()
        p.run(op)
        status = M.moe_check_error(p.ws)
        elapsed = time.time() - t0
    finally:
        M.moe_debug_stall_pipeline(0)
    assert status == M.MOE_ERR_TIMEOUT
    assert 0.9 < elapsed < 30
    p.check(op, p.run(op))


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_graph_replays_with_other_offsets(dtype, op):
    # captured once, replayed with other rows and another split of them
    s = torch.cuda.Stream()
    p = Problem([100, 0, 60, 200], 136, 200, dtype, seed=10)
    with torch.cuda.stream(s):
        p.run(op, stream=s)
    torch.cuda.synchronize()
    out = torch.empty((p.E, p.n, p.k) if op == "dw" else (p.R, p.n if op == "fwd" else p.k), dtype=dtype,
                      device="cuda")
    call = {"fwd": lambda: M.moe_grouped_matmul(p.x, p.offsets, p.w, out, p.ws, stream=s),
            "dx": lambda: M.moe_grouped_matmul_dx(p.dy, p.offsets, p.w, out, p.ws, stream=s),
            "dw": lambda: M.moe_grouped_matmul_dw(p.dy, p.x, p.offsets, out, p.ws, stream=s)}[op]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for seed, counts in ((11, [0, 359, 1, 0]), (12, [90, 90, 90, 90])):
        q = Problem(counts, 136, 200, dtype, seed=seed)
        for a, b in ((p.x, q.x), (p.dy, q.dy), (p.w, q.w), (p.offsets, q.offsets)):
            a.copy_(b)
        p.off = q.off
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        p.check(op, out)


def test_two_streams_with_their_own_workspaces():
    ps = [Problem([50, 300, 0, 120], 264, 520, BF, seed=13 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for i, (p, s) in enumerate(zip(ps, streams)):
            with torch.cuda.stream(s):
                outs[i].append([p.run(op) for op in ("fwd", "dx", "dw")])
    torch.cuda.synchronize()
    for p, rounds in zip(ps, outs):
        for o in rounds:
            for op, t in zip(("fwd", "dx", "dw"), o):
                p.check(op, t)
                assert torch.equal(t, rounds[0][("fwd", "dx", "dw").index(op)])   # the same bits every time


def test_gradients_against_differences():
    # f = sum(c * y) is linear in x and in w: its differences are the gradients
    p = Problem([3, 0, 17, 40], 20, 28, F32, seed=15)
    dx, dw = p.run("dx"), p.run("dw")
    c = p.dy.double()

    def f(x, w):
        y = torch.zeros(p.R, p.n, device="cuda")
        M.moe_grouped_matmul(x, p.offsets, w, y, p.ws)
        return (c * y.double()).sum().item()

    g = torch.Generator(device="cuda").manual_seed(16)
    for _ in range(3):
        d = torch.randn(p.x.shape, generator=g, device="cuda")
        want = (dx.double() * d.double()).sum().item()
        got = (f(p.x + d, p.w) - f(p.x - d, p.w)) / 2
        assert abs(got - want) <= 1e-4 * (dx.double() * d.double()).abs().sum().item()
        d = torch.randn(p.w.shape, generator=g, device="cuda")
        want = (dw.double() * d.double()).sum().item()
        got = (f(p.x, p.w + d) - f(p.x, p.w - d)) / 2
        assert abs(got - want) <= 1e-4 * (dw.double() * d.double()).abs().sum().item()


@pytest.mark.parametrize("at", [16, 32, 64, 112, 240])
def test_workspace_at_any_multiple_of_16_bytes(at):
    # dw's maps lie in the workspace: sliced out of a larger tensor, as a pool does
    p = Problem([40, 0, 129, 7, 300], 264, 520, BF, lead=1, tail=2, seed=17)
    n = p.ws.numel()
    pool = torch.full((n + 512,), 0xff, dtype=torch.uint8, device="cuda")
    p.ws = pool[at:at + n]
    assert p.ws.data_ptr() % 256 == at
    M.moe_workspace_init(p.ws)
    for op in ("fwd", "dx", "dw"):
        p.check(op, p.run(op))
    assert bool((pool[:at] == 0xff).all()) and bool((pool[at + n:] == 0xff).all())


def test_dw_of_more_rows_than_a_second_reads():
    # one expert of 2^30 rows, the most there may be: one tile, whose reduction
    # takes longer than the waits' second. Rows of zeros but for 4000
    R, n = 1 << 30, 8
    x = torch.zeros(R, n, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(18)
    rows = torch.cat([torch.randint(0, R, (3998,), generator=g, device="cuda"),
                      torch.tensor([0, R - 1], device="cuda")]).unique()
    x[rows] = torch.randn(len(rows), n, generator=g, device="cuda").to(BF)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    ws = M.alloc_workspace_grouped(R, 1, n, n, BF)
    dw = torch.full((1, n, n), 7.0, device="cuda")
    M.moe_grouped_matmul_dw(x, x, off, dw, ws)
    assert M.moe_check_error(ws) == M.MOE_OK
    v = x[rows].double()
    # (additions of zeros are exact)
    assert bool(((dw[0].double() - v.T @ v).abs() <= (len(rows) + 2) * 2.0 ** -23 * (v.abs().T @ v.abs())).all())


@pytest.mark.parametrize("dw_dtype", [F32, BF])
@pytest.mark.parametrize("n,k", [(72, 40), (200, 168), (264, 520)])
def test_dw_of_parts(n, k, dw_dtype):
    # reductions about the ends of the parts that are summed at once, and
    # accumulating ones
    p = Problem([767, 768, 769, 0, 832, 1536, 1537, 2305, 5], n, k, BF, lead=1, tail=2, seed=20)
    out = p.run("dw", dw_dtype=dw_dtype)
    p.check("dw", out)
    base = torch.randn(out.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).to(dw_dtype)
    acc = base.clone()
    M.moe_grouped_matmul_dw(p.dy, p.x, p.offsets, acc, p.ws, accumulate=True)
    p.check("dw", acc, base)


@pytest.mark.parametrize("dw_dtype", [F32, BF])
@pytest.mark.parametrize("n,k", [(72, 40), (264, 520)])
def test_dw_of_many_rows_keeps_its_precision(n, k, dw_dtype):
    # Positive rows, so that every error of a sum has one sign. Sums of 768 rows
    # at most may be truncated, an addition by 2^-23 of itself (768 rows and 2 as
    # above); the parts' sums are added up with a rounding of 2^-24 each
    counts = [769, 1 << 20, 0, 4099]
    p = Problem(counts, n, k, BF, lead=1, tail=1, seed=19)
    for t in (p.x, p.dy):
        t[1:-1] = t[1:-1].abs() + 0.5
    out = p.run("dw", dw_dtype=dw_dtype)
    base = torch.full_like(out, 1024.0)
    acc = base.clone()
    M.moe_grouped_matmul_dw(p.dy, p.x, p.offsets, acc, p.ws, accumulate=True)
    for got, first in ((out, 0.0), (acc, 1024.0)):
        for e, r in p.spans():
            rows = r.stop - r.start
            ref = p.dy[r].double().T @ p.x[r].double() + first
            tol = (770 * 2.0 ** -23 + (rows // 768 + 2) * 2.0 ** -24) * ref
            tol = tol + torch.finfo(dw_dtype).eps / 2 * (ref + tol)
            assert bool(((got[e].double() - ref).abs() <= tol).all()), (e, ((got[e].double() - ref).abs() / ref).max())
    assert M.moe_check_error(p.ws) == M.MOE_OK
