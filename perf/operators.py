"""Measured cases of the experts' grouped products and of their 4-bit form.

The operators, over the rows of an expert-ordered batch (expert e owns rows
[offsets[e], offsets[e + 1]), as the layer's dispatch writes them):

  matmul         y[r]  = W_e x[r]                    (W [E, n, k], x [R, k])
  matmul_dx      dx[r] = W_e^T dy[r]                 (dy [R, n])
  matmul_dw      dW_e  = sum over e's rows of dy[r] x[r]^T
  matvec_w4      y[r]  = W_e x[r], W_e in 4 bits with one scale per group of
                 `group` inputs of an output: W[i, j] = (code - 8) scale
  swiglu_w4      h[r]  = silu(W1_e x[src[r]]) * (W3_e x[src[r]]), the same form

With `own` false, run() computes them by elementary torch operations in fp32,
rounded once; with `own` true it calls the library.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the tiny fp32 layer's up-projection: a few microseconds, launch latency counts
        dict(name="matmul_tiny_f32", op="matmul", dtype="f32", T=64, topk=4, E=16, n=64, k=128, skew=0.0),
        # the down-projection of a decode batch: a few rows per expert, bound by the weights' bytes
        dict(name="matmul_decode_bf16", op="matmul", dtype="bf16", T=128, topk=8, E=256, n=7168, k=2048,
             skew=0.0),
        # the up-projection of a prefill (or training) batch: bound by the tensor cores
        dict(name="matmul_prefill_bf16", op="matmul", dtype="bf16", T=8192, topk=8, E=256, n=2048, k=7168,
             skew=0.0),
        # the input's gradient with expert popularity skewed: hot experts, near-empty ones, ragged tails
        dict(name="dx_skew_bf16", op="matmul_dx", dtype="bf16", T=8192, topk=8, E=256, n=2048, k=7168,
             skew=1.2),
        # the fp32 layer's training step at sizes that divide no tile
        dict(name="dx_odd_f32", op="matmul_dx", dtype="f32", T=1021, topk=4, E=16, n=1032, k=2052, skew=0.6),
        # the weights' gradient of the softmax layer's up-projection
        dict(name="dw_softmax_bf16", op="matmul_dw", dtype="bf16", dw_dtype="bf16", T=4096, topk=6, E=64,
             n=1408, k=2048, skew=0.0),
        # one expert-parallel rank's weights' gradient, kept in fp32 for the optimizer
        dict(name="dw_rank_f32out", op="matmul_dw", dtype="bf16", dw_dtype="f32", T=8192, topk=2, E=32,
             n=2048, k=7168, skew=0.6),
        # the fp32 layer's weights' gradient at sizes that divide no tile
        dict(name="dw_odd_f32", op="matmul_dw", dtype="f32", dw_dtype="f32", T=1021, topk=4, E=16, n=1032,
             k=2052, skew=0.6),
        # one token being decoded: its eight experts' weights once, latency counts
        dict(name="w4_up_token", op="swiglu_w4", dtype="bf16", T=1, topk=8, E=256, n=2048, k=7168, group=128,
             skew=0.0),
        dict(name="w4_down_token", op="matvec_w4", dtype="bf16", T=1, topk=8, E=256, n=7168, k=2048,
             group=128, skew=0.0),
        # a decode batch: every expert's weights once, a few rows each
        dict(name="w4_down_decode", op="matvec_w4", dtype="bf16", T=128, topk=8, E=256, n=7168, k=2048,
             group=128, skew=0.0),
        # a small odd layer with the finest groups and many rows per expert
        dict(name="w4_up_odd", op="swiglu_w4", dtype="bf16", T=37, topk=4, E=16, n=1000, k=1056, group=32,
             skew=0.6),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    while True:
        op = rng.choice(["matmul", "matmul_dx", "matmul_dw", "matvec_w4", "swiglu_w4"])
        E = _log_int(rng, 1, 256)
        c = dict(op=op, dtype="bf16", topk=rng.randint(1, min(8, E)), E=E, skew=rng.choice([0.0, 0.6, 1.2]))
        if op in ("matvec_w4", "swiglu_w4"):
            c["group"] = rng.choice([32, 64, 128])
            c["T"] = _log_int(rng, 1, 512)
            c["n"] = _log_int(rng, 64, 7168, 8)
            c["k"] = _log_int(rng, 128, 7168, c["group"])
            most_w, most_f = 3.8e9, 6e10
        else:
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            step = 8 if c["dtype"] == "bf16" else 4
            c["T"] = _log_int(rng, 1, 8192)
            c["n"] = _log_int(rng, 64, 7168, step)
            c["k"] = _log_int(rng, 64, 7168, step)
            most_w = 3.8e9 if op != "matmul_dw" else 4.8e8
            most_f = 1.93e12
            if c["dtype"] == "f32":
                most_w, most_f = 4.8e8, 2e10
            if op == "matmul_dw":
                c["dw_dtype"] = "f32" if c["dtype"] == "f32" else rng.choice(["bf16", "f32"])
        if c["E"] * c["n"] * c["k"] <= most_w and work(c)["flops"] <= most_f:
            return c


def _active(case):
    """Expected number of experts that get a row (their weights are read)."""
    return case["E"] * (1.0 - (1.0 - case["topk"] / case["E"]) ** case["T"])


def work(case):
    T, R, E, n, k = case["T"], case["T"] * case["topk"], case["E"], case["n"], case["k"]
    op = case["op"]
    if op in ("matvec_w4", "swiglu_w4"):
        m = 2 if op == "swiglu_w4" else 1
        w = _active(case) * m * (n * k / 2 + 2 * n * (k // case["group"]))
        rows = T if op == "swiglu_w4" else R
        return {"bytes": w + 2 * rows * k + 2 * R * n, "flops": 2.0 * m * R * n * k}
    s = 2 if case["dtype"] == "bf16" else 4
    if op == "matmul_dw":
        so = 2 if case["dw_dtype"] == "bf16" else 4
        return {"bytes": s * R * (n + k) + so * E * n * k, "flops": 2.0 * R * n * k}
    return {"bytes": s * (R * (n + k) + _active(case) * n * k), "flops": 2.0 * R * n * k}


def _route(case, gen):
    """A batch's assignment: topk distinct experts per token; counts, offsets
    and the token of each expert-ordered row."""
    T, E = case["T"], case["E"]
    pop = -case["skew"] * torch.log1p(torch.randperm(E, generator=gen, device="cuda").float())
    u = torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    idx = (pop - torch.log(-torch.log(u))).topk(case["topk"], dim=1).indices.reshape(-1)
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    src = (torch.argsort(idx, stable=True) // case["topk"]).to(torch.int32)
    return counts.tolist(), offsets, src


def _normal(gen, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _quantized(gen, E, n, k, group):
    """Normal weights in the 4-bit layout: codes [E, n, k / 2], two to a byte,
    the lower input in the low half; bf16 scales [E, k / group, n]."""
    q = torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, k // group, n, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 28) // (n * k))
    for e in range(0, E, step):
        w = torch.empty(min(step, E - e), n, k // group, group, device="cuda")
        w.normal_(0.0, k ** -0.5, generator=gen)
        sc = (w.abs().amax(-1) / 7).to(torch.bfloat16)
        c = (w / sc.float().unsqueeze(-1)).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
        c = c.reshape(-1, n, k // 2, 2)
        q[e:e + step] = c[..., 0] | (c[..., 1] << 4)
        s[e:e + step] = sc.transpose(1, 2)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DT[case["dtype"]]
    T, E, n, k = case["T"], case["E"], case["n"], case["k"]
    R = T * case["topk"]
    counts, offsets, src = _route(case, gen)
    st = dict(op=op, counts=counts, offsets=offsets, src=src, group=case.get("group"))
    if op in ("matvec_w4", "swiglu_w4"):
        st["q"], st["s"] = _quantized(gen, E, n, k, case["group"])
        if op == "swiglu_w4":
            st["q3"], st["s3"] = _quantized(gen, E, n, k, case["group"])
        st["x"] = _normal(gen, (T if op == "swiglu_w4" else R, k), 1.0, dt)
        st["out"] = torch.empty(R, n, dtype=dt, device="cuda")
        dtype_ws = dt
    else:
        if op != "matmul":
            st["dy"] = _normal(gen, (R, n), 0.01, dt)
        if op != "matmul_dx":
            st["x"] = _normal(gen, (R, k), 1.0, dt)
        if op != "matmul_dw":
            st["w"] = _normal(gen, (E, n, k), k ** -0.5, dt)
        shape, od = {"matmul": ((R, n), dt), "matmul_dx": ((R, k), dt),
                     "matmul_dw": ((E, n, k), DT[case.get("dw_dtype", "f32")])}[op]
        st["out"] = torch.empty(shape, dtype=od, device="cuda")
        dtype_ws = dt
    if own:
        from mixture_experts_layer_42_b200 import binding as M
        st["ws"] = M.alloc_workspace_grouped(R, E, n, k, dtype_ws)
    return st


def _spans(counts):
    b = 0
    for e, c in enumerate(counts):
        yield e, b, b + c
        b += c


def _dequant(q, s, group):
    """One expert's weights [n, k] in fp32 from codes [n, k / 2] and scales [k / group, n]."""
    c = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1, group)
    return ((c.float() - 8.0) * s.float().t().unsqueeze(-1)).reshape(q.shape[0], -1)


def _plain(st):
    op, out, counts = st["op"], st["out"], st["counts"]
    for e, b, z in _spans(counts):
        if op == "matmul_dw":
            out[e] = (st["dy"][b:z].float().t() @ st["x"][b:z].float()).to(out.dtype)
        elif b == z:
            continue
        elif op == "matmul":
            out[b:z] = (st["x"][b:z].float() @ st["w"][e].float().t()).to(out.dtype)
        elif op == "matmul_dx":
            out[b:z] = (st["dy"][b:z].float() @ st["w"][e].float()).to(out.dtype)
        elif op == "matvec_w4":
            w = _dequant(st["q"][e], st["s"][e], st["group"])
            out[b:z] = (st["x"][b:z].float() @ w.t()).to(out.dtype)
        else:
            x = st["x"][st["src"][b:z].long()].float()
            a = x @ _dequant(st["q"][e], st["s"][e], st["group"]).t()
            g = x @ _dequant(st["q3"][e], st["s3"][e], st["group"]).t()
            out[b:z] = (a / (1.0 + torch.exp(-a)) * g).to(out.dtype)
    return out


def run(st):
    if not own:
        return _plain(st)
    from mixture_experts_layer_42_b200 import binding as M
    op, out, off, ws = st["op"], st["out"], st["offsets"], st["ws"]
    if op == "matmul":
        M.moe_grouped_matmul(st["x"], off, st["w"], out, ws)
    elif op == "matmul_dx":
        M.moe_grouped_matmul_dx(st["dy"], off, st["w"], out, ws)
    elif op == "matmul_dw":
        M.moe_grouped_matmul_dw(st["dy"], st["x"], off, out, ws)
    elif op == "matvec_w4":
        M.moe_grouped_matvec_w4(st["x"], None, off, st["q"], st["s"], out, ws)
    else:
        M.moe_grouped_swiglu_w4(st["x"], st["src"], off, st["q"], st["s"], st["q3"], st["s3"], out, ws)
    return out


def exact(case, seed):
    """The outputs in float64, from the definitions."""
    st = prepare(case, seed)
    op, off = st["op"], st["offsets"].tolist()
    d = torch.float64
    res = torch.zeros(st["out"].shape, dtype=d, device="cuda")
    steps = torch.arange(16, device="cuda", dtype=d) - 8.0

    def weights(q, s, e):
        byte = q[e].long()
        n, k = byte.shape[0], 2 * byte.shape[1]
        w = torch.empty(n, k, dtype=d, device="cuda")
        w[:, 0::2] = steps[byte.remainder(16)]
        w[:, 1::2] = steps[byte.div(16, rounding_mode="floor")]
        for j in range(s.shape[1]):
            w[:, j * case["group"]:(j + 1) * case["group"]] *= s[e, j].to(d)[:, None]
        return w

    for e in range(case["E"]):
        rows = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        if op == "matmul":
            res[rows] = torch.einsum("rk,nk->rn", st["x"][rows].to(d), st["w"][e].to(d))
        elif op == "matmul_dx":
            res[rows] = torch.einsum("rn,nk->rk", st["dy"][rows].to(d), st["w"][e].to(d))
        elif op == "matmul_dw":
            res[e] = torch.einsum("rn,rk->nk", st["dy"][rows].to(d), st["x"][rows].to(d))
        elif op == "matvec_w4":
            res[rows] = torch.einsum("rk,nk->rn", st["x"][rows].to(d), weights(st["q"], st["s"], e))
        else:
            x = st["x"].index_select(0, st["src"][rows].long()).to(d)
            a = torch.einsum("rk,nk->rn", x, weights(st["q"], st["s"], e))
            res[rows] = a * torch.sigmoid(a) * torch.einsum("rk,nk->rn", x, weights(st["q3"], st["s3"], e))
    return res
