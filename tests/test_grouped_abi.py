"""Argument checks of the grouped products and of the 4-bit calls; no GPU
needed: every call here returns before touching the device."""

import ctypes

import pytest
import torch

from mixture_experts_layer_42_b200 import build as B


@pytest.fixture(scope="module")
def M():
    B.build()
    from mixture_experts_layer_42_b200 import binding
    return binding


P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def shape(M, **kw):
    base = dict(rows=64, n_experts=8, n=64, k=128, dtype=M.MOE_DT_BF16)
    base.update(kw)
    return M.moe_grouped_shape(**base)


def size(M, **kw):
    n = ctypes.c_size_t(0)
    st = M.raw_status("moe_grouped_workspace_size", ctypes.byref(shape(M, **kw)), ctypes.byref(n))
    return st, n.value


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(rows=0), 0), (dict(rows=1 << 30), 0),
    (dict(rows=-1), -1), (dict(n_experts=0), -1), (dict(n=0), -1), (dict(k=0), -1),
    (dict(n=12), -1), (dict(k=4), -1), (dict(dtype=2), -1),
    (dict(dtype=0, n=12, k=4), 0), (dict(dtype=0, n=6), -1),
    (dict(rows=(1 << 30) + 1), -2), (dict(rows=1 << 31), -2), (dict(n_experts=1025), -2), (dict(n=(1 << 20) + 8), -2),
    (dict(n_experts=1024, n=1 << 20, k=1 << 9), 0), (dict(n_experts=1024), 0),
    (dict(n_experts=1024, n=1 << 20, k=1 << 10), -2), (dict(n_experts=1, n=1 << 20, k=1 << 20), -2),
])
def test_shapes(M, kw, status):
    st, n = size(M, **kw)
    assert st == status
    assert st != 0 or n > 0


def test_null_shape_and_size(M):
    assert M.raw_status("moe_grouped_workspace_size", None, None) == -1
    assert M.raw_status("moe_grouped_workspace_size", ctypes.byref(shape(M)), None) == -1


@pytest.mark.parametrize("name", ["moe_grouped_matmul", "moe_grouped_matmul_dx"])
def test_product_arguments(M, name):
    ws = size(M)[1]
    g = ctypes.byref(shape(M))
    ok = [P, P, P, P]
    for i in range(4):
        for bad in (None, ODD):
            a = list(ok)
            a[i] = bad
            assert M.raw_status(name, g, *a, P, ws, None) == -1
    assert M.raw_status(name, g, *ok, None, ws, None) == -3
    assert M.raw_status(name, g, *ok, P, ws - 1, None) == -3
    assert M.raw_status(name, g, *ok, ODD, ws, None) == -1
    assert M.raw_status(name, None, *ok, P, ws, None) == -1
    assert M.raw_status(name, ctypes.byref(shape(M, k=4)), *ok, P, ws, None) == -1


def test_dw_arguments(M):
    ws = size(M)[1]
    g = ctypes.byref(shape(M))
    call = lambda *a, g=g: M.raw_status("moe_grouped_matmul_dw", g, *a, None)
    for i in range(4):
        a = [P, P, P, 0, 0, P]
        a[i if i < 3 else 5] = ODD
        assert call(*a, P, ws) == -1
    assert call(P, P, P, 2, 0, P, P, ws) == -1           # dw type
    assert call(P, P, P, 0, 2, P, P, ws) == -1           # accumulate
    assert call(P, P, P, 1, 0, P, P, ws, g=ctypes.byref(shape(M, dtype=0))) == -2   # bf16 dw of an fp32 layer
    assert call(P, P, P, 0, 0, P, None, ws) == -3
    assert call(P, P, P, 0, 0, P, P, ws - 1) == -3


def w4m(M, q=0x10000, s=0x10000):
    return ctypes.byref(M.moe_w4_matrix(q, s))


def test_w4_product_arguments(M):
    ws = size(M)[1]
    g = ctypes.byref(shape(M))

    def one(g=g, group=64, x_rows=64, x=P, src=None, off=P, m=w4m(M), y=P, w=P, n=ws):
        return M.raw_status("moe_grouped_matvec_w4", g, group, x_rows, x, src, off, m, y, w, n, None)

    def two(g=g, group=64, x_rows=9, x=P, src=P, off=P, m=w4m(M), m3=w4m(M), y=P, w=P, n=ws):
        return M.raw_status("moe_grouped_swiglu_w4", g, group, x_rows, x, src, off, m, m3, y, w, n, None)

    for f in (one, two):
        assert f(group=16) == -1 and f(group=0) == -1 and f(group=256) == -1
        assert f(g=ctypes.byref(shape(M, k=96))) == -1            # k not whole groups
        assert f(g=ctypes.byref(shape(M, dtype=0))) == -2         # fp32
        assert f(x=None) == -1 and f(x=ODD) == -1 and f(y=None) == -1 and f(off=ODD) == -1
        assert f(m=None) == -1 and f(m=w4m(M, q=0x10004)) == -1 and f(m=w4m(M, s=0)) == -1
        assert f(src=ODD) == -1 and f(x_rows=-1) == -1
        assert f(x_rows=1 << 31, src=P) == -2
        assert f(w=None) == -3 and f(n=ws - 1) == -3
    assert one(x_rows=63) == -1                                   # without src, one x row per row
    assert two(m3=None) == -1 and two(m3=w4m(M, q=0)) == -1


def test_w4_quantizer_arguments(M):
    f = lambda g=shape(M), group=64, w=P, q=P, s=P: M.raw_status("moe_quantize_w4", ctypes.byref(g), group, w, q, s,
                                                                 None)
    assert f(group=48) == -1 and f(w=None) == -1 and f(q=ODD) == -1 and f(s=None) == -1
    assert f(g=shape(M, dtype=0, n=12)) == -1                     # n not a multiple of 8
    assert f(g=shape(M, k=96)) == -1


def test_w4_layer_arguments(M):
    cfg = dict(dim=128, n_routed=16, n_groups=4, topk_groups=2, topk=4, moe_inter=64, shared_inter=64, score=0,
               route_scale=1.0, has_bias=1, dtype=1)
    n = ctypes.c_size_t(0)
    c = ctypes.byref(M.moe_config(**cfg))
    assert M.raw_status("moe_workspace_size_w4", c, 8, ctypes.byref(n)) == 0 and n.value > 0
    assert M.raw_status("moe_workspace_size_w4", c, 8, None) == -1
    assert M.raw_status("moe_workspace_size_w4", ctypes.byref(M.moe_config(**dict(cfg, dtype=0))), 8,
                        ctypes.byref(n)) == -2
    m = M.moe_w4_matrix(0x10000, 0x10000)

    def weights(group=64, **kw):
        return ctypes.byref(M.moe_w4_weights(**dict(dict(w1=m, w3=m, w2=m, ws1=m, ws3=m, ws2=m, group=group), **kw)))

    def f(c=c, x=P, r=P, b=P, w=weights(), y=P, wo=None, io=None, ws=P, nb=n.value):
        return M.raw_status("moe_forward_w4", c, 8, x, r, b, w, y, wo, io, ws, nb, None)

    none = M.moe_w4_matrix(None, None)
    assert f(w=None) == -1 and f(w=weights(group=128)) == -1 and f(w=weights(group=8)) == -1
    for name in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        assert f(w=weights(**{name: none})) == -1
    assert f(x=None) == -1 and f(r=ODD) == -1 and f(b=None) == -1 and f(y=None) == -1
    assert f(wo=ODD) == -1 and f(io=ODD) == -1
    assert f(ws=None) == -3 and f(nb=n.value - 1) == -3


def test_binding_checks_shapes(M):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    off = z(3, dtype=torch.int32)
    ws = z(4096, dtype=torch.uint8)
    w = z(2, 16, 24)
    bad = [
        lambda: M.moe_grouped_matmul(z(4, 16), off, w, z(4, 16), ws),
        lambda: M.moe_grouped_matmul(z(4, 24), off, w, z(5, 16), ws),
        lambda: M.moe_grouped_matmul(z(4, 24), z(2, dtype=torch.int32), w, z(4, 16), ws),
        lambda: M.moe_grouped_matmul(z(4, 24), z(3, dtype=torch.int64), w, z(4, 16), ws),
        lambda: M.moe_grouped_matmul(z(4, 24, dtype=torch.float32), off, w, z(4, 16, dtype=torch.float32), ws),
        lambda: M.moe_grouped_matmul(z(4, 24), off, w, z(4, 16, dtype=torch.float32), ws),
        lambda: M.moe_grouped_matmul(z(4, 24, dtype=torch.float16), off, w, z(4, 16, dtype=torch.float16), ws),
        lambda: M.moe_grouped_matmul(z(4, 24), off, w.transpose(1, 2).contiguous().transpose(1, 2), z(4, 16), ws),
        lambda: M.moe_grouped_matmul_dx(z(4, 24), off, w, z(4, 24), ws),
        lambda: M.moe_grouped_matmul_dw(z(4, 16), z(3, 24), off, w, ws),
        lambda: M.moe_grouped_matmul_dw(z(4, 16), z(4, 24), off, w.half(), ws),
        lambda: M.moe_quantize_w4(z(2, 8, 64), 32, z(2, 8, 64, dtype=torch.uint8), z(2, 2, 8)),
        lambda: M.moe_quantize_w4(z(2, 8, 64), 32, z(2, 8, 32, dtype=torch.uint8), z(2, 1, 8)),
    ]
    q, s = z(2, 8, 32, dtype=torch.uint8), z(2, 2, 8)
    bad += [
        lambda: M.moe_grouped_matvec_w4(z(4, 32), None, off, q, s, z(4, 8), ws),
        lambda: M.moe_grouped_matvec_w4(z(4, 64), None, off, q, z(2, 8, 2), z(4, 8), ws),
        lambda: M.moe_grouped_matvec_w4(z(4, 64), z(3, dtype=torch.int32), off, q, s, z(4, 8), ws),
        lambda: M.moe_grouped_matvec_w4(z(4, 64), None, off, q.to(torch.int8), s, z(4, 8), ws),
        lambda: M.moe_grouped_swiglu_w4(z(4, 64), None, off, q, s, z(2, 16, 32, dtype=torch.uint8), s, z(4, 8), ws),
    ]
    # right shapes, but on the host
    bad += [
        lambda: M.moe_grouped_matmul(z(4, 24), off, w, z(4, 16), ws),
        lambda: M.moe_grouped_matmul_dx(z(4, 16), off, w, z(4, 24), ws),
        lambda: M.moe_grouped_matmul_dw(z(4, 16), z(4, 24), off, w, ws),
        lambda: M.moe_quantize_w4(z(2, 8, 64), 32, q, s),
        lambda: M.moe_grouped_matvec_w4(z(4, 64), None, off, q, s, z(4, 8), ws),
        lambda: M.moe_grouped_swiglu_w4(z(4, 64), None, off, q, s, q, s, z(4, 8), ws),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")


@pytest.mark.parametrize("E", [1, 7, 8, 1024])
def test_workspace_holds_aligned_maps(M, E):
    # a workspace may begin at any multiple of 16 bytes; the 2 E maps of 128
    # bytes after its header begin at a multiple of 128
    n = size(M, n_experts=E)[1]
    for ws in range(0x10000, 0x10000 + 256, 16):
        first = -(-(ws + 256) // 128) * 128
        assert first + 2 * E * 128 <= ws + n


def w4_tensors(group=64, E=4, D=128, I=64, Is=64):
    """(codes, scales) of a layer's six matrices, on the host."""
    z = torch.zeros
    pair = lambda e, n, k: (z(e, n, k // 2, dtype=torch.uint8), z(e, k // group, n, dtype=torch.bfloat16))
    return dict(w1=pair(E, I, D), w3=pair(E, I, D), w2=pair(E, D, I), ws1=pair(1, Is, D), ws3=pair(1, Is, D),
                ws2=pair(1, D, Is))


def test_w4_weights_of_host_tensors_are_refused(M):
    with pytest.raises(ValueError, match="on a GPU"):
        M.w4_weights(64, **w4_tensors())


@pytest.mark.parametrize("name", ["w1", "w2", "ws3"])
def test_w4_weights_of_other_types_and_shapes_are_refused(M, name):
    def refused(what, group=64, **kw):
        with pytest.raises(ValueError, match=what):
            M.w4_weights(group, **dict(w4_tensors(), **kw))

    q, s = w4_tensors()[name]
    refused("codes must be uint8", **{name: (q.to(torch.int8), s)})
    refused("codes must be uint8", **{name: (q.flatten(), s)})
    refused("scales must be bfloat16", **{name: (q, s.float())})
    refused("scales must be bfloat16", **{name: (q, s.transpose(1, 2).contiguous())})
    refused("scales must be bfloat16", **{name: (q[..., :-16].contiguous(), s)})
    refused("scales must be bfloat16", group=32)
    refused("scales must be bfloat16", group=0)
    refused("contiguous", **{name: (q.transpose(0, 1).contiguous().transpose(0, 1) if q.shape[0] > 1 else
                                    torch.zeros(1, q.shape[1], 2 * q.shape[2], dtype=torch.uint8)[..., ::2], s)})
    if not name.startswith("ws"):
        refused("are needed", **{name: None})


def test_w4_layer_tensors_are_checked_against_the_configuration(M):
    cfg = M.moe_config(dim=128, n_routed=4, n_groups=1, topk_groups=1, topk=2, moe_inter=64, shared_inter=64, score=0,
                       route_scale=1.0, has_bias=1, dtype=1)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    F = torch.float32

    def weights(**kw):
        m = M.moe_w4_matrix(0x10000, 0x10000)
        w = M.moe_w4_weights(m, m, m, m, m, m, 64)
        w.shapes = dict(dict(w1=(4, 64, 128), w3=(4, 64, 128), w2=(4, 128, 64), ws1=(1, 64, 128), ws3=(1, 64, 128),
                             ws2=(1, 128, 64)), **kw)
        return w

    def refused(what, x=z(8, 128), r=z(4, 128), b=z(4, dtype=F), w=None, y=z(8, 128), wo=None, io=None):
        with pytest.raises(ValueError, match=what):
            M.moe_forward_w4(cfg, x, r, b, w or weights(), y, z(1 << 16, dtype=torch.uint8), wo, io)

    refused("x must be", x=z(8, 120))
    refused("x must be", x=z(8, 128, dtype=F))
    refused("w_router must be", r=z(5, 128))
    refused("w_router must be", r=z(4, 128, dtype=F))
    refused("bias must be", b=z(4))
    refused("y must be", y=z(7, 128))
    refused("y must be", y=z(8, 128, dtype=F))
    refused("weights_out must be", wo=z(8, 2))
    refused("weights_out must be", wo=z(7, 2, dtype=F))
    refused("idx_out must be", io=z(8, 2, dtype=torch.int64))
    for name, shape in (("w1", (4, 64, 64)), ("w3", (3, 64, 128)), ("w2", (4, 64, 128)), ("ws1", (1, 128, 128)),
                        ("ws2", None)):
        refused(name + ": 4-bit weights", w=weights(**{name: shape}))
    refused("on a GPU")                                           # right, but on the host
