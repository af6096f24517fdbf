"""The operators of the dense half of a block without a GPU: pins of their float64 oracle
(closed forms, and central differences for the gradients) and refusals of the C entries,
which come back as a status before anything touches the device."""
import ctypes

import numpy as np
import pytest

from oracle import block_oracle as B

NUL = ctypes.c_void_p(0)
P = ctypes.c_void_p(1 << 20)        # never dereferenced: the calls below stop before a launch
ODD = ctypes.c_void_p((1 << 20) + 8)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
EPS = 1e-5          # step of the central differences: truncation ~ EPS^2, rounding ~ 1e-16 / EPS
TOL = 1e-6          # a hundred times the larger of the two, for values of order 1


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routed_top_gb300 import build, lib
    build.build()
    return lib()


def _diff(f, v, direction):
    return (f(v + EPS * direction) - f(v - EPS * direction)) / (2 * EPS)


# ------------------------------------------------------------------ gated products
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_against_differences(act):
    g = np.random.default_rng(4)
    x, w, b, gh = g.normal(size=(5, 8)), g.normal(size=(6, 8)), g.normal(size=6), g.normal(size=(5, 3))
    _, z = B.gated_linear(x, w, b, act)
    dx, dw, db, _ = B.gated_linear_backward(gh, x, w, z, act)
    for val, grad, f in ((x, dx, lambda a: B.gated_linear(a, w, b, act)), (w, dw, lambda a: B.gated_linear(x, a, b, act)),
                         (b, db, lambda a: B.gated_linear(x, w, a, act))):
        u = g.normal(size=val.shape)
        assert abs(_diff(lambda a: (f(a)[0] * gh).sum(), val, u) - (grad * u).sum()) < TOL


def test_gated_closed_forms():
    x, w = np.array([[2.0, -3.0]]), np.array([[1.0, 0], [0, 1], [0, 1], [1, 0]])       # gates 2, -3; ups -3, 2
    h, z = B.gated_linear(x, w, activation="relu")
    assert z.tolist() == [[2.0, -3.0, -3.0, 2.0]] and h.tolist() == [[-6.0, 0.0]]
    assert B.gated_linear_backward([[1, 1]], x, w, z, "relu")[3].tolist() == [[-3.0, 0.0, 2.0, 0.0]]


X, W, Z = (ctypes.c_void_p(i << 24) for i in (1, 2, 3))


def gated(L, x=X, ld_x=64, w=W, ld_w=64, bias=NUL, bdt=0, act=0, T=4, K=64, I=32, out=P, ld_out=32, z=NUL, ws=P,
          wsb=1 << 30):
    return L.moe_gated_linear(x, ld_x, w, ld_w, bias, bdt, act, T, K, I, out, ld_out, z, ws, wsb, NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(I=-1), INVALID), (dict(K=0), UNSUPPORTED), (dict(K=60), UNSUPPORTED),
    (dict(ld_x=68), UNSUPPORTED), (dict(ld_w=56), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID),
    (dict(bias=P, bdt=2), INVALID), (dict(ld_out=31), INVALID), (dict(x=NUL), INVALID), (dict(w=NUL), INVALID),
    (dict(out=NUL), INVALID), (dict(x=ODD), INVALID), (dict(bias=ODD), INVALID), (dict(z=P), INVALID),
    (dict(out=X), INVALID), (dict(out=W), INVALID), (dict(z=X), INVALID),
    (dict(ws=NUL), INVALID), (dict(wsb=128), WORKSPACE), (dict(I=1 << 30, ld_out=1 << 30), UNSUPPORTED),
    (dict(T=0, x=NUL), OK), (dict(I=0, x=NUL), OK)])
def test_gated_linear_refusals(L, kw, status):
    assert gated(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(act=-1), INVALID), (dict(z=NUL), INVALID), (dict(K=60), UNSUPPORTED), (dict(ld_gh=31), INVALID),
    (dict(ld_z=63), INVALID), (dict(gh=NUL), INVALID), (dict(wsb=64), WORKSPACE), (dict(x=ODD), INVALID),
    (dict(dx=X), INVALID), (dict(dw=W), INVALID), (dict(dw=P, dx=P), INVALID)])
def test_gated_linear_backward_refusals(L, kw, status):
    need = L.moe_gated_linear_backward_workspace_size(4, 32)
    assert need >= 4 * 64 * 2 and L.moe_gated_linear_backward_workspace_size(4, 1 << 30) == 0
    a = dict(gh=Z, ld_gh=32, x=X, act=0, z=Z, ld_z=64, K=64, wsb=need, dx=P, dw=ctypes.c_void_p(1 << 21))
    a.update(kw)
    assert L.moe_gated_linear_backward(a["gh"], a["ld_gh"], a["x"], 64, W, 64, a["act"], a["z"], a["ld_z"], 4, a["K"],
                                       32, a["dx"], a["dw"], NUL, P, a["wsb"], NUL) == status


# ------------------------------------------------------------------ 8-bit products
def test_linear_fp8_closed_forms():
    qx, qw = np.full((1, 256), 0x38, np.uint8), np.full((130, 256), 0x38, np.uint8)       # ones
    y, z, mag = B.linear_fp8(qx, [[2.0, 0.5]], qw, [[1.0, 4.0], [8.0, 0.0]], bias=np.arange(130.0), activation="relu",
                             residual=np.ones((1, 130)))
    assert z[0, 0] == 128 * (2 + 2) and z[0, 129] == 128 * 16 + 129 and y[0, 129] == z[0, 129] + 1 and mag[0, 127] == 512


def rows8(L, x=P, ld_x=256, T=4, K=256, fmt=1, q=P, s=P, s_row=2, s_kb=1):
    return L.moe_quantize_fp8_rows(x, ld_x, T, K, fmt, q, s, s_row, s_kb, NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(K=0), UNSUPPORTED), (dict(K=200), UNSUPPORTED), (dict(ld_x=255), INVALID),
    (dict(ld_x=260), UNSUPPORTED), (dict(fmt=0), INVALID), (dict(fmt=3), INVALID), (dict(s_row=0), INVALID),
    (dict(s_kb=-1), INVALID), (dict(x=NUL), INVALID), (dict(q=NUL), INVALID), (dict(s=NUL), INVALID),
    (dict(x=ODD), INVALID), (dict(q=ODD), INVALID), (dict(s=ctypes.c_void_p((1 << 20) + 2)), INVALID),
    (dict(T=0, x=NUL), OK)])
def test_quantize_fp8_rows_refusals(L, kw, status):
    assert rows8(L, **kw) == status


def lin8(L, x=X, ld_x=256, xs=NUL, s_row=0, s_kb=0, w=W, ld_w=256, ws8=P, fmt=1, bias=NUL, bdt=0, act=-1, res=NUL,
         ld_res=0, T=4, K=256, N=32, out=P, odt=0, ld_out=32, ws=P, wsb=1 << 30):
    return L.moe_linear_fp8(x, ld_x, xs, s_row, s_kb, w, ld_w, ws8, fmt, bias, bdt, act, res, ld_res, T, K, N, out, odt,
                            ld_out, ws, wsb, NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), UNSUPPORTED), (dict(K=192), UNSUPPORTED),
    (dict(ld_x=260), UNSUPPORTED), (dict(ld_x=264, xs=P, s_row=2, s_kb=1), UNSUPPORTED), (dict(ld_w=255), INVALID),
    (dict(ld_w=264), UNSUPPORTED), (dict(fmt=0), INVALID), (dict(fmt=3), INVALID), (dict(xs=P, s_row=0, s_kb=1), INVALID),
    (dict(act=3), INVALID), (dict(odt=2), INVALID), (dict(bias=P, bdt=2), INVALID), (dict(ld_out=31), INVALID),
    (dict(res=P, ld_res=31), INVALID), (dict(res=P, ld_res=40), INVALID), (dict(x=NUL), INVALID), (dict(w=NUL), INVALID),
    (dict(ws8=NUL), INVALID), (dict(out=NUL), INVALID), (dict(out=X), INVALID), (dict(out=W), INVALID), (dict(x=ODD), INVALID), (dict(w=ODD), INVALID),
    (dict(ws=NUL), INVALID), (dict(wsb=128), WORKSPACE), (dict(T=0, x=NUL), OK), (dict(N=0, x=NUL), OK)])
def test_linear_fp8_refusals(L, kw, status):
    assert lin8(L, **kw) == status


def test_linear_fp8_workspace(L):
    """Given codes need the products' part alone; bf16 rows their codes and scales too."""
    small, need = L.moe_linear_workspace_size(), L.moe_linear_fp8_workspace_size(4, 256)
    assert need >= small + 4 * 256 + 4 * 2 * 4 and L.moe_linear_fp8_workspace_size(-1, 256) == 0
    assert lin8(L, wsb=need - 1) == WORKSPACE
    assert lin8(L, xs=P, s_row=2, s_kb=1, wsb=small - 1) == WORKSPACE


# ------------------------------------------------------------------ layer norm
def test_layer_norm_gradient_against_differences():
    g = np.random.default_rng(6)
    v = dict(residual=g.normal(size=(4, 10)) + 3, y=g.normal(size=(4, 10)), weight=g.normal(size=10), bias=g.normal(size=10))
    gr, gn = g.normal(size=(4, 10)), g.normal(size=(4, 10))

    def loss(**q):
        r, n = B.layer_norm(**q)
        return (r * gr).sum() + (n * gn).sum()
    dr, dw, db = B.layer_norm_backward(gr, gn, B.layer_norm(**v)[0], v["weight"])
    for name, d in (("residual", dr), ("y", dr), ("weight", dw), ("bias", db)):
        u = g.normal(size=v[name].shape)
        assert abs(_diff(lambda a: loss(**{**v, name: a}), v[name], u) - (d * u).sum()) < TOL, name


def test_layer_norm_closed_forms():
    r, n = B.layer_norm([[1.0, 2.0]], [[1.0, 4.0]], weight=[2.0, 3.0], bias=[1.0, -1.0], eps=0.0)
    assert r.tolist() == [[2.0, 6.0]] and n.tolist() == [[-1.0, 2.0]]
    # shifts and scales of the row have no gradient through the norm
    dr = B.layer_norm_backward(None, [[1.0, 5.0, -2.0]], [[1.0, 2.0, 4.0]], eps=0.0)[0]
    assert abs(dr.sum()) < 1e-12 and abs((dr * [[1.0, 2.0, 4.0]]).sum()) < 1e-12


def lnorm(L, res=P, res_dt=0, ld_res=64, y=P, ld_y=64, w=P, b=P, wdt=0, T=4, H=64, out=P, n=None):
    n = ctypes.c_void_p(1 << 21) if n is None else n
    return L.moe_layer_norm(res, res_dt, ld_res, y, ld_y, w, b, wdt, 1e-5, T, H, out, n, NUL)


Q = ctypes.c_void_p(1 << 22)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), UNSUPPORTED), (dict(H=16385, ld_res=16385, ld_y=16385), UNSUPPORTED),
    (dict(res_dt=3), INVALID), (dict(wdt=3), INVALID), (dict(ld_res=63), INVALID), (dict(ld_y=63), INVALID),
    (dict(res=NUL), INVALID), (dict(out=NUL), INVALID), (dict(n=NUL), INVALID), (dict(ld_res=72), INVALID),
    (dict(n=P), INVALID), (dict(y=Q, out=Q), INVALID), (dict(y=NUL, n=P), INVALID), (dict(y=ODD), INVALID),
    (dict(w=ODD), INVALID), (dict(b=ODD), INVALID), (dict(T=0, res=NUL), OK)])
def test_layer_norm_refusals(L, kw, status):
    a = dict(y=ctypes.c_void_p(1 << 23))
    a.update(kw)
    assert lnorm(L, **a) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), UNSUPPORTED), (dict(H=16385), UNSUPPORTED), (dict(res_dt=2), INVALID),
    (dict(ld_gr=63), INVALID), (dict(ld_gn=63), INVALID), (dict(ld_res=63), INVALID), (dict(gn=NUL), INVALID),
    (dict(res=NUL), INVALID), (dict(dr=NUL), INVALID), (dict(ws=NUL), INVALID), (dict(wsb=16), WORKSPACE),
    (dict(dr=Q, gr=Q, ld_gr=72), INVALID), (dict(dr=Q, res=Q), INVALID), (dict(dr=Q, dy=Q), INVALID),
    (dict(dr=Q, dy=P), INVALID), (dict(gr=ODD), INVALID), (dict(dw=ODD), INVALID)])
def test_layer_norm_backward_refusals(L, kw, status):
    a = dict(gr=P, ld_gr=64, gn=P, ld_gn=64, res=P, res_dt=0, ld_res=64, T=4, H=64, dr=Q, dy=NUL, dw=NUL, ws=P,
             wsb=L.moe_layer_norm_backward_workspace_size(64))
    a.update(kw)
    assert a["wsb"] == 16 or a["wsb"] >= 2 * 64 * 4
    assert L.moe_layer_norm_backward(a["gr"], a["ld_gr"], a["gn"], a["ld_gn"], a["res"], a["res_dt"], a["ld_res"], P, 0,
                                     1e-5, a["T"], a["H"], a["dr"], a["dy"], a["dw"], NUL, a["ws"], a["wsb"], NUL) == status


def test_packed_calls(L):
    """The calls of the dense half by number: each one's own refusals come back."""
    import struct

    def block(*v):
        return struct.pack("=" + "".join("d" if isinstance(x, float) else "q" for x in v), *v)
    p = P.value
    assert L.moe_call_packed(7, block(p, 60, p, 60, 0, 0, 0, 4, 60, 8, p, 8, 0, p, 1 << 25, 0)) == UNSUPPORTED
    assert L.moe_call_packed(8, block(p, 8, p, 64, p, 64, -1, p, 16, 4, 64, 8, p, p, 0, p, 1 << 25, 0)) == INVALID
    assert L.moe_call_packed(9, block(p, 64, 4, 64, 1, p, p, 1, 1, 0)) == UNSUPPORTED
    assert L.moe_call_packed(10, block(p, 128, 0, 0, 0, p, 128, p, 1, 0, 0, -1, 0, 0, 4, 128, 8, p, 0, 7, p, 1 << 25, 0)) == INVALID
    assert L.moe_call_packed(11, block(p, 0, 8, 0, 0, 0, 0, 0, 1e-5, 4, 0, 0, p, 0)) == UNSUPPORTED
    assert L.moe_call_packed(12, block(0, 0, p, 8, p, 0, 8, 0, 0, 1e-5, 1 << 33, 8, p, 0, 0, 0, p, 1 << 25, 0)) == UNSUPPORTED
    for call in (6, 13, 99):
        assert L.moe_call_packed(call, block(*([0] * 30))) == INVALID


def test_the_bindings_refuse_host_tensors():
    import torch

    import mixture_experts_routed_top_gb300 as m
    t = torch.zeros(4, 8)
    for call in (lambda: m.gated_linear(t, t), lambda: m.gated_linear_backward(t, t, t, t),
                 lambda: m.quantize_fp8_rows(t), lambda: m.linear_fp8(t, t, t), lambda: m.layer_norm(t),
                 lambda: m.layer_norm_backward(t, t, t)):
        with pytest.raises(ValueError):
            call()
