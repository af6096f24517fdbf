"""Refusals of the operators around the experts, checked without a GPU: every
bad argument comes back as a status before anything touches the device."""
import ctypes
import struct

import pytest

NUL = ctypes.c_void_p(0)
P = ctypes.c_void_p(1 << 20)        # never dereferenced: the calls below stop before a launch
ODD = ctypes.c_void_p((1 << 20) + 8)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routed_top_gb300 import build, lib
    build.build()
    return lib()


def route(L, logits=P, dt=1, ld=None, T=4, E=8, k=2, score=1, bias=NUL, n_group=1, topk_group=1, group_top=2,
          renorm=1, scale=1.0, idx=P, w=P):
    return L.moe_route_scored(logits, dt, E if ld is None else ld, T, E, k, score, bias, n_group, topk_group,
                              group_top, renorm, scale, idx, w, NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(k=0), UNSUPPORTED),
    (dict(k=9), UNSUPPORTED), (dict(E=64, k=33), UNSUPPORTED), (dict(dt=2), INVALID), (dict(score=2), INVALID),
    (dict(ld=7), INVALID), (dict(n_group=3), UNSUPPORTED), (dict(n_group=0), UNSUPPORTED),
    (dict(E=66, n_group=33), UNSUPPORTED), (dict(n_group=4, topk_group=5), UNSUPPORTED),
    (dict(n_group=4, topk_group=0), UNSUPPORTED), (dict(n_group=8, topk_group=1), UNSUPPORTED),
    (dict(group_top=3), INVALID), (dict(logits=NUL), INVALID), (dict(idx=NUL), INVALID), (dict(w=NUL), INVALID),
    (dict(bias=ODD), INVALID), (dict(logits=ODD), INVALID), (dict(T=0, logits=NUL), OK)])
def test_route_scored(L, kw, status):
    assert route(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), INVALID), (dict(k=9), UNSUPPORTED), (dict(ldo=7), INVALID), (dict(T=0), OK), (dict(dt=5), INVALID)])
def test_route_scored_backward(L, kw, status):
    a = dict(dt=1, T=4, E=8, k=2, ldo=8, g=NUL)
    a.update(kw)
    assert L.moe_route_scored_backward(P, a["dt"], a["E"], a["T"], a["E"], a["k"], 0, NUL, 1, 1.0, P, P, a["g"], P,
                                       a["ldo"], NUL) == status


def norm(L, res=P, res_dt=0, ld_res=64, y=P, ld_y=64, gate=NUL, kind=0, gate_dt=0, ld_gate=0, post=0, post_w=NUL,
         pre=1, pre_w=NUL, wdt=0, T=4, H=64, out=P, n=P):
    return L.moe_block_norm(res, res_dt, ld_res, y, ld_y, gate, kind, gate_dt, ld_gate, 1.0, post, post_w, pre,
                            pre_w, wdt, 1e-6, T, H, out, n, NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), UNSUPPORTED), (dict(H=16385, ld_res=16385, ld_y=16385), UNSUPPORTED),
    (dict(res_dt=3), INVALID), (dict(wdt=3), INVALID), (dict(kind=4), INVALID), (dict(kind=1), INVALID),
    (dict(gate=P), INVALID), (dict(gate=P, kind=3, ld_gate=63), INVALID), (dict(gate=P, kind=1, gate_dt=4), INVALID),
    (dict(y=NUL, post=1), INVALID), (dict(y=NUL, gate=P, kind=1), INVALID), (dict(post_w=P), INVALID),
    (dict(pre=0, pre_w=P, n=NUL), INVALID), (dict(y=NUL, pre=0, n=NUL), INVALID), (dict(ld_res=63), INVALID),
    (dict(ld_y=63), INVALID), (dict(res=NUL), INVALID), (dict(out=NUL), INVALID), (dict(n=NUL), INVALID),
    (dict(pre=0), INVALID), (dict(ld_res=72), INVALID), (dict(y=ODD), INVALID), (dict(T=0, res=NUL), OK)])
def test_block_norm(L, kw, status):
    assert norm(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(gr=NUL, gn=NUL), INVALID), (dict(H=0), UNSUPPORTED), (dict(ws=NUL), INVALID), (dict(wsb=16), WORKSPACE),
    (dict(dy=NUL), INVALID), (dict(gate=P, kind=1), INVALID), (dict(res=NUL), INVALID), (dict(dpost=P), INVALID),
    (dict(gn=NUL, dpre=P), INVALID), (dict(ws=ctypes.c_void_p((1 << 20) + 16)), INVALID)])
def test_block_norm_backward(L, kw, status):
    need = L.moe_block_norm_backward_workspace_size(64)
    assert need >= 3 * 64 * 4
    a = dict(gr=P, gn=P, res=P, y=P, gate=NUL, kind=0, T=4, H=64, dy=P, dgate=NUL, dpost=NUL, dpre=NUL, ws=P, wsb=need)
    a.update(kw)
    assert L.moe_block_norm_backward(a["gr"], 64, a["gn"], 64, a["res"], 0, 64, a["y"], 64, a["gate"], a["kind"], 0, 0,
                                     1.0, 0, NUL, NUL, 0, 1e-6, a["T"], a["H"], P, a["dy"], a["dgate"], a["dpost"],
                                     a["dpre"], a["ws"], a["wsb"], NUL) == status


def lin(L, x=P, ld_x=64, w=P, ld_w=64, bias=NUL, bdt=0, act=-1, res=NUL, ld_res=0, T=4, K=64, N=32, out=P, odt=0,
        ld_out=32, z=NUL, ws=P, wsb=1 << 30):
    return L.moe_linear(x, ld_x, w, ld_w, bias, bdt, act, res, ld_res, T, K, N, out, odt, ld_out, z, ws, wsb, NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), UNSUPPORTED), (dict(K=60), UNSUPPORTED),
    (dict(ld_x=68), UNSUPPORTED), (dict(ld_w=56), INVALID), (dict(act=3), INVALID), (dict(act=-2), INVALID),
    (dict(odt=2), INVALID), (dict(bias=P, bdt=2), INVALID), (dict(ld_out=31), INVALID), (dict(res=P, ld_res=31), INVALID),
    (dict(x=NUL), INVALID), (dict(w=NUL), INVALID), (dict(out=NUL), INVALID), (dict(x=ODD), INVALID),
    (dict(res=P, ld_res=40), INVALID), (dict(z=P), INVALID), (dict(ws=NUL), INVALID), (dict(wsb=128), WORKSPACE),
    (dict(T=0, x=NUL), OK), (dict(N=0, x=NUL), OK)])
def test_linear(L, kw, status):
    assert lin(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(act=0), INVALID), (dict(z=P), INVALID), (dict(K=60), UNSUPPORTED), (dict(ydt=2), INVALID),
    (dict(ld_gy=31), INVALID), (dict(gy=NUL), INVALID), (dict(wsb=64), WORKSPACE), (dict(x=ODD), INVALID)])
def test_linear_backward(L, kw, status):
    need = L.moe_linear_backward_workspace_size(4, 32)
    assert need >= 4 * 32 * 2
    a = dict(gy=P, ydt=0, ld_gy=32, x=P, act=-1, z=NUL, K=64, wsb=need)
    a.update(kw)
    assert L.moe_linear_backward(a["gy"], a["ydt"], a["ld_gy"], a["x"], 64, P, 64, a["act"], a["z"], 32, 4, a["K"], 32,
                                 P, P, NUL, P, a["wsb"], NUL) == status


def test_the_bindings_refuse_host_tensors():
    import torch

    import mixture_experts_routed_top_gb300 as m
    t = torch.zeros(4, 8)
    for call in (lambda: m.route_scored(t, 2), lambda: m.block_norm(t), lambda: m.linear(t, t),
                 lambda: m.linear_backward(t, t, t), lambda: m.block_norm_backward(t, t, t)):
        with pytest.raises(ValueError):
            call()


def test_packed_calls(L):
    """One block of 8-byte slots stands for the arguments; each call's own refusals come back."""
    def block(*v):
        return struct.pack("=" + "".join("d" if isinstance(x, float) else "q" for x in v), *v)

    p = P.value
    route_args = [p, 1, 8, 4, 8, 2, 1, 0, 1, 1, 2, 1, 1.0, p, p, 0]
    for call, at, value, status in [(0, 3, -1, INVALID), (0, 5, 9, UNSUPPORTED), (0, 3, 1 << 32, UNSUPPORTED),
                                    (0, 13, 0, INVALID), (0, 3, 0, OK), (6, 3, 0, INVALID), (-1, 3, 0, INVALID)]:
        a = list(route_args)
        a[at] = value
        assert L.moe_call_packed(call, block(*a)) == status
    # T, K, N of a product: a length that is no multiple of 8
    assert L.moe_call_packed(4, block(p, 12, p, 12, 0, 0, -1, 0, 0, 4, 12, 8, p, 0, 8, 0, p, 1 << 25, 0)) == UNSUPPORTED
    assert L.moe_call_packed(0, None) == INVALID
