"""Results of the dense half that share memory with operands or with each other are refused
before anything touches the device: by start address or only in part.  (Columns of one matrix
that lie beside each other share none: on the GPU, in test_gpu_dense_edges.py.)"""
import ctypes

import pytest

NUL = ctypes.c_void_p(0)
INVALID = 1


def at(i, more=0):
    """An address in the i-th of buffers far from each other; never dereferenced."""
    return ctypes.c_void_p((i << 30) + more)


X, W, OUT, Z, B, R, Y, S, WS = (at(i) for i in range(1, 10))


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routed_top_gb300 import build, lib
    build.build()
    return lib()


@pytest.mark.parametrize("kw", [
    dict(out=X), dict(out=at(1, 64)), dict(out=at(1, 3 * 128 + 112)), dict(out=W), dict(out=at(2, 63 * 128 + 96)),
    dict(z=OUT), dict(z=at(3, 2 * 64)), dict(z=at(1, 128)), dict(z=at(2, 4096)), dict(out=at(5, 16)), dict(z=B)])
def test_gated_linear(L, kw):
    a = dict(out=OUT, z=Z)
    a.update(kw)
    # T 4, K 64, I 32: x 512 bytes, w 8192, out 256, z 512, bias 256
    assert L.moe_gated_linear(X, 64, W, 64, B, 1, 0, 4, 64, 32, a["out"], 32, a["z"], WS, 1 << 30, NUL) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dx=X), dict(dx=at(1, 256)), dict(dx=at(7, 16)), dict(dx=at(4, 496)), dict(dw=at(2, 8176)), dict(dw=at(3, 496)),
    dict(db=at(3, 16)), dict(db=at(6, 128)), dict(db=at(4)), dict(dw=at(1, 16))])
def test_gated_linear_backward(L, kw):
    a = dict(dx=OUT, dw=R, db=S)
    a.update(kw)
    assert L.moe_gated_linear_backward(Y, 32, X, 64, W, 64, 0, Z, 64, 4, 64, 32, a["dx"], a["dw"], a["db"], WS, 1 << 30,
                                       NUL) == INVALID


@pytest.mark.parametrize("kw", [
    dict(q=X), dict(q=at(1, 2032)), dict(s=X), dict(s=at(1, 2044)), dict(s=OUT), dict(s=at(3, 1020)),
    dict(s=at(1, 4), s_row=1, s_kb=4), dict(s=OUT, s_row=7, s_kb=3)])
def test_quantize_fp8_rows(L, kw):
    a = dict(q=OUT, s=S, s_row=2, s_kb=1)
    a.update(kw)
    # T 4, K 256: x 2048 bytes, q 1024, scales 32
    assert L.moe_quantize_fp8_rows(X, 256, 4, 256, 1, a["q"], a["s"], a["s_row"], a["s_kb"], NUL) == INVALID


FP8 = [dict(out=X), dict(out=at(1, 1008)), dict(out=at(2, 32 * 256 - 16)), dict(out=W), dict(out=B),
       dict(out=at(8, 16), s=at(8, 12)), dict(out=at(6, 16)), dict(res=at(3, 64), ld_res=32), dict(res=at(3, 16), ld_res=40),
       dict(res=at(3), ld_res=40)]


@pytest.mark.parametrize("codes,kw", [(c, kw) for c in (False, True) for kw in FP8] + [(True, dict(out=Y))])
def test_linear_fp8(L, codes, kw):
    a = dict(out=OUT, res=R, ld_res=32, s=S)
    a.update(kw)
    # T 4, K 256, N 32: x 1024 bytes of codes, w 8192, out 256, residual 256, x's scales 32, w's 8 (a row of blocks)
    assert L.moe_linear_fp8(X, 256, Y if codes else NUL, 2, 1, W, 256, a["s"], 1, B, 1, -1, a["res"], a["ld_res"], 4, 256, 32,
                            a["out"], 0, 32, WS, 1 << 30, NUL) == INVALID


@pytest.mark.parametrize("kw", [
    dict(res_out=at(1, 128)), dict(res_out=Y), dict(res_out=at(7, 496)), dict(res_out=at(2, 112)), dict(n=X),
    dict(n=at(1, 16)), dict(n=at(7, 16)), dict(n=at(3, 496)), dict(n=W), dict(n=at(5, 16)), dict(n=at(1, 16), res_out=X),
    dict(y=NUL, n=at(1, 256))])
def test_layer_norm(L, kw):
    a = dict(y=Y, res_out=OUT, n=Z)
    a.update(kw)
    # T 4, H 64: rows of 128 bytes, 512 in all; weight and bias 128
    assert L.moe_layer_norm(X, 0, 64, a["y"], 64, W, B, 0, 1e-5, 4, 64, a["res_out"], a["n"], NUL) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dr=X), dict(dr=at(1, 16)), dict(dr=at(6, 128)), dict(dr=at(7, 16)), dict(dr=at(2, 16)), dict(dy=OUT),
    dict(dy=at(3, 128)), dict(dy=at(1, 128)), dict(dy=at(6, 16)), dict(dy=at(7, 16)), dict(dy=R, dr=R), dict(dw=S),
    dict(dw=at(3, 16)), dict(dw=at(8, 128))])
def test_layer_norm_backward(L, kw):
    a = dict(dr=OUT, dy=Z, dw=B)
    a.update(kw)
    # grad_residual R, grad_normed Y, residual X, weight W: rows of 128 bytes; d_bias S: 256
    assert L.moe_layer_norm_backward(R, 64, Y, 64, X, 0, 64, W, 0, 1e-5, 4, 64, a["dr"], a["dy"], a["dw"], S, WS, 1 << 30,
                                     NUL) == INVALID
