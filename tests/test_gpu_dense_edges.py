"""The dense half of a block where its calls could go wrong: kernels of CTA pairs again and again,
rows beyond whole tiles, buffers that overlap, values at the ends of the formats.

Tolerances as in test_gpu_dense_ops.py.
"""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import block_oracle as B
from test_gpu_dense_ops import _acc8, _close, _np, _rng, _rows8, _weights8, moe  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ 8-bit products
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_linear_fp8_pairs_again_and_again(moe, fmt):
    """Both CTAs of a pair hand their sums over 16 times a tile; each call gives the same bits,
    and rows of either CTA are right."""
    T, K, N = 2560, 2048, 1100
    g = _rng(T, K, N)
    x = _rows8(g, T, K)
    w, ws, wc, wsv = _weights8(g, N, K, fmt)
    q, s = moe.quantize_fp8_rows(x, fmt)
    y = moe.linear_fp8(q, w, ws, x_scale=s, out_dtype=torch.float32)
    at = torch.arange(0, T, 37)
    xc, _, xsv = O.quantize_blocks(_np(x)[at].astype(np.float32), 1, 128, fmt)
    ry, _, mag = B.linear_fp8(xc, xsv, wc, wsv)
    _close(y[at.cuda()], ry, mag, False, _acc8(K))
    for _ in range(40):
        assert torch.equal(moe.linear_fp8(q, w, ws, x_scale=s, out_dtype=torch.float32), y)
    moe.workspace_status(moe.default_workspace())


@pytest.mark.parametrize("T,K,N,launches", [
    (2051, 2048, 2112, 2), (2064, 4096, 2112, 2), (1032, 2048, 4090, 2),   # the last rows apart from whole tiles
    (2064, 2048, 2112, 1), (2065, 4096, 2112, 1), (2048, 2048, 2112, 1),   # too many, or none
    (1040, 512, 4096, 1), (272, 1024, 18432, 1), (528, 2048, 7168, 1)])    # a second reading of w costs more than the wave
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_linear_fp8_rows_beyond_whole_tiles(moe, T, K, N, launches, fmt):
    """Rows that would begin another wave of CTA pairs go to the kernel of few tokens only where
    that is cheaper, and are right either way."""
    g = _rng(T, K, N, 12)
    x = _rows8(g, T, K)
    w, ws, wc, wsv = _weights8(g, N, K, fmt)
    q, s = moe.quantize_fp8_rows(x, fmt)
    r = torch.from_numpy(g.normal(size=(T, N)).astype(np.float32)).cuda()
    b = torch.from_numpy(g.normal(size=N).astype(np.float32)).cuda()
    out = r.clone()
    n0 = moe.launch_count()
    moe.linear_fp8(q, w, ws, x_scale=s, bias=b, activation="silu", residual=out, out=out)
    assert moe.launch_count() - n0 == launches
    at = np.r_[0, 255, T // 256 * 256 - 1:T]          # rows of whole tiles, all beyond them
    xc, _, xsv = O.quantize_blocks(_np(x)[at].astype(np.float32), 1, 128, fmt)
    ry, rz, mag = B.linear_fp8(xc, xsv, wc, wsv, _np(b), "silu", _np(r)[at])
    _close(out[torch.from_numpy(at).cuda()], ry, 1.2 * (mag + np.abs(rz) + np.abs(_np(r)[at])), False, _acc8(K) + 2.0 ** -21)


def test_linear_fp8_rows_apart_in_a_graph_and_beside_it(moe):
    """Codes, whole tiles and the rows beyond them in one graph, replayed on new contents while another
    stream makes the same product of its own: each as by itself."""
    T, K, N = 2051, 2048, 2112
    g = _rng(T, K, N, 14)
    w, ws, _, _ = _weights8(g, N, K, "ue8m0")
    xs = [_rows8(g, T, K) for _ in range(4)]
    want = [moe.linear_fp8(x, w, ws) for x in xs]
    x, out = xs[0].clone(), torch.empty_like(want[0])
    one, two, side = moe.Workspace(), moe.Workspace(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        moe.linear_fp8(x, w, ws, out=out, workspace=one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.linear_fp8(x, w, ws, out=out, workspace=one)
    other = torch.cuda.Stream()
    for a, b in zip((0, 1, 2, 3, 1, 0), (3, 2, 1, 0, 3, 2)):
        x.copy_(xs[a])
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            y = [moe.linear_fp8(xs[b], w, ws, workspace=two) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want[a]) and all(torch.equal(v, want[b]) for v in y)
    moe.workspace_status(one)
    moe.workspace_status(two)


@pytest.mark.parametrize("T,N", [(3, 40), (12, 40), (40, 40), (2050, 1540)])
@pytest.mark.parametrize("fmt,down", [("f32", 0), ("f32", 20), ("f32", 33), ("ue8m0", 0), ("ue8m0", 20), ("ue8m0", 33)])
def test_linear_fp8_ends_of_the_range(moe, T, N, fmt, down):
    """Tokens of the smallest and the largest values against the oracle, with weights of ordinary size
    and 2^-20 and 2^-33 of it.  The scales' product is made in fp32: where it is below 2^-126 it is off
    by at most 2^-150, which times the block's sum of codes is far below the smallest result of
    ordinary tokens; so is a result below 2^-126."""
    K = 256
    g = _rng(T, N, 5, down)
    x = _rows8(g, T, K)
    w, ws, wc, wsv = _weights8(g, N, K, fmt)
    ws, wsv = (ws * 2.0 ** -down if fmt == "f32" else ws - down), wsv * 2.0 ** -down
    x[0], x[2] = 0, 0
    x[1] = torch.where(torch.arange(K, device="cuda") % 3 == 0, -(2.0 ** -132), 2.0 ** -131)
    x[2, :4] = torch.tensor([3.3e38, -3.3e38, 1e38, 3.3e38])
    q, s = moe.quantize_fp8_rows(x, fmt)
    sx = s.double().cpu().numpy() if fmt == "f32" else np.exp2(s.double().cpu().numpy() - 127)
    assert (sx[1] == 2.0 ** -126).all() and sx[2, 1] == 1                      # the least scale; a block of zeros
    largest = _np(x)[2, 0] / 448
    assert sx[2, 0] == (np.float32(largest) if fmt == "f32" else np.exp2(np.ceil(np.log2(largest))))
    xc = q.cpu().numpy()
    assert set(xc[1]) == {0x88, 0x10} and (xc[0] == 0).all()                   # -2^-6 and 2^-5, exactly
    ry, _, mag = B.linear_fp8(xc, sx, wc, wsv)
    codes = np.abs(O.moe_oracle.e4m3_decode(xc).astype(np.float64)) @ np.abs(O.moe_oracle.e4m3_decode(wc).astype(np.float64)).T
    tol = _acc8(K) * mag + 2.0 ** -23 * np.abs(ry) + (codes + 3) * 2.0 ** -150
    for dt, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        y = moe.linear_fp8(x, w, ws, out_dtype=dt)
        assert torch.equal(moe.linear_fp8(q, w, ws, x_scale=s, out_dtype=dt), y)
        got, lim = _np(y), tol + half * (np.abs(ry) + tol) + (2.0 ** -134 if half else 0)
        over = np.abs(ry) - lim >= torch.finfo(dt).max                         # infinities, with their sign
        assert (got[over] == np.sign(ry[over]) * np.inf).all()
        near = (np.abs(ry) + lim >= torch.finfo(dt).max) & ~over               # either is right
        ok = ~(over | near)
        assert (np.abs(got - ry)[ok] <= lim[ok]).all()
        assert (got[0] == 0).all() and np.isfinite(got[1]).all() and not np.isnan(got).any()
    # the bound leaves row 1, of some 2^-131 with ordinary weights, its signs and sizes
    assert down > 0 or (np.abs(ry[1]) > 8 * tol[1]).mean() > 0.8


@pytest.mark.parametrize("N,K", [(2112, 7168), (1, 128), (300, 384)])
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_linear_fp8_of_weights_that_end_inside_a_block(moe, N, K, fmt):
    """Weights of any N from quantize_fp8_blocks as documented: padded with rows of zeros, and the
    first N rows of the codes; a partial last row by itself is refused."""
    g = _rng(N, K, 21)
    x, w = _rows8(g, 9, K), torch.from_numpy(g.normal(size=(N, K)) / K ** 0.5).bfloat16().cuda()
    codes, ws = moe.quantize_fp8_blocks(torch.nn.functional.pad(w, (0, 0, 0, -N % 128)), fmt)
    padded = np.zeros((-(-N // 128) * 128, K), np.float32)
    padded[:N] = _np(w)
    wc, stored, wsv = O.quantize_blocks(padded, 128, 128, fmt)
    assert np.array_equal(codes.cpu().numpy(), wc) and np.array_equal(ws.cpu().numpy(), stored)
    xc, _, xsv = O.quantize_blocks(_np(x).astype(np.float32), 1, 128, fmt)
    ry, _, mag = B.linear_fp8(xc, xsv, wc[:N], wsv)
    _close(moe.linear_fp8(x, codes[:N], ws, out_dtype=torch.float32), ry, mag, False, _acc8(K))
    with pytest.raises(moe.MoEError):
        moe.quantize_fp8_blocks(w, fmt)


# ------------------------------------------------------------------ columns of one matrix
def test_columns_side_by_side_share_nothing(moe):
    """Results among the columns of the matrix that their operands are columns of."""
    T, K, I, N = 300, 256, 40, 72
    g = _rng(T, K, I, N)
    x, w = _rows8(g, T, K), torch.from_numpy(g.normal(size=(2 * I, K)) / 16).bfloat16().cuda()
    big = torch.zeros(T, K + I + N + 32, dtype=torch.bfloat16, device="cuda")
    big[:, :K] = x
    a, b, c = big[:, :K], big[:, K:K + I], big[:, K + I:K + I + N]
    moe.gated_linear(a, w, out=b)
    assert torch.equal(b, moe.gated_linear(x, w)) and torch.equal(a, x)
    w8, ws, _, _ = _weights8(g, N, K, "f32")
    moe.linear_fp8(a, w8, ws, out=c)
    y = moe.linear_fp8(x, w8, ws)
    assert torch.equal(c, y)
    moe.linear_fp8(a, w8, ws, residual=c, out=c)
    assert torch.equal(c, moe.linear_fp8(x, w8, ws, residual=y)) and torch.equal(a, x)
    assert (big[:, K + I + N:] == 0).all()
    # every other row of a matrix, and rows in front of and behind others
    rows = torch.zeros(2 * T, N, dtype=torch.bfloat16, device="cuda")
    rows[1::2] = y
    moe.linear_fp8(x, w8, ws, residual=rows[1::2], out=rows[::2])
    assert torch.equal(rows[::2], c) and torch.equal(rows[1::2], y)
    two = torch.zeros(2 * T, K, dtype=torch.bfloat16, device="cuda")
    two[:T] = x
    r, n = moe.layer_norm(two[:T], x, out=(None, two[T:]))
    assert torch.equal(two[:T], x) and torch.equal(n, moe.layer_norm(x, x)[1]) and n.data_ptr() == two[T:].data_ptr()
    for bad in (lambda: moe.linear_fp8(a, w8, ws, out=big[:, K - 8:K - 8 + N]), lambda: moe.gated_linear(a, w, out=big[:, K - 8:K - 8 + I]),
                lambda: moe.layer_norm(two[:T], x, out=(None, two[T - 1:-1])), lambda: moe.layer_norm(two[8:T + 8], x, out=(two[:T], None)),
                lambda: moe.quantize_fp8_rows(x, out=(x.view(torch.uint8).view(-1)[:T * K].view(T, K), torch.zeros(T, 2, device="cuda"))),
                lambda: moe.linear_fp8(x, w8, ws, residual=rows[1:T + 1], out=rows[:T])):
        with pytest.raises(moe.MoEError):
            bad()
    assert torch.equal(a, x) and torch.equal(two[:T], x)


# ------------------------------------------------------------------ layer norm
def test_layer_norm_without_a_sum_has_no_residual_out(moe):
    """A buffer that would stay unwritten is refused; residual itself or none are not."""
    x = torch.randn(5, 64, device="cuda")
    n = torch.empty(5, 64, dtype=torch.bfloat16, device="cuda")
    ref = moe.layer_norm(x)[1]
    for buf in (None, x, x[:]):
        r, got = moe.layer_norm(x, out=(buf, n))
        assert r is x and got is n and torch.equal(n, ref)
    with pytest.raises(ValueError):
        moe.layer_norm(x, out=(torch.empty_like(x), n))


# ------------------------------------------------------------------ gated products
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("T", [1, 40])
def test_gated_gradient_of_x_far_from_zero(moe, act, T):
    """dx where each dz has a column of its own: activation and slope go to 0 on the left and to z and 1
    on the right, as far as bf16 goes.  A rounding of dz and one of dx that finds it exact, or of few dz
    two parts (2^-17 is left) and a rounding; fp32 arithmetic; where e^-z leaves fp32 81 e^-80."""
    far = [-3e38, -1e33, -1e20, -1000.0, -88.5, -80.5, -79.0, -20.0, -1.0, 0.0, 0.5, 20.0, 90.0, 1000.0, 1e33]
    I, K = len(far), 64
    z = torch.cat([torch.tensor(far), torch.linspace(-2, 2, I)]).bfloat16().cuda().repeat(T, 1).contiguous()
    x, w = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"), torch.eye(2 * I, K, dtype=torch.bfloat16, device="cuda")
    gh = torch.linspace(-1, 1.5, T * I, device="cuda").view(T, I).bfloat16()
    dx, dw, _ = moe.gated_linear_backward(gh, x, w, z, activation=act)
    zg, zu = _np(z)[:, :I], _np(z)[:, I:]
    with np.errstate(over="ignore", invalid="ignore"):
        terms = np.concatenate([zu * np.nan_to_num(B._slope(zg, act)), B._act(zg, act)], 1)
    ref = np.concatenate([_np(gh), _np(gh)], 1) * terms
    assert (np.abs(_np(dx)[:, :2 * I] - ref) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(ref) + 250 * np.exp(-80.0)).all()
    assert (dx[:, 2 * I:] == 0).all() and (dw == 0).all()
