"""The dense half of a block on the GPU against the float64 oracle: gated products, 8-bit
products with block scales, layer norm.

Tolerances as in test_gpu_block_ops.py, from the arithmetic: a bf16 result is one
rounding, at most 2^-8 of it (BF); a tensor-core sum of K products is off by at most
(K / 16 + 16) 2^-23 of the sum of magnitudes (_acc); fp32 arithmetic over a row or
a column stays within 2^-18 of the sum of magnitudes (F32).
"""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8
F32 = 2.0 ** -18


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routed_top_gb300 as m
    m.lib()
    return m


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rng(*seed):
    return np.random.default_rng(list(seed))


def _dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _close(got, ref, mag, bf16, f32=F32):
    """|got - ref| within one rounding of ref, plus fp32 arithmetic on mag."""
    err = np.abs(_np(got) - ref)
    # half a unit of the highest binade the value before rounding can be in
    half = np.exp2(np.floor(np.log2(np.abs(ref) + f32 * mag + 1e-300)) - 8)
    tol = (half * 1.01 if bf16 else 2.0 ** -23 * np.abs(ref)) + f32 * mag + 1e-30
    bad = ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(err / tol):.2f} of the tolerance"


def _acc(K):
    return (K / 16 + 16) * 2.0 ** -23


# ------------------------------------------------------------------ gated products
GATED = [  # T, K, I: one token, few tokens, one tile and less, ragged edges, split contractions, CTA pairs
    (1, 8, 1), (1, 2056, 512), (2, 2056, 1000), (8, 1024, 131), (12, 7168, 40), (16, 72, 8), (30, 1032, 500),
    (17, 512, 1025), (31, 136, 513), (9, 64, 1), (100, 72, 33), (129, 1024, 129), (300, 520, 264), (257, 136, 3),
    (256, 2048, 64), (640, 1032, 704), (2050, 192, 768), (2049, 328, 801), (1301, 2056, 1020), (3000, 64, 384)]


@pytest.mark.parametrize("T,K,I", GATED)
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_gated_linear_and_gradient(moe, T, K, I, act):
    g = _rng(T, K, I)
    x, w = _dev(g.normal(size=(T, K)), torch.bfloat16), _dev(g.normal(size=(2 * I, K)) / K ** 0.5, torch.bfloat16)
    mag = np.abs(_np(x)) @ np.abs(_np(w)).T
    for bdt in (torch.float32, torch.bfloat16, None):
        b = None if bdt is None else _dev(g.normal(size=2 * I), bdt)
        h, z = moe.gated_linear(x, w, bias=b, activation=act, preact=True)
        rh, rz = B.gated_linear(_np(x), _np(w), None if b is None else _np(b), act)
        m = mag + np.abs(rz)
        _close(z, rz, m, True, _acc(K))
        # errors of both factors: |act'| < 1.2, act's own arithmetic 2^-19 of it
        mg, mu = m[:, :I], m[:, I:]
        rg, ru = np.abs(rz[:, :I]), np.abs(rz[:, I:])
        _close(h, rh, 1.2 * (mg * ru + mu * rg) + _acc(K) * mg * mu, True, _acc(K) + 2.0 ** -19)
        assert torch.equal(moe.gated_linear(x, w, bias=b, activation=act), h)
        gh = _dev(g.normal(size=(T, I)), torch.bfloat16)
        dx, dw, db = moe.gated_linear_backward(gh, x, w, z, bias=b, activation=act)
        rdx, rdw, rdb, dz = B.gated_linear_backward(_np(gh), _np(x), _np(w), _np(z), act)
        az = np.abs(dz)
        # dz enters the products rounded to bf16; its own arithmetic is 2^-19 of the terms act' is made of
        raw = np.abs(np.concatenate([_np(gh) * _np(z)[:, I:], _np(gh) * np.abs(_np(z)[:, :I])], 1))
        _close(dx, rdx, az @ np.abs(_np(w)) + 2.0 ** -10 * (raw @ np.abs(_np(w))), True, _acc(2 * I) + BF)
        _close(dw, rdw, az.T @ np.abs(_np(x)) + 2.0 ** -10 * (raw.T @ np.abs(_np(x))), True, _acc(T) + BF)
        if b is None:
            assert db is None
        else:
            _close(db, rdb, 1.2 * raw.sum(0), False)
    moe.workspace_status(moe.default_workspace())


@pytest.mark.parametrize("T,K,I", [(1, 5392, 24), (2, 136, 256), (3, 64, 7), (500, 72, 1), (31, 2048, 16)])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_gated_gradient_of_few_dz(moe, T, K, I, act):
    """Up to 1024 dz enter the products as two bf16 numbers: 2^-17 of dz is left, and
    2^-18 of rounding the smaller product, beside the result's own rounding."""
    g = _rng(T, K, I, 11)
    x, w = _dev(g.normal(size=(T, K)), torch.bfloat16), _dev(g.normal(size=(2 * I, K)) / K ** 0.5, torch.bfloat16)
    gh, z = _dev(g.normal(size=(T, I)), torch.bfloat16), _dev(g.normal(size=(T, 2 * I)) * 2, torch.bfloat16)
    dx, dw, _ = moe.gated_linear_backward(gh, x, w, z, activation=act)
    rdx, rdw, _, dz = B.gated_linear_backward(_np(gh), _np(x), _np(w), _np(z), act)
    zg, zu = np.abs(_np(z)[:, :I]), np.abs(_np(z)[:, I:])
    # the slope's terms cancel where it crosses zero
    az = np.abs(dz) + 2.0 ** -5 * np.concatenate([np.abs(_np(gh)) * zu, np.abs(_np(gh)) * zg], 1)
    _close(dx, rdx, az @ np.abs(_np(w)), True, _acc(2 * I) + 2.0 ** -16)
    _close(dw, rdw, az.T @ np.abs(_np(x)), True, _acc(T) + 2.0 ** -16)


def test_gated_linear_strides_parts_and_empty(moe):
    g = _rng(21)
    big = _dev(g.normal(size=(70, 400)), torch.bfloat16)
    x, w = big[:, 16:216], _dev(g.normal(size=(180, 256)) / 14, torch.bfloat16)[:, 8:208]
    ref, z = moe.gated_linear(x.contiguous(), w.contiguous(), preact=True)
    assert torch.equal(moe.gated_linear(x, w), ref)
    out = torch.zeros(70, 104, dtype=torch.bfloat16, device="cuda")
    assert moe.gated_linear(x, w, out=out[:, :90]).data_ptr() == out.data_ptr()
    assert torch.equal(out[:, :90], ref) and (out[:, 90:] == 0).all()
    wide = torch.zeros(70, 200, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:188] = z
    gh, b = out[:, :90], torch.zeros(180, device="cuda")
    full = moe.gated_linear_backward(gh.contiguous(), x.contiguous(), w.contiguous(), z, bias=b)
    for got, want in zip(moe.gated_linear_backward(gh, x, w, wide[:, 8:188], bias=b), full):
        assert torch.equal(got, want)
    a = moe.gated_linear_backward(gh, x, w, z, need_w=False)
    c = moe.gated_linear_backward(gh, x, w, z, bias=b, need_x=False)
    d = moe.gated_linear_backward(gh, x, w, z, bias=b, need_x=False, need_w=False)
    assert a[1] is None and a[2] is None and torch.equal(a[0], full[0])
    assert c[0] is None and torch.equal(c[1], full[1]) and torch.equal(c[2], full[2])
    assert d[0] is None and d[1] is None and torch.equal(d[2], full[2])
    assert moe.gated_linear(x[:0], w).shape == (0, 90) and moe.gated_linear(x, w[:0]).shape == (70, 0)
    e = moe.gated_linear_backward(gh[:0], x[:0], w, z[:0], bias=b)
    assert e[0].shape == (0, 200) and (e[1] == 0).all() and (e[2] == 0).all()
    e = moe.gated_linear_backward(gh[:, :0], x, w[:0], z[:, :0], bias=b[:0])
    assert (e[0] == 0).all() and e[0].shape == (70, 200) and e[1].shape == (0, 200) and e[2].shape == (0,)
    for bad in (lambda: moe.gated_linear(x, w, activation="tanh"), lambda: moe.gated_linear(x, w, activation=None),
                lambda: moe.gated_linear(x, w[:179]), lambda: moe.gated_linear(x, w, bias=b[:90]),
                lambda: moe.gated_linear(x, w, out=out), lambda: moe.gated_linear(x.float(), w),
                lambda: moe.gated_linear_backward(gh, x, w, z[:, :90]),
                lambda: moe.gated_linear_backward(gh.float(), x, w, z)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError):
        moe.gated_linear(big[:, :196], big[:6, :196])             # K not a multiple of 8


@pytest.mark.parametrize("T,K,I", [(1, 64, 24), (5, 72, 7), (40, 64, 24), (40, 1032, 33), (2050, 64, 768), (2050, 64, 771)])
def test_gated_linear_not_finite(moe, T, K, I):
    """A NaN of a token or of a gate or up row is in all it is multiplied into, and nowhere else."""
    g = _rng(T, K, I, 3)
    x, w = _dev(g.normal(size=(T, K)), torch.bfloat16), _dev(g.normal(size=(2 * I, K)), torch.bfloat16)
    x[T // 2, 3] = float("nan")
    w[I // 2, K - 1] = float("nan")
    w[I + I // 3, 0] = float("nan")
    h, z = moe.gated_linear(x, w, activation="relu", preact=True)
    want = np.zeros((T, 2 * I), bool)
    want[T // 2], want[:, I // 2], want[:, I + I // 3] = True, True, True
    assert np.array_equal(np.isnan(_np(z)), want)
    assert np.array_equal(np.isnan(_np(h)), want[:, :I] | want[:, I:])


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("T", [1, 40])
def test_gated_gradient_far_from_zero(moe, act, T):
    """The gate's activation and slope go to 0 on the left and to z and 1 on the right, as far as bf16 goes."""
    far = [-3e38, -1e33, -1e20, -1000.0, -88.5, -80.5, -79.0, -20.0, 0.0, 20.0, 90.0, 1000.0, 1e33]
    I, K = len(far), 64
    z = torch.cat([torch.tensor(far), torch.ones(I)]).bfloat16().cuda().repeat(T, 1).contiguous()
    x, w = _dev(np.ones((T, K)), torch.bfloat16), _dev(np.ones((2 * I, K)), torch.bfloat16)
    gh = torch.ones(T, I, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = moe.gated_linear_backward(gh, x, w, z, bias=torch.zeros(2 * I, device="cuda"), activation=act)
    with np.errstate(over="ignore", invalid="ignore"):
        zg = _np(z)[0, :I]
        ref = np.concatenate([np.nan_to_num(B._slope(zg, act)), B._act(zg, act)])
    # fp32 arithmetic, and where e^-z leaves fp32 less than 81 e^-80
    assert (np.abs(_np(db) - T * ref) <= T * (2.0 ** -18 * np.abs(ref) + 81 * np.exp(-80.0))).all()
    assert (np.abs(_np(dw)[:, 0] - T * ref) <= T * (2.0 ** -7 * np.abs(ref) + 81 * np.exp(-80.0))).all()


# ------------------------------------------------------------------ 8-bit products
def _acc8(K):
    """Sums of 128 on the tensor core (at most 128 / 16 + 16 additions, 2^-23 each of the sum of
    magnitudes), then K / 128 fp32 products and additions, half of 2^-23 each."""
    return (24 + K / 128 + 1) * 2.0 ** -23


def _weights8(g, N, K, fmt):
    w = g.normal(size=(-(-N // 128) * 128, K)) / K ** 0.5 * (1 + 9 * (g.random((1, K)) < 0.02))
    w[N:] = 0
    codes, stored, scale = O.quantize_blocks(w.astype(np.float32), 128, 128, fmt)
    return torch.from_numpy(codes[:N].copy()).cuda(), torch.from_numpy(stored).cuda(), codes[:N], scale


def _rows8(g, T, K):
    return _dev(g.normal(size=(T, K)) * (0.1 + 3 * g.random((T, 1))) * (1 + 20 * (g.random((1, K)) < 0.02)), torch.bfloat16)


@pytest.mark.parametrize("T,K", [(1, 128), (31, 640), (33, 512), (64, 128), (7, 1152), (129, 2048)])
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_quantize_fp8_rows(moe, T, K, fmt):
    """Codes and scales bit for bit, in both orders of the scales and from strided rows."""
    g = _rng(T, K)
    x = _rows8(g, T, K)
    x[T // 2, :128] = 0
    codes, stored, _ = O.quantize_blocks(_np(x).astype(np.float32), 1, 128, fmt)
    q, s = moe.quantize_fp8_rows(x, fmt)
    assert q.is_contiguous() and s.is_contiguous()
    assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), stored)
    big = torch.zeros(T, K + 24, dtype=torch.bfloat16, device="cuda")
    big[:, 8:8 + K] = x
    o = (torch.zeros(T, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(K // 128, T, dtype=s.dtype, device="cuda").t())
    moe.quantize_fp8_rows(big[:, 8:8 + K], fmt, out=o)
    assert torch.equal(o[0].view(torch.uint8), q) and torch.equal(o[1], s)


FP8 = [  # T, K, N: a token, few tokens, tiles and split contractions, ragged, CTA pairs
    (1, 128, 1), (1, 2048, 7168), (2, 256, 33), (8, 7168, 100), (9, 128, 16), (16, 1152, 129), (17, 640, 1025),
    (30, 384, 700), (32, 512, 17), (33, 128, 130), (100, 7168, 576), (129, 1024, 129), (300, 512, 264), (257, 256, 3),
    (700, 2048, 1000), (2050, 256, 1536), (2049, 384, 1601), (1301, 2048, 2041), (4500, 128, 900),
    (2562, 256, 1700), (1298, 384, 3300)]         # the last two: their last rows apart from whole tiles


@pytest.mark.parametrize("T,K,N", FP8)
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_linear_fp8(moe, T, K, N, fmt):
    g = _rng(T, K, N, 8)
    x = _rows8(g, T, K)
    w, ws, wc, wsv = _weights8(g, N, K, fmt)
    q, s = moe.quantize_fp8_rows(x, fmt)
    xc, xs, xsv = O.quantize_blocks(_np(x).astype(np.float32), 1, 128, fmt)
    for act, dt, bdt, res in (("silu", torch.bfloat16, torch.float32, True), (None, torch.float32, None, False),
                              ("gelu", torch.float32, torch.bfloat16, True), ("relu", torch.bfloat16, None, False),
                              ("silu", torch.float32, torch.bfloat16, False), (None, torch.bfloat16, None, True),
                              ("gelu", torch.bfloat16, None, False), ("relu", torch.float32, None, True)):
        b = None if bdt is None else _dev(g.normal(size=N), bdt)
        r = _dev(g.normal(size=(T, N)), dt) if res else None
        ry, rz, mag = B.linear_fp8(xc, xsv, wc, wsv, None if b is None else _np(b), act, None if r is None else _np(r))
        m = mag + np.abs(rz) + (0 if r is None else np.abs(_np(r)))
        y = moe.linear_fp8(x, w, ws, bias=b, activation=act, residual=r, out_dtype=dt)
        _close(y, ry, 1.2 * m, dt == torch.bfloat16, _acc8(K) + 2.0 ** -21)     # |act'| < 1.2
        # the same codes, however they come
        for qq, ss in ((q, s), (q.view(torch.float8_e4m3fn), s.t().contiguous().t())):
            y2 = moe.linear_fp8(qq, w.view(torch.float8_e4m3fn), ws, x_scale=ss, bias=b, activation=act, residual=r, out_dtype=dt)
            assert torch.equal(y2, y)
    moe.workspace_status(moe.default_workspace())


def test_linear_fp8_strides_in_place_and_empty(moe):
    g = _rng(31)
    x = _rows8(g, 70, 256)
    w, ws, wc, wsv = _weights8(g, 90, 256, "f32")
    ref = moe.linear_fp8(x, w, ws)
    big, wbig = torch.zeros(70, 400, dtype=torch.bfloat16, device="cuda"), torch.zeros(90, 320, dtype=torch.uint8, device="cuda")
    big[:, 16:272], wbig[:, 32:288] = x, w
    out = torch.zeros(70, 104, dtype=torch.bfloat16, device="cuda")
    moe.linear_fp8(big[:, 16:272], wbig[:, 32:288], ws, out=out[:, :90])
    assert torch.equal(out[:, :90], ref) and (out[:, 90:] == 0).all()
    q, s = moe.quantize_fp8_rows(x)
    qbig = torch.zeros(70, 288, dtype=torch.uint8, device="cuda")
    qbig[:, 16:272] = q
    sbig = torch.zeros(141, 5, device="cuda")
    sbig[1::2, 1:5:2] = s
    assert torch.equal(moe.linear_fp8(qbig[:, 16:272], w, ws, x_scale=sbig[1::2, 1:5:2]), ref)      # apart from each other
    acc = ref.clone()
    moe.linear_fp8(x, w, ws, residual=acc, out=acc)
    _close(acc, 2 * _np(ref), 4 * np.abs(_np(ref)), True, BF)
    assert moe.linear_fp8(x[:0], w, ws).shape == (0, 90) and moe.linear_fp8(x, w[:0], ws[:0]).shape == (70, 0)
    q0, s0 = moe.quantize_fp8_rows(x[:0])
    assert q0.shape == (0, 256) and s0.shape == (0, 2)
    e8 = torch.zeros(1, 2, dtype=torch.uint8, device="cuda")
    for bad in (lambda: moe.linear_fp8(x, w, ws[:, :1]), lambda: moe.linear_fp8(x, w, ws, x_scale=s),
                lambda: moe.linear_fp8(q, w, ws), lambda: moe.linear_fp8(q, w, e8, x_scale=s),
                lambda: moe.linear_fp8(x, w, ws, activation="tanh"), lambda: moe.linear_fp8(x, w.float(), ws),
                lambda: moe.linear_fp8(x, w, ws, out=out), lambda: moe.quantize_fp8_rows(x, "none"),
                lambda: moe.quantize_fp8_rows(x.float()), lambda: moe.quantize_fp8_rows(x, out=(q, s[:, :1]))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError):
        moe.quantize_fp8_rows(x[:, :136])             # K not a multiple of 128
    with pytest.raises(moe.MoEError):
        moe.linear_fp8(q, w, ws, x_scale=s[:1].expand(70, 2))     # one scale for all rows: a stride of 0


@pytest.mark.parametrize("T,N", [(3, 40), (40, 40), (2050, 1540)])
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_linear_fp8_extremes(moe, T, N, fmt):
    """Rows of zeros give zeros, the smallest and largest bf16 values keep their sign and size, and
    an infinity or NaN stays in its row; a NaN code of w stays in its column."""
    K = 256
    g = _rng(T, N)
    x = _rows8(g, T, K)
    w, ws, wc, wsv = _weights8(g, N, K, fmt)
    x[0] = 0
    x[1] = 2.0 ** -132                                  # below the smallest scale's reach: a code of 2^-6 or none
    x[2] = 0
    x[2, :4] = 3.3e38
    y = moe.linear_fp8(x, w, ws, out_dtype=torch.float32)
    assert (y[0] == 0).all() and (y[1].abs() <= K * 2.0 ** -126 * 20).all()
    assert (torch.isfinite(y[2]) | (y[2].abs() == float("inf"))).all()
    rows = torch.ones(T, dtype=torch.bool)
    x[T - 1, 5], x[2, 7] = float("nan"), float("inf")
    rows[T - 1], rows[2] = False, False
    wn = w.clone()
    wn[N // 2, 3] = 0x7F
    y2 = moe.linear_fp8(x, wn, ws, out_dtype=torch.float32)
    cols = torch.arange(N) != N // 2
    assert torch.isnan(y2[T - 1]).all() and torch.isnan(y2[:, N // 2]).all() and not torch.isfinite(y2[2]).any()
    a, b = y[rows.cuda()][:, cols.cuda()], y2[rows.cuda()][:, cols.cuda()]
    assert torch.equal(a, b)


def test_linear_fp8_long_rows_of_one_sign(moe):
    """Without cancellation the sums stay as near as fp32 ones: 2^-19 of the result over 7168."""
    g = _rng(5)
    for T, N in ((4, 64), (64, 256), (2048, 1536)):
        x = _dev(np.abs(g.normal(size=(T, 7168))), torch.bfloat16)
        w, ws, wc, wsv = _weights8(g, N, 7168, "f32")
        y = moe.linear_fp8(x, w & 0x7F, ws, out_dtype=torch.float32)
        xc, _, xsv = O.quantize_blocks(_np(x).astype(np.float32), 1, 128, "f32")
        ry = B.linear_fp8(xc, xsv, wc & 0x7F, wsv)[0]
        assert np.linalg.norm(_np(y) - ry) < 2.0 ** -19 * np.linalg.norm(ry)


# ------------------------------------------------------------------ layer norm
NORMS = [  # T, H: rows in part of a warp, a block's several rows, odd widths, one row, the widest, several turns of the ring
    (1, 1), (1, 7168), (3, 8), (5, 7), (37, 72), (64, 2048), (33, 2049), (19, 2056), (2, 8192), (9, 7167), (130, 264),
    (2600, 2048), (700, 7168), (5000, 77), (320, 4100), (3, 8200), (200, 12288), (170, 8193), (2, 16384), (2, 16383)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_layer_norm_and_gradient(moe, T, H, dt):
    g = _rng(T, H)
    bf = dt == torch.bfloat16
    for i, (wdt, bdt, add) in enumerate(((torch.bfloat16, True, True), (torch.float32, True, False), (None, False, True),
                                         (torch.float32, False, True), (None, True, False))):
        x = _dev(g.normal(size=(T, H)) * 2 + 4 * g.normal(size=(T, 1)), dt)
        y = _dev(g.normal(size=(T, H)), torch.bfloat16) if add else None
        w = None if wdt is None else _dev(1 + 0.3 * g.normal(size=H), wdt)
        b = _dev(g.normal(size=H), torch.float32 if wdt is None else wdt) if bdt else None
        r, n = moe.layer_norm(x, y, weight=w, bias=b)
        f = lambda t: None if t is None else _np(t)
        rr, rn = B.layer_norm(_np(x), f(y), f(w), f(b))
        if add:
            _close(r, rr, np.abs(_np(x)) + np.abs(_np(y)), bf, 2.0 ** -23)
        else:
            assert r is x
        # the mean is off by F32 of the row's magnitudes, and with it every difference from it
        aw = 1.0 if w is None else np.abs(_np(w))
        rs = 1 / np.sqrt(rr.var(1, keepdims=True) + 1e-5)
        hm = (np.abs(rr) + np.abs(rr).mean(1, keepdims=True)) * rs
        _close(n, rn, hm * aw + np.abs(rn) + (0 if b is None else np.abs(_np(b))), True)
        gn, gr = _dev(g.normal(size=(T, H)), torch.bfloat16), _dev(g.normal(size=(T, H)), dt) if i % 2 == 0 else None
        need = add or not bf
        dr, dy, dw, db = moe.layer_norm_backward(gr, gn, r, weight=w, bias=b, need_y=need)
        rdr, rdw, rdb = B.layer_norm_backward(f(gr), _np(gn), _np(r), f(w))
        v = _np(r)
        rs = 1 / np.sqrt(v.var(1, keepdims=True) + 1e-5)
        hm = (np.abs(v) + np.abs(v).mean(1, keepdims=True)) * rs
        q = np.abs(_np(gn)) * aw
        mag = rs * (q + q.mean(1, keepdims=True) + hm * (q * hm).mean(1, keepdims=True)) + (0 if gr is None else np.abs(_np(gr)))
        _close(dr, rdr, mag, bf)
        assert (dy is dr) if bf and need else (dy is None) if not need else torch.equal(dy, dr.bfloat16())
        if w is None:
            assert dw is None
        else:
            _close(dw, rdw, (np.abs(_np(gn)) * hm).sum(0), False)
        if b is None:
            assert db is None
        else:
            _close(db, rdb, np.abs(_np(gn)).sum(0), False)


def test_layer_norm_far_from_zero(moe):
    """A stream at 4096 with a spread of one: the variance is that of the differences, not a difference of squares."""
    g = _rng(9)
    for T, H in ((5, 300), (4, 2048), (3, 7167), (2, 12288)):
        x = _dev(4096 + np.round(g.normal(size=(T, H)) * 64) / 64)
        _, n = moe.layer_norm(x)
        # the mean is off by at most 2^-18 of 4096 = 2^-6; on average by the trees' few roundings of 2^-12
        ref = B.layer_norm(_np(x))[1]
        assert np.abs(_np(n) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -9


def test_layer_norm_strides_in_place_and_empty(moe):
    g = _rng(41)
    for H, lead, T in ((264, 8, 37), (264, 16, 37), (77, 8, 300)):
        x, y = _dev(g.normal(size=(T, H)), torch.bfloat16), _dev(g.normal(size=(T, H)), torch.bfloat16)
        w, b = _dev(g.normal(size=H)), _dev(g.normal(size=H))
        r, n = moe.layer_norm(x, y, weight=w, bias=b)
        big = torch.zeros(T, 400, dtype=torch.bfloat16, device="cuda")
        big[:, lead:lead + H] = x
        r2, n2 = moe.layer_norm(big[:, lead:lead + H], y, weight=w, bias=b)
        assert torch.equal(r2, r) and torch.equal(n2, n)
        copy, nn = x.clone(), torch.empty_like(n)
        r3, n3 = moe.layer_norm(copy, y, weight=w, bias=b, out=(copy, nn))
        assert r3 is copy and n3 is nn and torch.equal(copy, r) and torch.equal(nn, n)
        gr, gn = _dev(g.normal(size=(T, H)), torch.bfloat16), _dev(g.normal(size=(T, H)), torch.bfloat16)
        full = moe.layer_norm_backward(gr, gn, r, weight=w, bias=b)
        big2 = torch.zeros(T, 408, dtype=torch.bfloat16, device="cuda")
        big2[:, lead:lead + H] = gn
        again = moe.layer_norm_backward(gr, big2[:, lead:lead + H], r, weight=w, bias=b)
        assert all(torch.equal(p, q) for p, q in zip((full[0], *full[2:]), (again[0], *again[2:])))
        e = moe.layer_norm_backward(gr[:0], gn[:0], r[:0], weight=w, bias=b, need_y=True)
        assert e[0].shape == (0, H) and (e[2] == 0).all() and (e[3] == 0).all()
        assert moe.layer_norm(x[:0], y[:0])[1].shape == (0, H)
    for bad in (lambda: moe.layer_norm(x, y.float()), lambda: moe.layer_norm(x, weight=w[1:]),
                lambda: moe.layer_norm(x, weight=w, bias=b.bfloat16()), lambda: moe.layer_norm(x.half()),
                lambda: moe.layer_norm_backward(gr.float(), gn, r), lambda: moe.layer_norm_backward(gr, gn[1:], r)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError):
        moe.layer_norm(torch.zeros(2, 16392, device="cuda"))


def test_layer_norm_rows_stay_apart(moe):
    """Equal columns have variance 0 and give the bias; a NaN or an infinity stays in its row."""
    for H in (64, 77, 7168, 12288):
        x = torch.full((6, H), 3.0, device="cuda")
        x[1, H // 2], x[4, H - 1] = float("nan"), float("inf")
        b = torch.arange(H, device="cuda") * 1.0
        _, n = moe.layer_norm(x, bias=b)
        assert torch.isnan(n[1]).all() and torch.isnan(n[4]).any() and not torch.isfinite(n[4, H - 1])
        for i in (0, 2, 3, 5):
            assert torch.equal(n[i], b.bfloat16())
