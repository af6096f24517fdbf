"""The operators around the experts on the GPU against the float64 oracle.

Tolerances, from the arithmetic: a bf16 result is one rounding of a value
held in fp32, half a unit in the last of its 8 significant bits, at most 2^-8
of it (BF); fp32 arithmetic over a row of H <= 16384
terms in trees of at most 16 levels stays within 2^-18 of the sum of the
terms' magnitudes (F32); a tensor-core sum of K products adds them 16 at a
time, each addition off by at most 2^-23 of the running sum, which the sum of
magnitudes bounds: (K / 16 + 16) 2^-23 of that (ACC).  Indices have to be equal
wherever the oracle's margin is above SURE = 2^-18, 64 roundings, of the row's
largest score and bias.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8
F32 = 2.0 ** -18
SURE = 2.0 ** -18


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


# ------------------------------------------------------------------ routing
ROUTES = [  # T, E, k, n_group, topk_group, group_top
    (1, 256, 8, 8, 4, 2), (513, 256, 8, 8, 4, 2), (300, 60, 4, 1, 1, 2), (33, 8, 2, 2, 1, 1), (70, 160, 6, 8, 3, 2),
    (9, 1024, 32, 32, 8, 2), (5, 1, 1, 1, 1, 1), (64, 128, 8, 1, 1, 2), (17, 33, 32, 1, 1, 2), (40, 384, 8, 6, 2, 2),
    (21, 96, 5, 4, 2, 1), (8, 513, 7, 1, 1, 2), (12, 64, 2, 32, 2, 2)]


@pytest.mark.parametrize("T,E,k,ng,tg,gt", ROUTES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_scored(moe, T, E, k, ng, tg, gt, score, dtype):
    g = _rng(T, E, k)
    x = _dev(g.normal(size=(T, E)) * 2, dtype)
    for bias in (None, _dev(np.round(g.normal(size=E) * 30) * 1e-3)):
        for renorm, scale in ((True, 2.5), (False, 1.0)):
            kw = dict(score=score, n_group=ng, topk_group=tg, group_top=gt, renormalise=renorm, scale=scale)
            idx, w = moe.route_scored(x, k, bias=bias, **kw)
            ridx, rw, margin = B.route_scored(_np(x), k, bias=None if bias is None else _np(bias), **kw)
            top = B.scores(_np(x), score).max(1) + (0 if bias is None else np.abs(_np(bias)).max())
            sure = margin > SURE * top
            # nearly every row is decided
            assert sure.sum() >= T // 2
            assert np.array_equal(idx.cpu().numpy()[sure], ridx[sure])
            _close(w[torch.from_numpy(sure).cuda()], rw[sure], np.abs(rw[sure]), False)


def test_route_scored_ties_and_masks(moe):
    inf = float("inf")
    rows = [[0.5] * 8, [-inf] * 8, [float("nan")] * 8, [-inf, 1, -inf, 1, 1, float("nan"), -inf, 0],
            [inf, 0, 1, -inf, 0, 0, 0, 0], [-200.0] * 8, [200.0, 100.0, 3, 2, 1, 0, -1, -2],
            [-inf, -inf, -inf, -inf, -inf, -inf, -inf, -3.0]]
    x = torch.tensor(rows)
    for score in ("sigmoid", "softmax"):
        for ng, tg in ((1, 1), (4, 2), (2, 1)):
            for renorm in (True, False):
                kw = dict(score=score, n_group=ng, topk_group=tg, renormalise=renorm)
                idx, w = moe.route_scored(x.cuda(), 3, **kw) if ng != 4 else moe.route_scored(x.cuda(), 3, **kw)
                ridx, rw, _ = B.route_scored(x.numpy(), 3, **kw)
                if score == "sigmoid":  # in 32 bits 200 and 100 both score exactly 1 and tie: index order
                    assert ridx[6, 0] == 0
                assert np.array_equal(idx.cpu().numpy(), ridx), (score, ng, renorm)
                np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-6, atol=1e-37)
    bias = torch.tensor([0, -inf, float("nan"), 0, 5, 0, 0, 0.0])
    idx, w = moe.route_scored(x[:1].cuda(), 8, bias=bias.cuda(), renormalise=False)
    assert idx.cpu().tolist() == [[4, 0, 3, 5, 6, 7, 1, 2]]
    assert (w.cpu()[0, 6:] == 0).all() and (w.cpu()[0, :6] > 0.6).all()


def test_route_scored_rows_apart_and_streams(moe):
    g = _rng(5)
    big = _dev(g.normal(size=(50, 200)))
    for cut in (slice(8, 72), slice(3, 63)):        # aligned and unaligned row starts
        x = big[:, cut]
        if x.data_ptr() % 16:
            with pytest.raises(moe.MoEError):
                moe.route_scored(x, 4)
            x = big[:, cut.start - cut.start % 4:][:, : 60]
        a = moe.route_scored(x, 4)
        b = moe.route_scored(x.contiguous(), 4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = (torch.empty(50, 4, dtype=torch.int32, device="cuda"), torch.empty(50, 4, device="cuda"))
    moe.route_scored(x, 4, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out[0], b[0]) and torch.equal(out[1], b[1])
    assert moe.route_scored(x[:0], 4)[0].shape == (0, 4)


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (130, 60, 4), (17, 1024, 32), (9, 33, 5), (6, 8, 8), (3, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_scored_backward(moe, T, E, k, score, renorm, dtype):
    g = _rng(T, E, k, 7)
    x = _dev(g.normal(size=(T, E)) * 2, dtype)
    if E > 40:
        x[0, 3:9] = float("-inf")
    gw = _dev(g.normal(size=(T, k)))
    idx, w = moe.route_scored(x, k, score=score, renormalise=renorm, scale=2.0)
    d = moe.route_scored_backward(x, idx, w, gw, score=score, renormalise=renorm, scale=2.0)
    ref = B.route_scored_backward(_np(x), idx.cpu().numpy(), _np(w), _np(gw), score, None, renorm, 2.0)
    mag = np.abs(_np(gw)).sum(1, keepdims=True) * 2 * (1.0 if renorm else np.abs(_np(w)).max(1, keepdims=True))
    _close(d, ref, mag, dtype == torch.bfloat16, 2.0 ** -20)


def test_route_scored_backward_masked_rows(moe):
    inf = float("inf")
    x = torch.tensor([[-inf] * 4, [0.0, -inf, -inf, -inf], [90.0, -90.0, 0, 0]]).cuda()
    gw = torch.tensor([[1.0, -2.0]] * 3).cuda()
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            idx, w = moe.route_scored(x, 2, score=score, renormalise=renorm)
            d = moe.route_scored_backward(x, idx, w, gw, score=score, renormalise=renorm)
            ref = B.route_scored_backward(_np(x), idx.cpu().numpy(), _np(w), _np(gw), score, None, renorm)
            assert torch.isfinite(d).all()
            np.testing.assert_allclose(_np(d), ref, rtol=1e-5, atol=1e-6)
    bad = torch.tensor([[0, 7], [-1, 1], [2, 3]], dtype=torch.int32).cuda()     # outside [0, E): no gradient
    d = moe.route_scored_backward(x, bad, torch.ones(3, 2, device="cuda"), gw, renormalise=False)
    assert d[1].abs().sum() == 0 and d[2, 0] == 0 and d[2, 2] != 0


# ------------------------------------------------------------------ norms
NORMS = [(1, 7168), (5, 2048), (700, 128), (3, 1000), (4, 1001), (2, 16384), (9, 72), (2, 1), (3, 9000), (1, 24)]


def _norm_case(T, H, stream, wdtype, gate, post, seed):
    g = _rng(T, H, seed)
    v = dict(residual=_dev(g.normal(size=(T, H)) * 2, stream), y=_dev(g.normal(size=(T, H)), torch.bfloat16),
             pre_weight=_dev(1 + 0.2 * g.normal(size=H), wdtype),
             post_weight=_dev(1 + 0.2 * g.normal(size=H), wdtype) if post else None,
             gate={"none": lambda: None, "channel": lambda: _dev(g.normal(size=H)),
                   "token": lambda: _dev(g.normal(size=(T, 1)), torch.bfloat16),
                   "element": lambda: _dev(g.normal(size=(T, H)), torch.bfloat16)}[gate]())
    return g, v


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate,post", [("none", True), ("channel", True), ("token", False), ("element", True)])
def test_block_norm_and_gradient(moe, T, H, stream, gate, post):
    wdtype = torch.bfloat16 if H % 16 else torch.float32
    g, v = _norm_case(T, H, stream, wdtype, gate, post, 1)
    if T == H and gate == "token":
        pytest.skip("a [T, 1] gate of T = H = 1 is per channel")
    bf = stream == torch.bfloat16
    kw = dict(gate=v["gate"], scale=0.5, post_norm=post, post_weight=v["post_weight"], pre_weight=v["pre_weight"])
    r, n = moe.block_norm(v["residual"], v["y"], **kw)
    nkw = {k: (_np(t) if torch.is_tensor(t) else t) for k, t in kw.items()}
    rr, rn = B.block_norm(_np(v["residual"]), _np(v["y"]), **nkw)
    _close(r, rr, np.abs(rr) + np.abs(_np(v["residual"])) + 4, bf, 2.0 ** -20)
    _close(n, rn, (np.abs(_np(v["residual"])) + 4) * np.abs(rn / np.where(rr == 0, 1, rr)), True, 2.0 ** -20)
    gr, gn = _dev(g.normal(size=(T, H)), stream), _dev(g.normal(size=(T, H)), torch.bfloat16)
    got = moe.block_norm_backward(gr, gn, r, v["y"], **kw)
    ref = B.block_norm_backward(_np(gr), _np(gn), _np(r), _np(v["y"]), **nkw)
    d = np.abs(ref["d_residual"]).max() + 1
    gmax = 1.0 if v["gate"] is None else np.abs(nkw["gate"]).max() + 1
    _close(got[0], ref["d_residual"], d, bf)
    _close(got[1], ref["d_y"], np.abs(ref["d_y"]).max() + d * gmax, True)
    if gate != "none":
        terms = {"channel": T, "token": H, "element": 1}[gate]
        _close(got[2], ref["d_gate"], d * 6 * terms, gate in ("token", "element"))
    else:
        assert got[2] is None
    if post:
        _close(got[3], ref["d_post_weight"], d * gmax * 6 * T, False)
    _close(got[4], ref["d_pre_weight"], 6 * np.abs(_np(gn)).max() * T, False)
    again = moe.block_norm_backward(gr, gn, r, v["y"], **kw)      # sums over tokens in a fixed order
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("T,H,pad", [(2000, 77, 0), (3000, 7, 1), (1500, 1001, 3), (700, 264, 1), (500, 2051, 0),
                                     (330, 7167, 2), (320, 8192, 5)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["channel", "element"])
def test_block_norm_ragged_rows(moe, T, H, pad, stream, gate):
    """Several rows per block at every alignment of their starts; rows of a wider matrix."""
    g, v = _norm_case(T, H, stream, torch.bfloat16, gate, True, 3)

    def rows(t, extra):      # the same rows inside a matrix whose other columns are NaN
        big = torch.full((T, H + extra), float("nan"), dtype=t.dtype, device="cuda")
        big[:, :H] = t
        return big[:, :H]

    res, y = rows(v["residual"], pad), rows(v["y"], 2 * pad)
    kw = dict(gate=rows(v["gate"], pad) if gate == "element" else v["gate"], scale=0.5, post_norm=True,
              post_weight=v["post_weight"], pre_weight=v["pre_weight"])
    nkw = {k: (_np(t) if torch.is_tensor(t) else t) for k, t in kw.items()}
    r, n = moe.block_norm(res, y, **kw)
    rr, rn = B.block_norm(_np(res), _np(y), **nkw)
    bf = stream == torch.bfloat16
    _close(r, rr, np.abs(rr) + np.abs(_np(res)) + 4, bf, 2.0 ** -20)
    _close(n, rn, (np.abs(_np(res)) + 4) * np.abs(rn / np.where(rr == 0, 1, rr)), True, 2.0 ** -20)
    gr, gn = rows(_dev(g.normal(size=(T, H)), stream), pad), rows(_dev(g.normal(size=(T, H)), torch.bfloat16), 3 * pad)
    got = moe.block_norm_backward(gr, gn, rows(r, pad), y, **kw)
    ref = B.block_norm_backward(_np(gr), _np(gn), _np(r), _np(y), **nkw)
    d, gmax = np.abs(ref["d_residual"]).max() + 1, np.abs(nkw["gate"]).max() + 1
    _close(got[0], ref["d_residual"], d, bf)
    _close(got[1], ref["d_y"], np.abs(ref["d_y"]).max() + d * gmax, True)
    _close(got[2], ref["d_gate"], d * 6 * (T if gate == "channel" else 1), gate == "element")
    _close(got[3], ref["d_post_weight"], d * gmax * 6 * T, False)
    _close(got[4], ref["d_pre_weight"], 6 * np.abs(_np(gn)).max() * T, False)
    for a, b in zip(got, moe.block_norm_backward(gr, gn, rows(r, pad), y, **kw)):
        assert torch.equal(a, b)


def test_block_norm_parts(moe):
    g, v = _norm_case(7, 264, torch.bfloat16, torch.bfloat16, "none", False, 2)
    r, y, w = v["residual"], v["y"], v["pre_weight"]
    # the norm alone: the stream comes back as it is
    out, n = moe.block_norm(r, pre_weight=w)
    assert out is r
    _close(n, B.block_norm(_np(r), pre_weight=_np(w))[1], np.abs(_np(n)), True, 2.0 ** -20)
    # the sum alone, in place, and rows of a larger matrix
    big = torch.zeros(7, 300, dtype=torch.bfloat16, device="cuda")
    big[:, 3:267] = y
    ref = B.block_norm(_np(r), _np(y), scale=0.25, pre_norm=False)[0]
    for yy in (y, big[:, 3:267]):
        if yy.data_ptr() % 16:
            with pytest.raises(moe.MoEError):
                moe.block_norm(r, yy, scale=0.25, pre_norm=False)
            big[:, 8:272] = y
            yy = big[:, 8:272]
        s, none = moe.block_norm(r, yy, scale=0.25, pre_norm=False)
        assert none is None
        _close(s, ref, np.abs(ref), True, 2.0 ** -20)
    copy = r.clone()
    moe.block_norm(copy, y, scale=0.25, pre_norm=False, out=(copy, None))
    assert torch.equal(copy, s)
    # a gradient of the sum alone
    d = moe.block_norm_backward(r, None, r, y, scale=0.25)
    assert torch.equal(d[0], r) and d[2] is None and d[4] is None
    _close(d[1], 0.25 * _np(r), np.abs(_np(r)), True)
    # no rows
    e = moe.block_norm_backward(r[:0], y[:0], r[:0], y[:0], post_norm=True, post_weight=w, pre_weight=w)
    assert e[0].shape == (0, 264) and e[3].abs().sum() == 0 and e[4].abs().sum() == 0


def test_block_norm_zero_rows_and_non_finite(moe):
    z = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    r, n = moe.block_norm(z, z, post_norm=True, eps=1e-6)
    assert (r == 0).all() and (n == 0).all()
    bad = z.clone()
    bad[0, 5] = float("nan")
    r, n = moe.block_norm(z, bad)
    assert torch.isnan(r[0, 5]) and torch.isnan(n[0]).all() and (n[1] == 0).all()   # rows stay apart


# ------------------------------------------------------------------ products
def _acc(K):
    return (K / 16 + 16) * 2.0 ** -23


LINEARS = [  # T, K, N: one tile and less, ragged edges, a split contraction, several tiles, both tile kernels
    (1, 8, 1), (1, 2048, 512), (2, 2056, 1000), (12, 7168, 40), (15, 136, 4001), (30, 1032, 700), (32, 64, 17),
    (17, 512, 1025), (3, 264, 77), (8, 1024, 130), (9, 64, 1), (16, 7168, 256), (100, 72, 33),
    (129, 1024, 129), (300, 520, 264), (257, 136, 3), (2050, 192, 1536), (2049, 328, 1601),
    (1301, 2056, 2041)]


@pytest.mark.parametrize("T,K,N", LINEARS)
@pytest.mark.parametrize("act", [None, "silu", "gelu", "relu"])
def test_linear_and_gradient(moe, T, K, N, act):
    g = _rng(T, K, N)
    x, w = _dev(g.normal(size=(T, K)), torch.bfloat16), _dev(g.normal(size=(N, K)) / K ** 0.5, torch.bfloat16)
    mag = np.abs(_np(x)) @ np.abs(_np(w)).T
    for dt, bdt, res, bias in ((torch.bfloat16, torch.float32, True, True), (torch.float32, torch.bfloat16, False, True),
                               (torch.bfloat16, None, False, False)):
        bf = dt == torch.bfloat16
        b = _dev(g.normal(size=N), bdt) if bias else None
        r = _dev(g.normal(size=(T, N)), dt) if res else None
        y, z = moe.linear(x, w, bias=b, activation=act, residual=r, out_dtype=dt, preact=True)
        ry, rz = B.linear(_np(x), _np(w), None if b is None else _np(b), act, None if r is None else _np(r))
        m = mag + np.abs(rz) + (0 if r is None else np.abs(_np(r)))
        _close(z, rz, m, bf, _acc(K))
        _close(y, ry, 1.2 * m, bf, _acc(K) + 2.0 ** -21)     # |act'| < 1.2
        assert torch.equal(moe.linear(x, w, bias=b, activation=act, residual=r, out_dtype=dt), y)
        gy = _dev(g.normal(size=(T, N)), dt)
        pre = None if act is None else z
        dx, dw, db = moe.linear_backward(gy, x, w, bias=b, activation=act, preact=pre)
        rdx, rdw, rdb, dz = B.linear_backward(_np(gy), _np(x), _np(w), act, None if pre is None else _np(pre))
        # dz enters the products rounded to bf16 (it is exact where it is a bf16 gradient itself)
        az = np.abs(dz)
        _close(dx, rdx, az @ np.abs(_np(w)), True, _acc(N) + BF)
        _close(dw, rdw, az.T @ np.abs(_np(x)), True, _acc(T) + BF)
        if bias:
            _close(db, rdb, 1.2 * np.abs(_np(gy)).sum(0), False)     # the terms of act' are at most 1.2
        else:
            assert db is None
    moe.workspace_status(moe.default_workspace())


@pytest.mark.parametrize("T,K,N", [(1, 5392, 24), (2, 136, 512), (3, 64, 7), (1024, 72, 1), (31, 2048, 33)])
@pytest.mark.parametrize("act,dt", [("silu", torch.bfloat16), ("gelu", torch.bfloat16), ("relu", torch.float32),
                                    (None, torch.float32)])
def test_linear_gradient_of_few_dz(moe, T, K, N, act, dt):
    """Up to 1024 dz enter the products as two bf16 numbers: 2^-17 of dz is left, and
    2^-18 of rounding the smaller product, beside the result's own rounding."""
    g = _rng(T, K, N, 11)
    x, w = _dev(g.normal(size=(T, K)), torch.bfloat16), _dev(g.normal(size=(N, K)) / K ** 0.5, torch.bfloat16)
    gy = _dev(g.normal(size=(T, N)), dt)
    z = None if act is None else _dev(g.normal(size=(T, N)) * 2, dt)
    dx, dw, _ = moe.linear_backward(gy, x, w, activation=act, preact=z)
    rdx, rdw, _, dz = B.linear_backward(_np(gy), _np(x), _np(w), act, None if z is None else _np(z))
    az = np.abs(dz) + 2.0 ** -5 * np.abs(_np(gy))      # the slope's terms cancel where it crosses zero
    _close(dx, rdx, az @ np.abs(_np(w)), True, _acc(N) + 2.0 ** -16)
    _close(dw, rdw, az.T @ np.abs(_np(x)), True, _acc(T) + 2.0 ** -16)


@pytest.mark.parametrize("T,K,N,act", [(1800, 4104, 1000, "silu"), (2300, 5000, 1030, "gelu"), (130, 7168, 260, None),
                                       (600, 6152, 1500, "relu")])
def test_linear_fp32_results_of_long_contractions(moe, T, K, N, act):
    """fp32 results: at most 1024 of the contraction is added in one tensor-core
    accumulator, whatever its length; the sums of those parts are fp32 (F32)."""
    g = _rng(T, K, N)
    x, w = _dev(g.normal(size=(T, K)), torch.bfloat16), _dev(g.normal(size=(N, K)) / K ** 0.5, torch.bfloat16)
    b, r = _dev(g.normal(size=N)), _dev(g.normal(size=(T, N)))
    ry, rz = B.linear(_np(x), _np(w), _np(b), act, _np(r))
    y, z = moe.linear(x, w, bias=b, activation=act, residual=r, out_dtype=torch.float32, preact=True)
    mag = np.abs(_np(x)) @ np.abs(_np(w)).T + np.abs(rz) + np.abs(_np(r))
    _close(z, rz, mag, False, _acc(1024))
    _close(y, ry, 1.2 * mag, False, _acc(1024) + 2.0 ** -21)
    # truncation of 1024 / 16 additions, half a unit on average, is 2^-18 of the result at most
    assert np.linalg.norm(_np(z) - rz) < 2.0 ** -18 * np.linalg.norm(rz)
    moe.workspace_status(moe.default_workspace())


def test_linear_strides_in_place_and_parts(moe):
    g = _rng(11)
    big = _dev(g.normal(size=(70, 400)), torch.bfloat16)
    x, w = big[:, 16:216], _dev(g.normal(size=(90, 256)), torch.bfloat16)[:, 8:208]
    ref = moe.linear(x.contiguous(), w.contiguous())
    assert torch.equal(moe.linear(x, w), ref)
    out = torch.zeros(70, 104, dtype=torch.bfloat16, device="cuda")
    moe.linear(x, w, out=out[:, :90])
    assert torch.equal(out[:, :90], ref) and (out[:, 90:] == 0).all()
    acc = ref.clone()
    moe.linear(x, w, residual=acc, out=acc)                 # in place on the residual
    _close(acc, 2 * _np(ref), np.abs(_np(x)) @ np.abs(_np(w)).T, True, BF)
    gy = out[:, :90]
    a = moe.linear_backward(gy, x, w, need_w=False)
    b = moe.linear_backward(gy.contiguous(), x.contiguous(), w.contiguous(), bias=torch.zeros(90, device="cuda"), need_x=False)
    full = moe.linear_backward(gy, x, w)
    assert a[1] is None and b[0] is None and torch.equal(a[0], full[0]) and torch.equal(b[1], full[1])
    _close(b[2], _np(gy).sum(0), np.abs(_np(gy)).sum(0), False)
    e = moe.linear_backward(gy[:0], x[:0], w, bias=torch.zeros(90, device="cuda"))
    assert e[0].shape == (0, 200) and (e[1] == 0).all() and (e[2] == 0).all()
    assert moe.linear(x[:0], w).shape == (0, 90) and moe.linear(x, w[:0]).shape == (70, 0)
    with pytest.raises(ValueError):
        moe.linear(x, w, activation="tanh")
    with pytest.raises(moe.MoEError):
        moe.linear(big[:, :196], big[:5, :196])             # K not a multiple of 8


def test_linear_non_finite_rows_stay_apart(moe):
    for T in (2, 40):
        x = torch.ones(T, 64, dtype=torch.bfloat16, device="cuda")
        w = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
        x[1, 7] = float("inf")
        w[2, 9] = float("nan")
        y = moe.linear(x, w, activation="relu", out_dtype=torch.float32)
        assert (y[0, :2] == 64).all() and torch.isinf(y[1, :2]).all()
        z = moe.linear(x, w, out_dtype=torch.float32)
        assert torch.isnan(z[:, 2]).all()


def test_operators_in_a_graph(moe):
    """Every operator can be captured: no allocation or synchronisation of its own."""
    g = _rng(12)
    x, w = _dev(g.normal(size=(64, 256)), torch.bfloat16), _dev(g.normal(size=(32, 256)) / 16, torch.bfloat16)
    r = _dev(g.normal(size=(64, 256)), torch.bfloat16)

    def step():
        s, n = moe.block_norm(r, x, post_norm=True)
        idx, p = moe.route_scored(moe.linear(n, w, out_dtype=torch.float32), 4, n_group=4, topk_group=2)
        return s, idx, p, *moe.linear_backward(moe.linear(n, w), n, w)[:2], moe.block_norm_backward(s, n, s, x)[1]
    want = step()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
