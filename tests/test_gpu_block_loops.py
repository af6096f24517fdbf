"""The operators around the experts where their kernels loop: several rows per block and
turns of the ring in the norms, several tiles per CTA pair in the products, and the
combinations of gates, norms and gradients that share a loop.

Tolerances as in test_gpu_block_ops.py: one rounding of a bf16 result, fp32 arithmetic
over a row (F32), (K / 16 + 16) 2^-23 of the terms' magnitudes for a sum on the tensor
core (_acc); and norm-wise the same, which one lost group of 16 terms out of a few
thousand would exceed many times over.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

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
    err = np.abs(_np(got) - ref)
    half = np.exp2(np.floor(np.log2(np.abs(ref) + f32 * mag + 1e-300)) - 8)
    tol = (half * 1.01 if bf16 else 2.0 ** -23 * np.abs(ref)) + f32 * mag + 1e-30
    bad = ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(err / tol):.2f} of the tolerance"


def _near(got, ref, mag, bf16, f32):
    """The same as norms: rounding is at most 2^-8 of each result, arithmetic f32 of mag."""
    err = np.linalg.norm(_np(got) - ref)
    assert err <= (2.0 ** -8 if bf16 else 2.0 ** -23) * np.linalg.norm(ref) + f32 * np.linalg.norm(mag)


# ------------------------------------------------------------------ norms
# rows per step over all blocks (forward / backward): 152 or 304 blocks x rows of a block; four to eight
# steps each, the last one partly filled
STEPS = [(20000, 72), (11000, 264), (2600, 2048), (800, 4096), (700, 7168), (21000, 77), (900, 7167)]
GATES = ["none", "channel", "token", "token32", "element", "element32"]


def _gate(g, kind, T, H):
    if kind == "none":
        return None
    shape = H if kind == "channel" else (T, 1) if kind.startswith("token") else (T, H)
    return _dev(g.normal(size=shape), torch.bfloat16 if kind in ("token", "element") else torch.float32)


@pytest.mark.parametrize("T,H", STEPS)
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate,post,weights", [("channel", True, True), ("token", True, True), ("token32", True, False),
                                               ("element32", True, True), ("none", False, True)])
def test_block_norm_over_many_steps(moe, T, H, stream, gate, post, weights):
    g = _rng(T, H, GATES.index(gate), post)
    bf = stream == torch.bfloat16
    r, y = _dev(g.normal(size=(T, H)) * 2, stream), _dev(g.normal(size=(T, H)), torch.bfloat16)
    kw = dict(gate=_gate(g, gate, T, H), scale=0.5, post_norm=post,
              post_weight=_dev(1 + 0.2 * g.normal(size=H)) if post and weights else None,
              pre_weight=_dev(1 + 0.2 * g.normal(size=H)) if weights else None)
    nkw = {k: (_np(t) if torch.is_tensor(t) else t) for k, t in kw.items()}
    out, n = moe.block_norm(r, y, **kw)
    rr, rn = B.block_norm(_np(r), _np(y), **nkw)
    _close(out, rr, np.abs(rr) + np.abs(_np(r)) + 4, bf, 2.0 ** -20)
    _close(n, rn, (np.abs(_np(r)) + 4) * np.abs(rn / np.where(rr == 0, 1, rr)), True, 2.0 ** -20)
    gr, gn = _dev(g.normal(size=(T, H)), stream), _dev(g.normal(size=(T, H)), torch.bfloat16)
    got = moe.block_norm_backward(gr, gn, out, y, **kw)
    ref = B.block_norm_backward(_np(gr), _np(gn), _np(out), _np(y), **nkw)
    d = np.abs(ref["d_residual"]).max() + 1
    gmax = 1.0 if kw["gate"] is None else np.abs(nkw["gate"]).max() + 1
    _close(got[0], ref["d_residual"], d, bf)
    _close(got[1], ref["d_y"], np.abs(ref["d_y"]).max() + d * gmax, True)
    if kw["gate"] is None:
        assert got[2] is None
    else:
        terms = {"channel": T, "token": H, "token32": H}.get(gate, 1)
        _close(got[2], ref["d_gate"], d * 6 * terms, gate in ("token", "element"))
        # sums of terms of either sign: a lost or doubled row is 1 / T of the norm's square
        _near(got[2], ref["d_gate"], np.abs(ref["d_gate"]) * terms ** 0.5, gate in ("token", "element"), F32)
    if kw["post_weight"] is not None:
        _close(got[3], ref["d_post_weight"], d * gmax * 6 * T, False)
        _near(got[3], ref["d_post_weight"], np.abs(ref["d_post_weight"]) * T ** 0.5, False, F32)
    if weights:
        _close(got[4], ref["d_pre_weight"], 6 * np.abs(_np(gn)).max() * T, False)
        _near(got[4], ref["d_pre_weight"], np.abs(ref["d_pre_weight"]) * T ** 0.5, False, F32)
    else:
        assert got[3] is None and got[4] is None
    for a, b in zip(got, moe.block_norm_backward(gr, gn, out, y, **kw)):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(2600, 2048), (11000, 264), (800, 4096), (21000, 77)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_block_norm_parts_over_many_steps(moe, T, H, stream):
    """A norm or a gradient left out: the kernels' other loops."""
    g = _rng(T, H, 9)
    bf = stream == torch.bfloat16
    r, y = _dev(g.normal(size=(T, H)) * 2, stream), _dev(g.normal(size=(T, H)), torch.bfloat16)
    w = _dev(1 + 0.2 * g.normal(size=H))
    gate = _gate(g, "channel", T, H)
    _, n = moe.block_norm(r, pre_weight=w)                       # the norm alone
    rn = B.block_norm(_np(r), pre_weight=_np(w))[1]
    _close(n, rn, np.abs(rn), True, 2.0 ** -20)
    s, none = moe.block_norm(r, y, scale=0.25, gate=gate, post_norm=True, post_weight=w, pre_norm=False)
    rs = B.block_norm(_np(r), _np(y), gate=_np(gate), scale=0.25, post_norm=True, post_weight=_np(w), pre_norm=False)[0]
    assert none is None
    _close(s, rs, np.abs(rs) + np.abs(_np(r)) + 4, bf, 2.0 ** -20)
    gr, gn = _dev(g.normal(size=(T, H)), stream), _dev(g.normal(size=(T, H)), torch.bfloat16)
    for agr, agn in ((None, gn), (gr, None)):
        kw = dict(gate=gate, scale=0.25, post_norm=True, post_weight=w, pre_weight=None if agn is None else w)
        nkw = {k: (_np(t) if torch.is_tensor(t) else t) for k, t in kw.items()}
        got = moe.block_norm_backward(agr, agn, s, y, **kw)
        ref = B.block_norm_backward(None if agr is None else _np(agr), None if agn is None else _np(agn), _np(s), _np(y),
                                    **nkw)
        d, gmax = np.abs(ref["d_residual"]).max() + 1, np.abs(_np(gate)).max() + 1
        _close(got[0], ref["d_residual"], d, bf)
        _close(got[1], ref["d_y"], np.abs(ref["d_y"]).max() + d * gmax, True)
        _close(got[2], ref["d_gate"], d * 6 * T, False)
        _near(got[2], ref["d_gate"], np.abs(ref["d_gate"]) * T ** 0.5, False, F32)
        _close(got[3], ref["d_post_weight"], d * gmax * 6 * T, False)
        assert (got[4] is None) == (agn is None)
    d = moe.block_norm_backward(gr, gn, r, pre_weight=w)         # no block: the norm's gradient alone
    ref = B.block_norm_backward(_np(gr), _np(gn), _np(r), pre_weight=_np(w))
    _close(d[0], ref["d_residual"], np.abs(ref["d_residual"]).max() + 1, bf)
    _close(d[4], ref["d_pre_weight"], 6 * np.abs(_np(gn)).max() * T, False)
    assert d[1] is None and d[2] is None and d[3] is None


# ------------------------------------------------------------------ products
def _acc(K):
    return (K / 16 + 16) * 2.0 ** -23


def _case(T, K, N):
    g = _rng(T, K, N)
    return g, _dev(g.normal(size=(T, K)), torch.bfloat16), _dev(g.normal(size=(N, K)) / K ** 0.5, torch.bfloat16)


# 289 tiles of 256 x 256 on 76 pairs: three or four each, of one to nine stages (the ring has three)
@pytest.mark.parametrize("T,K,N", [(4100, 72, 4100), (4097, 520, 4104), (4100, 1160, 4099)])
@pytest.mark.parametrize("dt,act", [(torch.bfloat16, None), (torch.bfloat16, "silu"), (torch.float32, None),
                                    (torch.float32, "gelu")])
def test_linear_of_several_tiles_per_pair(moe, T, K, N, dt, act):
    g, x, w = _case(T, K, N)
    b, r = _dev(g.normal(size=N)), _dev(g.normal(size=(T, N)), dt)
    y, z = moe.linear(x, w, bias=b, activation=act, residual=r, out_dtype=dt, preact=True)
    ry, rz = B.linear(_np(x), _np(w), _np(b), act, _np(r))
    mag = np.abs(_np(x)) @ np.abs(_np(w)).T + np.abs(rz) + np.abs(_np(r))
    bf = dt == torch.bfloat16
    acc = _acc(K if bf else min(K, 1024))       # fp32 results: at most 1024 of K in one accumulator
    _close(z, rz, mag, bf, acc)
    _close(y, ry, 1.2 * mag, bf, acc + 2.0 ** -21)
    _near(z, rz, mag, bf, acc)
    moe.workspace_status(moe.default_workspace())


# dx of many tiles; dw of many tiles; both in split tiles over a long contraction
@pytest.mark.parametrize("T,K,N", [(4100, 4104, 264), (264, 4104, 4100), (4097, 1160, 1029), (513, 264, 4096)])
def test_linear_gradient_of_several_tiles_per_pair(moe, T, K, N):
    """A bf16 gradient without an activation enters the products as it is: nothing but the
    results' own rounding and the sums'."""
    g, x, w = _case(T, K, N)
    gy = _dev(g.normal(size=(T, N)), torch.bfloat16)
    dx, dw, db = moe.linear_backward(gy, x, w, bias=torch.zeros(N, device="cuda"))
    rdx, rdw, rdb, dz = B.linear_backward(_np(gy), _np(x), _np(w))
    mx, mw = np.abs(dz) @ np.abs(_np(w)), np.abs(dz).T @ np.abs(_np(x))
    _close(dx, rdx, mx, True, _acc(N))
    _close(dw, rdw, mw, True, _acc(T))
    _near(dx, rdx, mx, True, _acc(N))
    _near(dw, rdw, mw, True, _acc(T))
    _close(db, rdb, np.abs(dz).sum(0), False)
    moe.workspace_status(moe.default_workspace())


@pytest.mark.parametrize("T,K,N", [(300, 520, 264), (1301, 2056, 1000), (100, 72, 33), (17, 512, 1025)])
@pytest.mark.parametrize("act", [None, "relu"])
def test_linear_gradient_of_exact_dz(moe, T, K, N, act):
    """The same in tiles and split tiles; relu's slope is 0 or 1, so its dz is exact too."""
    g, x, w = _case(T, K, N)
    gy = _dev(g.normal(size=(T, N)), torch.bfloat16)
    z = _dev(g.normal(size=(T, N)), torch.bfloat16) if act else None
    dx, dw, _ = moe.linear_backward(gy, x, w, activation=act, preact=z)
    rdx, rdw, _, dz = B.linear_backward(_np(gy), _np(x), _np(w), act, None if z is None else _np(z))
    mx, mw = np.abs(dz) @ np.abs(_np(w)), np.abs(dz).T @ np.abs(_np(x))
    _close(dx, rdx, mx, True, _acc(N))
    _close(dw, rdw, mw, True, _acc(T))
    _near(dx, rdx, mx, True, _acc(N))
    _near(dw, rdw, mw, True, _acc(T))


@pytest.mark.parametrize("T,K,N", [(5, 264, 90), (70, 200, 90), (2050, 192, 1536)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_preact_beside_a_result_with_rows_apart(moe, T, K, N, dt):
    g, x, w = _case(T, K, N)
    big = torch.zeros(T, N + 14, dtype=dt, device="cuda")
    y, z = moe.linear(x, w, activation="silu", preact=True, out=big[:, :N])
    y2, z2 = moe.linear(x, w, activation="silu", preact=True, out_dtype=dt)
    assert y.data_ptr() == big.data_ptr() and z.shape == (T, N)
    assert torch.equal(y, y2) and torch.equal(z, z2) and (big[:, N:] == 0).all()


# ------------------------------------------------------------------ routing
@pytest.mark.parametrize("T,E,k,ng,tg,gt", [(37, 256, 20, 8, 4, 2), (300, 96, 17, 4, 2, 1), (9, 1024, 32, 4, 1, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_slots_in_groups(moe, T, E, k, ng, tg, gt, score):
    """More slots than the ranking takes, with groups out of the choice."""
    g = _rng(T, E, k, 3)
    x, bias = _dev(g.normal(size=(T, E)) * 2), _dev(np.round(g.normal(size=E) * 30) * 1e-3)
    kw = dict(score=score, n_group=ng, topk_group=tg, group_top=gt, scale=2.5)
    idx, w = moe.route_scored(x, k, bias=bias, **kw)
    ridx, rw, margin = B.route_scored(_np(x), k, bias=_np(bias), **kw)
    sure = margin > 2.0 ** -18 * (B.scores(_np(x), score).max(1) + np.abs(_np(bias)).max())
    assert sure.sum() >= T // 2
    assert np.array_equal(idx.cpu().numpy()[sure], ridx[sure])
    _close(w[torch.from_numpy(sure).cuda()], rw[sure], np.abs(rw[sure]), False)


# ------------------------------------------------------------------ wide rows
# a row per block forward; backward two or three rows per block, whole vectors and not
@pytest.mark.parametrize("T,H", [(700, 9000), (650, 8193), (340, 12289), (310, 16383), (310, 16384)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["channel", "token", "element32"])
def test_block_norm_of_wide_rows(moe, T, H, stream, gate):
    test_block_norm_over_many_steps(moe, T, H, stream, gate, True, True)


# fp32 streams with a gate per element above 2048 columns: rows that have no ring in the backward pass
@pytest.mark.parametrize("T,H", [(700, 2049), (700, 4096), (650, 4099), (320, 7168), (320, 8191)])
@pytest.mark.parametrize("gate", ["element", "element32"])
def test_block_norm_of_fp32_streams_with_element_gates(moe, T, H, gate):
    test_block_norm_over_many_steps(moe, T, H, torch.float32, gate, True, True)
