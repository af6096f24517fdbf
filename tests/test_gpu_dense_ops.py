"""The dense half of a block on the GPU against the float64 oracle: gated products.

Tolerances as in test_gpu_block_ops.py, from the arithmetic: a bf16 result is one
rounding, at most 2^-8 of it (BF); a tensor-core sum of K products is off by at most
(K / 16 + 16) 2^-23 of the sum of magnitudes (_acc); fp32 arithmetic over a row or
a column stays within 2^-18 of the sum of magnitudes (F32).
"""
import numpy as np
import pytest
import torch

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
