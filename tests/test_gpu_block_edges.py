"""The operators around the experts on values that are not finite or far from one,
against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

# a token, few tokens, split tiles, whole vectors and not, CTA pairs, pairs with sums in registers
SHAPES = [(1, 64, 24), (5, 64, 24), (5, 72, 7), (40, 64, 24), (40, 1032, 33), (2050, 64, 1536)]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routed_top_gb300 as m
    m.lib()
    return m


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_relu_keeps_nan(moe, T, K, N, dt):
    """max(z, 0) of a NaN is a NaN: a diverged row or weight shows in the result."""
    g = np.random.default_rng([T, K, N])
    x = torch.from_numpy(g.normal(size=(T, K))).bfloat16().cuda()
    w = torch.from_numpy(g.normal(size=(N, K))).bfloat16().cuda()
    w[N // 2, K - 1] = float("nan")
    x[T // 2, 3] = float("nan")
    y, z = moe.linear(x, w, activation="relu", out_dtype=dt, preact=True)
    want = np.zeros((T, N), bool)
    want[T // 2], want[:, N // 2] = True, True
    assert np.array_equal(np.isnan(_np(z)), want)
    assert np.array_equal(np.isnan(_np(y)), want)
    rest = ~want
    assert np.array_equal(_np(y)[rest], np.maximum(_np(z)[rest], 0.0))


@pytest.mark.parametrize("T", [2, 300])      # the small-token kernels and the grouped products
def test_reglu_experts_keep_nan(moe, T):
    """A NaN that only the gate has: the rows of that expert show it."""
    g = np.random.default_rng(5)
    H, I, E = 128, 128, 2
    x = torch.from_numpy(g.normal(size=(T, H))).bfloat16().cuda()
    wgu = torch.from_numpy(g.normal(size=(E, 2 * I, H)) / H ** 0.5).bfloat16().cuda()
    wd = torch.from_numpy(g.normal(size=(E, H, I)) / I ** 0.5).bfloat16().cuda()
    wgu[1, 7, 5] = float("nan")
    idx = (torch.arange(T, dtype=torch.int32, device="cuda") % 2)[:, None].contiguous()
    y = moe.experts_forward(x, idx, torch.ones(T, 1, device="cuda"), wgu, wd, activation="relu")
    moe.workspace_status(moe.default_workspace())
    assert torch.isnan(y[1::2]).all() and torch.isfinite(y[0::2]).all()


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_silu_far_from_zero(moe, T, K, N, dt):
    """silu and its slope go to 0 on the left and to z and 1 on the right, as far as the type goes."""
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    far = [-3e38, -1e36, -1e33, -1e20, -1000.0, -88.5, -87.0, -80.5, -79.0, -20.0, 0.0, 20.0, 90.0, 1000.0, 1e33, 3e38]
    x[:, 0] = 1
    w[:, 0] = torch.tensor([far[i % len(far)] for i in range(N)]).bfloat16()
    y, z = moe.linear(x, w, activation="silu", out_dtype=dt, preact=True)
    assert torch.equal(z, w[:, 0].to(dt).expand(T, N))
    with np.errstate(over="ignore"):
        ry = _np(z) / (1 + np.exp(-_np(z)))
        p = 1 / (1 + np.exp(-_np(z)))
        slope = np.where(_np(z) < -700, 0.0, p * (1 + _np(z) * (1 - p)))
    # a result of 8 bits or fp32 arithmetic, and where e^-z leaves fp32 (|z| above 87) less than 88 e^-87
    tol = (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -18) * np.abs(ry) + 88 * np.exp(-80.0)
    assert (np.abs(_np(y) - ry) <= tol).all()
    gy = torch.ones(T, N, dtype=dt, device="cuda")
    _, dw, db = moe.linear_backward(gy, x, w, bias=torch.zeros(N, device="cuda"), activation="silu", preact=z)
    assert (np.abs(_np(db) - T * slope[0]) <= T * (2.0 ** -18 * np.abs(slope[0]) + 81 * np.exp(-80.0))).all()
    assert (np.abs(_np(dw)[:, 0] - T * slope[0]) <= T * (2.0 ** -7 * np.abs(slope[0]) + 81 * np.exp(-80.0))).all()


@pytest.mark.parametrize("T,N", [(16, 64), (17, 64), (1, 1024), (1, 1032), (3, 7)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), 3.4e38])
@pytest.mark.parametrize("act", [None, "silu"])
def test_infinite_gradients_of_few_and_many_dz(moe, T, N, value, act):
    """A gradient beyond bf16 makes its row of dx and of dw infinite, with the signs of what it
    multiplies, on either side of the number of dz that enter the products in two parts."""
    K = 72
    g = np.random.default_rng([T, N])
    x, w = (torch.from_numpy(np.where(g.random(s) < 0.5, -1, 1) * (0.5 + g.random(s))).bfloat16().cuda()
            for s in ((T, K), (N, K)))
    gy = torch.from_numpy(g.normal(size=(T, N))).float().cuda()
    gy[T // 2, N // 3] = value
    z = torch.full((T, N), 20.0, device="cuda") if act else None     # silu's slope is 1 there, to 2^-24
    dx, dw, _ = moe.linear_backward(gy, x, w, activation=act, preact=z)
    big = torch.full((K,), float("inf"), device="cuda") * (1 if value > 0 else -1)
    assert torch.equal(dx[T // 2].float(), big * w[N // 3].float())
    assert torch.equal(dw[N // 3].float(), big * x[T // 2].float())
    gy[T // 2, N // 3] = 0
    zdx, zdw, _ = moe.linear_backward(gy, x, w, activation=act, preact=z)
    rows, cols = torch.arange(T, device="cuda") != T // 2, torch.arange(N, device="cuda") != N // 3
    assert torch.equal(dx[rows], zdx[rows]) and torch.equal(dw[cols], zdw[cols])


@pytest.mark.parametrize("T,N", [(16, 64), (17, 64), (1, 1024), (1, 1032), (3, 7), (1024, 1), (1100, 1)])
@pytest.mark.parametrize("K", [72, 4104])
def test_infinite_operands_of_few_and_many_dz(moe, T, N, K):
    """An infinite token or weight makes infinities of what it is multiplied into and no NaN."""
    g = np.random.default_rng([T, N, K])
    x, w = (torch.from_numpy(g.normal(size=s)).bfloat16().cuda() for s in ((T, K), (N, K)))
    gy = torch.from_numpy(np.where(g.random((T, N)) < 0.5, -1, 1) * (0.5 + g.random((T, N)))).float().cuda()
    x[T // 2, 5], w[N // 3, 9] = float("inf"), -float("inf")
    dx, dw, _ = moe.linear_backward(gy, x, w)
    assert torch.equal(dx[:, 9].float(), -gy[:, N // 3] * float("inf"))
    assert torch.equal(dw[:, 5].float(), gy[T // 2] * float("inf"))
    cols = torch.arange(K, device="cuda")
    assert torch.isfinite(dx[:, cols != 9]).all() and torch.isfinite(dw[:, cols != 5]).all()
