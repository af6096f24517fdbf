"""Pins of the float64 oracle of the operators around the experts: closed
forms and, for every gradient, central differences of the forward."""
import numpy as np
import pytest

from oracle import block_oracle as B

EPS = 1e-5          # step of the central differences: truncation ~ EPS^2, rounding ~ 1e-16 / EPS
TOL = 1e-7          # ten times the larger of the two, for values of order 1


def _diff(f, v, direction):
    return (f(v + EPS * direction) - f(v - EPS * direction)) / (2 * EPS)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    g = np.random.default_rng(1)
    x, gw = g.normal(size=(5, 12)), g.normal(size=(5, 3))
    idx, w, margin = B.route_scored(x, 3, score, renormalise=renorm, scale=2.5)
    assert margin.min() > 1e-3          # the differences do not move the choice

    def loss(v):
        s = np.take_along_axis(B.scores(v, score), idx, 1)
        s = s / s.sum(1, keepdims=True) if renorm else s
        return 2.5 * (s * gw).sum()
    d = B.route_scored_backward(x, idx, w, gw, score, renormalise=renorm, scale=2.5)
    for _ in range(4):
        u = g.normal(size=x.shape)
        assert abs(_diff(loss, x, u) - (d * u).sum()) < TOL * 10


def test_route_closed_forms():
    x = np.zeros((1, 8))
    idx, w, _ = B.route_scored(x, 3)
    assert idx.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 3)
    # the bias moves the choice, not the weights
    idx, w, _ = B.route_scored(x, 2, bias=np.eye(8)[5], renormalise=False)
    assert idx.tolist() == [[5, 0]] and np.allclose(w, 0.5)
    # group 1 wins by the sum of its two best, although group 0 holds the best expert
    x = np.array([[3.0, -9, -9, -9, 2, 2, -9, -9]])
    assert B.route_scored(x, 2, n_group=2, topk_group=1)[0].tolist() == [[4, 5]]
    assert B.route_scored(x, 2, n_group=2, topk_group=1, group_top=1)[0].tolist() == [[0, 1]]
    # masked experts: never before a live one, weight 0; nothing live: 1/k
    x = np.array([[-np.inf, np.nan, 1.0, -np.inf]])
    idx, w, _ = B.route_scored(x, 2)
    assert idx.tolist() == [[2, 0]] and w.tolist() == [[1.0, 0.0]]
    idx, w, _ = B.route_scored(np.full((1, 4), -np.inf), 4, score="softmax")
    assert idx.tolist() == [[0, 1, 2, 3]] and np.allclose(w, 0.25)


def test_route_agrees_with_the_softmax_router():
    import oracle as O
    x = np.random.default_rng(3).normal(size=(64, 60)).astype(np.float32)
    idx, w, _ = B.route_scored(x, 4, score="softmax")
    ridx, rw = O.route(x, 4)
    assert np.array_equal(idx, ridx) and np.allclose(w, rw, rtol=1e-6)


@pytest.mark.parametrize("gate", [None, "channel", "token", "element"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_gradient_against_differences(gate, post):
    g = np.random.default_rng(2)
    T, H = 4, 10
    v = dict(residual=g.normal(size=(T, H)), y=g.normal(size=(T, H)), pre_weight=g.normal(size=H))
    if post:
        v["post_weight"] = g.normal(size=H)
    if gate:
        v["gate"] = g.normal(size={"channel": (H,), "token": (T, 1), "element": (T, H)}[gate])
    gr, gn = g.normal(size=(T, H)), g.normal(size=(T, H))

    def loss(**q):
        r, n = B.block_norm(scale=0.5, post_norm=post, **q)
        return (r * gr).sum() + (n * gn).sum()
    r_out, _ = B.block_norm(scale=0.5, post_norm=post, **v)
    kw = {k: v[k] for k in ("gate", "post_weight", "pre_weight") if k in v}
    d = B.block_norm_backward(gr, gn, r_out, v["y"], scale=0.5, post_norm=post, **kw)
    for name in v:
        u = g.normal(size=v[name].shape)
        num = _diff(lambda a: loss(**{**v, name: a}), v[name], u)
        assert abs(num - (d["d_" + name] * u).sum()) < TOL * 10, name


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_linear_gradient_against_differences(act):
    g = np.random.default_rng(4)
    x, w, b, r = g.normal(size=(5, 8)), g.normal(size=(3, 8)), g.normal(size=3), g.normal(size=(5, 3))
    gy = g.normal(size=(5, 3))
    _, z = B.linear(x, w, b, act, r)
    dx, dw, db, _ = B.linear_backward(gy, x, w, act, z)
    for val, grad, f in ((x, dx, lambda a: B.linear(a, w, b, act, r)), (w, dw, lambda a: B.linear(x, a, b, act, r)),
                         (b, db, lambda a: B.linear(x, w, a, act, r))):
        u = g.normal(size=val.shape)
        assert abs(_diff(lambda a: (f(a)[0] * gy).sum(), val, u) - (grad * u).sum()) < TOL * 10


def test_linear_closed_forms():
    x = np.array([[1.0, -2.0]])
    w = np.eye(2)
    assert B.linear(x, w, activation="relu")[0].tolist() == [[1.0, 0.0]]
    y, z = B.linear(x, w, bias=[1, 1], residual=[[10, 10]])
    assert y.tolist() == [[12.0, 9.0]] and z.tolist() == [[2.0, -1.0]]
    assert B.linear_backward([[1, 1]], x, w, "relu", x)[0].tolist() == [[1.0, 0.0]]
