"""CPU oracle of the operators around the experts, in float64: scored
routing, the norms after and before a block, dense products with their
epilogue, and the gradient of each.

Definitions (the tests pin them against finite differences and closed forms):

* route_scored: s = softmax(l) or 1/(1+exp(-l)); choice c = s + bias, -inf for
  masked experts (logit or bias -inf or NaN); group score = sum of a group's
  one or two largest unmasked c; the topk_group best groups keep their c; the
  k largest c, ties to the lower index; weights s (0 where c = -inf),
  renormalised (1/k where they sum to 0) and scaled.
* block_norm: z = y/rms(y) w_post (or y), r' = r + scale g z,
  n = r'/rms(r') w_pre, rms(v) = sqrt(mean v^2 + eps).
* linear: residual + act(x w^T + b).
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["scores", "route_scored", "route_scored_backward", "block_norm", "block_norm_backward",
           "linear", "linear_backward"]

_erf = np.vectorize(math.erf, otypes=[np.float64])


# ------------------------------------------------------------------ routing
def _masked(logits):
    return ~(logits > -np.inf)


def scores(logits, score):
    x = np.asarray(logits, np.float64)
    dead = _masked(x)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            top = np.where(dead, -np.inf, x).max(1, keepdims=True)
            e = np.where(dead, 0.0, np.exp(np.where(x == top, 0.0, x - top)))
            tot = e.sum(1, keepdims=True)
            s = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
    return np.where(dead, 0.0, s)


def route_scored(logits, k, score="sigmoid", bias=None, n_group=1, topk_group=1, group_top=2,
                 renormalise=True, scale=1.0):
    """-> (idx [T,k], w [T,k], margin [T]): margin is the smallest gap between
    choices (or group scores) that the result depends on; an implementation
    in 32 bits may differ only where it is of the order of rounding."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    s = scores(x, score)
    c = s if bias is None else s + np.asarray(bias, np.float64)
    c = np.where(_masked(x) | ~(c > -np.inf), -np.inf, c)
    margin = np.full(T, np.inf)
    if n_group > 1:
        g = -np.sort(-c.reshape(T, n_group, -1), axis=2)
        gs = g[:, :, 0].copy()
        if group_top == 2 and g.shape[2] > 1:
            gs += np.where(g[:, :, 1] > -np.inf, g[:, :, 1], 0.0)
        order = np.argsort(-gs, axis=1, kind="stable")
        keep = np.zeros((T, n_group), bool)
        np.put_along_axis(keep, order[:, :topk_group], True, 1)
        if topk_group < n_group:
            ranked = np.take_along_axis(gs, order, 1)
            with np.errstate(invalid="ignore"):
                gap = ranked[:, topk_group - 1] - ranked[:, topk_group]
            margin = np.minimum(margin, np.where(np.isfinite(gap), gap, np.inf))
        c = np.where(np.repeat(keep, E // n_group, axis=1), c, -np.inf)
    order = np.argsort(-c, axis=1, kind="stable")
    ranked = np.take_along_axis(c, order, 1)[:, : k + 1]
    with np.errstate(invalid="ignore"):
        gaps = ranked[:, :-1] - ranked[:, 1:]
    same = np.take_along_axis(x, order, 1)[:, : k + 1]
    # exactly equal logits with equal biases tie exactly in any precision
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    tied = (same[:, :-1] == same[:, 1:]) & (b[order][:, : k + 1][:, :-1] == b[order][:, : k + 1][:, 1:])
    gaps = np.where(np.isfinite(gaps) & ~tied, gaps, np.inf)
    if gaps.shape[1]:
        margin = np.minimum(margin, gaps.min(1))
    idx = order[:, :k]
    w = np.where(np.take_along_axis(c, idx, 1) > -np.inf, np.take_along_axis(s, idx, 1), 0.0)
    if renormalise:
        tot = w.sum(1, keepdims=True)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), 1.0 / k)
    return idx.astype(np.int32), w * scale, margin


def route_scored_backward(logits, idx, w, grad_w, score="sigmoid", bias=None, renormalise=True, scale=1.0):
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    s = scores(x, score)
    dead = _masked(x)
    if bias is not None:
        dead = dead | ~(np.asarray(bias, np.float64) > -np.inf)
    ok = (np.asarray(w) != 0) & ~np.take_along_axis(dead, idx, 1)
    sj = np.where(ok, np.take_along_axis(s, idx, 1), 0.0)
    g = np.where(ok, np.asarray(grad_w, np.float64) * scale, 0.0)
    if renormalise:
        tot = sj.sum(1, keepdims=True)
        inv = np.where(tot > 0, 1.0 / np.where(tot > 0, tot, 1.0), 0.0)
        g = np.where(ok, (g - (g * sj).sum(1, keepdims=True) * inv) * inv, 0.0)
    ds = np.zeros((T, E))
    np.put_along_axis(ds, idx, g, 1)
    if score == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdims=True))


# ------------------------------------------------------------------ norms
def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def _f64(v):
    return None if v is None else np.asarray(v, np.float64)


def block_norm(residual, y=None, gate=None, scale=1.0, post_norm=False, post_weight=None, pre_norm=True,
               pre_weight=None, eps=1e-6):
    """gate broadcastable to [T,H] -> (r', n or None)."""
    r = _f64(residual)
    if y is not None:
        z = _f64(y)
        if post_norm:
            z = z * _rstd(z, eps) * (1.0 if post_weight is None else _f64(post_weight))
        r = r + scale * (1.0 if gate is None else _f64(gate)) * z
    n = r * _rstd(r, eps) * (1.0 if pre_weight is None else _f64(pre_weight)) if pre_norm else None
    return r, n


def block_norm_backward(grad_residual, grad_normed, residual, y=None, gate=None, scale=1.0, post_norm=False,
                        post_weight=None, pre_weight=None, eps=1e-6):
    """-> dict of d_residual, d_y, d_gate (of gate's shape), d_post_weight, d_pre_weight."""
    out = dict(d_y=None, d_gate=None, d_post_weight=None, d_pre_weight=None)
    d = 0.0 if grad_residual is None else _f64(grad_residual)
    if grad_normed is not None:
        r, dn = _f64(residual), _f64(grad_normed)
        rs = _rstd(r, eps)
        q = dn * rs * (1.0 if pre_weight is None else _f64(pre_weight))
        out["d_pre_weight"] = (dn * r * rs).sum(0)
        d = d + q - r * rs * rs * (q * r).mean(1, keepdims=True)
    out["d_residual"] = d
    if y is not None:
        v = _f64(y)
        rs = _rstd(v, eps) if post_norm else 1.0
        w = 1.0 if post_weight is None else _f64(post_weight)
        g = 1.0 if gate is None else _f64(gate)
        dz = scale * g * d
        if gate is not None:
            dg = scale * v * rs * w * d
            shape = np.shape(gate)
            if len(shape) == 1:
                dg = dg.sum(0)
            elif shape[1] == 1 and dg.shape[1] != 1:
                dg = dg.sum(1, keepdims=True)
            out["d_gate"] = dg
        q = dz * w * rs
        if post_norm:
            out["d_post_weight"] = (dz * v * rs).sum(0)
            q = q - v * rs * rs * (q * v).mean(1, keepdims=True)
        out["d_y"] = q
    return out


# ------------------------------------------------------------------ products
def _act(z, act):
    if act == "silu":
        with np.errstate(over="ignore"):
            return z / (1 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if act == "relu":
        return np.maximum(z, 0.0)
    return z


def _slope(z, act):
    if act == "silu":
        p = 1 / (1 + np.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "relu":
        return (z > 0).astype(np.float64)
    return np.ones_like(z)


def linear(x, w, bias=None, activation=None, residual=None):
    """-> (y, z) with z = x w^T + bias."""
    z = _f64(x) @ _f64(w).T
    if bias is not None:
        z = z + _f64(bias)
    y = _act(z, activation)
    return (y if residual is None else y + _f64(residual)), z


def linear_backward(grad_y, x, w, activation=None, preact=None):
    """-> (dx, dw, dbias, dz)."""
    dz = _f64(grad_y)
    if activation is not None:
        dz = dz * _slope(_f64(preact), activation)
    return dz @ _f64(w), dz.T @ _f64(x), dz.sum(0), dz
