"""The block example against the oracle, and its training step."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mixture_experts_routed_top_gb300 as moe
import oracle as O
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T", [1, 70])
def test_forward_against_the_oracle(example, T):
    b = example.RoutedBlock(H=256, I=128, E=16, k=3, n_group=4, topk_group=2, shared=192)
    b.bias += 0.01 * torch.arange(16, device="cuda")
    x = torch.randn(T, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).bfloat16()
    keep = {}
    out, nxt = b.forward(x, keep)
    _, n = B.block_norm(_np(x), pre_weight=_np(b.pre_weight))
    # each stage from the stage before as it was stored (bf16), so that a near-tie of the router does not count
    n = _np(keep["n"])
    logits = B.linear(n, _np(b.w_router))[0]
    idx, p, margin = B.route_scored(logits, 3, bias=_np(b.bias), n_group=4, topk_group=2)
    sure = margin > 1e-4          # fp32 logits of 256 products: 1e-5 of their size
    assert sure.sum() >= T * 0.8 and np.array_equal(keep["idx"].cpu().numpy()[sure], idx[sure])
    gi, gp = keep["idx"].cpu().numpy(), _np(keep["p"])
    y = O.forward(n.astype(np.float32), gi, gp, b.w_gate_up.float().cpu().numpy(), b.w_down.float().cpu().numpy())
    y = y + B.linear(_np(keep["h"]), _np(b.w_out))[0]
    # the routed sum is rounded to bf16 before the shared expert joins it, then the whole: 2 halves of 2^-7; the
    # experts' own tolerance (2e-2 of the rms) covers their bf16 intermediate
    assert np.abs(_np(keep["y"]) - y).max() < 2e-2 * np.sqrt((y * y).mean()) + 2.0 ** -7 * np.abs(y).max()
    r, nx = B.block_norm(_np(x), _np(keep["y"]), scale=0.5, post_norm=True, post_weight=_np(b.post_weight),
                         pre_weight=_np(b.next_weight))
    assert np.abs(_np(out) - r).max() <= 2.0 ** -8 * np.abs(r).max() * 1.01
    assert np.abs(_np(nxt) - nx).max() <= 2.0 ** -8 * np.abs(nx).max() * 1.01


def test_training_step_lowers_the_loss(example):
    losses = example.main(["--tokens", "256", "--steps", "6"])
    assert all(np.isfinite(losses)) and losses[-1] < losses[0]


def test_router_gradient_against_differences(example):
    """dL/d w_router of a loss that is linear in the stream, along the gradient
    itself: the loss moves by what the gradient says, for a step that changes no choice."""
    b = example.RoutedBlock(H=256, I=128, E=16, k=3, n_group=4, topk_group=2, shared=192)
    x = torch.randn(64, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    gy = torch.randn(64, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()
    _, n = moe.block_norm(x, pre_weight=b.pre_weight)
    w = _np(b.w_router)
    nn = _np(n)
    idx, p, _ = B.route_scored(nn @ w.T, 3, n_group=4, topk_group=2)
    ids = torch.from_numpy(idx).cuda()
    one = torch.ones(64, 1, device="cuda")
    outs = np.stack([_np(moe.experts_forward(n, ids[:, j:j + 1].contiguous(), one, b.w_gate_up, b.w_down))
                     for j in range(3)], 1)
    dp = (outs * _np(gy)[:, None, :]).sum(2)

    def loss(wr):
        s = np.take_along_axis(B.scores(nn @ wr.T, "sigmoid"), idx, 1)
        return (s / s.sum(1, keepdims=True) * dp).sum()
    logits = moe.linear(n, b.w_router, out_dtype=torch.float32)
    dl = moe.route_scored_backward(logits, ids, torch.from_numpy(p).float().cuda(), torch.from_numpy(dp).float().cuda())
    dw = _np(moe.linear_backward(dl, n, b.w_router)[1])
    u = dw / np.linalg.norm(dw)
    num = (loss(w + 1e-4 * u) - loss(w - 1e-4 * u)) / 2e-4
    # dl and dw are rounded to bf16 (2^-9 each on average, 2^-8 at most)
    assert abs(num - (dw * u).sum()) < 2.0 ** -7 * np.linalg.norm(dw)
