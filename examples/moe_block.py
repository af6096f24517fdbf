"""A routed-expert block as a model runs it: norms and residual stream, router,
routed experts, a shared expert beside them; one forward pass and one training
step of everything but the routed experts' own weights.

    python examples/moe_block.py [--tokens T] [--steps N]

The block, for a residual stream r [T, H]:

    n      = norm(r) * pre_weight                                  block_norm
    logits = n w_router^T, fp32                                    linear
    idx, p = top-k of sigmoid scores + balance bias, in groups     route_scored
    y      = sum_j p_j expert_idx_j(n)                             experts_forward
    y     += shared expert(n)                                      linear, linear (residual = y)
    r'     = r + scale * norm(y) * post_weight;  n' = norm(r') * next_weight     block_norm

The training step has the gradients of r' and n', keeps the routed experts
frozen, and updates the router, the shared expert and the norms' weights; the
balance bias follows the experts' loads, not a gradient.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import mixture_experts_routed_top_gb300 as moe

BF16, F32 = torch.bfloat16, torch.float32


class RoutedBlock:
    """Weights of one block; activations are bf16, the router's logits fp32."""

    def __init__(self, H=2048, I=512, E=64, k=6, n_group=8, topk_group=4, shared=1024, scale=0.5, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(BF16)

        self.k, self.E, self.n_group, self.topk_group, self.scale = k, E, n_group, topk_group, scale
        self.pre_weight = torch.ones(H, device=device)
        self.post_weight = torch.ones(H, device=device)
        self.next_weight = torch.ones(H, device=device)
        self.w_router = w(E, H)
        self.bias = torch.zeros(E, device=device)
        self.w_gate_up, self.w_down = w(E, 2 * I, H), w(E, H, I)
        self.w_up, self.b_up, self.w_out = w(shared, H), torch.zeros(shared, device=device), w(H, shared)

    def forward(self, residual, keep=None):
        """-> (residual stream, input of the next block); keep: a dict that takes
        what the training step needs."""
        _, n = moe.block_norm(residual, pre_weight=self.pre_weight)
        logits = moe.linear(n, self.w_router, out_dtype=F32)
        idx, p = moe.route_scored(logits, self.k, bias=self.bias, n_group=self.n_group, topk_group=self.topk_group)
        y = moe.experts_forward(n, idx, p, self.w_gate_up, self.w_down)
        train = keep is not None
        h = moe.linear(n, self.w_up, bias=self.b_up, activation="silu", preact=train)
        h, z = h if train else (h, None)
        y = moe.linear(h, self.w_out, residual=y, out=y)
        out, nxt = moe.block_norm(residual, y, scale=self.scale, post_norm=True, post_weight=self.post_weight,
                                  pre_weight=self.next_weight)
        if train:
            keep.update(residual=residual, n=n, logits=logits, idx=idx, p=p, h=h, z=z, y=y, out=out)
        return out, nxt

    def gradients(self, keep, grad_out, grad_next):
        """Gradients of the trained weights, by name."""
        k = keep
        _, dy, _, d_post, d_next = moe.block_norm_backward(
            grad_out, grad_next, k["out"], k["y"], scale=self.scale, post_norm=True, post_weight=self.post_weight,
            pre_weight=self.next_weight)
        dh, d_w_out, _ = moe.linear_backward(dy, k["h"], self.w_out)
        dn, d_w_up, d_b_up = moe.linear_backward(dh, k["n"], self.w_up, bias=self.b_up, activation="silu",
                                                 preact=k["z"])
        # dL/dp_j = <dy, output of slot j's expert>: a forward of each slot with weight one
        one = torch.ones(dy.shape[0], 1, device=dy.device)
        dp = torch.stack([(moe.experts_forward(k["n"], k["idx"][:, j:j + 1].contiguous(), one, self.w_gate_up,
                                               self.w_down).float() * dy.float()).sum(1)
                          for j in range(self.k)], 1)
        dlogits = moe.route_scored_backward(k["logits"], k["idx"], k["p"], dp, bias=self.bias)
        dn_router, d_router, _ = moe.linear_backward(dlogits, k["n"], self.w_router)
        # the routed experts are frozen, so n's gradient is the shared expert's and the router's
        d_pre = moe.block_norm_backward(None, dn + dn_router, k["residual"], pre_weight=self.pre_weight)[4]
        return dict(w_router=d_router, w_up=d_w_up, b_up=d_b_up, w_out=d_w_out, pre_weight=d_pre,
                    post_weight=d_post, next_weight=d_next)

    def step(self, grads, lr, idx, bias_rate=1e-3):
        for name, g in grads.items():
            v = getattr(self, name)
            v.copy_((v.float() - lr * g.float()).to(v.dtype))
        counts = moe.dispatch(idx, self.E)[0].float()
        self.bias += bias_rate * torch.sign(counts.mean() - counts)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args(argv)
    block = RoutedBlock()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(a.tokens, 2048, generator=g, device="cuda").to(BF16)
    target = torch.randn(a.tokens, 2048, generator=g, device="cuda")
    losses = []
    for i in range(a.steps):
        keep = {}
        _, nxt = block.forward(x, keep)
        diff = nxt.float() - target
        losses.append(diff.square().mean().item())
        grads = block.gradients(keep, torch.zeros_like(x), (2 / diff.numel() * diff * 4096).to(BF16))
        block.step(grads, lr=0.05, idx=keep["idx"])
        print(f"step {i}: loss {losses[-1]:.5f}")
    # serving: one token at a time through the same block
    out, nxt = block.forward(x[:1])
    moe.workspace_status(moe.default_workspace())
    print(f"one token: stream rms {out.float().square().mean().sqrt().item():.4f}")
    return losses


if __name__ == "__main__":
    main()
