"""Fitting the norm weights around a quantised MoE layer to recorded outputs, on one GPU.

    python examples/fit_norms.py [--tokens 512] [--steps 300]

Quantising a layer shifts its outputs; its block can take part of that back by adjusting the two norm
weights beside it, block by block, without a gradient of the layer itself. For tokens with the quantised
layer's output y and the residual stream r, and the recorded r* and x* of the block in full precision,

    r', x' = residual_norm(y, r; w_post, w_pre)
    loss   = mean |r' - r*|^2 + mean |x' - x*|^2
    dw_post, dw_pre = residual_norm_backward(y, r, d loss / d r', d loss / d x')

and Adam on float32 copies of both weights. The program makes the recorded outputs itself, from other
norm weights: it shows the calls, their types and their buffers.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from nvfp4_mixture_experts_02_gb300 import ftmoe  # noqa: E402

EPS = 1e-6


class NormFit:
    """Adam on w_post and w_pre (float32 masters, bf16 in the calls). y, target_x bf16 [T, H]; residual and
    target_r float32 [T, H]; gate as residual_norm takes it, not fitted."""

    def __init__(self, y, residual, target_r, target_x, w_post, w_pre, gate=None, scale=1.0, lr=0.02):
        self.y, self.residual, self.target_r, self.target_x = y, residual, target_r, target_x
        self.gate, self.scale, self.lr, self.t = gate, scale, lr, 0
        self.masters = [w_post.float().clone(), w_pre.float().clone()]
        self.first = [torch.zeros_like(w) for w in self.masters]
        self.second = [torch.zeros_like(w) for w in self.masters]

    def step(self):
        """One step; returns the loss before it (a tensor)."""
        w_post, w_pre = (w.bfloat16() for w in self.masters)
        kw = dict(w_post=w_post, w_pre=w_pre, gate=self.gate, scale=self.scale, eps=EPS)
        r, x = ftmoe.residual_norm(self.y, self.residual, **kw)
        off_r, off_x = r - self.target_r, x.float() - self.target_x.float()
        # gradients of the sums over the channels, means over the tokens: bf16 keeps their range
        mean = 2.0 / len(self.y)
        got = ftmoe.residual_norm_backward(self.y, self.residual, off_r * mean, (off_x * mean).bfloat16(), **kw)
        self.t += 1
        for w, g, m, v in zip(self.masters, (got.dw_post, got.dw_pre), self.first, self.second):
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.01)
            w -= self.lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-12)
        return off_r.square().mean() + off_x.square().mean()

    def weights(self):
        return tuple(w.bfloat16() for w in self.masters)


def random_block(tokens, device, H=1024, E=16, k=4, I=512):
    """Inputs of a NormFit: the layer's outputs for random tokens, and outputs recorded with other weights."""
    byte = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device=device)  # noqa: E731
    block = lambda *s: torch.randint(0x28, 0x38, s, dtype=torch.uint8, device=device)  # noqa: E731
    g = torch.full((E,), 0.03, device=device)
    experts = ftmoe.NvFP4Experts(byte(E, 2 * I, H // 2), block(E, 2 * I, H // 16), g,
                                 byte(E, H, I // 2), block(E, H, I // 16), g)
    residual = torch.randn(tokens, H, device=device)
    ones = torch.ones(H, dtype=torch.bfloat16, device=device)
    _, x = ftmoe.residual_norm(torch.zeros_like(residual, dtype=torch.bfloat16), residual, w_pre=ones)
    idx, w = ftmoe.route(torch.randn(tokens, E, device=device), k)
    y = ftmoe.prefill(x, idx, w, experts)
    recorded = [(1 + 0.2 * torch.randn(H, device=device)).bfloat16() for _ in range(2)]
    target_r, target_x = ftmoe.residual_norm(y, residual, w_post=recorded[0], w_pre=recorded[1], scale=0.5, eps=EPS)
    return NormFit(y, residual, target_r, target_x, ones, ones, scale=0.5), recorded


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=300)
    args = ap.parse_args()
    torch.manual_seed(0)
    fit, _ = random_block(args.tokens, torch.device("cuda"))
    losses = torch.stack([fit.step() for _ in range(args.steps)])
    print(f"{args.steps} steps on {args.tokens} tokens: loss {losses[0].item():.3e} -> {losses[-1].item():.3e}")


if __name__ == "__main__":
    main()
