"""An embedding and a mixture-of-experts layer on the one-hot operators: a few
training steps, then one decoding step.

    python examples/moe_layer.py [--tokens T --experts E --top K --width H --hidden F --vocab V --steps N]

The layer is y = x + sum over a token's experts e of w_e W2_e silu(W1_e x) with
x = embed(token).  Rows are bf16, weights of the experts fp32; the router, the
activation and the loss are ordinary torch operations.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_dense_matrix_spmm_gb300 as spmm  # noqa: E402


@dataclass
class Layer:
    table: torch.Tensor   # V x H embedding
    router: torch.Tensor  # E x H
    W1: torch.Tensor      # E x F x H
    W2: torch.Tensor      # E x H x F
    top: int

    @staticmethod
    def random(V, E, H, F, top, seed=0, device="cuda", dtype=torch.bfloat16):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)

        return Layer(normal(V, H, scale=1.0), normal(E, H, scale=H ** -0.5), normal(E, F, H, scale=H ** -0.5),
                     normal(E, H, F, scale=F ** -0.5), top)


def forward(layer: Layer, tokens: torch.Tensor):
    """y and what the backward pass needs."""
    x = spmm.spmm_embed(layer.table, tokens)
    scores = torch.topk(x.float() @ layer.router.float().t(), layer.top, dim=1)
    w = torch.softmax(scores.values, dim=1).contiguous()
    R = spmm.spmm_build_route(scores.indices, layer.W1.shape[0])
    xs = spmm.spmm_dispatch(R, x)
    h = spmm.spmm_experts(R, xs, layer.W1)
    a = torch.nn.functional.silu(h.float()).to(h.dtype)
    ys = spmm.spmm_experts(R, a, layer.W2)
    y = x + spmm.spmm_combine(R, ys, w)
    return y, (tokens, x, R, w, scores.indices, xs, h, a, ys)


def backward(layer: Layer, saved, dy: torch.Tensor):
    """Gradients of the table, the router, W1 and W2 for the gradient dy of y."""
    tokens, x, R, w, chosen, xs, h, a, ys = saved
    dys, dw = spmm.spmm_combine_grad(R, dy, ys, w)
    da, dW2 = spmm.spmm_experts_grad(R, dys, a, layer.W2)
    s = torch.sigmoid(h.float())
    dh = (da.float() * s * (1 + h.float() * (1 - s))).to(h.dtype)
    dxs, dW1 = spmm.spmm_experts_grad(R, dh, xs, layer.W1)
    dx = dy.float() + spmm.spmm_dispatch_grad(R, dxs).float()
    # softmax over the chosen scores, then the scores' product with the router
    dscore = w * (dw - (dw * w).sum(1, keepdim=True))
    dlogits = torch.zeros(x.shape[0], layer.router.shape[0], device=x.device).scatter_(1, chosen, dscore)
    dx += dlogits @ layer.router.float()
    drouter = dlogits.t() @ x.float()
    V = spmm.spmm_build_route(tokens, layer.table.shape[0])
    dtable = spmm.spmm_embed_grad(V, dx.to(x.dtype))
    return dtable, drouter.to(x.dtype), dW1, dW2


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("experts", 32), ("top", 4), ("width", 1024), ("hidden", 768),
                        ("vocab", 8000), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    o = ap.parse_args(argv)
    layer = Layer.random(o.vocab, o.experts, o.width, o.hidden, o.top)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, o.vocab, (o.tokens,), generator=g, device="cuda")
    tokens[-o.tokens // 16:] = -1  # padding
    goal = torch.randn(o.tokens, o.width, generator=g, device="cuda")
    losses = []
    for step in range(o.steps):
        y, saved = forward(layer, tokens)
        diff = y.float() - goal
        losses.append(diff.square().mean().item())
        print(f"step {step}: loss {losses[-1]:.4f}")
        grads = backward(layer, saved, (diff * (2.0 / o.width)).to(y.dtype))
        for p, d in zip((layer.table, layer.router, layer.W1, layer.W2), grads):
            p -= (0.25 * d.float()).to(p.dtype)
    y, _ = forward(layer, tokens[:1])
    print(f"one decoded token: |y| = {y.float().norm().item():.3f}, device error word {spmm.last_device_error()}")
    return losses


if __name__ == "__main__":
    main()
