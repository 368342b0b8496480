"""A mixture of gated experts on the library's operators: training steps whose
activations are kept in 8 bits, then decoding steps of one token.

    python examples/gated_moe_layer.py [--tokens T --experts E --top K --width H --hidden F --steps N --keep packed|rows]

The layer is y = x + sum over a token's experts e of w_e D_e (silu(G_e x) * U_e x), the
weights w the softmax over the chosen experts' logits.  What a training step keeps for
the way back is the rows of the experts' inputs and [G x, U x]: with --keep packed both
in 8 bits, 17/16 bytes a value instead of 2; the hidden rows are computed again from them.
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
    router: torch.Tensor  # E x H
    up: torch.Tensor      # E x 2F x H: the gate's rows, then the up projection's
    down: torch.Tensor    # E x H x F
    top: int

    @staticmethod
    def random(E, H, F, top, seed=0, device="cuda", dtype=torch.bfloat16):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)

        return Layer(normal(E, H, scale=H ** -0.5), normal(E, 2 * F, H, scale=H ** -0.5), normal(E, H, F, scale=F ** -0.5), top)


def forward(layer: Layer, x: torch.Tensor, keep=None):
    """y, and with keep ("packed" or "rows") what the backward pass needs."""
    logits = (x @ layer.router.t()).float()
    ids, w = spmm.spmm_topk(logits, layer.top)
    R = spmm.spmm_build_route(ids, layer.router.shape[0])
    xs = spmm.spmm_dispatch(R, x)
    if keep is None:
        h = spmm.spmm_experts_gated(R, xs, layer.up)
        return x + spmm.spmm_combine(R, spmm.spmm_experts(R, h, layer.down), w), None
    h, gu = spmm.spmm_experts_gated(R, xs, layer.up, save=keep)
    ys = spmm.spmm_experts(R, h, layer.down)
    y = x + spmm.spmm_combine(R, ys, w)
    return y, (x, logits, ids, w, R, spmm.spmm_pack_rows(xs) if keep == "packed" else xs, gu, ys)


def backward(layer: Layer, saved, dy: torch.Tensor):
    """Gradients of x, the router, up and down for the gradient dy of y."""
    x, logits, ids, w, R, xs, gu, ys = saved
    dys, dw = spmm.spmm_combine_grad(R, dy, ys, w)
    dh = spmm.spmm_experts_dx(R, dys, layer.down)
    dgu, h = spmm.spmm_gated_grad(R, dh, gu, with_h=True)  # the hidden rows come back with it
    ddown = spmm.spmm_experts_dw(R, dys, h)
    dxs = spmm.spmm_experts_dx(R, dgu, layer.up)
    rows = spmm.spmm_unpack_rows(xs) if isinstance(xs, spmm.Rows8) else xs
    dup = spmm.spmm_experts_dw(R, dgu, rows)
    dlogits = spmm.spmm_topk_grad(logits, ids, w, dw).to(x.dtype)
    dx = dy.float() + spmm.spmm_dispatch_grad(R, dxs).float() + (dlogits @ layer.router).float()
    return dx.to(x.dtype), dlogits.t() @ x, dup, ddown


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("experts", 32), ("top", 4), ("width", 1024), ("hidden", 768), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--keep", choices=("packed", "rows"), default="packed")
    o = ap.parse_args(argv)
    layer = Layer.random(o.experts, o.width, o.hidden, o.top)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(o.tokens, o.width, generator=g, device="cuda").to(torch.bfloat16)
    goal = torch.randn(o.tokens, o.width, generator=g, device="cuda")
    losses = []
    for step in range(o.steps):
        y, saved = forward(layer, x, o.keep)
        diff = y.float() - goal
        losses.append(diff.square().mean().item())
        print(f"step {step}: loss {losses[-1]:.4f}")
        grads = backward(layer, saved, (diff * (2.0 / o.width)).to(y.dtype))
        for p, d in zip((layer.router, layer.up, layer.down), grads[1:]):
            p -= (0.25 * d.float()).to(p.dtype)
    for _ in range(2):
        y, _ = forward(layer, x[:1])
    print(f"one decoded token: |y| = {y.float().norm().item():.3f}, device error word {spmm.last_device_error()}")
    return losses


if __name__ == "__main__":
    main()
