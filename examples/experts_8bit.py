"""Block-scaled 8-bit training of a projection, then decoding with a mixture of experts on 8-bit weights.

    python examples/experts_8bit.py

The projection learns to imitate a fixed one: blocks.linear quantizes activations and gradients in 1 x 128 blocks and
the weight in 128 x 128 blocks, each once per use in the two layouts that its products need, and runs the forward and
both gradient products on the codes.  The trained rows then feed a mixture-of-experts layer, once with bfloat16 experts
and once with the same experts in 8 bits, one sequence and a small batch at a time.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from hpc_linear_algebra_amd import blocks                              # noqa: E402
from hpc_linear_algebra_amd.moe import MoELayer, quantize_experts      # noqa: E402


def train(steps: int = 30, tokens: int = 512, width: int = 512, features: int = 640, seed: int = 0):
    """(weight, losses) of a bfloat16 projection after `steps` of gradient descent on a float32 master weight."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    target = torch.randn(features, width, generator=g, device="cuda") / width ** 0.5
    w = torch.zeros(features, width, device="cuda", requires_grad=True)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
        y = blocks.linear(x, w, fast=True)
        loss = (y.float() - x.float() @ target.t()).square().mean()
        loss.backward()
        with torch.no_grad():
            w -= 0.2 * features * w.grad
            w.grad = None
        losses.append(float(loss.detach()))
    return w.detach(), losses


def decode(x: torch.Tensor, experts: int = 32, inter: int = 384, topk: int = 4, seed: int = 1):
    """(outputs with bfloat16 experts, with 8-bit experts, ids) for the rows of x."""
    hidden = x.shape[1]
    g = torch.Generator(device="cuda").manual_seed(seed)
    router = (torch.randn(experts, hidden, generator=g, device="cuda") / hidden ** 0.5).bfloat16()
    gate_up = (torch.randn(experts, 2 * inter, hidden, generator=g, device="cuda") / hidden ** 0.5).bfloat16()
    down = (torch.randn(experts, hidden, inter, generator=g, device="cuda") / inter ** 0.5).bfloat16()
    wide = MoELayer(router, gate_up, down, topk=topk, max_tokens=x.shape[0])
    (c1, s1), (c2, s2) = quantize_experts(gate_up), quantize_experts(down)
    narrow = MoELayer(router, c1, c2, topk=topk, max_tokens=x.shape[0], gate_up_scales=s1, down_scales=s2)
    y, ids, _ = wide(x)
    z, ids8, _ = narrow(x)
    assert torch.equal(ids, ids8)          # the router is the same one
    return y, z, ids


def main():
    w, losses = train()
    print(f"projection: mean squared error {losses[0]:.4f} -> {losses[-1]:.6f} in {len(losses)} steps")
    out = []
    for tokens in (1, 24):
        x = torch.randn(tokens, w.shape[1], device="cuda").bfloat16()
        w8, _ = blocks.quantize(w, block=blocks.BLOCK)
        x8, _ = blocks.quantize(x)
        hidden = blocks.gemm(w8, x8, fast=True)
        y, z, ids = decode(hidden)
        rel = float((z.float() - y.float()).norm() / y.float().norm())
        out.append(rel)
        print(f"{tokens:3d} tokens through {ids.unique().numel()} of 32 experts: 8-bit against bfloat16 weights, "
              f"relative difference {rel:.4f}")
    return losses, out


if __name__ == "__main__":
    main()
