"""A layer of experts trained in 8 bits, then served on 8-bit integers.

    python examples/train_experts.py

The router is a plain product with a softmax; its choices are sorted by expert, each expert runs on its rows (blocks.linear:
products on block-scaled codes; blocks.gated: the activation, its input kept for the backward pass as 8-bit integers with a
scale for every 128 entries), and the rows go back to their tokens with the router's weights.  Gradients reach tokens,
router and experts.  The trained weights then become 8-bit integers with a scale for each output channel, and the same
layer runs on those for a batch of any size, without a gradient.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from hpc_linear_algebra_amd import blocks, int8, moe      # noqa: E402


class Experts(torch.nn.Module):
    """A mixture of gated experts with float32 master weights."""

    def __init__(self, experts: int = 8, hidden: int = 256, inter: int = 384, topk: int = 2, seed: int = 0):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.nn.Parameter(torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5)   # noqa: E731
        self.router, self.gate_up, self.down = rn(experts, hidden), rn(experts, 2 * inter, hidden), rn(experts, hidden, inter)
        self.topk = topk

    def choose(self, x):
        """(ids, weights): the router's choices for the rows of x and their probabilities."""
        top = torch.topk(x.float() @ self.router.t(), self.topk, dim=1)
        return top.indices, torch.softmax(top.values, dim=1)

    def forward(self, x):
        ids, weights = self.choose(x)
        order = moe.sort(ids, len(self.gate_up))
        ends = order.offsets.tolist()            # the experts' rows, as sizes of the products below
        xs = moe.gather(x, order)
        rows = [blocks.linear(blocks.gated(blocks.linear(xs[a:b], up, fast=True)), down, fast=True)
                for a, b, up, down in zip(ends, ends[1:], self.gate_up, self.down)]
        return moe.combine(torch.cat(rows), weights, order)

    def served(self):
        """The experts on 8-bit integers."""
        return moe.Int8Experts(int8.quantize(self.gate_up.detach()), int8.quantize(self.down.detach()))


def train(model: Experts, steps: int = 20, tokens: int = 1024, rate: float = 20.0, seed: int = 1):
    """Losses of gradient descent towards a fixed linear map."""
    hidden = model.router.shape[1]
    g = torch.Generator(device="cuda").manual_seed(seed)
    target = torch.randn(hidden, hidden, generator=g, device="cuda") / hidden ** 0.5
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
        loss = (model(x).float() - x.float() @ target.t()).square().mean()
        model.zero_grad(set_to_none=True)
        loss.backward()
        with torch.no_grad():
            for p in model.parameters():
                p -= rate * p.grad
        losses.append(float(loss.detach()))
    return losses


def main():
    model = Experts()
    losses = train(model)
    print(f"mean squared error {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    serve, out = model.served(), []
    with torch.no_grad():
        for tokens in (1, 50, 3000):
            x = torch.randn(tokens, model.router.shape[1], device="cuda").bfloat16()
            y, z = model(x), serve(x, *model.choose(x))
            out.append(float((z.float() - y.float()).norm() / y.float().norm()))
            print(f"{tokens:5d} tokens: 8-bit integers against block-scaled codes, relative difference {out[-1]:.4f}")
    return losses, out


if __name__ == "__main__":
    main()
