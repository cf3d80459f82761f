"""Results of blocks.linear as autograd sees them, on the CPU: its quantizer and product replaced by plain ones."""
import pytest
import torch

from hpc_linear_algebra_amd import blocks
from test_linear_autograd_host import plain_gemm, plain_quantize


@pytest.mark.parametrize("shape", [(5, 40), (2, 5, 40), (2, 1, 5, 40), (0, 5, 40)])
def test_results_can_be_changed_in_place(shape, monkeypatch):
    monkeypatch.setattr(blocks, "quantize", plain_quantize)
    monkeypatch.setattr(blocks, "gemm", plain_gemm)
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randint(-3, 4, s, generator=g).float().requires_grad_() for s in (shape, (24, 40)))       # codes hold these
    y = blocks.linear(x, w)
    want = torch.autograd.grad(y, [x, w], torch.ones_like(y))
    y = blocks.linear(x, w)
    y += 1.0
    assert torch.equal(y, x @ w.t() + 1.0)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, [x, w], torch.ones_like(y)), want))
