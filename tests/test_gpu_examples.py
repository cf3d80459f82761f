"""The examples run and do what they say."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_experts_8bit():
    losses, rel = load("experts_8bit").main()
    # gradient descent on a quadratic with steps of 0.4 of the inverse curvature (2 / features per output, unit inputs)
    # shrinks the error by a factor of 0.6 a step until the quantization noise of x and w is left: codes of 4 bits
    # (2^-4 relative, uniform: 2^-4 / sqrt 3 rms of a step's half) on both operands, squared and summed
    noise = 2 * (2.0 ** -4 / 3 ** 0.5) ** 2
    assert losses[-1] < 2 * noise < losses[0] / 20
    # weights off by at most 2^-4 of themselves through two products and a gate
    assert all(0 < r < 3 * 2.0 ** -4 for r in rel)


def test_quantize_experts_is_quantize_of_each():
    import torch

    from hpc_linear_algebra_amd import blocks
    from hpc_linear_algebra_amd.moe import quantize_experts
    w = torch.randn(3, 200, 272, generator=torch.Generator().manual_seed(1)).cuda()
    codes, scales = quantize_experts(w)
    assert codes.shape == (3, 200, 272) and scales.shape == (3, 3, 2) and codes.is_contiguous()
    for e in range(3):
        q, _ = blocks.quantize(w[e], block=128)
        assert torch.equal(codes[e].view(torch.uint8), q.codes.view(torch.uint8)) and torch.equal(scales[e], q.scales)
    with pytest.raises(ValueError):
        quantize_experts(w[:, :, :270].contiguous())
