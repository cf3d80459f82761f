"""A mixture-of-experts layer and the memory of its weights."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_layer_keeps_the_memory_that_it_was_made_with():
    from hpc_linear_algebra_amd.moe import MoELayer
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()   # noqa: E731
    x, router, gate_up, down = rn(3, 64), rn(8, 64), rn(8, 64, 64) / 8, rn(8, 64, 32) / 8
    layer = MoELayer(router, gate_up, down, 2)
    want = layer(x)
    at = down.data_ptr()
    down.data = torch.zeros_like(down)               # other memory for the name; the layer's stays
    taken = [torch.full((8, 64, 32), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    assert at not in [t.data_ptr() for t in taken]
    assert all(torch.equal(a, b) for a, b in zip(layer(x), want))
    gate_up.mul_(2)                                  # in place: seen
    assert not torch.equal(layer(x)[0], want[0])
    assert layer.c.hidden == 64 and layer.ws.is_cuda
