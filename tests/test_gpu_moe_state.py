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


@pytest.mark.parametrize("tokens,experts", [(1, 8), (3, 8), (17, 8), (2, 300)])
@pytest.mark.parametrize("x2,w2", [(-80, -80), (100, 60), (127, 127)])
def test_the_choice_holds_over_bfloat16s_range(tokens, experts, x2, w2):
    """Logits whose products lie outside float's range order the experts as 64-bit sums do."""
    from hpc_linear_algebra_amd.moe import MoELayer
    hidden, topk = 64, 4
    x = torch.zeros(tokens, hidden)
    x[:, 5] = 2.0 ** x2
    router = torch.zeros(experts, hidden)
    router[:, 5] = (1 + torch.arange(experts) % 64 / 64) * 2.0 ** w2        # 8 bits: exact in bfloat16
    router[experts - 2, 5] = 1.75 * 2.0 ** w2 if experts < 64 else 1.9921875 * 2.0 ** w2
    logits = x.bfloat16().double() @ router.bfloat16().double().t()
    want = torch.tensor([sorted(range(experts), key=lambda e: (-float(row[e]), e))[:topk] for row in logits])
    zero = torch.zeros(experts, 2 * 16, hidden, dtype=torch.bfloat16, device="cuda")
    layer = MoELayer(router.bfloat16().cuda(), zero, zero[:, :16].transpose(1, 2).contiguous(), topk, tokens)
    _, ids, p = layer(x.bfloat16().cuda())
    assert torch.equal(ids.cpu().long(), want)
    top = torch.softmax(logits, 1).gather(1, want)
    assert torch.all((p.cpu().double() - top / top.sum(1, keepdim=True)).abs() <= 80 * 2.0 ** -24)


def test_a_layer_cuts_no_graph_without_a_word():
    from hpc_linear_algebra_amd.moe import MoELayer
    g = torch.Generator(device="cuda").manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()   # noqa: E731
    x, router, gate_up, down = rn(3, 64), rn(8, 64), rn(8, 64, 64) / 8, rn(8, 64, 32) / 8
    layer = MoELayer(router, gate_up, down, 2)
    want = layer(x)
    x.requires_grad_()
    with pytest.raises(RuntimeError, match="no backward"):
        layer(x)
    assert all(torch.equal(a, b) for a, b in zip(layer(x.detach()), want))
    with torch.no_grad():
        assert all(torch.equal(a, b) for a, b in zip(layer(x), want))
    trained = MoELayer(router, gate_up.requires_grad_(), down, 2)
    with pytest.raises(RuntimeError, match="no backward"):
        trained(x.detach())
    with torch.inference_mode():
        assert all(torch.equal(a, b) for a, b in zip(trained(x), want))
