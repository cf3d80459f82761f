"""What torch is told of the operators on sorted rows, of the gated activation and of the linear layers: tangents, traces,
results changed in place, memory that waits for the backward pass."""
import pytest
import torch
import torch.autograd.forward_ad as forward

from hpc_linear_algebra_amd import blocks, int8, moe

pytestmark = pytest.mark.gpu


def order_of(tokens, topk, experts):
    return moe.sort(torch.randint(0, experts, (tokens, topk), device="cuda"), experts)


def test_tangents_are_refused():
    """A result without its tangent would be a derivative of zero."""
    order = order_of(5, 2, 3)
    x, y, w, z = (torch.randn(*s, device="cuda") for s in ((5, 16), (10, 16), (5, 2), (2, 3, 64)))
    W, x8 = int8.quantize(torch.randn(8, 16, device="cuda")), int8.quantize(x)
    G, D = int8.quantize(torch.randn(3, 32, 16, device="cuda")), int8.quantize(torch.randn(3, 16, 16, device="cuda"))
    _, codes, scales = blocks.gated_forward(z[0])
    layer = moe.MoELayer(torch.randn(4, 16, device="cuda").half(), torch.randn(4, 32, 16, device="cuda").half(),
                         torch.randn(4, 16, 16, device="cuda").half(), 2)
    ids = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    calls = [(lambda v: moe.gather(v, order), x), (lambda v: moe.combine(v, w, order), y), (lambda v: moe.combine(y, v, order), w),
             (lambda v: moe.combine(v, None, order), y), (blocks.gated, z), (blocks.gated, z[0]), (blocks.gated_forward, z[0]),
             (lambda v: blocks.gated_backward(v, codes, scales), torch.randn(3, 32, device="cuda")), (lambda v: int8.linear(v, W), x),
             (lambda v: int8.gemm(int8.RowScaled(W.codes, v, 16), x8), W.scales), (lambda v: int8.gemm(W, x8, out=v), torch.zeros(5, 8, device="cuda")),
             (lambda v: moe.Int8Experts(G, D)(v, ids, w), x), (lambda v: moe.Int8Experts(G, D)(x, ids, v), w), (layer, x.half())]
    for call, v in calls:
        with forward.dual_level():
            for leaf in (v, v.detach().requires_grad_()):
                with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode derivative"):
                    call(forward.make_dual(leaf, torch.ones_like(leaf)))
            with torch.no_grad():
                call(v)


def test_traces_are_refused():
    order = order_of(5, 2, 3)
    W = int8.quantize(torch.randn(8, 16, device="cuda"))
    x, y = torch.randn(5, 16, device="cuda"), torch.randn(10, 16, device="cuda")
    for call, v in ((lambda v: moe.gather(v, order), x), (lambda v: moe.combine(v, None, order), y), (blocks.gated, x), (lambda v: int8.linear(v, W), x),
                    (lambda v: int8.quantize(v).scales, x), (lambda v: moe.sort(v, 3).place, order.place)):
        for leaf in (v, v.clone().requires_grad_()) if v.is_floating_point() else (v,):
            with torch.no_grad(), pytest.raises(RuntimeError, match="cannot be traced"):
                torch.jit.trace(call, (leaf,), check_trace=False)
        call(v)


@pytest.mark.parametrize("weights", ["none", "given", "trained"])
def test_rows_are_kept_for_gradients_of_the_weights_alone(weights):
    """The gradient of the rows needs the weights, not the rows."""
    tokens, topk, hidden = 512, 4, 256
    order = order_of(tokens, topk, 8)
    base = torch.randn(tokens * topk, hidden, device="cuda", requires_grad=True)
    w = None if weights == "none" else torch.rand(tokens, topk, device="cuda", requires_grad=weights == "trained")
    dout = torch.randn(tokens, hidden, device="cuda")
    want, = torch.autograd.grad(moe.combine(base, w, order), [base], dout)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    out = moe.combine(base * 1.0, w, order)
    kept = torch.cuda.memory_allocated() - before - 4 * tokens * hidden - (4 * tokens * topk if w is None else 0)
    assert kept == (4 * tokens * topk * hidden if weights == "trained" else 0)
    got, = torch.autograd.grad(out, [base], dout)
    assert torch.equal(got, want)
    y = torch.zeros(hidden, tokens * topk, device="cuda").t().copy_(base.detach()).requires_grad_()          # columns, not rows
    got, = torch.autograd.grad(moe.combine(y, w, order), [y], dout)
    assert torch.equal(got, want)


@pytest.mark.parametrize("trained", [True, False])
def test_changes_in_place_are_noticed_whether_rows_are_kept_or_not(trained):
    order = order_of(5, 2, 3)
    base, w = torch.randn(10, 16, device="cuda", requires_grad=True), torch.rand(5, 2, device="cuda", requires_grad=trained)
    y = base * 1.0
    out = moe.combine(y, w, order)
    y.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    y = base * 1.0
    out = moe.combine(y, w, order)
    with torch.no_grad():
        w.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


@pytest.mark.parametrize("shape", [(64,), (3, 64), (2, 3, 64), (2, 1, 3, 64)])
def test_gated_results_can_be_changed_in_place(shape):
    """A result that were a view of another tensor could not be, of any number of dimensions but two."""
    x = torch.randn(*shape, device="cuda", requires_grad=True)
    dy = torch.randn(*shape[:-1], 32, device="cuda")
    y = blocks.gated(x)
    want, = torch.autograd.grad(y, [x], 2.0 * dy)
    kept = y.detach().clone()
    y = blocks.gated(x)
    y.mul_(2.0).add_(1.0)
    got, = torch.autograd.grad(y, [x], dy)
    assert torch.equal(got, want) and torch.equal(y.detach(), 2.0 * kept + 1.0)
    with torch.no_grad():
        z = blocks.gated(x)
    assert torch.equal(z.add_(1.0), kept + 1.0)


@pytest.mark.parametrize("shape", [(48,), (3, 48), (2, 3, 48), (2, 1, 30, 48)])
def test_results_without_gradients_take_some_in_place(shape):
    """A frozen layer's result, made without gradients, and what is trained beside it."""
    x, W = torch.randn(*shape, device="cuda"), int8.quantize(torch.randn(16, 48, device="cuda"))
    for frozen in (lambda: int8.linear(x, W), lambda: blocks.gated(x[..., :32])):
        with torch.no_grad():
            y = frozen()
        beside = torch.randn_like(y).requires_grad_()
        kept = y.clone()
        y += 2.0 * beside
        got, = torch.autograd.grad(y.sum(), [beside])
        assert torch.equal(got, torch.full_like(got, 2.0)) and torch.equal(y.detach(), kept + 2.0 * beside.detach())


@pytest.mark.parametrize("shape", [(3, 48), (2, 3, 48), (2, 1, 3, 48), (0, 3, 48)])
def test_linear_results_can_be_changed_in_place(shape):
    x, w = torch.randn(*shape, device="cuda", requires_grad=True), torch.randn(16, 48, device="cuda", requires_grad=True)
    dy = torch.randn(*shape[:-1], 16, device="cuda")
    y = blocks.linear(x, w)
    want = torch.autograd.grad(y, [x, w], dy)
    kept = y.detach().clone()
    y = blocks.linear(x, w)
    y += 1.0
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, [x, w], dy), want)) and torch.equal(y.detach(), kept + 1.0)


def test_traces_of_layers_are_refused():
    layer = moe.MoELayer(torch.randn(4, 16, device="cuda").half(), torch.randn(4, 32, 16, device="cuda").half(),
                         torch.randn(4, 16, 16, device="cuda").half(), 2)
    G, D = int8.quantize(torch.randn(3, 32, 16, device="cuda")), int8.quantize(torch.randn(3, 16, 16, device="cuda"))
    x, ids, w = torch.randn(5, 16, device="cuda").half(), torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.rand(5, 2, device="cuda")
    for call in (lambda v: layer(v)[0], lambda v: moe.Int8Experts(G, D)(v, ids, w)):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            torch.jit.trace(call, (x,), check_trace=False)
        assert torch.equal(call(x), call(x))
    # a product within a function of autograd is recorded as that function
    v = torch.randn(8, 16, device="cuda")
    with torch.no_grad():
        traced = torch.jit.trace(lambda z: blocks.linear(z, v) + 1.0, (torch.zeros(5, 16, device="cuda"),), check_trace=False)
        z = torch.randn(5, 16, device="cuda")
        assert torch.equal(traced(z), blocks.linear(z, v) + 1.0)
