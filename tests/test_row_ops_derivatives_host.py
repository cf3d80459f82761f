"""Calls that torch cannot follow: tangents of forward mode and torch.jit.trace are refused before anything is launched,
so that they run without a GPU."""
import pytest
import torch
import torch.autograd.forward_ad as forward

from hpc_linear_algebra_amd import blocks, int8, moe

W = int8.RowScaled(torch.zeros(4, 48, dtype=torch.int8), torch.zeros(4), 40)
PLACE = torch.zeros(3, 2, dtype=torch.int32)
ORDER = moe.Order(torch.zeros(5, dtype=torch.int32), PLACE, None)
E1, E2 = (int8.RowScaled(torch.zeros(2, r, 48, dtype=torch.int8), torch.zeros(2, r), k) for r, k in ((64, 40), (40, 32)))
ROW, SORTED, WEIGHTS, GATED_CODES, GATED_SCALES = (torch.zeros(3, 40), torch.zeros(6, 40), torch.zeros(3, 2), torch.zeros(3, 2, 48, dtype=torch.int8),
                                                   torch.zeros(3, 2, 1))
# each with one float operand that could carry a tangent
CALLS = {
    "linear": (lambda x: int8.linear(x, W), ROW),
    "linear scales": (lambda s: int8.linear(ROW, int8.RowScaled(W.codes, s, 40)), W.scales),
    "gemm scales": (lambda s: int8.gemm(int8.RowScaled(W.codes, s, 40), W), W.scales),
    "gemm scales of B": (lambda s: int8.gemm(W, int8.RowScaled(W.codes, s, 40)), W.scales),
    "gemm out": (lambda out: int8.gemm(W, W, out=out), torch.zeros(4, 4)),
    "gather": (lambda x: moe.gather(x, ORDER), ROW),
    "combine": (lambda y: moe.combine(y, None, ORDER), SORTED),
    "combine weights": (lambda w: moe.combine(SORTED, w, ORDER), WEIGHTS),
    "gated": (blocks.gated, ROW),
    "gated rows": (lambda x: blocks.gated(x[None]), ROW),
    "gated_forward": (blocks.gated_forward, ROW),
    "gated_backward": (lambda dy: blocks.gated_backward(dy, GATED_CODES, GATED_SCALES), ROW),
    "experts": (lambda x: moe.Int8Experts(E1, E2)(x, PLACE, WEIGHTS), ROW),
    "experts' weights": (lambda w: moe.Int8Experts(E1, E2)(ROW, PLACE, w), WEIGHTS),
}


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("name", CALLS)
def test_tangents_are_refused(name, grad):
    """no_grad says nothing about forward mode: a tangent travels there too."""
    call, x = CALLS[name]
    with forward.dual_level(), torch.set_grad_enabled(grad):
        with pytest.raises(RuntimeError, match="forward-mode derivative"):
            call(forward.make_dual(x, torch.ones_like(x)))
        with pytest.raises(ValueError):                       # the same call without a tangent: on the host, nothing else
            call(x)
        with forward._set_fwd_grad_enabled(False), pytest.raises(ValueError):
            call(forward.make_dual(x, torch.ones_like(x)))


@pytest.mark.parametrize("name", [*CALLS, "sort", "quantize", "quantize of rows"])
def test_traces_are_refused(name):
    """torch.jit.trace records torch's own operations alone: of these calls that would be an empty result."""
    call, x = CALLS.get(name) or {"sort": (lambda ids: moe.sort(ids, 4), PLACE), "quantize": (int8.quantize, ROW),
                                  "quantize of rows": (lambda r: int8.quantize(ROW, rows=r), PLACE[0])}[name]

    def traced(v):
        got = call(v)
        return got if torch.is_tensor(got) else got[0]

    with pytest.raises(RuntimeError, match="cannot be traced"):
        torch.jit.trace(traced, (x,), check_trace=False)
    with pytest.raises(ValueError):                            # and later calls are what they were
        call(x)
