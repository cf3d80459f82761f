"""Gradients of the example's layer of experts against the layer in 64 bits, within what its 8-bit codes can be off; and that
mistakes in them would not pass."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EXPERTS, WIDE, TOKENS = 4, 128, 300

# An e4m3 code is off by up to 2^-4 of its entry, uniformly within a step: 2^-4 / sqrt(3) of the power of two below it, 2.65%
# rms of entries spread evenly over their binade.  Errors of independent entries add in squares, so that a sum of products
# of two codes is off by 3.75% of its norm.  In that way: gate and up 3.75%; the activation, a product of the two (its
# first factor with a slope of up to 1.1), 5.5%; its code and down's on top, the experts' results 6.6%, and with them the router's
# gradient.  Backward: the gradient of the activation 3.75%; times slopes at gates and ups off by 3.75% and by the
# checkpoint's 0.7%, 6.8%; with a code of its own and the other operand's, 7.8% for x and gate_up; dout's code and the
# activation's with its 5.5%, 6.7% for down.  Twice the largest of them:
MOST = 0.16


def inputs():
    g = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    leaves = [rn(TOKENS, WIDE).bfloat16(), *(rn(*s) / s[-1] ** 0.5 for s in ((EXPERTS, WIDE), (EXPERTS, 2 * WIDE, WIDE), (EXPERTS, WIDE, WIDE)))]
    return leaves, rn(TOKENS, WIDE).bfloat16()


def gradients(leaves, ids, dout, mistake=None):
    """Of x, router, gate_up and down, in doubles; `mistake`: a term that is left out."""
    ref = [t.detach().cpu().double().requires_grad_() for t in leaves]
    x, router, gate_up, down = ref
    logits = x @ router.t()
    weights = torch.softmax(logits.gather(1, ids), dim=1)
    if mistake == "router":
        weights = weights.detach()
    if mistake == "softmax":
        weights = torch.exp(logits.gather(1, ids)) / torch.exp(logits.gather(1, ids)).sum(dim=1, keepdim=True).detach()
    out = torch.zeros(TOKENS, WIDE, dtype=torch.float64)
    for e in range(EXPERTS):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ gate_up[e].t()
        g, u = gu[:, :WIDE], gu[:, WIDE:]
        s = torch.sigmoid(g)
        if mistake == "slope":
            s = s.detach()
        if mistake == "up":
            u = u.detach()
        y = (g * s * u) @ down[e].t()
        if mistake == "expert" and e == 2:
            y = y.detach()
        out = out.index_add(0, t, y * weights[t, slot].unsqueeze(1))
    return torch.autograd.grad(out, ref, dout.cpu().double(), materialize_grads=True)


def off(got, want):
    return [float((a.detach().cpu().double() - b).norm() / b.norm()) for a, b in zip(got, want)]


@pytest.mark.parametrize("mistake", ["router", "softmax", "slope", "up", "expert"])
def test_a_term_that_is_left_out_is_seen(mistake):
    leaves, dout = inputs()
    ids = torch.topk(leaves[0].float() @ leaves[1].t(), 2, dim=1).indices
    want = gradients(leaves, ids, dout)
    assert max(off(gradients(leaves, ids, dout), want)) == 0.0
    assert max(off(gradients(leaves, ids, dout, mistake), want)) > MOST          # codes add to it in squares


@pytest.mark.gpu
def test_gradients_are_within_their_codes_errors():
    spec = importlib.util.spec_from_file_location("train_experts", os.path.join(ROOT, "examples", "train_experts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    (x, *weights), dout = inputs()
    model = example.Experts(experts=EXPERTS, hidden=WIDE, inter=WIDE, topk=2)
    with torch.no_grad():
        for p, w in zip(model.parameters(), weights):
            p.copy_(w)
    x = x.cuda().requires_grad_()
    leaves = [x, *model.parameters()]
    got = torch.autograd.grad(model(x), leaves, dout.cuda())
    want = gradients(leaves, model.choose(x)[0].cpu(), dout)
    assert all(v < MOST for v in off(got, want)), off(got, want)
