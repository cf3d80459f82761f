"""The example of a trained layer of experts: it runs, and its gradients are the layer's."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("train_experts", os.path.join(ROOT, "examples", "train_experts.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_it_runs():
    losses, out = example().main()
    assert len(losses) == 20 and all(v == v and 0 < v < float("inf") for v in losses)
    # block-scaled codes are off by up to 2^-4 of each entry in two operands and two products, integers by a 254th of a row's largest
    assert all(0 < r < 4 * 2.0 ** -4 for r in out)


def test_gradients_are_the_layers():
    """Against the same layer in 64 bits: e4m3 codes of tokens, weights and gradients are off by at most 2^-4 each (3% rms),
    through two products forward and two backward."""
    model = example().Experts(experts=4, hidden=128, inter=128, topk=2)
    x = torch.randn(300, 128, generator=torch.Generator().manual_seed(2)).cuda().bfloat16().requires_grad_()
    dout = torch.randn(300, 128, generator=torch.Generator().manual_seed(3)).cuda().bfloat16()
    leaves = [x, *model.parameters()]
    got = torch.autograd.grad(model(x), leaves, dout)
    ref = [t.detach().cpu().double().requires_grad_() for t in leaves]
    ids, _ = model.choose(x)
    ids = ids.cpu()
    weights = torch.softmax((ref[0] @ ref[1].t()).gather(1, ids), dim=1)
    out = torch.zeros(300, 128, dtype=torch.float64)
    for e in range(4):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        gu = ref[0][t] @ ref[2][e].t()
        h = torch.nn.functional.silu(gu[:, :128]) * gu[:, 128:]
        out = out.index_add(0, t, (h @ ref[3][e].t()) * weights[t, slot].unsqueeze(1))
    want = torch.autograd.grad(out, ref, dout.cpu().double())
    for a, b in zip(got, want):
        assert a.dtype in (torch.float32, torch.bfloat16)
        assert float((a.cpu().double() - b).norm() / b.norm()) < 8 * 2.0 ** -4
