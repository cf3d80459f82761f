"""blocks.linear as autograd sees it, on the CPU: its quantizer and product replaced by plain ones."""
import gc
import weakref

import pytest
import torch

from hpc_linear_algebra_amd import blocks


def plain_quantize(x, block=1, fmt="e4m3", straight=True, transposed=False):
    def one(v):
        rows, k = v.shape
        ld, nr = -(-k // 16) * 16, rows if block == 1 else -(-rows // 128)
        codes = torch.zeros(rows, ld, dtype=blocks.FORMATS[fmt])
        codes[:, :k] = v.float().to(codes.dtype)
        return blocks._made(codes, torch.ones(-(-k // 128), nr), rows, k, block)
    return one(x) if straight else None, one(x.t()) if transposed else None


def plain_gemm(A, B, out=None, alpha=1.0, beta=0.0, dtype="bf16", fast=False):
    out.copy_(alpha * (B.dequantize() @ A.dequantize().t()))
    return out


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    monkeypatch.setattr(blocks, "quantize", plain_quantize)
    monkeypatch.setattr(blocks, "gemm", plain_gemm)


def leaves():
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randint(-3, 4, s, generator=g).float()   # noqa: E731  (codes hold these)
    return rn(5, 40).requires_grad_(), rn(24, 40).requires_grad_(), rn(5, 24)


def test_gradients():
    x, w, dy = leaves()
    blocks.linear(x, w).backward(dy)
    assert torch.equal(x.grad, dy @ w.detach()) and torch.equal(w.grad, dy.t() @ x.detach())


@pytest.mark.parametrize("need_x,need_w", [(True, True), (True, False), (False, True)])
def test_saved_tensor_hooks_see_the_codes(need_x, need_w):
    """What the backward pass needs goes through the hooks, and what they give back is what it uses."""
    x, w, dy = leaves()
    x.requires_grad_(need_x), w.requires_grad_(need_w)
    packed, back = [], []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: packed.append(t) or (len(packed) - 1),
                                                  lambda i: back.append(i) or packed[i].clone()):
        y = blocks.linear(x, w)
    assert len(packed) == 2 * (need_x + need_w) and not back
    y.backward(dy)
    assert sorted(back) == list(range(len(packed)))
    if need_x:
        assert torch.equal(x.grad, dy @ w.detach())
    if need_w:
        assert torch.equal(w.grad, dy.t() @ x.detach())


def test_a_second_backward_needs_the_graph_kept():
    x, w, dy = leaves()
    y = blocks.linear(x, w)
    y.backward(dy, retain_graph=True)
    y.backward(dy)
    assert torch.equal(x.grad, 2 * dy @ w.detach())
    with pytest.raises(RuntimeError):
        y.backward(dy)


def test_codes_are_freed_by_the_backward_pass(monkeypatch):
    alive = []

    def watched(*args, **kwargs):
        got = plain_quantize(*args, **kwargs)
        alive.extend(weakref.ref(t) for q in got if q is not None for t in (q.codes, q.scales))
        return got

    monkeypatch.setattr(blocks, "quantize", watched)
    x, w, dy = leaves()
    y = blocks.linear(x, w)
    y.backward(dy)
    gc.collect()
    assert y.grad_fn is not None and not any(r() is not None for r in alive)
