"""blocks.linear in every type against the definition in 64 bits: output and both gradients, with float sums and with
those of the 8-bit instructions, gradients coded in e4m3 and e5m2."""
import numpy as np
import pytest
import torch

from test_gpu_blocks import TD, largest

pytestmark = pytest.mark.gpu


def stands_for(q):
    """The matrix of a BlockScaled in 64 bits, on the host."""
    s = q.scales.double().cpu().t().repeat_interleave(128, dim=1)[:, :q.k]
    if q.block == 128:
        s = s.repeat_interleave(128, dim=0)[:q.rows]
    return (q.codes[:, :q.k].float().double().cpu() * s).numpy()


def check(got, a, b, k, dtype, fast):
    """Float accumulation of the k products of b a^T: min(k, 128) + k / 128 additions and four roundings of 2^-24 of
    the sum of magnitudes; `fast`: 2^-13 of the block's largest product for each of its products besides; up to eight
    parts add as many floats; one rounding to the result's type."""
    ref, mag = b @ a.T, np.abs(b) @ np.abs(a).T
    t = torch.finfo(TD[dtype])
    tol = (min(k, 128) + k / 128 + 4 + 9) * 2.0 ** -24 * mag
    if fast:
        tol = tol + 2.0 ** -13 * largest(a, b, k)
    tol = tol + t.eps / 2 * (np.abs(ref) + tol) + t.smallest_normal * t.eps
    worst = float(np.max(np.abs(got.detach().double().cpu().numpy() - ref) / tol))
    assert worst <= 1.0, f"error {worst:.3f} of its bound"


def operands(tokens, k, features, xt, wt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, k, generator=g)
    x[:, ::64] *= 30.0                              # a strong channel or two in every block
    w = torch.randn(features, k, generator=g) / k ** 0.5
    dy = torch.randn(tokens, features, generator=g) * torch.exp(torch.randn(tokens, 1, generator=g))
    return (x.to(TD[xt]).cuda().requires_grad_(), w.to(TD[wt]).cuda().requires_grad_(), dy.to(TD[xt]).cuda())


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("grad_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("tokens,k,features", [(150, 260, 200), (1, 128, 144), (515, 1040, 392)])
def test_linear_is_the_definition(tokens, k, features, xt, wt, grad_fmt, fast):
    from hpc_linear_algebra_amd import blocks
    x, w, dy = operands(tokens, k, features, xt, wt, tokens + k)
    y = blocks.linear(x, w, grad_fmt=grad_fmt, fast=fast)
    y.backward(dy)
    assert (y.dtype, x.grad.dtype, w.grad.dtype) == (TD[xt], TD[xt], TD[wt])
    x8, x8t = (stands_for(q) for q in blocks.quantize(x.detach(), transposed=True))
    w8, w8t = (stands_for(q) for q in blocks.quantize(w.detach(), block=128, transposed=True))
    d8, d8t = (stands_for(q) for q in blocks.quantize(dy, fmt=grad_fmt, transposed=True))
    check(y, w8, x8, k, xt, fast and xt != "f32")
    check(x.grad, w8t, d8, features, xt, fast and xt != "f32")
    check(w.grad, x8t, d8t, tokens, wt, fast and wt != "f32")


def test_linear_cuts_no_product_unless_asked():
    """Products of 448^2 that cancel beside others of 2^-14 of them, which the 8-bit instructions cut to nothing: sums
    in float are exact here but for the result's rounding."""
    from hpc_linear_algebra_amd import blocks
    x = torch.full((3, 128), 448.0 * 2.0 ** -14)
    x[:, 0::4], x[:, 2::4] = 448.0, -448.0
    w = torch.full((16, 128), 1.0)
    x8, w8 = stands_for(blocks.quantize(x.cuda())[0]), stands_for(blocks.quantize(w.cuda(), block=128)[0])
    y = blocks.linear(x.half().cuda(), w.half().cuda())
    check(y, w8, x8, 128, "f16", False)
    assert torch.all((y - 64 * 448.0 * 2.0 ** -14).abs() <= 2.0 ** -11 * 2)


def test_saved_codes_through_host_memory():
    """Codes that a saved-tensor hook moves away and back give the same gradients; a second backward needs them kept."""
    from hpc_linear_algebra_amd import blocks
    x, w, dy = operands(150, 260, 200, "bf16", "f32", 9)
    y = blocks.linear(x, w)
    want = torch.autograd.grad(y, (x, w), dy)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, (x, w), dy)
    with torch.autograd.graph.save_on_cpu():
        y = blocks.linear(x, w)
    for keep in (True, False):
        got = torch.autograd.grad(y, (x, w), dy, retain_graph=keep)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
