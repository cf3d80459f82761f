"""What a product on the GPU takes from its operands: the tensors as they are when it is called."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_product_takes_the_tensors_that_its_operands_hold_now():
    from hpc_linear_algebra_amd import blocks
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    A = blocks.quantize(rn(300, 260), block=128)[0]
    B, other = (blocks.quantize(rn(40, 260))[0] for _ in range(2))
    first, want = blocks.gemm(A, B, dtype="f32"), blocks.gemm(A, other, dtype="f32")
    kept = B.codes, B.scales
    B.codes, B.scales = other.codes.clone(), other.scales.clone()
    assert torch.equal(blocks.gemm(A, B, dtype="f32"), want) and not torch.equal(first, want)
    B.codes = kept[0][:39]
    with pytest.raises(ValueError):
        blocks.gemm(A, B)
    B.codes, B.scales = kept
    assert torch.equal(blocks.gemm(A, B, dtype="f32"), first)


def test_a_product_into_a_saved_tensor_is_noticed():
    from hpc_linear_algebra_amd import blocks
    g = torch.Generator(device="cuda").manual_seed(2)
    A, B = (blocks.quantize(torch.randn(n, 64, generator=g, device="cuda"))[0] for n in (16, 8))
    out = torch.randn(8, 16, generator=g, device="cuda")
    w = torch.randn(8, 16, generator=g, device="cuda").requires_grad_()
    before = out._version
    loss = (w * out).sum()                       # saves out for the gradient of w
    blocks.gemm(A, B, out=out)
    assert out._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_a_product_cuts_no_graph_without_a_word():
    from hpc_linear_algebra_amd import blocks
    g = torch.Generator(device="cuda").manual_seed(3)
    A, B = (blocks.quantize(torch.randn(n, 64, generator=g, device="cuda"))[0] for n in (16, 8))
    want = blocks.gemm(A, B, dtype="f32")
    out = torch.zeros(8, 16, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        blocks.gemm(A, B, out=out)
    with pytest.raises(ValueError, match="gradient"):
        blocks.gemm(A, B, out=out * 1.0)
    assert not out.any()
    with torch.no_grad():
        assert torch.equal(blocks.gemm(A, B, out=out), want)
    A.scales.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        blocks.gemm(A, B)
    with torch.no_grad():
        assert torch.equal(blocks.gemm(A, B, dtype="f32"), want)
    with torch.inference_mode():
        made_there = torch.zeros(8, 16, device="cuda")
        assert torch.equal(blocks.gemm(A, B, out=made_there), want)
