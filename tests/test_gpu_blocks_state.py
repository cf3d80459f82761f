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
