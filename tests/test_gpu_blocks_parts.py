"""Every kernel of the block-scaled product in every number of parts that the library chooses, with both block heights
on A's side, added into a C at odd columns."""
import numpy as np
import pytest
import torch

import block_gemm_shapes
from test_gpu_blocks import TD, codes, largest

pytestmark = pytest.mark.gpu

CASES = [(want, shape, True) for want, shape in block_gemm_shapes.FAST.items()] + \
        [(want, shape, False) for want, shape in block_gemm_shapes.EXACT.items()]


@pytest.mark.parametrize("ablk,afmt,bfmt", [(128, "e4m3", "e4m3"), (1, "e5m2", "e4m3")])
@pytest.mark.parametrize("want,shape,fast", CASES)
def test_kernel(want, shape, fast, ablk, afmt, bfmt):
    """Bound as in test_gpu_blocks: min(k, 128) + k / 128 additions and four roundings of 2^-24 of the sum of magnitudes,
    nine more for halves and parts, 2^-13 of the block's largest product a product with `fast`; alpha and beta: two
    more; a rounding to the type."""
    from hpc_linear_algebra_amd import blocks
    from hpc_linear_algebra_amd import tlrgemm as T
    m, n, k = shape
    c = T.tlr_block_gemm_plan(m, n, k, T.TLR_BLOCK_FAST if fast else 0)
    assert (c.rows, c.cols, c.threads, c.halves, c.parts) == want
    dtype = "bf16" if fast else "f32"
    A, a = codes(m, k, afmt, ablk, m + n)
    B, b = codes(n, k, bfmt, 1, m + n + 1, pad=16)
    i, j = sorted({*range(0, m, max(1, m // 23)), m - 1}), sorted({*range(0, n, max(1, n // 19)), n - 1})
    a, b = a[i], b[j]
    ref, mag = b @ a.T, np.abs(b) @ np.abs(a).T
    tol = (min(k, 128) + k / 128 + 4 + 9) * 2.0 ** -24 * mag + (2.0 ** -13 * largest(a, b, k) if fast else 0.0)
    t = torch.finfo(TD[dtype])

    def compare(got, ref, tol):
        tol = tol + t.eps / 2 * (np.abs(ref) + tol) + t.smallest_normal * t.eps
        worst = float(np.max(np.abs(got[j][:, i].double().cpu().numpy() - ref) / tol))
        assert worst <= 1.0, f"error {worst:.3f} of its bound"

    got = blocks.gemm(A, B, dtype=dtype, fast=fast)
    assert torch.isfinite(got).all()
    compare(got, ref, tol)
    assert torch.equal(got, blocks.gemm(A, B, dtype=dtype, fast=fast))
    g = torch.Generator(device="cuda").manual_seed(m)
    big = torch.randn(n + 2, m + 7, generator=g, device="cuda").to(TD[dtype])
    keep = big.clone()
    out = big[1:n + 1, 3:m + 3]
    c0 = out[j][:, i].double().cpu().numpy()
    blocks.gemm(A, B, out=out, alpha=0.75, beta=-1.5, fast=fast)
    compare(out, 0.75 * ref - 1.5 * c0, 0.75 * tol + 2 * 2.0 ** -24 * (0.75 * mag + 1.5 * np.abs(c0)))
    big[1:n + 1, 3:m + 3] = keep[1:n + 1, 3:m + 3]
    assert torch.equal(big, keep)
