"""Which kernel the block-scaled product takes: known before any launch, so checked without a GPU."""
import random

import pytest

import block_gemm_shapes
from hpc_linear_algebra_amd import tlrgemm as T

FAST = T.TLR_BLOCK_FAST


def grid(m, n, k, flags):
    c = T.tlr_block_gemm_plan(m, n, k, flags)
    y = c.grid_y * c.parts
    assert c.grid_x * c.threads < 1 << 32 and y < 1 << 16, (m, n, k, c.rows, c.cols, c.grid_x, y)
    # every entry of C has its workgroup
    across = -(-m // c.rows)
    assert c.grid_x * c.grid_y == across * -(-n // c.cols)
    return c


@pytest.mark.parametrize("flags", [0, FAST])
@pytest.mark.parametrize("m,n,k", [
    (1 << 30, 1, 16), ((1 << 31) - 512, 1, 16), (1, (1 << 31) - 512, 16), ((1 << 31) - 512, 64, 128), (1 << 26, 16, 128),
    ((1 << 26) - 1, 17, 4096), (1 << 27, 100, 4096), (1 << 28, 800, 4096), (1 << 19, 1 << 17, 4096), (1, 1 << 20, 128),
    (16, 1 << 21, 1 << 21), (200, 1 << 26, 1 << 20)])
def test_every_launch_of_an_accepted_size_fits(m, n, k, flags):
    grid(m, n, k, flags)


def test_every_launch_of_a_sampled_size_fits():
    rng = random.Random(1)
    for _ in range(4000):
        m, n = (int(2 ** rng.uniform(0, 31)) for _ in range(2))
        k = int(2 ** rng.uniform(0, 22))
        try:
            T.tlr_block_gemm_plan(m, n, k)
        except T.TLRError as e:
            # only what the header excludes
            assert e.status == T.TLR_ERR_INVALID_ARG
            assert max(m, n) > (1 << 31) - 512 or -(-m // 128) * -(-n // 128) >= 1 << 24
            continue
        grid(m, n, k, 0)
        grid(m, n, k, FAST)


def test_refusals():
    for args in ((-1, 1, 1), (1, 1 << 31, 1), (1 << 30, 1 << 15, 128), (1 << 28, 1000, 4096), (1, 1, 1, 2)):
        with pytest.raises(T.TLRError) as e:
            T.tlr_block_gemm_plan(*args)
        assert e.value.status == T.TLR_ERR_INVALID_ARG
    with pytest.raises(T.TLRError) as e:
        T.tlr_block_gemm_workspace_bytes(1 << 30, 1 << 15, 128)
    assert e.value.status == T.TLR_ERR_INVALID_ARG
    assert T.tlr_block_gemm_plan(0, 5, 5).grid_x == 0 and T.tlr_block_gemm_plan(5, 5, 0).threads == 0


def test_a_quantizer_of_too_many_tiles_is_refused():
    """2^24 tiles of 256 threads are one more than a launch takes."""
    with pytest.raises(T.TLRError) as e:
        T.tlr_block_quantize("bf16", "e4m3", 1, 1, (1 << 31) - 1, 0x10000, (1 << 31) - 1, 0x10000, 1 << 31, 0x10000, 1, 0, 0, 0, 0)
    assert e.value.status == T.TLR_ERR_INVALID_ARG and "tiles" in str(e.value)


def test_a_call_needs_the_workspace_of_its_own_mode_and_only_for_a_product():
    """Sizes whose float sums run in parts and whose fast ones do not."""
    from hpc_linear_algebra_amd import blocks
    m, n, k = 2560, 4096, 11008
    exact, fast = T.tlr_block_gemm_plan(m, n, k), T.tlr_block_gemm_plan(m, n, k, FAST)
    assert exact.parts > 1 == fast.parts
    assert exact.workspace == 4 * exact.parts * m * n == T.tlr_block_gemm_workspace_bytes(m, n, k) and fast.workspace == 0
    assert blocks._gemm_workspace(m, n, k, 0) == exact.workspace and blocks._gemm_workspace(m, n, k, FAST) == 0

    def call(alpha, flags, workspace=0, size=0):
        none = T.tlr_block_matrix(None, None, k, n, 1, T.TLR_E4M3)
        T.tlr_block_gemm("f32", m, n, k, alpha, none, none, 1.0, 0x10000, m, flags, workspace, size)

    call(0.0, 0)                                    # C <- C
    with pytest.raises(T.TLRError, match="A: null"):
        call(1.0, FAST)
    with pytest.raises(T.TLRError, match="workspace"):
        call(1.0, 0)
    with pytest.raises(T.TLRError) as e:
        call(1.0, 0, 0x10000, exact.workspace - 1)
    assert e.value.status == T.TLR_ERR_WORKSPACE
    with pytest.raises(T.TLRError, match="A: null"):
        call(1.0, 0, 0x10000, exact.workspace)


@pytest.mark.parametrize("flags,shapes", [(0, block_gemm_shapes.EXACT), (FAST, block_gemm_shapes.FAST)])
def test_the_shapes_that_stand_for_each_kernel_take_it_and_leave_none_out(flags, shapes):
    """The tests on the GPU run these shapes: a kernel that another choice of constants brings in needs one."""
    def kind(m, n, k):
        c = T.tlr_block_gemm_plan(m, n, k, flags)
        return c.rows, c.cols, c.threads, c.halves, c.parts

    for want, shape in shapes.items():
        assert kind(*shape) == want, shape
    rng = random.Random(2)
    seen = set()
    for _ in range(150000):
        m, n = (int(2 ** rng.uniform(0, 15.5)) for _ in range(2))
        seen.add(kind(m, n, int(2 ** rng.uniform(4, 15.5))))
    assert seen <= set(shapes), seen - set(shapes)
