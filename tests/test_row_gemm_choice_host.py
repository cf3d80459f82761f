"""Which kernel the 8-bit integer product takes: known before any launch, so checked without a GPU."""
import random

import pytest

import row_gemm_shapes
from hpc_linear_algebra_amd import tlrgemm as T


def grid(m, n, k, groups=0):
    c = T.tlr_row_gemm_plan(m, n, k, groups)
    assert c.grid_x * c.threads < 1 << 32 and c.grid_y * c.parts < 1 << 16, (m, n, k, groups, c.rows, c.cols, c.grid_x, c.grid_y)
    # every entry of C has its workgroup; whatever groups' sizes: all but one piece of each, of the rows before the first
    # and of those behind the last are whole.  One workgroup a CU goes through tiles of 256 x 256.
    tiles = -(-m // c.rows) * (min(n, (n + (groups + 2) * (c.cols - 1)) // c.cols) if groups else -(-n // c.cols))
    assert c.grid_x * c.grid_y == (tiles if c.rows < 256 else min(tiles, 256)) and (c.parts == 1 or groups == 0)
    return c


@pytest.mark.parametrize("groups", [0, 1, 64, 1024])
@pytest.mark.parametrize("m,n,k", [
    (1 << 30, 1, 16), ((1 << 31) - 512, 1, 16), (1, (1 << 31) - 512, 16), (1 << 26, 16, 128), ((1 << 26) - 1, 17, 4096),
    (1 << 19, 1 << 17, 4096), (1, 1 << 20, 128), (16, 1 << 21, 1 << 16), (200, 1 << 26, 1 << 15), (5, 5, 0), (1000, 1, 131071)])
def test_every_launch_of_an_accepted_size_fits(m, n, k, groups):
    try:
        grid(m, n, k, groups)
    except T.TLRError as e:
        pieces = min(n, (n + (groups + 2) * 127) // 128) if groups else -(-n // 128)
        assert e.status == T.TLR_ERR_INVALID_ARG and -(-m // 128) * pieces >= 1 << 24


def test_every_launch_of_a_sampled_size_fits():
    rng = random.Random(1)
    for _ in range(4000):
        m, n = (int(2 ** rng.uniform(0, 31)) for _ in range(2))
        k, groups = int(2 ** rng.uniform(0, 16.9)), rng.choice([0, 0, int(2 ** rng.uniform(0, 10))])
        try:
            T.tlr_row_gemm_plan(m, n, k, groups)
        except T.TLRError as e:
            pieces = min(n, (n + (groups + 2) * 127) // 128) if groups else -(-n // 128)
            assert e.status == T.TLR_ERR_INVALID_ARG
            assert max(m, n) > (1 << 31) - 512 or -(-m // 128) * pieces >= 1 << 24
            continue
        grid(m, n, k, groups)


def test_refusals():
    for args in ((-1, 1, 1), (1, 1 << 31, 1), (1 << 30, 1 << 15, 128), (1, 1, -1), (1, 1, 1, -1), (1, 1, 1, 1025)):
        with pytest.raises(T.TLRError) as e:
            T.tlr_row_gemm_plan(*args)
        assert e.value.status == T.TLR_ERR_INVALID_ARG
    with pytest.raises(T.TLRError) as e:
        T.tlr_row_gemm_plan(5, 5, 131072)
    assert e.value.status == T.TLR_ERR_UNSUPPORTED
    assert T.tlr_row_gemm_plan(0, 5, 5).grid_x == 0 and T.tlr_row_gemm_plan(5, 0, 5, 3).threads == 0


def test_workspaces():
    """Of parts for the product; of x's codes, its scales and parts for the linear layer, none for a few tokens."""
    m, n, k = row_gemm_shapes.ONE[(128, 64, 512, 4)]
    c = T.tlr_row_gemm_plan(m, n, k)
    assert c.parts == 4 and c.workspace == 16 * m * n == T.tlr_row_gemm_workspace_bytes(m, n, k)
    up = lambda x: -(-x // 256) * 256   # noqa: E731
    assert T.tlr_row_linear_workspace_bytes(m, n, k) == up(n * -(-k // 16) * 16) + up(4 * n) + c.workspace
    assert T.tlr_row_gemm_workspace_bytes(m, n, k, 3) == 0
    def two_launches(m, n, k):
        return up(n * -(-k // 16) * 16) + up(4 * n) + T.tlr_row_gemm_plan(m, n, k).workspace

    for tokens, most in ((1, 16384), (2, 8192), (3, 4096), (4, 4096), (5, 2048), (8, 2048)):
        assert T.tlr_row_linear_workspace_bytes(2048, tokens, most) == 0
        assert T.tlr_row_linear_workspace_bytes(2048, tokens, most + 1) == two_launches(2048, tokens, most + 1) > 0
    assert T.tlr_row_linear_workspace_bytes(24576, 1, 4096) == 0             # three rounds of workgroups, a vector a lane
    assert T.tlr_row_linear_workspace_bytes(24577, 1, 4096) == two_launches(24577, 1, 4096) > 0
    assert T.tlr_row_linear_workspace_bytes(2048, 9, 64) > 0
    assert T.tlr_row_linear_workspace_bytes(0, 9, 64) == T.tlr_row_linear_workspace_bytes(9, 0, 64) == 0


def test_the_shapes_that_stand_for_each_kernel_take_it_and_leave_none_out():
    """The tests on the GPU run these shapes: a kernel that another choice of constants brings in needs one."""
    def kind(*shape):
        c = T.tlr_row_gemm_plan(*shape)
        return c.rows, c.cols, c.threads, c.parts

    for shapes in (row_gemm_shapes.ONE, row_gemm_shapes.GROUPS):
        for want, shape in shapes.items():
            assert kind(*shape) == want, shape
    for shape in row_gemm_shapes.SEVERAL + row_gemm_shapes.SEVERAL_GROUPS:
        c = T.tlr_row_gemm_plan(*shape)
        assert c.rows == c.cols == 256 and -(-shape[0] // 256) * -(-shape[1] // 256) > c.grid_x == 256, shape
    rng = random.Random(2)
    one, groups = set(), set()
    for _ in range(60000):
        m, n = (int(2 ** rng.uniform(0, 15.5)) for _ in range(2))
        k = int(2 ** rng.uniform(4, 15.5))
        one.add(kind(m, n, k))
        groups.add(kind(m, n, k, int(2 ** rng.uniform(0, 10))))
    assert one <= set(row_gemm_shapes.ONE), one - set(row_gemm_shapes.ONE)
    assert groups <= set(row_gemm_shapes.GROUPS), groups - set(row_gemm_shapes.GROUPS)
