"""Every kernel of the 8-bit integer product in every number of parts, and the linear layer's one-launch form, against
exact sums."""
import itertools

import pytest
import torch

import row_gemm_shapes
from hpc_linear_algebra_amd import int8
from hpc_linear_algebra_amd import tlrgemm as T

pytestmark = pytest.mark.gpu

# three roundings of float, the last one of the result's type
TOL = {"f32": 3.01 * 2.0 ** -24, "f16": 2.0 ** -11 + 3.01 * 2.0 ** -24, "bf16": 2.0 ** -8 + 3.01 * 2.0 ** -24}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def operand(g, *shape, k):
    """Codes with anything behind column k, and scales."""
    codes = torch.randint(-128, 128, (*shape, -(-k // 16) * 16), generator=g, dtype=torch.int8, device="cuda")
    return codes, torch.exp(torch.randn(shape, generator=g, device="cuda")) * 2.0 ** -10


def exact(a, sa, b, sb, k):
    """Doubles hold these sums, whatever their order."""
    return (b[:, :k].double() @ a[:, :k].double().t().contiguous()) * sb.double().unsqueeze(1) * sa.double()


def check(got, want, dtype):
    assert bool(((got.double() - want).abs() <= TOL[dtype] * want.abs() + 2.0 ** -126).all())


@pytest.mark.parametrize("kind,shape", [*row_gemm_shapes.ONE.items(), *((None, s) for s in row_gemm_shapes.SEVERAL)])
def test_every_kernel(kind, shape):
    m, n, k = shape
    c = T.tlr_row_gemm_plan(m, n, k)
    assert (c.rows, c.cols, c.threads, c.parts) == (kind or (256, 256, 512, 1))
    g = torch.Generator(device="cuda").manual_seed(m)
    a, sa = operand(g, m, k=k)
    b, sb = operand(g, n, k=k)
    want = exact(a, sa, b, sb, k)
    A, B = int8.RowScaled(a, sa, k), int8.RowScaled(b, sb, k)
    for dtype in ("f32", "bf16"):
        check(int8.gemm(A, B, dtype=dtype), want, dtype)
    whole = torch.full((n + 1, m + 5), 3.0, device="cuda")            # odd rows into a larger tensor
    int8.gemm(A, B, out=whole[:n, 5:])
    check(whole[:n, 5:], want, "f32")
    assert (whole[n] == 3.0).all() and (whole[:, :5] == 3.0).all()


@pytest.mark.parametrize("kind,shape", [*row_gemm_shapes.GROUPS.items(), *((None, s) for s in row_gemm_shapes.SEVERAL_GROUPS)])
def test_every_kernel_of_groups(kind, shape):
    m, n, k, groups = shape
    c = T.tlr_row_gemm_plan(m, n, k, groups)
    assert (c.rows, c.cols, c.threads, c.parts) == (kind or (256, 256, 512, 1))
    g = torch.Generator(device="cuda").manual_seed(m)
    a, sa = operand(g, groups, m, k=k)
    b, sb = operand(g, n, k=k)
    # uneven: some empty, one with half the rows, a few rows behind the last
    parts = torch.rand(groups, generator=g, device="cuda")
    parts[::4] = 0.0
    parts[groups // 2] = float(parts.sum()) + 0.1
    counts = (parts / parts.sum() * (n - 3)).long().tolist()
    ends = [0, *itertools.accumulate(counts)]
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    want = torch.zeros(n, m, dtype=torch.float64, device="cuda")
    for e in range(groups):
        if counts[e]:
            lo, hi = ends[e], ends[e + 1]
            want[lo:hi] = exact(a[e], sa[e], b[lo:hi], sb[lo:hi], k)
    A, B = int8.RowScaled(a, sa, k), int8.RowScaled(b, sb, k)
    for dtype in ("f32", "bf16"):
        check(int8.gemm(A, B, offsets=offsets, dtype=dtype), want, dtype)
    whole = torch.full((n, m), 3.0, device="cuda")
    int8.gemm(A, B, offsets=offsets, out=whole)
    check(whole[:ends[-1]], want[:ends[-1]], "f32")
    assert (whole[ends[-1]:] == 3.0).all()


@pytest.mark.parametrize("shape", [(6000, 4500, 130), (4096, 8192, 1024), (5001, 5000, 2000), (2816, 12000, 700, 30), (2050, 15000, 640, 9)])
def test_large_products_are_the_same_every_time(shape):
    """On two streams at once: stores of one tile and loads of the next are under way together."""
    m, n, k, groups = (*shape, 0)[:4]
    assert T.tlr_row_gemm_plan(m, n, k, groups).rows == 256
    g = torch.Generator(device="cuda").manual_seed(k)
    a, sa = operand(g, *([groups] if groups else []), m, k=k)
    b, sb = operand(g, n, k=k)
    offsets = torch.arange(groups + 1, dtype=torch.int32, device="cuda") * (n // groups) if groups else None
    A, B = int8.RowScaled(a, sa, k), int8.RowScaled(b, sb, k)
    first = {dtype: int8.gemm(A, B, offsets=offsets, dtype=dtype) for dtype in DT}
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for dtype, want in first.items():
        got = []
        for i in range(8):
            with torch.cuda.stream(streams[i % 2]):
                got.append(int8.gemm(A, B, offsets=offsets, dtype=dtype))
        torch.cuda.synchronize()
        assert all(torch.equal(c, want) for c in got)


@pytest.mark.parametrize("shape", [*row_gemm_shapes.GROUPS.values(), *row_gemm_shapes.SEVERAL_GROUPS])
def test_groups_that_begin_later(shape):
    """Offsets of some of the experts: rows before the first and behind the last are of no group."""
    m, n, k, groups = shape
    g = torch.Generator(device="cuda").manual_seed(n)
    a, sa = operand(g, groups, m, k=k)
    b, sb = operand(g, n, k=k)
    for first, last in ((n // 3, n - n // 4), (n // 2, n // 2), (n, n), (1, n)):
        ends = [first + (last - first) * i // groups for i in range(groups + 1)]
        offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
        want = torch.zeros(n, m, dtype=torch.float64, device="cuda")
        for e in range(groups):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                want[lo:hi] = exact(a[e], sa[e], b[lo:hi], sb[lo:hi], k)
        A, B = int8.RowScaled(a, sa, k), int8.RowScaled(b, sb, k)
        check(int8.gemm(A, B, offsets=offsets, dtype="f32"), want, "f32")
        whole = torch.full((n, m), 3.0, device="cuda")
        int8.gemm(A, B, offsets=offsets, out=whole)
        check(whole[first:last], want[first:last], "f32")
        assert (whole[:first] == 3.0).all() and (whole[last:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k", [(1, 1), (1, 127), (1, 2570), (1, 4096), (1, 4097), (1, 16384), (1, 16385), (2, 100), (2, 8192), (3, 4090),
                                 (4, 2049), (5, 2048), (6, 7), (7, 130), (8, 2048), (8, 2049), (9, 512)])
def test_linear_of_a_few_tokens(n, k, dtype):
    """One launch up to four vectors a lane, two beyond: the same values as quantizer and product."""
    g = torch.Generator(device="cuda").manual_seed(n + k)
    m = 133
    x = (torch.randn(n, k + 3, generator=g, device="cuda") * torch.exp(torch.randn(k + 3, generator=g, device="cuda"))).to(DT[dtype])[:, 1:k + 1]
    a, sa = operand(g, m, k=k)
    W = int8.RowScaled(a, sa, k)
    got = int8.linear(x, W)
    assert torch.equal(got, int8.gemm(W, int8.quantize(x), dtype=dtype))
    x8 = int8.quantize(x)
    want = exact(a, sa, x8.codes, x8.scales, k)
    check(torch.where(want.abs() < 65000, got.double(), 0.0), torch.where(want.abs() < 65000, want, 0.0), dtype)


def test_linear_of_special_tokens():
    """A token of zeros, one with an infinity, one with a NaN, and their neighbours."""
    g = torch.Generator(device="cuda").manual_seed(1)
    a, sa = operand(g, 70, k=300)
    x = torch.randn(6, 300, generator=g, device="cuda")
    x[1], x[2, 299], x[4, 0] = 0.0, float("inf"), float("nan")
    got = int8.linear(x, int8.RowScaled(a, sa, 300))
    assert not got[1].any() and torch.isnan(got[2]).all() and torch.isnan(got[4]).all() and torch.isfinite(got[[0, 3, 5]]).all()
    for j in (0, 3, 5):
        assert torch.equal(got[j], int8.linear(x[j], int8.RowScaled(a, sa, 300)))


def test_far_operands():
    """Weights and results whose offsets pass 2^32 bytes."""
    m, k = 70000, 65536                    # 4.6 GB of weights
    w = torch.empty(m, k, dtype=torch.int8, device="cuda")
    w.copy_((torch.arange(m, device="cuda") % 101).to(torch.int8).unsqueeze(1).expand(m, k))
    x = torch.ones(1, k, device="cuda", dtype=torch.bfloat16)
    W = int8.RowScaled(w, torch.ones(m, device="cuda"), k)
    want = (torch.arange(m, device="cuda") % 101).double() * k
    for n in (1, 20):                      # both of them strips, the quantizer in front
        got = int8.linear(x.expand(n, k).float(), W)
        assert bool(((got.double() - want).abs() <= 1.01 * 2.0 ** -22 * want).all())
    n, m, k = 90000, 13000, 32             # 4.7 GB of results
    x8 = int8.RowScaled(torch.ones(n, 32, dtype=torch.int8, device="cuda"), torch.arange(1, n + 1, device="cuda", dtype=torch.float32), k)
    W = int8.RowScaled(torch.ones(m, 32, dtype=torch.int8, device="cuda"), torch.ones(m, device="cuda"), k)
    got = int8.gemm(W, x8, dtype="f32")
    for c in (0, 6000, m - 1):
        assert torch.equal(got[:, c], 32.0 * torch.arange(1, n + 1, device="cuda", dtype=torch.float32))


@pytest.mark.parametrize("m,n,groups", [(70000, 1500, 0), (4096, 20000, 20)])
def test_far_operands_of_large_tiles(m, n, groups):
    """Rows and groups of weights whose offsets pass 2^32 bytes.  Sums stay below 2^24, scales are 1: exact."""
    k, all_rows = 65536, m * max(groups, 1)
    assert T.tlr_row_gemm_plan(m, n, k, groups).rows == 256
    a = (torch.arange(all_rows, device="cuda") % 101).to(torch.int8)
    b = (torch.arange(n, device="cuda") % 5 - 2).to(torch.int8)
    shape = (groups, m) if groups else (m,)
    A = int8.RowScaled(a.unsqueeze(1).repeat(1, k).view(*shape, k), torch.ones(shape, device="cuda"), k)
    B = int8.RowScaled(b.unsqueeze(1).repeat(1, k), torch.ones(n, device="cuda"), k)
    offsets = torch.arange(groups + 1, dtype=torch.int32, device="cuda") * (n // groups) if groups else None
    got = int8.gemm(A, B, offsets=offsets, dtype="f32")
    for e in range(max(groups, 1)):
        rows = slice(e * (n // groups), (e + 1) * (n // groups)) if groups else slice(0, n)
        want = b[rows].float().unsqueeze(1) * a[e * m:(e + 1) * m].float() * k
        assert torch.equal(got[rows], want)
