"""Sizes from which results pass the caches, and products whose columns begin with a cache line: kernels of their own, against
the definitions in 64 bits."""
import itertools

import pytest
import torch

from hpc_linear_algebra_amd import int8, moe
from hpc_linear_algebra_amd import tlrgemm as T

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}            # half a step, relative
LEAST = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}       # half a step of the smallest numbers, or their flushing
EPS = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def numbers(g, rows, cols, dtype):
    return (torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(torch.randn(cols, generator=g, device="cuda"))).to(DT[dtype])


def same_codes(q, x):
    x = x.double()
    s = (x.abs().amax(dim=1) / 127.0).float().double().clamp_min(2.0 ** -100)
    assert torch.equal(q.scales.double(), s)
    want = torch.round((x / s.unsqueeze(1)).float().double()).clamp_(-127.0, 127.0)
    assert torch.equal(q.codes[:, :q.k].double(), want) and not q.codes[:, q.k:].any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("k", [130, 512, 1037, 2048, 2049, 4096, 4100, 8192, 8193])
def test_quantizer_past_the_caches(k, dtype):
    """From 2^24 entries on, each width of the registers."""
    rows = (1 << 24) // k + 3
    g = gen(k)
    x = numbers(g, rows, k, dtype)
    x[7] = 0.0
    same_codes(int8.quantize(x), x)
    if k <= 2049:
        index = torch.randint(-1, rows + 1, (rows,), generator=g, dtype=torch.int32, device="cuda")
        none = (index < 0) | (index >= rows)
        same_codes(int8.quantize(x, rows=index), x[index.clamp(0, rows - 1).long()].masked_fill(none.unsqueeze(1), 0.0))


@pytest.mark.parametrize("tokens,topk,hidden,dtype", [(1003, 4, 4201, "f32"), (1003, 8, 4201, "f16"), (701, 9, 5400, "bf16"), (4200, 8, 1000, "bf16"),
                                                      (70000, 1, 500, "bf16"), (524, 64, 1024, "f16")])
def test_rows_and_gradients_past_the_caches(tokens, topk, hidden, dtype):
    """Rows of 64 MB and more."""
    assert tokens * topk * hidden * torch.finfo(DT[dtype]).bits // 8 >= 1 << 26
    g = gen(tokens)
    experts = 37
    ids = torch.randint(-3, experts + 1, (tokens, topk), generator=g, device="cuda")
    order = moe.sort(ids, experts)
    flat = torch.where((ids < 0) | (ids >= experts), experts, ids).reshape(-1)
    at = torch.sort(flat, stable=True).indices
    place = torch.empty_like(at)
    place[at] = torch.arange(tokens * topk, device="cuda")
    place, end = place.view(tokens, topk), int((flat < experts).sum())
    assert torch.equal(order.place.long(), place) and int(order.offsets[-1]) == end
    x, y, dxs, dout = (numbers(g, rows, hidden, dtype) for rows in (tokens, tokens * topk, tokens * topk, tokens))
    w = torch.randn(tokens, topk, generator=g, device="cuda")
    y[end:] = float("nan")                                   # rows of no expert are not read
    leaves = [t.requires_grad_() for t in (x, y, w)]
    xs, out = moe.gather(x, order), moe.combine(y, w, order)
    dx, dy, dw = torch.autograd.grad([xs, out], leaves, [dxs, dout])
    x, y, w, xs, out = (t.detach() for t in (x, y, w, xs, out))

    def check(got, want, terms, count):
        # `count` float additions, each off by at most half a step of the sum of the magnitudes, and the last rounding
        bound = HALF[dtype] * want.abs() * (1 + count * EPS) + 1.01 * count * EPS * terms + LEAST[dtype]
        assert bool(((got.double() - want).abs() <= bound).all())

    sums = [torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda") for _ in range(4)]
    for s in range(topk):                                    # one assignment of each token at a time
        p, ws = place[:, s], w[:, s].double().unsqueeze(1)
        real = (p < end).unsqueeze(1)
        assert torch.equal(xs[p], torch.where(real, x, 0.0))
        picked = torch.where(real, y[p], 0.0).double()
        want = torch.where(real, dout.double() * ws, 0.0)
        check(dy[p], want, want.abs(), 1)
        back = torch.where(real, dxs[p], 0.0).double()
        for total, v in zip(sums, (picked * ws, (picked * ws).abs(), back, back.abs())):
            total += v
        t = picked * dout.double()
        # a lane's entries one after another, then 6 + 2 additions
        bound = 1.01 * (8 * -(-hidden // 2048) + 8) * EPS * t.abs().sum(dim=1) + 2.0 ** -149
        assert bool(((dw[:, s].double() - t.sum(dim=1)).abs() <= bound).all())
    check(out, sums[0], sums[1], topk)
    check(dx, sums[2], sums[3], topk)


def operand(g, *shape, k):
    """Codes with anything behind column k, and scales."""
    codes = torch.randint(-128, 128, (*shape, -(-k // 16) * 16), generator=g, dtype=torch.int8, device="cuda")
    return codes, torch.exp(torch.randn(shape, generator=g, device="cuda")) * 2.0 ** -10


def exact(a, sa, b, sb, k):
    """Doubles hold these sums, whatever their order."""
    return (b[:, :k].double() @ a[:, :k].double().t().contiguous()) * sb.double().unsqueeze(1) * sa.double()


def check_product(got, want, dtype):
    """Three roundings of float, the last one of the result's type."""
    half = 3.01 * EPS + (HALF[dtype] if dtype != "f32" else 0.0)
    assert float(want.abs().max()) < 60000.0                  # a number in each of the types
    assert bool(((got.double() - want).abs() <= half * want.abs() + LEAST[dtype]).all())


@pytest.mark.parametrize("m,n,k", [(4096, 8192, 1024), (6016, 4500, 130), (4224, 8200, 16), (5120, 4608, 0), (8192, 4101, 385), (3008, 3501, 600)])
def test_large_products_of_whole_lines(m, n, k):
    """256 x 256 tiles whose columns of C begin with a cache line: m is a multiple of 64, C a new tensor."""
    assert m % 64 == 0 and T.tlr_row_gemm_plan(m, n, k).rows == 256
    g = gen(m)
    (a, sa), (b, sb) = operand(g, m, k=k), operand(g, n, k=k)
    want = exact(a, sa, b, sb, k)
    A, B = int8.RowScaled(a, sa, k), int8.RowScaled(b, sb, k)
    for dtype in DT:
        check_product(int8.gemm(A, B, dtype=dtype), want, dtype)
        whole = torch.full((n + 1, m + 128), 3.0, dtype=DT[dtype], device="cuda")         # lines of a larger tensor
        int8.gemm(A, B, out=whole[:n, 64:64 + m])
        check_product(whole[:n, 64:64 + m], want, dtype)
        assert (whole[n] == 3.0).all() and (whole[:, :64] == 3.0).all() and (whole[:, 64 + m:] == 3.0).all()


@pytest.mark.parametrize("m,n,k,groups", [(1088, 20000, 100, 20), (4096, 9000, 130, 7), (1088, 20000, 0, 20), (2048, 15000, 640, 9), (704, 60000, 500, 130)])
def test_large_products_of_groups_of_whole_lines(m, n, k, groups):
    assert m % 64 == 0 and T.tlr_row_gemm_plan(m, n, k, groups).rows == 256
    g = gen(m + n)
    (a, sa), (b, sb) = operand(g, groups, m, k=k), operand(g, n, k=k)
    # uneven: some empty, one with half the rows, a few rows before the first and behind the last
    parts = torch.rand(groups, generator=g, device="cuda")
    parts[::4] = 0.0
    parts[groups // 2] = float(parts.sum()) + 0.1
    counts = (parts / parts.sum() * (n - 8)).long().tolist()
    ends = [5, *(5 + e for e in itertools.accumulate(counts))]
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    want = torch.zeros(n, m, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            want[lo:hi] = exact(a[e], sa[e], b[lo:hi], sb[lo:hi], k)
    A, B = int8.RowScaled(a, sa, k), int8.RowScaled(b, sb, k)
    for dtype in DT:
        check_product(int8.gemm(A, B, offsets=offsets, dtype=dtype), want, dtype)
        whole = torch.full((n, m), 3.0, dtype=DT[dtype], device="cuda")
        int8.gemm(A, B, offsets=offsets, out=whole)
        check_product(whole[5:ends[-1]], want[5:ends[-1]], dtype)
        assert (whole[:5] == 3.0).all() and (whole[ends[-1]:] == 3.0).all()
