"""8-bit integers with a scale for each row: quantizer and product against the definition in 64 bits."""
import pytest
import torch

from hpc_linear_algebra_amd import int8
from hpc_linear_algebra_amd import tlrgemm as T

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# A result is the exact sum rounded to float, multiplied by two scales and rounded to its type: a half step of
# float for each of the first three (the last product is the float result itself), and one of the type.
TOL = {"f32": 3.01 * 2.0 ** -24, "f16": 2.0 ** -11 + 3.01 * 2.0 ** -24, "bf16": 2.0 ** -8 + 3.01 * 2.0 ** -24}
LEAST = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}       # half a step of the smallest numbers


def gen(seed):
    return torch.Generator().manual_seed(seed)


def numbers(g, *shape):
    x = torch.randn(*shape, generator=g, dtype=torch.float64)
    return x * torch.exp(torch.randn(shape[-1], generator=g, dtype=torch.float64))


def plain_quantize(x):
    """Codes and scales in 64 bits: scale and quotient are rounded to float, the quotient then to an integer."""
    x = x.double()
    s = (x.abs().amax(dim=-1) / 127.0).float().double().clamp_min(2.0 ** -100) if x.shape[-1] else torch.full(x.shape[:-1], 2.0 ** -100)
    q = (x / s.unsqueeze(-1)).float().double()
    return torch.round(q).clamp(-127, 127), s


def same_codes(q, x):
    codes, s = plain_quantize(x)
    assert torch.equal(q.scales.cpu().double(), s.double())
    assert torch.equal(q.codes[..., :q.k].cpu().double(), codes.double())
    assert not q.codes[..., q.k:].any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 8), (3, 17), (5, 512), (9, 513), (2, 2047), (7, 2048), (4, 2049), (3, 4096),
                                    (2, 4097), (3, 8191), (2, 8193), (5, 20011), (1030, 40)])
def test_quantize(dtype, rows, k):
    x = numbers(gen(rows * 31 + k), rows, k).to(DT[dtype])
    same_codes(int8.quantize(x.cuda()), x)


def test_quantize_ties_and_ends():
    """Quotients halfway between integers go to the even one; the largest entry gets 127 or -127."""
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -127.0, 126.5, -126.5, 3.49999976]])
    q = int8.quantize(x.cuda())
    assert q.codes[0, :11].tolist() == [127, 0, 2, 2, 0, -2, -2, -127, 126, -126, 3]
    same_codes(q, x)


def test_quantize_zero_tiny_and_special_rows():
    x = torch.randn(8, 100, generator=gen(0))
    x[0] = 0.0
    x[1] *= 1e-38
    x[2] *= 1e37
    x[3, 7] = float("inf")
    x[4, 99] = float("nan")
    x[5, 0] = -float("inf")
    q = int8.quantize(x.cuda())
    fine = [0, 1, 2, 6, 7]
    same_codes(int8.RowScaled(q.codes[fine], q.scales[fine], 100), x[fine])
    assert torch.isnan(q.scales[3:6]).all() and not q.codes[3:6].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k,off,ld", [(40, 0, 64), (40, 1, 41), (513, 3, 777), (2100, 5, 2105)])
def test_quantize_strides(dtype, k, off, ld):
    base = numbers(gen(k), 7 * ld + off).to(DT[dtype])
    x = base[off:off + 7 * ld].view(7, ld)[:, :k]
    dev = base.cuda()[off:off + 7 * ld].view(7, ld)[:, :k]
    same_codes(int8.quantize(dev), x)
    same_codes(int8.quantize(dev[::2]), x[::2])
    same_codes(int8.quantize(dev.t()), x.t())                                 # columns: copied first
    same_codes(int8.quantize(dev[:1].expand(5, k)), x[:1].expand(5, k))


def test_quantize_picks_rows():
    x = numbers(gen(3), 6, 130).bfloat16()
    rows = torch.tensor([5, 0, 0, -1, 3, 6, 2, -2147483648, 2147483647], dtype=torch.int32)
    want = torch.zeros(9, 130)
    for i, r in enumerate(rows.tolist()):
        if 0 <= r < 6:
            want[i] = x[r].float()
    same_codes(int8.quantize(x.cuda(), rows=rows.cuda()), want)
    both = torch.stack([rows, rows], dim=1).cuda()[:, 0]                      # a strided index
    same_codes(int8.quantize(x.cuda(), rows=both), want)
    none = int8.quantize(x.cuda(), rows=rows[:0].cuda())
    assert tuple(none.codes.shape) == (0, 144)
    empty = int8.quantize(x[:0].cuda(), rows=rows.cuda())                     # no row to pick
    assert not empty.codes.any() and (empty.scales == 2.0 ** -100).all()


def test_quantize_three_dimensions_and_empty():
    x = numbers(gen(4), 3, 5, 70)
    same_codes(int8.quantize(x.float().cuda()), x.float())
    for shape in ((0, 40), (4, 0), (0, 0)):
        q = int8.quantize(torch.zeros(shape, device="cuda"))
        assert q.scales.shape == shape[:1] and (q.scales == 2.0 ** -100).all()


def operand(g, rows, k, ld=None, experts=None):
    """Random codes in rows of ld bytes with anything behind column k, and scales over a wide range."""
    shape = (rows,) if experts is None else (experts, rows)
    ld = ld or -(-k // 16) * 16
    codes = torch.randint(-127, 128, (*shape, ld), generator=g, dtype=torch.int8)
    scales = torch.exp(3.0 * torch.randn(shape, generator=g))
    return codes, scales


def exact(a, sa, b, sb, k):
    return (b[:, :k].double() @ a[:, :k].double().t()) * sb.double().unsqueeze(1) * sa.double()


def check(got, want, dtype):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= TOL[dtype] * want.abs() + LEAST[dtype]).all()), float((err / want.abs().clamp_min(1e-300)).max())


SIZES = [(1, 1, 1), (16, 1, 128), (17, 3, 129), (100, 16, 1000), (130, 17, 255), (5, 33, 16), (300, 40, 77), (128, 128, 128),
         (129, 127, 384), (257, 200, 500), (700, 300, 1200), (260, 1030, 130), (512, 512, 2048), (2100, 9, 4100), (1030, 66, 3000),
         (300, 700, 5000)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm(m, n, k, dtype):
    g = gen(m + 7 * n + 13 * k)
    a, sa = operand(g, m, k, -(-k // 16) * 16 + 32)
    b, sb = operand(g, n, k)
    if dtype == "f16":
        sa, sb = sa * 2.0 ** -12, sb * 2.0 ** -12
    got = int8.gemm(int8.RowScaled(a.cuda(), sa.cuda(), k), int8.RowScaled(b.cuda(), sb.cuda(), k), dtype=dtype)
    assert got.shape == (n, m) and got.dtype == DT[dtype]
    want = exact(a, sa, b, sb, k)
    if dtype == "f16":
        fits = want.abs() < 65000
        got, want = torch.where(fits.cuda(), got, 0.0), torch.where(fits, want, 0.0)
    check(got, want, dtype)


def test_gemm_largest_sums():
    """Sums that need all of 31 bits: 131071 products of -128 and -128, and of 127 and -127."""
    k = 131071
    for x, y in ((-128, -128), (127, -127)):
        a = torch.full((3, 131072), x, dtype=torch.int8)
        b = torch.full((2, 131072), y, dtype=torch.int8)
        one = lambda n: torch.ones(n)   # noqa: E731
        got = int8.gemm(int8.RowScaled(a.cuda(), one(3).cuda(), k), int8.RowScaled(b.cuda(), one(2).cuda(), k), dtype="f32")
        assert (got.cpu() == torch.tensor(float(k * x * y))).all()
        a, b = a.expand(3, -1).repeat(50, 1), b.repeat(40, 1)
        got = int8.gemm(int8.RowScaled(a.cuda(), one(150).cuda(), k), int8.RowScaled(b.cuda(), one(80).cuda(), k), dtype="f32")
        assert (got.cpu() == torch.tensor(float(k * x * y))).all()


def test_gemm_into_slices_and_nothing_else():
    g = gen(9)
    for m, n, k in ((37, 5, 100), (201, 150, 300)):
        a, sa = operand(g, m, k)
        b, sb = operand(g, n, k)
        for off, wide in ((0, m), (3, m + 9)):
            whole = torch.full((n + 2, wide), 7.0, dtype=torch.bfloat16, device="cuda")
            out = whole[1:n + 1, off:off + m]
            version = out._version
            got = int8.gemm(int8.RowScaled(a.cuda(), sa.cuda(), k), int8.RowScaled(b.cuda(), sb.cuda(), k), out=out)
            assert got.data_ptr() == out.data_ptr() and out._version > version
            check(out, exact(a, sa, b, sb, k), "bf16")
            whole[1:n + 1, off:off + m] = 7.0
            assert (whole == 7.0).all()


def test_gemm_operand_strides():
    g = gen(10)
    m, n, k = 90, 140, 200
    a, sa = operand(g, 2 * m, k, 256)
    b, sb = operand(g, 2 * n, k, 272)
    A = int8.RowScaled(a.cuda()[::2], sa.cuda()[::2].contiguous(), k)
    B = int8.RowScaled(b.cuda()[1::2], sb.cuda()[1::2].contiguous(), k)
    check(int8.gemm(A, B, dtype="f32"), exact(a[::2], sa[::2], b[1::2], sb[1::2], k), "f32")


def test_gemm_special_scales():
    g = gen(11)
    a, sa = operand(g, 40, 64)
    b, sb = operand(g, 30, 64)
    sa[3], sb[7] = float("nan"), float("nan")
    sb[8] = 0.0
    got = int8.gemm(int8.RowScaled(a.cuda(), sa.cuda(), 64), int8.RowScaled(b.cuda(), sb.cuda(), 64), dtype="f32").cpu()
    bad = torch.zeros(30, 40, dtype=torch.bool)
    bad[:, 3] = True
    bad[7] = True
    assert torch.equal(torch.isnan(got), bad) and (got[8][~bad[8]] == 0).all()


@pytest.mark.parametrize("m,n,k", [(0, 3, 16), (3, 0, 16), (3, 4, 0), (200, 150, 0)])
def test_gemm_empty(m, n, k):
    A = int8.RowScaled(torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.ones(m, device="cuda"), k)
    B = int8.RowScaled(torch.zeros(n, k, dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda"), k)
    got = int8.gemm(A, B, dtype="f32")
    assert got.shape == (n, m) and not got.any()


@pytest.mark.parametrize("groups,m,n", [(1, 3, 4), (5, 1030, 40), (3, 7, 2)])
def test_groups_of_no_columns(groups, m, n):
    """Their codes have strides that are no multiple of 16."""
    A = int8.RowScaled(torch.zeros(groups, m, 0, dtype=torch.int8, device="cuda"), torch.ones(groups, m, device="cuda"), 0)
    B = int8.RowScaled(torch.zeros(n, 0, dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda"), 0)
    offsets = torch.tensor([0] * groups + [n - 1], dtype=torch.int32, device="cuda")
    got = int8.gemm(A, B, offsets=offsets, dtype="f32")
    assert got.shape == (n, m) and not got.any()


def test_one_group_whatever_its_step():
    g = torch.Generator(device="cuda").manual_seed(4)
    m, n, k = 20, 9, 48
    a = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8, device="cuda")
    b = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8, device="cuda")
    sa, sb = torch.rand(m, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    A = int8.RowScaled(a.as_strided((1, m, k), (7, k, 1)), sa.as_strided((1, m), (3, 1)), k)
    got = int8.gemm(A, int8.RowScaled(b, sb, k), offsets=offsets, dtype="f32")
    assert torch.equal(got, int8.gemm(int8.RowScaled(a, sa, k), int8.RowScaled(b, sb, k), dtype="f32"))


def grouped(a, sa, b, sb, k, offsets, m):
    want = torch.zeros(b.shape[0], m, dtype=torch.float64)
    for e in range(a.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            want[lo:hi] = exact(a[e], sa[e], b[lo:hi], sb[lo:hi], k)
    return want


COUNTS = [[0], [1], [5, 0, 0, 3], [0, 0, 17], [16, 16, 1, 33, 0, 2], [128, 127, 129, 0, 1], [300, 0, 5, 260, 64], [1] * 70, [0] * 200 + [9, 1],
          [700, 500], [3] * 130]


@pytest.mark.parametrize("behind", [0, 1, 200])
@pytest.mark.parametrize("counts", COUNTS)
def test_gemm_grouped(counts, behind):
    m, k = 150, 210
    g = gen(sum(counts) + behind)
    experts, n = len(counts), sum(counts) + behind
    a, sa = operand(g, m, k, experts=experts)
    b, sb = operand(g, n, k)
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    offsets = torch.tensor(ends, dtype=torch.int32)
    want = grouped(a, sa, b, sb, k, ends, m)
    A, B = int8.RowScaled(a.cuda(), sa.cuda(), k), int8.RowScaled(b.cuda(), sb.cuda(), k)
    check(int8.gemm(A, B, offsets=offsets.cuda(), dtype="f32"), want, "f32")
    out = torch.full((n + 1, m + 3), 5.0, device="cuda")
    int8.gemm(A, B, offsets=offsets.cuda(), out=out[:n, 1:m + 1])
    check(out[:ends[-1], 1:m + 1], want[:ends[-1]], "f32")
    assert (out[ends[-1]:] == 5.0).all() and (out[:, 0] == 5.0).all() and (out[:, m + 1:] == 5.0).all()


@pytest.mark.parametrize("ends", [[0, 50, 20, 60], [-5, 10, 400, 1000], [60, 60, 60, 60], [3, 2, 1, 0], [0, 0, 0, -1], [10, 30, 30, 60]])
def test_gemm_bad_offsets_stay_in_bounds(ends):
    """Offsets out of order or range are cut; rows that they leave in one group are that group's."""
    for m, n in ((40, 60), (150, 600)):
        g = gen(2)
        a, sa = operand(g, m, 64, experts=3)
        b, sb = operand(g, n, 64)
        whole = torch.full((n + 64, m), 5.0, device="cuda")
        int8.gemm(int8.RowScaled(a.cuda(), sa.cuda(), 64), int8.RowScaled(b.cuda(), sb.cuda(), 64),
                  offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), out=whole[:n])
        assert (whole[n:] == 5.0).all()
        if ends == [10, 30, 30, 60]:
            check(whole[10:30], exact(a[0], sa[0], b[10:30], sb[10:30], 64), "f32")
            check(whole[30:60], exact(a[2], sa[2], b[30:60], sb[30:60], 64), "f32")
            assert (whole[:10] == 5.0).all()


def test_gemm_grouped_strided_experts():
    g = gen(12)
    a, sa = operand(g, 60, 100, 128, experts=6)
    b, sb = operand(g, 50, 100)
    ends = [0, 20, 20, 50]
    A = int8.RowScaled(a.cuda()[::2], sa.cuda()[::2], 100)
    got = int8.gemm(A, int8.RowScaled(b.cuda(), sb.cuda(), 100), offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), dtype="f32")
    check(got, grouped(a[::2], sa[::2], b, sb, 100, ends, 60), "f32")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,m,k", [(1, 200, 300), (3, 500, 4096), (20, 130, 2049), (150, 260, 130)])
def test_linear(n, m, k, dtype):
    g = gen(n + m)
    x = numbers(g, n, k).to(DT[dtype])
    w = torch.randn(m, k, generator=g) / k ** 0.5
    W8 = int8.quantize(w.cuda())
    got = int8.linear(x.cuda(), W8)
    x8, sx = plain_quantize(x)
    w8, sw = plain_quantize(w)
    check(got, (x8 @ w8.t()) * sx.unsqueeze(1) * sw, dtype)
    assert torch.equal(got, int8.gemm(W8, int8.quantize(x.cuda()), dtype=dtype))
    assert torch.equal(got, int8.linear(x.cuda().reshape(1, n, 1, k), W8).reshape(n, m))
    if n == 1:
        assert torch.equal(got[0], int8.linear(x.cuda()[0], W8))


def test_every_kernel_is_reached():
    kinds = set()
    for m, n, k in SIZES:
        c = T.tlr_row_gemm_plan(m, n, k)
        kinds.add((c.rows, c.cols, c.threads))
    assert len(kinds) >= 2


def test_other_stream_and_graph():
    g = gen(13)
    m, n, k = 300, 70, 600
    x = numbers(g, n, k).bfloat16().cuda()
    W8 = int8.quantize(torch.randn(m, k, generator=g).cuda())
    a, sa = operand(g, m, k, experts=4)
    A = int8.RowScaled(a.cuda(), sa.cuda(), k)
    offsets = torch.tensor([0, 10, 10, 50, 66], dtype=torch.int32, device="cuda")

    def run():
        x8 = int8.quantize(x)
        return int8.linear(x, W8), int8.gemm(W8, x8, dtype="f32"), int8.gemm(A, x8, offsets=offsets)

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    for w, t in zip(want, got):
        assert torch.equal(w, t)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = run()
    keep = x.clone()
    for i in range(3):
        x.copy_(keep * (i + 1))
        offsets.copy_(torch.tensor([0, 10 + i, 20, 50 - i, 66 + i], dtype=torch.int32))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for w, t in zip(want, got):
            assert torch.equal(w, t)
