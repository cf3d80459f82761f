"""What calls leave behind and take from each other: second derivatives, views, inference tensors, several graphs, streams
of their own, empty parts."""
import pytest
import torch

from hpc_linear_algebra_amd import blocks, int8, moe

pytestmark = pytest.mark.gpu


def test_no_second_derivative_through_rows():
    ids = torch.tensor([[0, 1], [1, 0]], device="cuda")
    order = moe.sort(ids, 2)
    x = torch.randn(2, 8, device="cuda", requires_grad=True)
    y, w = torch.randn(4, 8, device="cuda", requires_grad=True), torch.rand(2, 2, device="cuda", requires_grad=True)
    dx, = torch.autograd.grad(moe.gather(x, order).square().sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        dx.sum().backward()
    dy, dw = torch.autograd.grad(moe.combine(y, w, order).square().sum(), [y, w], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (dy.sum() + dw.sum()).backward()
    # asked for, not used: no error
    torch.autograd.grad(moe.combine(y, w, order).sum(), [w], create_graph=True)


def test_gradients_accumulate_and_repeat():
    ids = torch.randint(0, 3, (20, 2), device="cuda")
    order = moe.sort(ids, 3)
    x = torch.randn(20, 64, device="cuda", requires_grad=True)
    for i in (1, 2):
        moe.combine(moe.gather(x, order), None, order).sum().backward()
        assert torch.equal(x.grad, torch.full_like(x, 2.0 * i))            # two rows a token
    out = blocks.gated(x)
    a, = torch.autograd.grad(out.sum(), [x], retain_graph=True)
    b, = torch.autograd.grad(out.sum(), [x])
    assert torch.equal(a, b)


def test_inputs_changed_in_place_are_noticed():
    """combine keeps y and weights themselves; gated and gather do not need x again."""
    ids = torch.randint(0, 3, (5, 2), device="cuda")
    order = moe.sort(ids, 3)
    base = torch.randn(10, 16, device="cuda", requires_grad=True)
    y = base * 1.0
    out = moe.combine(y, None, order)
    y.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    x = torch.randn(4, 32, device="cuda", requires_grad=True)
    z = x * 1.0
    out = blocks.gated(z)
    want, = torch.autograd.grad(out.sum(), [x], retain_graph=True)
    z.detach().zero_()
    got, = torch.autograd.grad(out.sum(), [x])
    assert torch.equal(got, want)


def test_inference_mode():
    with torch.inference_mode():
        x = torch.randn(6, 64, device="cuda").bfloat16()
        W = int8.quantize(torch.randn(32, 64, device="cuda"))
        out = torch.empty(6, 32, device="cuda")
        order = moe.sort(torch.randint(0, 4, (6, 2), device="cuda"), 4)
        a = int8.gemm(W, int8.quantize(x), out=out)
        b = moe.combine(moe.gather(x, order), None, order)
        c = blocks.gated(x)
    assert torch.equal(a, int8.gemm(W, int8.quantize(x), dtype="f32")) and c.shape == (6, 32)
    assert torch.equal(b, (x.float() * 2).bfloat16())


def test_out_that_requires_a_gradient_is_refused():
    W, x8 = int8.quantize(torch.randn(8, 32, device="cuda")), int8.quantize(torch.randn(3, 32, device="cuda"))
    out = torch.zeros(3, 8, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        int8.gemm(W, x8, out=out)
    with torch.no_grad():
        int8.gemm(W, x8, out=out)
    for bad in (torch.zeros(3, 9, device="cuda"), torch.zeros(3, 8, device="cuda", dtype=torch.float64), torch.zeros(3, 8),
                torch.zeros(8, 3, device="cuda").t()):
        with pytest.raises(ValueError):
            int8.gemm(W, x8, out=bad)
    scales = x8.scales.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        int8.gemm(W, int8.RowScaled(x8.codes, scales, 32))


def test_groups_belong_to_a_weight_for_each():
    W = int8.quantize(torch.randn(8, 32, device="cuda"))
    E = int8.quantize(torch.randn(3, 8, 32, device="cuda"))
    x8 = int8.quantize(torch.randn(5, 32, device="cuda"))
    off = torch.tensor([0, 2, 4, 5], dtype=torch.int32, device="cuda")
    for A, o in ((W, off), (E, None), (E, off[:3]), (E, off.long()), (E, off.cpu())):
        with pytest.raises(ValueError):
            int8.gemm(A, x8, offsets=o)
    with pytest.raises(ValueError):
        int8.linear(torch.randn(5, 32, device="cuda"), E)
    got = int8.gemm(E, x8, offsets=off.repeat_interleave(2)[::2])            # a strided view
    assert torch.equal(got, int8.gemm(E, x8, offsets=off))


def test_misaligned_codes_are_refused():
    base = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.ones(4, device="cuda")
    x8 = int8.quantize(torch.randn(3, 32, device="cuda"))
    for codes in (base[:, 1:33], base.view(-1)[:4 * 40].view(4, 40)):        # off by one byte; rows of 40 bytes
        with pytest.raises(RuntimeError, match="aligned"):
            int8.gemm(int8.RowScaled(codes, s, 32), x8)
    short = torch.zeros(4 * 32 - 1, dtype=torch.int8, device="cuda").as_strided((4, 31), (32, 1))
    with pytest.raises(ValueError, match="readable"):
        int8.gemm(int8.RowScaled(short, s, 31), int8.RowScaled(x8.codes, x8.scales, 31))


def test_two_graphs_and_eager_calls_between():
    g = torch.Generator().manual_seed(1)
    m, n, k = 362, 548, 4009                    # a product in parts, with a workspace
    W = int8.quantize(torch.randn(m, k, generator=g).cuda())
    xs = [torch.randn(n, k, generator=g).bfloat16().cuda() for _ in range(2)]
    ids = [torch.randint(0, 9, (3000, 2), generator=g).cuda() for _ in range(2)]      # a sort in parts

    def run(i):
        return (int8.linear(xs[i], W), *moe.sort(ids[i], 9))

    want = [run(i) for i in (0, 1)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in (0, 1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run(i))
        graphs.append(graph)
    for _ in range(3):
        for i in (1, 0):
            graphs[i].replay()
            run(1 - i)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_streams_at_once():
    g = torch.Generator().manual_seed(2)
    W = int8.quantize(torch.randn(300, 5000, generator=g).cuda())
    xs = [torch.randn(400, 5000, generator=g).bfloat16().cuda() for _ in range(2)]
    ids = [torch.randint(0, 40, (6000, 2), generator=g).cuda() for _ in range(2)]
    want = [(int8.linear(x, W), *moe.sort(i, 40)) for x, i in zip(xs, ids)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((int8.linear(xs[i], W), *moe.sort(ids[i], 40)))
    torch.cuda.synchronize()
    for i in (0, 1):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i]))


def test_no_tokens():
    order = moe.sort(torch.zeros(0, 3, dtype=torch.int64, device="cuda"), 5)
    assert not order.offsets.any() and order.place.shape == (0, 3) and order.rows.shape == (0,)
    x = torch.zeros(0, 32, device="cuda", requires_grad=True)
    w = torch.zeros(0, 3, device="cuda", requires_grad=True)
    xs = moe.gather(x, order)
    out = moe.combine(xs, w, order)
    dx, dw = torch.autograd.grad(out, [x, w], torch.zeros_like(out))
    assert xs.shape == out.shape == dx.shape == (0, 32) and dw.shape == (0, 3)
    W = int8.quantize(torch.randn(4, 64, 32, device="cuda"))
    D = int8.quantize(torch.randn(4, 32, 32, device="cuda"))
    order = torch.zeros(0, 3, dtype=torch.int64, device="cuda")
    assert moe.Int8Experts(W, D)(torch.zeros(0, 32, device="cuda"), order, torch.zeros(0, 3, device="cuda")).shape == (0, 32)
    assert int8.linear(torch.zeros(0, 32, device="cuda"), int8.quantize(torch.randn(7, 32, device="cuda"))).shape == (0, 7)
    # an expert without rows on the way to a trained one
    w = torch.randn(16, 32, device="cuda", requires_grad=True)
    y = blocks.gated(blocks.linear(torch.zeros(0, 32, device="cuda"), w))
    assert y.shape == (0, 8)
    dw, = torch.autograd.grad(y.sum(), [w])
    assert dw.shape == w.shape and not dw.any()
