"""The gated activation, its 8-bit checkpoint and the gradient from it, against the definitions in 64 bits."""
import pytest
import torch

from hpc_linear_algebra_amd import blocks

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}            # half a step, relative
LEAST = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}        # floats below may be flushed on the way
EPS = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def plain_codes(x):
    """The values that a checkpoint of x (rows, inter) stands for, its codes and its scales."""
    rows, inter = x.shape
    nq = -(-inter // 128)
    codes, scales = torch.zeros(rows, inter, dtype=torch.float64), torch.zeros(rows, nq, dtype=torch.float64)
    for q in range(nq):
        piece = x[:, 128 * q:128 * q + 128].double()
        s = (piece.abs().amax(dim=1) / 127.0).float().double().clamp_min(2.0 ** -100)
        codes[:, 128 * q:128 * q + 128] = torch.round((piece / s.unsqueeze(1)).float().double()).clamp(-127, 127)
        scales[:, q] = s
    return codes * scales.repeat_interleave(128, dim=1)[:, :inter], codes, scales


TINY = 2.0 ** -126          # the hardware's exponential has no smaller results but 0


def silu_bound(g, u):
    """Float errors of g sigmoid(g) u: exponential one step, sum, reciprocal one step and product of the sigmoid (8 half
    steps together), two products; one more for a g that is itself a rounded product, which moves exp(g) by |g| half steps;
    and a sigmoid below TINY is 0."""
    return (12.0 + 2.0 * g.abs()) * EPS * (g * torch.sigmoid(g) * u).abs() + TINY * (g * u).abs()


def check(got, want, off, dtype):
    bound = HALF[dtype] * (want.abs() + off) + off + LEAST[dtype]
    err = (got.detach().cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def gradient(x, dy):
    inter = dy.shape[1]
    (g, _, _), (u, _, _) = plain_codes(x[:, :inter]), plain_codes(x[:, inter:])
    dy = dy.double()
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)
    dg, du = dy * u * s * (1.0 + g * rest), dy * g * s
    # dg's last factor is a difference near g = -1.3: its own error is absolute
    off_g = (16.0 + 2.0 * g.abs()) * EPS * (dy * u * s).abs() * (1.0 + g.abs() * rest) + TINY * (dy * u).abs() * (1.0 + g.abs())
    return torch.cat([dg, du], dim=1), torch.cat([off_g, silu_bound(g, dy)], dim=1)


SIZES = [(1, 1), (1, 128), (3, 7), (2, 129), (5, 200), (17, 1001), (33, 1024), (4, 5003), (700, 130), (9, 16)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,inter", SIZES)
def test_values_checkpoint_and_gradient(rows, inter, dtype):
    gn = gen(rows + inter)
    x = (3.0 * torch.randn(rows, 2 * inter, generator=gn) * torch.exp(torch.randn(2 * inter, generator=gn))).to(DT[dtype])
    dy = torch.randn(rows, inter, generator=gn).to(DT[dtype])
    leaf = x.cuda().requires_grad_()
    y = blocks.gated(leaf)
    g, u = x[:, :inter].double(), x[:, inter:].double()
    check(y, g * torch.sigmoid(g) * u, silu_bound(g, u), dtype)
    assert y.dtype == DT[dtype] and torch.equal(y, blocks.gated(x.cuda()))
    y2, codes, scales = blocks.gated_forward(x.cuda())
    assert torch.equal(y2, y)
    for h in (0, 1):
        _, c, s = plain_codes(x[:, h * inter:(h + 1) * inter])
        assert torch.equal(codes[:, h, :inter].cpu().double(), c) and torch.equal(scales[:, h].cpu().double(), s)
    dx, = torch.autograd.grad(y, [leaf], dy.cuda())
    want, off = gradient(x, dy)
    check(dx, want, off, dtype)
    assert torch.equal(dx, blocks.gated_backward(dy.cuda(), codes, scales))


def test_gradient_against_differences():
    """Where the checkpoint is exact (x are multiples of their block's scale), the gradient is the function's."""
    gn = gen(1)
    codes = torch.randint(-127, 128, (6, 200), generator=gn)
    codes[:, [0, 100]] = 127                       # both halves' scale is 2^-5
    x = codes.float() / 32.0
    dy = torch.randn(6, 100, generator=gn)
    leaf = x.cuda().requires_grad_()
    dx, = torch.autograd.grad(blocks.gated(leaf), [leaf], dy.cuda())
    x64, h = x.double(), 1e-6

    def f(v):
        return (v[:, :100] * torch.sigmoid(v[:, :100]) * v[:, 100:] * dy.double()).sum(dim=1)

    for c in (0, 1, 57, 99, 100, 131, 199):
        step = torch.zeros(200, dtype=torch.float64)
        step[c] = h
        want = (f(x64 + step) - f(x64 - step)) / (2 * h)
        # third derivative of silu is below 1 and |u|, |dy| below 4: the quotient is off by 1e-11, its doubles by 1e-8
        assert float((dx[:, c].cpu().double() - want).abs().max()) < 1e-7 + 20 * EPS * 16


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_far_gates(dtype):
    """Gates where the exponential over- or underflows, and the ends of the type."""
    top = 65504.0 if dtype == "f16" else 3e38
    gates = [0.0, -0.0, 1.0, -1.0, -1.2784645, 16.0, -16.0, 20.0, -20.0, 87.0, -87.0, 89.0, -89.0, 104.0, -104.0, 200.0, -200.0, top, -top]
    x = torch.zeros(len(gates), 256)
    x[:, 0] = torch.tensor(gates)                  # alone in its block: held exactly
    x[:, 128] = 1.0
    x = x.to(DT[dtype])
    leaf = x.cuda().requires_grad_()
    y = blocks.gated(leaf)
    g = x[:, :128].double()
    check(y, g * torch.sigmoid(g) * x[:, 128:].double(), silu_bound(g, x[:, 128:].double()), dtype)
    dy = torch.ones(len(gates), 128, dtype=DT[dtype])
    dx, = torch.autograd.grad(y, [leaf], dy.cuda())
    want, off = gradient(x, dy)
    check(dx, want, off, dtype)


def test_special_values():
    inf, nan = float("inf"), float("nan")
    x = torch.ones(4, 600)
    x[0, 5], x[1, 299], x[2, 300], x[3, 599] = inf, nan, nan, -inf
    leaf = x.cuda().requires_grad_()
    y = blocks.gated(leaf)
    one = float(torch.sigmoid(torch.ones(1)))
    bad = torch.zeros(4, 300, dtype=torch.bool)
    bad[0, 5] = bad[1, 299] = bad[2, 0] = bad[3, 299] = True
    assert y[0, 5] == inf and torch.isnan(y[1, 299]) and torch.isnan(y[2, 0]) and y[3, 299] == -inf
    assert float((y.detach().cpu()[~bad] - one).abs().max()) < 1e-6
    dx, = torch.autograd.grad(y, [leaf], torch.ones(4, 300, device="cuda"))
    dx = dx.cpu()
    assert torch.isnan(dx[0, :128]).all() and torch.isfinite(dx[0, 128:300]).all()          # its block of 128
    assert torch.isnan(dx[1, 256:300]).all() and torch.isfinite(dx[1, :256]).all()
    assert torch.isnan(dx[2, :128]).all() and torch.isfinite(dx[2, 300:]).all()             # u touches dg only
    assert torch.isnan(dx[3, 256:300]).all() and torch.isfinite(dx[3, 300:]).all()
    zero = torch.zeros(3, 64, device="cuda", requires_grad=True)
    dx, = torch.autograd.grad(blocks.gated(zero), [zero], torch.ones(3, 32, device="cuda"))
    assert not dx.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_shapes_and_empty(dtype):
    gn = gen(3)
    x = torch.randn(6, 2 * 133, generator=gn).to(DT[dtype]).cuda()
    y = blocks.gated(x)
    big = torch.zeros(12, 300, dtype=DT[dtype], device="cuda")
    big[::2, 1:267] = x
    assert torch.equal(blocks.gated(big[::2, 1:267]), y)
    assert torch.equal(blocks.gated(x.t().contiguous().t()), y)
    assert torch.equal(blocks.gated(x.reshape(2, 3, 266)), y.reshape(2, 3, 133)) and torch.equal(blocks.gated(x[0]), y[0])
    for shape in ((0, 20), (4, 0), (2, 0, 6)):
        leaf = torch.zeros(shape, dtype=DT[dtype], device="cuda", requires_grad=True)
        out = blocks.gated(leaf)
        assert out.shape == (*shape[:-1], shape[-1] // 2)
        assert torch.autograd.grad(out, [leaf], torch.zeros_like(out))[0].shape == shape
    leaf = x.reshape(2, 3, 266).clone().requires_grad_()
    a, = torch.autograd.grad(blocks.gated(leaf).float().sum(), [leaf])                       # an expanded gradient
    b, = torch.autograd.grad(blocks.gated(leaf), [leaf], torch.ones(2, 3, 133, dtype=DT[dtype], device="cuda"))
    assert torch.equal(a, b) and a.shape == leaf.shape
    wide = torch.randn(6, 400, generator=gn).to(DT[dtype]).cuda()
    leaf = x.clone().requires_grad_()
    a, = torch.autograd.grad(blocks.gated(leaf), [leaf], wide[:, 5:138])
    b, = torch.autograd.grad(blocks.gated(leaf), [leaf], wide[:, 5:138].contiguous())
    assert torch.equal(a, b)


def test_far_rows():
    """Rows whose offset passes 2^32 bytes, in the input and in the gradient."""
    rows, inter = 140000, 8192
    x = torch.empty(rows, 2 * inter, dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(rows, device="cuda") % 100 / 16).unsqueeze(1))
    y, codes, scales = blocks.gated_forward(x)
    g = (torch.arange(rows, device="cuda") % 100 / 16).bfloat16().double()
    want = g * torch.sigmoid(g) * g
    for c in (0, 5000, inter - 1):
        assert bool(((y[:, c].double() - want).abs() <= want * 2.0 ** -8 * 1.01).all())
    dx = blocks.gated_backward(y, codes, scales)
    assert torch.equal(dx[:, 0], dx[:, inter - 1]) and torch.equal(dx[:, inter], dx[:, -1])
    first, last = dx[:100], dx[rows - 100:]                    # the same rows of x, 100 dividing rows
    assert torch.equal(first, last)


def test_memory_kept_for_the_backward_pass():
    x = torch.randn(512, 2048, device="cuda").bfloat16().requires_grad_()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = blocks.gated(x)
    assert torch.cuda.memory_allocated() - before == y.numel() * 2 + 512 * 2048 + 512 * 2 * 8 * 4


def test_no_second_derivative():
    x = torch.randn(4, 32, device="cuda", requires_grad=True)
    dx, = torch.autograd.grad(blocks.gated(x).sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        dx.sum().backward()


def test_streams_and_graphs():
    gn = gen(4)
    x = torch.randn(300, 600, generator=gn).bfloat16().cuda()
    dy = torch.randn(300, 300, generator=gn).bfloat16().cuda()

    def run():
        leaf = x.detach().requires_grad_()
        y = blocks.gated(leaf)
        return y.detach(), torch.autograd.grad(y, [leaf], dy)[0]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    keep = x.clone()
    for i in range(3):
        x.copy_(keep * (i + 1))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
