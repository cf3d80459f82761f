"""The mixture-of-experts layer on the GPU against its definition in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TD = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(tokens, hidden, inter, experts, dtype, weights, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    t = dict(x=(rn(tokens, hidden) * spread).to(TD[dtype]), router=(rn(experts, hidden) / hidden ** 0.5).to(TD[dtype]))
    for name, rows, cols in (("gate_up", 2 * inter, hidden), ("down", hidden, inter)):
        if weights == "e4m3":
            c = (rn(experts, rows, cols) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            s = torch.exp(0.5 * rn(experts, -(-cols // 128), -(-rows // 128))) / (60 * cols ** 0.5)
            t[name], t[name + "_scales"] = c, s
        else:
            t[name] = (rn(experts, rows, cols) / cols ** 0.5).to(TD[dtype])
    return t


def values(t, name):
    w = t[name]
    if w.dtype != torch.float8_e4m3fn:
        return w.double()
    s = t[name + "_scales"].double().transpose(1, 2)
    s = s.repeat_interleave(128, dim=1)[:, :w.shape[1]].repeat_interleave(128, dim=2)[:, :, :w.shape[2]]
    return w.float().double() * s


def reference(t, topk, normalize):
    """(y, ids, weights, bound of |error| of y) in 64 bits."""
    x, wr, w1, w2 = t["x"].double(), t["router"].double(), values(t, "gate_up"), values(t, "down")
    u = torch.finfo(t["x"].dtype).eps / 2
    inter, hidden = w2.shape[2], w2.shape[1]
    logits = x @ wr.t()
    ids = torch.tensor([sorted(range(wr.shape[0]), key=lambda e: (-float(row[e]), e))[:topk] for row in logits])
    p = torch.softmax(logits, 1).gather(1, ids)
    if normalize:
        p = p / p.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    bound = torch.zeros_like(x)
    e32 = 2.0 ** -24
    for r in range(x.shape[0]):
        for j in range(topk):
            e = int(ids[r, j])
            a, m = w1[e] @ x[r], w1[e].abs() @ x[r].abs()
            # float sums of `hidden` exact products, one scale rounding a block: (hidden + 2) e32 of the magnitudes
            da = (hidden + 2) * e32 * m
            g, up, dg, du = a[:inter], a[inter:], da[:inter], da[inter:]
            s = g * torch.sigmoid(g)
            h = s * up
            # |silu'| <= 1.1; exp, sum, quotient and product in float: 8 units; hi + lo: u^2 (and a subnormal's half step)
            dh = 1.1 * dg * up.abs() + (s.abs() + 1.1 * dg) * du + 8 * e32 * h.abs() + 2 * u * u * h.abs()
            dh = dh + torch.finfo(t["x"].dtype).smallest_normal * u
            d, md = w2[e] @ h, w2[e].abs() @ h.abs()
            y[r] += p[r, j] * d
            # float sums of 2 inter products; the probability: 16 units; the sum over the experts: topk
            bound[r] += p[r, j] * (w2[e].abs() @ dh + (2 * inter + 18 + topk) * e32 * (md + w2[e].abs() @ dh))
    return y, ids, p, bound + u * (y.abs() + bound) + torch.finfo(t["x"].dtype).smallest_normal * u


def layer_of(t, topk, normalize=True, max_tokens=64):
    from hpc_linear_algebra_amd.moe import MoELayer
    c = {k: v.cuda() for k, v in t.items()}
    return MoELayer(c["router"], c["gate_up"], c["down"], topk, max_tokens, normalize, c.get("gate_up_scales"),
                    c.get("down_scales")), c["x"]


def check(got, ref):
    y, ids, p = (v.cpu() for v in got)
    ry, rids, rp, bound = ref
    assert torch.equal(ids.long(), rids)
    # exp and the logit's rounding to float: 2^-24 of |l - max| (below 64) each, and the divisions
    assert torch.all((p.double() - rp).abs() <= rp * (64 + 16) * 2.0 ** -24 + 1e-38)
    err = (y.double() - ry).abs() / bound
    assert float(err.max()) <= 1.0, f"error {float(err.max()):.3f} of its bound"


CASES = [  # tokens, hidden, inter, experts, topk
    (1, 16, 16, 1, 1), (1, 64, 32, 8, 2), (2, 144, 80, 5, 5), (3, 512, 272, 16, 4), (7, 272, 128, 3, 2),
    (17, 256, 144, 4, 4), (33, 128, 64, 2, 1), (40, 400, 208, 24, 6), (64, 256, 128, 64, 8), (130, 64, 48, 7, 3),
    (256, 48, 32, 300, 16)]


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", CASES)
@pytest.mark.parametrize("dtype,weights,normalize", [("bf16", "bf16", True), ("f16", "f16", False), ("bf16", "e4m3", False),
                                                     ("f16", "e4m3", True)])
def test_layer(tokens, hidden, inter, experts, topk, dtype, weights, normalize):
    t = make(tokens, hidden, inter, experts, dtype, weights, tokens + hidden)
    layer, x = layer_of(t, topk, normalize, tokens)
    got = layer(x)
    check(got, reference(t, topk, normalize))
    for _ in range(3):                                  # the workspace is reused, and no order changes a result
        again = layer(x)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_fewer_tokens_than_the_workspace_and_varying():
    t = make(48, 128, 64, 12, "bf16", "bf16", 9)
    layer, x = layer_of(t, 3, True, 64)
    for n in (48, 1, 5, 0, 17, 2, 48):
        part = dict(t, x=t["x"][:n])
        y, ids, p = layer(x[:n])
        assert y.shape == (n, 128) and ids.shape == (n, 3)
        if n:
            check((y, ids, p), reference(part, 3, True))


def test_ties_go_to_the_lowest_index():
    t = make(5, 64, 32, 16, "bf16", "bf16", 1)
    t["router"] = t["router"][:1].repeat(16, 1)
    layer, x = layer_of(t, 4)
    y, ids, p = layer(x)
    assert torch.equal(ids.cpu(), torch.arange(4, dtype=torch.int32).repeat(5, 1))
    check((y, ids, p), reference(t, 4, True))


def test_one_expert_takes_every_token():
    t = make(64, 128, 48, 32, "f16", "f16", 2)
    t["x"][:, 0] = 8.0
    t["router"][:, 0] = 0.0
    t["router"][7, 0] = 4.0
    layer, x = layer_of(t, 1)
    y, ids, p = layer(x)
    assert torch.all(ids == 7)
    check((y, ids, p), reference(t, 1, True))


def test_non_finite_tokens_stay_their_own():
    """A token with a NaN or an infinity gives a NaN row; the other rows are as without it."""
    t = make(6, 128, 64, 8, "bf16", "bf16", 3)
    layer, x = layer_of(t, 2)
    want = layer(x)
    bad = x.clone()
    bad[2, 5] = float("nan")
    bad[4, 9] = float("inf")
    y, ids, p = layer(bad)
    assert torch.isnan(y[2]).all() and torch.isnan(p[2]).all() and torch.isnan(y[4]).any()
    assert int(ids.min()) >= 0 and int(ids.max()) < 8
    for r in (0, 1, 3, 5):
        assert torch.equal(y[r], want[0][r]) and torch.equal(ids[r], want[1][r]) and torch.equal(p[r], want[2][r])


def test_strided_tokens_and_another_stream():
    t = make(9, 96, 64, 8, "bf16", "bf16", 4)
    layer, x = layer_of(t, 2)
    wide = torch.zeros(9, 120, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:112] = x
    want = reference(t, 2, True)
    check(layer(wide[:, 16:112]), want)                  # 16-byte rows, taken as they are
    wide2 = torch.zeros(9, 101, dtype=torch.bfloat16, device="cuda")
    wide2[:, 3:99] = x
    check(layer(wide2[:, 3:99]), want)                   # copied first
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer(x)
    s.synchronize()
    check(got, want)


def test_captured_into_a_graph():
    t = make(4, 256, 128, 16, "bf16", "e4m3", 5)
    layer, x = layer_of(t, 4)
    want = layer(x)
    torch.cuda.synchronize()
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer(static)
    for k in range(5):
        static.copy_(x.roll(k, 0))
        for v in got:
            v.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b.roll(k, 0)) for a, b in zip(got, want))
        eager = layer(x)                                 # the same workspace, in order
        assert all(torch.equal(a, b) for a, b in zip(eager, want))


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [
    (8, 64, 256, 64, 8), (16, 64, 1024, 16, 2), (17, 64, 1024, 16, 2),
    (8, 128, 512, 64, 8),     # routed one by one, sorted, parts added by a launch
    (16, 64, 2048, 16, 2),    # routed one by one, sorted, parts added by the down product
    (16, 96, 64, 32, 3),      # routed one by one, lists by the experts
    (12, 64, 48, 64, 4),      # routed together, lists by the experts, parts added by the down product
    (13, 256, 48, 64, 4),     # routed together, lists by the experts, parts added by a launch
    (17, 64, 2048, 32, 2),    # routed together, sorted, parts added by the down product
    (33, 400, 64, 24, 8)])    # routed together, sorted, parts added by a launch
@pytest.mark.parametrize("weights", ["bf16", "e4m3"])
def test_every_way_through_the_kernels(tokens, hidden, inter, experts, topk, weights):
    t = make(tokens, hidden, inter, experts, "bf16", weights, tokens + experts)
    layer, x = layer_of(t, topk)
    want = reference(t, topk, True)
    for _ in range(3):                                   # the counters are back at 0
        check(layer(x), want)


def test_expanded_and_transposed_tokens():
    t = make(6, 80, 48, 8, "f16", "f16", 9)
    layer, x = layer_of(t, 2)
    want = layer(x)
    back = x.t().contiguous().t()
    assert not back.is_contiguous() and all(torch.equal(a, b) for a, b in zip(layer(back), want))
    one = layer(x[:1].expand(5, 80).contiguous())
    assert all(torch.equal(a, b) for a, b in zip(layer(x[:1].expand(5, 80)), one))
