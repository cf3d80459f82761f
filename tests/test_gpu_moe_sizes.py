"""The mixture-of-experts layer against its definition in 64 bits where test_gpu_moe does not go: small activations in
half precision, and sizes whose loops run more than once."""
import pytest
import torch

from test_gpu_moe import check, layer_of, make, values

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
# What the two numbers that carry silu(g) u lose of it: relative, and half the step below which it is cut.
CARRY = {torch.float16: (2.0 ** -22, 2.0 ** -36), torch.bfloat16: (2.0 ** -16, 2.0 ** -134)}


def reference(t, topk, normalize):
    """(y, ids, weights, bound of |error| of y) in 64 bits: the bound's terms are those of test_gpu_moe's reference,
    with what the carried numbers lose as CARRY has it.  Expert by expert."""
    x, wr, w1, w2 = t["x"].double(), t["router"].double(), values(t, "gate_up"), values(t, "down")
    dtype = t["x"].dtype
    u, (rel, cut) = torch.finfo(dtype).eps / 2, CARRY[dtype]
    inter, hidden = w2.shape[2], w2.shape[1]
    logits = x @ wr.t()
    ids = torch.tensor([sorted(range(wr.shape[0]), key=lambda e: (-float(row[e]), e))[:topk] for row in logits])
    p = torch.softmax(logits, 1).gather(1, ids)
    if normalize:
        p = p / p.sum(1, keepdim=True)
    y, bound = torch.zeros_like(x), torch.zeros_like(x)
    for e in ids.unique().tolist():
        rows, slots = torch.nonzero(ids == e, as_tuple=True)
        a, da = x[rows] @ w1[e].t(), (hidden + 2) * E32 * (x[rows].abs() @ w1[e].abs().t())
        g, up, dg, du = a[:, :inter], a[:, inter:], da[:, :inter], da[:, inter:]
        s = g * torch.sigmoid(g)
        h = s * up
        dh = 1.1 * dg * up.abs() + (s.abs() + 1.1 * dg) * du + (8 * E32 + rel) * h.abs() + cut
        d, md, dd = h @ w2[e].t(), h.abs() @ w2[e].abs().t(), dh @ w2[e].abs().t()
        q = p[rows, slots].unsqueeze(1)
        y[rows] += q * d
        bound[rows] += q * (dd + (2 * inter + 18 + topk) * E32 * (md + dd))
    return y, ids, p, bound + u * (y.abs() + bound) + torch.finfo(dtype).smallest_normal * u


@pytest.mark.parametrize("tokens", [1, 3, 40])
@pytest.mark.parametrize("weights", ["f16", "e4m3"])
def test_small_activations_in_half_precision(tokens, weights):
    """silu(g) u about 2^-24, half precision's last step, and down weights that bring y back to its normal range."""
    t = make(tokens, 128, 64, 6, "f16", weights, tokens + 7)
    up, down = 2.0 ** -11, 2.0 ** 12
    for name, by in (("gate_up", up), ("down", down)):
        if weights == "e4m3":
            t[name + "_scales"] = t[name + "_scales"] * by
        else:
            t[name] = (t[name].float() * by).half()
    layer, x = layer_of(t, 3)
    want = reference(t, 3, True)
    assert float(want[0].abs().median()) > 2.0 ** -14        # normal numbers of half precision
    check(layer(x), want)


def uneven(t, seed):
    """Scales of neighbouring blocks that differ by up to 2^6: another block's is no answer."""
    g = torch.Generator().manual_seed(seed)
    for name in ("gate_up_scales", "down_scales"):
        if name in t:
            t[name] = t[name] * 2.0 ** torch.randint(-3, 4, t[name].shape, generator=g)
    return t


# splits of the router's columns: one for every 512 of hidden, up to four, where tokens are not routed one by one
SIZES = [  # tokens, hidden, inter, experts, topk
    (1, 1168, 400, 6, 4),       # one token: several passes over a row, every block of scales
    (1, 2064, 1040, 12, 5),     # and over the pairs of the down product
    (1, 528, 4112, 3, 2),
    (2, 1040, 272, 9, 3), (5, 704, 144, 33, 4),                 # routed one by one, several passes
    (3, 528, 48, 176, 3), (17, 528, 64, 72, 4),                 # two splits
    (3, 1040, 32, 200, 4), (17, 1040, 64, 66, 3),               # three
    (3, 2064, 48, 190, 5), (17, 2064, 32, 70, 2), (40, 2576, 32, 65, 6),      # four
    (7, 656, 656, 20, 3), (24, 1168, 784, 10, 2),               # two column groups in flight, both products
    (40, 1296, 1168, 6, 2), (70, 912, 400, 12, 4), (256, 1040, 144, 24, 4)]


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", SIZES)
@pytest.mark.parametrize("dtype,weights,normalize", [("bf16", "bf16", True), ("bf16", "e4m3", True), ("f16", "e4m3", False),
                                                     ("f16", "f16", True)])
def test_sizes_of_real_layers(tokens, hidden, inter, experts, topk, dtype, weights, normalize):
    t = uneven(make(tokens, hidden, inter, experts, dtype, weights, tokens + hidden + inter), tokens)
    layer, x = layer_of(t, topk, normalize, tokens)
    want = reference(t, topk, normalize)
    for _ in range(2):                                   # the counters are back at 0
        check(layer(x), want)


def test_the_reference_tells_blocks_apart():
    """Block 0's scale in every place is far outside the bound, in either product."""
    for name in ("gate_up_scales", "down_scales"):
        t = uneven(make(1, 1168, 400, 6, "bf16", "e4m3", 1), 1)
        want = reference(t, 4, True)
        t[name] = t[name][:, :1, :1].expand_as(t[name]).contiguous()
        off = (reference(t, 4, True)[0] - want[0]).abs()
        assert float((off > 4 * want[3]).float().mean()) > 0.5
