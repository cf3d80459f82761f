"""The mixture-of-experts layer against its definition in 64 bits where test_gpu_moe does not go: small activations in
half precision, and sizes whose loops run more than once."""
import pytest
import torch

from test_gpu_moe import TD, check, layer_of, make, values

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
