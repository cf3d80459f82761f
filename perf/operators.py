"""Cases of the block-scaled 8-bit operators and of the mixture-of-experts layer, with their plain forms.

Three operators:

* ``quantize``: a matrix to 8-bit floating point codes (e4m3 or e5m2) with one float scale for every 128
  consecutive entries of a row (block 1), or for every 128 x 128 tile (block 128); as it is, transposed, or
  both from one read.
* ``product``: C = B A^T for two such matrices, contraction index contiguous in both, each 128-long piece of
  the contraction weighted by the two scales that belong to it.  Forward and input gradient (128 x 128 weight
  scales against 1 x 128 activation scales) and weight gradient (1 x 128 on both sides).
* ``moe``: a whole mixture-of-experts layer for a few tokens: router product, softmax, top-k, gated experts
  (silu), weighted sum; weights in half, bfloat16, or e4m3 with 128 x 128 scales.

``own`` is set by whoever imports the file: false runs the plain forms below, true the framework's operators.
"""
import math

import torch

own = False

BLK = 128
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SMALLEST = 2.0 ** -100          # the smallest scale


# ---- cases ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode batch's activations before a product: latency
        dict(name="quantize_decode", kind="quantize", rows=32, cols=2048, dtype="bf16", block=1, fmt="e4m3",
             straight=True, transposed=False),
        # a training batch's activations, for the forward product and for the weight gradient
        dict(name="quantize_train", kind="quantize", rows=8192, cols=4096, dtype="bf16", block=1, fmt="e4m3",
             straight=True, transposed=True),
        # a float master weight, ragged, once a step: forward and input-gradient layouts
        dict(name="quantize_weight", kind="quantize", rows=5000, cols=4136, dtype="f32", block=128, fmt="e4m3",
             straight=True, transposed=True),
        # a projection of one token
        dict(name="product_token", kind="product", m=8192, n=1, k=4096, a_block=128, a_fmt="e4m3", b_fmt="e4m3",
             out="bf16"),
        # a small ragged decode batch
        dict(name="product_decode", kind="product", m=4608, n=37, k=2568, a_block=128, a_fmt="e4m3", b_fmt="e4m3",
             out="bf16"),
        # a ragged prompt
        dict(name="product_ragged", kind="product", m=2501, n=1111, k=1747, a_block=128, a_fmt="e4m3", b_fmt="e4m3",
             out="f16"),
        # a training or prefill batch through a projection
        dict(name="product_forward", kind="product", m=8192, n=4096, k=4096, a_block=128, a_fmt="e4m3", b_fmt="e4m3",
             out="bf16"),
        # the weight gradient of a 4096 x 4096 projection over 8192 tokens, gradients in e5m2
        dict(name="product_wgrad", kind="product", m=4096, n=4096, k=8192, a_block=1, a_fmt="e4m3", b_fmt="e5m2",
             out="f32"),
        # the largest product
        dict(name="product_large", kind="product", m=8192, n=8192, k=8192, a_block=128, a_fmt="e4m3", b_fmt="e4m3",
             out="bf16"),
        # decoding one sequence
        dict(name="moe_token", kind="moe", tokens=1, hidden=2048, inter=1024, experts=64, topk=8, dtype="bf16",
             weights="bf16", normalize=True),
        # a small batch on 8-bit weights, ragged sizes
        dict(name="moe_batch_e4m3", kind="moe", tokens=13, hidden=2064, inter=1168, experts=96, topk=6, dtype="bf16",
             weights="e4m3", normalize=True),
        # a decode batch that reaches nearly every expert
        dict(name="moe_batch", kind="moe", tokens=64, hidden=2048, inter=1024, experts=128, topk=8, dtype="bf16",
             weights="bf16", normalize=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "product", "moe"])
    if kind == "quantize":
        straight, transposed = rng.choice([(True, False), (False, True), (True, True)])
        return dict(kind=kind, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192), dtype=rng.choice(["bf16", "f16", "f32"]),
                    block=rng.choice([1, 1, 128]), fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), straight=straight,
                    transposed=transposed)
    if kind == "product":
        n = rng.choice([_log(rng, 1, 64), _log(rng, 64, 8192)])
        grad = rng.random() < 0.25
        return dict(kind=kind, m=_log(rng, 256, 8192), n=n, k=_log(rng, 128, 8192), a_block=1 if grad else 128,
                    a_fmt="e4m3", b_fmt="e5m2" if grad and rng.random() < 0.5 else "e4m3",
                    out="f32" if grad else rng.choice(["bf16", "bf16", "f16", "f32"]))
    weights = rng.choice(["bf16", "f16", "e4m3"])
    experts = _log(rng, 8, 128)
    hidden, inter = 16 * _log(rng, 32, 128), 16 * _log(rng, 16, 64)
    return dict(kind=kind, tokens=_log(rng, 1, 64), hidden=hidden, inter=inter, experts=experts,
                topk=rng.randint(1, min(8, experts)), dtype="f16" if weights == "f16" else "bf16", weights=weights,
                normalize=rng.random() < 0.7)


# ---- inputs --------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols):
    """Normal entries, channels of uneven strength (a few strong ones), rows of uneven strength."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    ch = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    ch = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.004, ch * 20.0, ch)
    return x.mul_(ch).mul_(torch.exp(0.3 * torch.randn(rows, 1, generator=g, device="cuda")))


def _ceil(a, b):
    return -(-a // b)


def _amax_blocks(x, block):
    """Largest magnitude of every block of x (..., rows, cols): (..., col blocks, row blocks)."""
    r, c = x.shape[-2:]
    rb = BLK if block == 128 else 1
    x = torch.nn.functional.pad(x.abs(), (0, _ceil(c, BLK) * BLK - c, 0, _ceil(r, rb) * rb - r))
    x = x.reshape(*x.shape[:-2], _ceil(r, rb), rb, _ceil(c, BLK), BLK).amax(dim=(-3, -1))
    return x.transpose(-1, -2).contiguous()


def _spread(scales, rows, cols, block):
    """The scale of every entry of a (..., rows, cols) matrix from its (..., col blocks, row blocks) scales."""
    s = scales.transpose(-1, -2).repeat_interleave(BLK, dim=-1)[..., :cols]
    return s.repeat_interleave(BLK, dim=-2)[..., :rows, :] if block == 128 else s


def _quantize(x, block, fmt):
    """(codes, scales) of a float (..., rows, cols) matrix, both unpadded.  A scale is the float nearest to the
    block's largest magnitude over the format's largest number, a code the number of the format nearest to the
    float quotient of entry and scale (ties to even)."""
    # divided by a tensor: by a Python number torch multiplies with its reciprocal, which is not the same float
    scales = (_amax_blocks(x, block) / torch.full((), TOP[fmt], device="cuda")).clamp_min(SMALLEST)
    q = x / _spread(scales, x.shape[-2], x.shape[-1], block)
    return q.clamp_(-TOP[fmt], TOP[fmt]).to(F8[fmt]), scales


def _padded(codes, k):
    """Codes with rows of a multiple of 16 bytes, zero codes after the k-th."""
    ld = _ceil(k, 16) * 16
    out = torch.zeros(*codes.shape[:-1], ld, dtype=torch.uint8, device="cuda")
    out[..., :k] = codes.view(torch.uint8)
    return out.view(codes.dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["kind"] == "quantize":
        x = _activations(g, case["rows"], case["cols"])
        if case["rows"] > 8:
            x[torch.randint(case["rows"], (1 + case["rows"] // 500,), generator=g, device="cuda")] = 0.0   # padding
        s["x"] = x.to(DT[case["dtype"]])
    elif case["kind"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        if case["a_block"] == 128:
            a = torch.randn(m, k, generator=g, device="cuda") * 0.02
        else:
            a = _activations(g, m, k)
        b = _activations(g, n, k)
        for name, x, block, fmt in (("a", a, case["a_block"], case["a_fmt"]), ("b", b, 1, case["b_fmt"])):
            codes, scales = _quantize(x, block, fmt)
            s[name + "_codes"], s[name + "_scales"] = _padded(codes, k), scales
        if own:
            from hpc_linear_algebra_amd import blocks
            s["A"] = blocks.BlockScaled(s["a_codes"], s["a_scales"], m, k, case["a_block"])
            s["B"] = blocks.BlockScaled(s["b_codes"], s["b_scales"], n, k, 1)
    else:
        t, h, i, e = case["tokens"], case["hidden"], case["inter"], case["experts"]
        dt = DT[case["dtype"]]
        s["x"] = (torch.randn(t, h, generator=g, device="cuda")).to(dt)
        s["router"] = (torch.randn(e, h, generator=g, device="cuda") / math.sqrt(h)).to(dt)
        w1 = torch.empty(e, 2 * i, h, dtype=dt, device="cuda").normal_(0.0, 1.0 / math.sqrt(h), generator=g)
        w2 = torch.empty(e, h, i, dtype=dt, device="cuda").normal_(0.0, 1.0 / math.sqrt(i), generator=g)
        if case["weights"] == "e4m3":
            c1, s["gate_up_scales"] = _quantize(w1.float(), 128, "e4m3")
            c2, s["down_scales"] = _quantize(w2.float(), 128, "e4m3")
            w1, w2 = c1, c2
        s["gate_up"], s["down"] = w1, w2
        if own:
            from hpc_linear_algebra_amd import moe
            s["layer"] = moe.MoELayer(s["router"], s["gate_up"], s["down"], topk=case["topk"], max_tokens=t,
                                      normalize=case["normalize"], gate_up_scales=s.get("gate_up_scales"),
                                      down_scales=s.get("down_scales"))
    return s


# ---- one pass ------------------------------------------------------------------------------------------

def _plain_quantize(s):
    x, out = s["x"].float(), []
    if s["straight"]:
        out += _quantize(x, s["block"], s["fmt"])
    if s["transposed"]:
        out += _quantize(x.t(), s["block"], s["fmt"])
    return out


def _own_quantize(s):
    from hpc_linear_algebra_amd import blocks
    got = blocks.quantize(s["x"], block=s["block"], fmt=s["fmt"], straight=s["straight"], transposed=s["transposed"])
    out = []
    for q in got:
        if q is not None:
            out += [q.codes[:, :q.k], q.scales]
    return out


def _plain_product(s):
    m, n, k = s["m"], s["n"], s["k"]
    a = s["a_codes"][:, :k].float() * _spread(s["a_scales"], m, k, s["a_block"])
    b = s["b_codes"][:, :k].float() * _spread(s["b_scales"], n, k, 1)
    return (b @ a.t()).to(DT[s["out"]])


def _own_product(s):
    from hpc_linear_algebra_amd import blocks
    # 16-bit results take the 8-bit matrix instructions' sums, float ones (weight gradients) sums in float
    return blocks.gemm(s["A"], s["B"], dtype=s["out"], fast=s["out"] != "f32")


def _plain_moe(s):
    t, h, i, e, k = s["tokens"], s["hidden"], s["inter"], s["experts"], s["topk"]
    x = s["x"].float()
    logits = s["x"].double() @ s["router"].double().t()
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]     # ties: the lower index first
    z = torch.exp((logits - logits.amax(dim=1, keepdim=True)).float())
    p = (z / z.sum(dim=1, keepdim=True)).gather(1, ids)
    if s["normalize"]:
        p = p / p.sum(dim=1, keepdim=True)
    if t * k <= e:             # the chosen experts' weights, once for every choice
        pick = ids.reshape(-1)
        xs = x.repeat_interleave(k, dim=0).unsqueeze(1)
    else:                      # every expert on every token
        pick = torch.arange(e, device="cuda")
        xs = x.unsqueeze(0).expand(e, t, h).contiguous()
    w1, w2 = s["gate_up"][pick].float(), s["down"][pick].float()
    if s["weights"] == "e4m3":
        w1 = w1 * _spread(s["gate_up_scales"][pick], 2 * i, h, 128)
        w2 = w2 * _spread(s["down_scales"][pick], h, i, 128)
    g, u = torch.bmm(xs, w1.transpose(1, 2)).split(i, dim=2)
    y = torch.bmm(g / (1.0 + torch.exp(-g)) * u, w2.transpose(1, 2))
    if t * k <= e:
        y = (y.reshape(t, k, h) * p.unsqueeze(2)).sum(dim=1)
    else:
        gate = torch.zeros(t, e, device="cuda").scatter_(1, ids, p)
        y = (y * gate.t().unsqueeze(2)).sum(dim=0)
    return y.to(s["x"].dtype), ids.to(torch.int32), p


def _own_moe(s):
    return s["layer"](s["x"])


def run(state):
    kind = state["kind"]
    if own:
        return {"quantize": _own_quantize, "product": _own_product, "moe": _own_moe}[kind](state)
    return {"quantize": _plain_quantize, "product": _plain_product, "moe": _plain_moe}[kind](state)


# ---- the work a pass cannot do without -----------------------------------------------------------------

def _scale_bytes(rows, cols, block):
    return 4 * _ceil(cols, BLK) * (_ceil(rows, BLK) if block == 128 else rows)


def work(case):
    if case["kind"] == "quantize":
        r, c = case["rows"], case["cols"]
        b = r * c * (4 if case["dtype"] == "f32" else 2)
        for on, p, q in ((case["straight"], r, c), (case["transposed"], c, r)):
            if on:
                b += r * c + _scale_bytes(p, q, case["block"])
        return {"bytes": b, "flops": 2 * r * c}
    if case["kind"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        b = m * k + n * k + _scale_bytes(m, k, case["a_block"]) + _scale_bytes(n, k, 1)
        return {"bytes": b + m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}
    t, h, i, e, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
    # experts that t independent choices of k out of e reach, on average
    reached = e * (1.0 - (1.0 - k / e) ** t)
    per = 3 * h * i * (1 if case["weights"] == "e4m3" else 2)
    if case["weights"] == "e4m3":
        per += _scale_bytes(2 * i, h, 128) + _scale_bytes(h, i, 128)
    return {"bytes": reached * per + 2 * e * h + 4 * t * h + 8 * t * k, "flops": 2 * t * e * h + 6 * t * k * h * i}


# ---- the same from the definitions, in 64 bits ---------------------------------------------------------

def _exact_codes(x, scale, fmt):
    """The float x / scale to the nearest number of the format (ties to even), as a double."""
    q = (x / scale).float().double()     # the quotient is a float number
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** low))).clamp_min(low) - bits)
    return (torch.round(q / step) * step).clamp(-TOP[fmt], TOP[fmt])


def _exact_quantize(x, block, fmt):
    r, c = x.shape
    scales = torch.empty(_ceil(c, BLK), _ceil(r, BLK) if block == 128 else r, dtype=torch.float64, device="cuda")
    codes = torch.empty_like(x)
    for j in range(scales.shape[0]):
        piece = x[:, j * BLK:(j + 1) * BLK]
        top = piece.abs().amax(dim=1)
        if block == 128:
            top = torch.stack([v.amax() for v in top.split(BLK)])
        # so is a scale
        scales[j] = (top / TOP[fmt]).clamp_min(SMALLEST).float().double()
        each = scales[j].repeat_interleave(BLK)[:r] if block == 128 else scales[j]
        codes[:, j * BLK:(j + 1) * BLK] = _exact_codes(piece, each.unsqueeze(1), fmt)
    return [codes, scales]


def _exact_values(codes, scales, rows, k, block):
    v = codes[:, :k].float().double()
    for j in range(scales.shape[0]):
        each = scales[j].double()
        each = each.repeat_interleave(BLK)[:rows] if block == 128 else each
        v[:, j * BLK:(j + 1) * BLK] *= each.unsqueeze(1)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "quantize":
        x, out = s["x"].double(), []
        if case["straight"]:
            out += _exact_quantize(x, case["block"], case["fmt"])
        if case["transposed"]:
            out += _exact_quantize(x.t().contiguous(), case["block"], case["fmt"])
        return out
    if case["kind"] == "product":
        a = _exact_values(s["a_codes"], s["a_scales"], case["m"], case["k"], case["a_block"])
        b = _exact_values(s["b_codes"], s["b_scales"], case["n"], case["k"], 1)
        return torch.mm(b, a.t())
    t, h, i, e, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
    x = s["x"].double()
    logits = torch.stack([(x * w).sum(dim=1) for w in s["router"].double()], dim=1).cpu()
    prob = torch.softmax(logits, dim=1)
    ids = torch.empty(t, k, dtype=torch.int64)
    for r in range(t):
        ids[r] = torch.tensor(sorted(range(e), key=lambda c: (-float(logits[r, c]), c))[:k])
    p = prob.gather(1, ids)
    if case["normalize"]:
        p = p / p.sum(dim=1, keepdim=True)
    y = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    for c in sorted(set(ids.reshape(-1).tolist())):
        rows, slots = torch.nonzero(ids == c, as_tuple=True)
        if case["weights"] == "e4m3":
            w1 = _exact_values(s["gate_up"][c], s["gate_up_scales"][c], 2 * i, h, 128)
            w2 = _exact_values(s["down"][c], s["down_scales"][c], h, i, 128)
        else:
            w1, w2 = s["gate_up"][c].double(), s["down"][c].double()
        a = x[rows.cuda()] @ w1.t()
        z = a[:, :i] * torch.sigmoid(a[:, :i]) * a[:, i:]
        y[rows.cuda()] += (z @ w2.t()) * p[rows, slots].cuda().unsqueeze(1)
    return y, ids.to(torch.int32), p
