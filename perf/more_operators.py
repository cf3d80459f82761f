"""Cases of the 8-bit integer product, of sorting tokens by expert, and of the gated activation with an 8-bit
checkpoint, with their plain forms.

Four kinds of case:

* ``linear``: y = x W^T for a weight in 8-bit integers with a scale for each output channel; x is quantized within the
  call, with a scale for each token.
* ``experts``: the same with one weight per expert.  Tokens are sorted by the experts that a router chose, quantized
  on the way to their rows, and each expert's rows are multiplied with its weight.
* ``route``: tokens sorted by expert (a copy for each choice) and the experts' results added back with the router's
  weights; ``train``: with the gradients of x, of the results and of the weights.
* ``gated``: silu(gate) * up for rows that hold gate and up halves; ``train``: the input is kept for the backward pass
  as 8-bit integers with a scale for every 128 entries of a row, and the gradient is computed from those.

``own`` is set by whoever imports the file: false runs the plain forms below, true the framework's operators.
"""
import math

import torch

own = False

BLK = 128
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SMALLEST = 2.0 ** -100          # the smallest scale


# ---- cases ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token through a projection: latency, and the weight's bytes
        dict(name="linear_token", kind="linear", n=1, m=8192, k=4096, dtype="bf16"),
        # a small ragged decode batch
        dict(name="linear_decode", kind="linear", n=37, m=4608, k=2568, dtype="bf16"),
        # a ragged prompt in half precision
        dict(name="linear_ragged", kind="linear", n=1111, m=2501, k=1747, dtype="f16"),
        # the largest product: many prompts at once
        dict(name="linear_large", kind="linear", n=8192, m=8192, k=8192, dtype="bf16"),
        # a decode batch through its experts' first product
        dict(name="experts_decode", kind="experts", tokens=24, topk=4, experts=32, m=2048, k=2048, dropped=False,
             dtype="bf16"),
        # prompts through many experts, padded tokens among them
        dict(name="experts_prompt", kind="experts", tokens=4096, topk=8, experts=64, m=2816, k=2048, dropped=True,
             dtype="bf16"),
        # one decoded token: to its experts' rows and back
        dict(name="route_token", kind="route", tokens=1, topk=8, experts=64, hidden=2048, dropped=False, train=False,
             dtype="bf16"),
        # a ragged batch with padding, rows that are not whole vectors
        dict(name="route_ragged", kind="route", tokens=1003, topk=6, experts=96, hidden=1037, dropped=True, train=True,
             dtype="f16"),
        # a training batch
        dict(name="route_train", kind="route", tokens=8192, topk=8, experts=64, hidden=4096, dropped=False, train=True,
             dtype="bf16"),
        # a decode batch's activations, nothing kept
        dict(name="gated_decode", kind="gated", rows=96, inter=1408, train=False, dtype="bf16"),
        # a ragged training batch in float
        dict(name="gated_ragged", kind="gated", rows=1333, inter=1001, train=True, dtype="f32"),
        # a training batch
        dict(name="gated_train", kind="gated", rows=16384, inter=4096, train=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "experts", "route", "gated"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "linear":
        n = rng.choice([_log(rng, 1, 64), _log(rng, 64, 8192)])
        return dict(kind=kind, n=n, m=_log(rng, 256, 8192), k=_log(rng, 128, 8192), dtype=dtype)
    experts = _log(rng, 4, 128)
    topk, dropped = rng.randint(1, min(8, experts)), rng.random() < 0.4
    if kind == "experts":
        return dict(kind=kind, tokens=_log(rng, 1, 4096), topk=topk, experts=experts, m=_log(rng, 256, 4096),
                    k=_log(rng, 256, 4096), dropped=dropped, dtype=dtype)
    train = rng.random() < 0.6
    if kind == "route":
        return dict(kind=kind, tokens=_log(rng, 1, 8192), topk=topk, experts=experts, hidden=_log(rng, 256, 4096),
                    dropped=dropped, train=train, dtype="bf16" if dtype == "f32" else dtype)
    return dict(kind=kind, rows=_log(rng, 1, 16384), inter=_log(rng, 128, 4096), train=train,
                dtype=dtype)


# ---- inputs --------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ceil(a, b):
    return -(-a // b)


def _activations(g, rows, cols):
    """Normal entries, channels of uneven strength (a few strong ones), rows of uneven strength."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    ch = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    ch = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.004, ch * 20.0, ch)
    return x.mul_(ch).mul_(torch.exp(0.3 * torch.randn(rows, 1, generator=g, device="cuda")))


def _choices(g, tokens, topk, experts, dropped):
    """(ids, weights) of a router with experts of uneven popularity; with `dropped` the last eighth of the tokens is
    padding (ids -1)."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    logits += 0.5 * torch.randn(experts, generator=g, device="cuda")
    top = torch.topk(logits, topk, dim=1)
    ids = top.indices.to(torch.int32)
    if dropped:
        ids[tokens - tokens // 8:] = -1
    return ids.contiguous(), torch.softmax(top.values, dim=1).contiguous()


def _divide(x, s):
    # by a tensor: by a Python number torch multiplies with its reciprocal, which is not the same float
    return x / (s if torch.is_tensor(s) else torch.full((), s, device="cuda"))


def _codes(x):
    """(codes, scales) of the rows of a float tensor, the codes as floats: a scale is the float nearest to the row's
    largest magnitude over 127, a code the integer nearest to the float quotient of entry and scale (ties to even)."""
    s = _divide(x.abs().amax(dim=-1), 127.0).clamp_min(SMALLEST)
    return torch.round(_divide(x, s.unsqueeze(-1))).clamp_(-127.0, 127.0), s


def _weight(g, m, k):
    """(codes, scales) of a random m x k weight: rows of a multiple of 16 bytes, zeros after the k-th."""
    codes, scales = _codes(torch.randn(m, k, generator=g, device="cuda") / math.sqrt(k))
    padded = torch.zeros(m, _ceil(k, 16) * 16, dtype=torch.int8, device="cuda")
    padded[:, :k] = codes.to(torch.int8)
    return padded, scales


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dt = DT[case["dtype"]]
    if case["kind"] == "linear":
        s["x"] = _activations(g, case["n"], case["k"]).to(dt)
        s["w"], s["w_scales"] = _weight(g, case["m"], case["k"])
    elif case["kind"] == "experts":
        s["x"] = _activations(g, case["tokens"], case["k"]).to(dt)
        s["ids"], _ = _choices(g, case["tokens"], case["topk"], case["experts"], case["dropped"])
        parts = [_weight(g, case["m"], case["k"]) for _ in range(case["experts"])]
        s["w"], s["w_scales"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    elif case["kind"] == "route":
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        s["x"] = torch.randn(t, h, generator=g, device="cuda").to(dt)
        s["y"] = torch.randn(t * k, h, generator=g, device="cuda").to(dt)        # the experts' results, by row
        s["ids"], s["weights"] = _choices(g, t, k, case["experts"], case["dropped"])
        if case["train"]:
            s["dxs"] = torch.randn(t * k, h, generator=g, device="cuda").to(dt)
            s["dout"] = torch.randn(t, h, generator=g, device="cuda").to(dt)
            if own:
                for name in ("x", "y", "weights"):
                    s[name].requires_grad_()
    else:
        s["x"] = (1.5 * _activations(g, case["rows"], 2 * case["inter"])).to(dt)
        if case["train"]:
            s["dy"] = torch.randn(case["rows"], case["inter"], generator=g, device="cuda").to(dt)
            if own:
                s["x"].requires_grad_()
    if own and case["kind"] in ("linear", "experts"):
        from hpc_linear_algebra_amd import int8
        s["W"] = int8.RowScaled(s["w"], s["w_scales"], case["k"])
    return s


# ---- one pass ------------------------------------------------------------------------------------------

def _plain_sort(ids, experts):
    """(offsets, rows, place) of the assignments ids (tokens, topk) in the order of their experts, those of one expert
    in the order of the tokens: where each expert's rows begin, the assignment that stands at each row, and the row of
    each assignment.  Assignments to no expert come last."""
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < experts), flat, experts)
    at = torch.sort(flat, stable=True).indices
    place = torch.empty_like(at)
    place[at] = torch.arange(at.numel(), device="cuda")
    counts = (flat.unsqueeze(1) == torch.arange(experts, device="cuda")).sum(dim=0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)])
    return offsets, at, place.reshape(ids.shape)


def _plain_linear(s):
    codes, scales = _codes(s["x"].float())
    y = codes @ s["w"][:, :s["k"]].float().t()
    return (y * scales.unsqueeze(1) * s["w_scales"]).to(s["x"].dtype)


def _own_linear(s):
    from hpc_linear_algebra_amd import int8
    return int8.linear(s["x"], s["W"])


def _plain_experts(s):
    k, dt = s["k"], s["x"].dtype
    offsets, at, _ = _plain_sort(s["ids"], s["experts"])
    codes, scales = _codes(s["x"].float())
    at = at // s["topk"]
    y = torch.zeros(at.numel(), s["m"], dtype=dt, device="cuda")
    ends = offsets.tolist()
    for e in range(s["experts"]):
        mine = at[ends[e]:ends[e + 1]]
        if mine.numel():
            part = codes[mine] @ s["w"][e, :, :k].float().t()
            y[ends[e]:ends[e + 1]] = (part * scales[mine].unsqueeze(1) * s["w_scales"][e]).to(dt)
    return offsets.to(torch.int32), y


def _own_experts(s):
    from hpc_linear_algebra_amd import int8, moe
    order = moe.sort(s["ids"], s["experts"])
    x8 = int8.quantize(s["x"], rows=order.rows)
    return order.offsets, int8.gemm(s["W"], x8, offsets=order.offsets, dtype=s["dtype"])


def _plain_route(s):
    x, y, w = s["x"].float(), s["y"].float(), s["weights"]
    t, k, dt = s["tokens"], s["topk"], s["x"].dtype
    offsets, _, place = _plain_sort(s["ids"], s["experts"])
    real = (place < offsets[-1]).unsqueeze(2)
    xs = torch.zeros_like(y)
    xs[place] = torch.where(real, x.unsqueeze(1), 0.0)
    picked = torch.where(real, y[place], 0.0)
    out = offsets.to(torch.int32), place.to(torch.int32), xs.to(dt), (picked * w.unsqueeze(2)).sum(dim=1).to(dt)
    if not s["train"]:
        return out
    dxs, dout = s["dxs"].float(), s["dout"].float()
    dx = torch.where(real, dxs[place], 0.0).sum(dim=1)
    dy = torch.zeros_like(y)
    dy[place] = torch.where(real, dout.unsqueeze(1) * w.unsqueeze(2), 0.0)
    dw = (picked * dout.unsqueeze(1)).sum(dim=2)
    return *out, dx.to(dt), dy.to(dt), dw


def _own_route(s):
    from hpc_linear_algebra_amd import moe
    order = moe.sort(s["ids"], s["experts"])
    xs = moe.gather(s["x"], order)
    out = moe.combine(s["y"], s["weights"], order)
    got = order.offsets, order.place, xs, out
    if not s["train"]:
        return got
    return *got, *torch.autograd.grad([xs, out], [s["x"], s["y"], s["weights"]], [s["dxs"], s["dout"]])


def _plain_gated(s):
    x, inter = s["x"].float(), s["inter"]
    dt = s["x"].dtype
    g, u = x[:, :inter], x[:, inter:]
    y = (g / (1.0 + torch.exp(-g)) * u).to(dt)
    if not s["train"]:
        return y
    kept = []
    for half in (g, u):
        blocks = torch.nn.functional.pad(half, (0, _ceil(inter, BLK) * BLK - inter)).reshape(s["rows"], -1, BLK)
        codes, scales = _codes(blocks)
        kept.append((codes * scales.unsqueeze(2)).reshape(s["rows"], -1)[:, :inter])
    g, u = kept
    dy = s["dy"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    rest = 1.0 / (1.0 + torch.exp(g))
    return y, torch.cat([dy * u * sig * (1.0 + g * rest), dy * g * sig], dim=1).to(dt)


def _own_gated(s):
    from hpc_linear_algebra_amd import blocks
    y = blocks.gated(s["x"])
    if not s["train"]:
        return y
    return y, torch.autograd.grad(y, s["x"], s["dy"])[0]


def run(state):
    kind = state["kind"]
    if own:
        return {"linear": _own_linear, "experts": _own_experts, "route": _own_route, "gated": _own_gated}[kind](state)
    return {"linear": _plain_linear, "experts": _plain_experts, "route": _plain_route, "gated": _plain_gated}[kind](state)


# ---- the work a pass cannot do without -----------------------------------------------------------------

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["kind"] == "linear":
        n, m, k = case["n"], case["m"], case["k"]
        return {"bytes": es * n * k + m * k + 4 * m + es * n * m, "flops": 2 * n * m * k}
    if case["kind"] == "gated":
        r, i = case["rows"], case["inter"]
        b = 3 * es * r * i
        if case["train"]:       # the checkpoint is written and read: holding it is what the operator is for
            b += 3 * es * r * i + 2 * (2 * r * i + 8 * r * _ceil(i, BLK))
        return {"bytes": b, "flops": (24 if case["train"] else 6) * r * i}
    t, k, e = case["tokens"], case["topk"], case["experts"]
    live = t - t // 8 if case["dropped"] else t
    if case["kind"] == "experts":
        m, n = case["m"], case["k"]
        # experts that `live` independent choices of k out of e reach, on average
        reached = e * (1.0 - (1.0 - k / e) ** live)
        return {"bytes": es * t * n + reached * m * (n + 4) + es * t * k * m + 4 * t * k, "flops": 2 * live * k * m * n}
    h = case["hidden"]
    b = 8 * t * k + es * h * (t + t * k + live * k + t) + 4 * t * k
    if case["train"]:           # y is read once for both directions
        b += es * h * (live * k + t + t + t * k) + 4 * t * k
    return {"bytes": b, "flops": (7 if case["train"] else 2) * live * k * h}


# ---- the same from the definitions, in 64 bits ---------------------------------------------------------

def _exact_codes(x):
    """Codes and scales of rows of doubles: scale and quotient are float numbers."""
    s = (x.abs().amax(dim=1) / 127.0).float().double().clamp_min(SMALLEST)
    q = (x / s.unsqueeze(1)).float().double()
    low = torch.floor(q)
    up = (q - low > 0.5) | ((q - low == 0.5) & (torch.remainder(low, 2.0) == 1.0))
    return (low + up).clamp(-127.0, 127.0), s


def _exact_order(ids, experts):
    """Per expert the list of its assignments, and the list of those of none."""
    lists = [[] for _ in range(experts + 1)]
    for a, e in enumerate(ids.reshape(-1).tolist()):
        lists[e if 0 <= e < experts else experts].append(a)
    return lists


def _exact_offsets(lists):
    ends = [0]
    for one in lists[:-1]:
        ends.append(ends[-1] + len(one))
    return torch.tensor(ends, dtype=torch.int32)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "linear":
        codes, scales = _exact_codes(s["x"].double())
        w = s["w"][:, :case["k"]].double() * s["w_scales"].double().unsqueeze(1)
        return torch.mm(codes * scales.unsqueeze(1), w.t())
    if case["kind"] == "experts":
        lists = _exact_order(s["ids"], case["experts"])
        codes, scales = _exact_codes(s["x"].double())
        x = codes * scales.unsqueeze(1)
        y = torch.zeros(case["tokens"] * case["topk"], case["m"], dtype=torch.float64, device="cuda")
        at = 0
        for e, mine in enumerate(lists[:-1]):
            if mine:
                w = s["w"][e, :, :case["k"]].double() * s["w_scales"][e].double().unsqueeze(1)
                tokens = torch.tensor(mine, device="cuda") // case["topk"]
                y[at:at + len(mine)] = torch.mm(x[tokens], w.t())
                at += len(mine)
        return _exact_offsets(lists), y
    if case["kind"] == "route":
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        lists = _exact_order(s["ids"], case["experts"])
        order = [a for one in lists for a in one]
        place = torch.empty(t * k, dtype=torch.int64)
        place[torch.tensor(order, dtype=torch.int64)] = torch.arange(t * k)
        end = t * k - len(lists[-1])
        at = torch.tensor(order[:end], dtype=torch.int64, device="cuda")
        token, w = at // k, s["weights"].detach().double().reshape(-1)[at].unsqueeze(1)
        x, y = s["x"].detach().double(), s["y"].detach().double()[:end]
        xs = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        xs[:end] = x[token]
        out = torch.zeros(t, h, dtype=torch.float64, device="cuda").index_add_(0, token, y * w)
        got = [_exact_offsets(lists), place.reshape(t, k).to(torch.int32), xs, out]
        if case["train"]:
            dout = s["dout"].double()[token]
            dx = torch.zeros(t, h, dtype=torch.float64, device="cuda").index_add_(0, token, s["dxs"].double()[:end])
            dy = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
            dy[:end] = dout * w
            dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
            dw[at] = (dout * y).sum(dim=1)
            got += [dx, dy, dw.reshape(t, k)]
        return tuple(got)
    inter = case["inter"]
    x = s["x"].detach().double()
    y = x[:, :inter] * torch.sigmoid(x[:, :inter]) * x[:, inter:]
    if not case["train"]:
        return y
    kept = torch.empty_like(x)
    for first in (0, inter):
        for c in range(0, inter, BLK):
            piece = slice(first + c, first + min(c + BLK, inter))
            codes, scales = _exact_codes(x[:, piece])
            kept[:, piece] = codes * scales.unsqueeze(1)
    g, u, dy = kept[:, :inter], kept[:, inter:], s["dy"].double()
    sig = torch.sigmoid(g)
    return y, torch.cat([dy * u * sig * (1.0 + g * torch.sigmoid(-g)), dy * g * sig], dim=1)
