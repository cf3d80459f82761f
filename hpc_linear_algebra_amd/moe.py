"""Mixtures of experts (torch plumbing around tlr_moe and tlr_expert_*,
include/tlrgemm.h).

MoELayer is a whole layer for a few tokens: router, softmax, top-k, gated experts
(silu), weighted sum.  For any number of tokens, trained ones among them:

    order = moe.sort(ids, experts)              # a row for each choice, by expert
    xs = moe.gather(x, order)                   # tokens to their rows; differentiable
    ...                                         # each expert on its rows
    out = moe.combine(y, weights, order)        # rows back to tokens; differentiable

and Int8Experts, which runs the experts between the two on 8-bit integers.  Within
torch.jit.trace, which records torch's own operations alone, these are refused.  A backward
pass in a captured graph takes torch.autograd.grad, or leaves that no live eager graph
holds: their accumulation belongs to its stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import tlrgemm as T
from . import int8
from .blocks import binding, gated, quantize

MAX_TOKENS = 256
_DT = {torch.float16: T.TLR_F16, torch.bfloat16: T.TLR_BF16}
_NAME = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}


def quantize_experts(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of expert weights (experts, rows, k), k a multiple of 16,
    as MoELayer takes them: e4m3 with 128 x 128 block scales, done once when
    the weights are loaded."""
    if w.dim() != 3 or w.shape[2] % 16:
        raise ValueError("quantize_experts: weights are (experts, rows, k), k a multiple of 16")
    parts = [quantize(e, block=128)[0] for e in w]
    return torch.stack([p.codes.view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn), torch.stack([p.scales for p in parts])


class MoELayer:
    """One layer's weights with the workspace of up to ``max_tokens`` tokens.

    router     (experts, hidden), float16 or bfloat16: the type of x and y
    gate_up    (experts, 2*inter, hidden): inter gate rows, then inter up rows
    down       (experts, hidden, inter)
    The expert weights have the router's type, or are float8_e4m3fn codes with
    128 x 128 block scales (as blocks.quantize gives them for one expert):
    gate_up_scales (experts, ceil(hidden/128), ceil(2*inter/128)) and
    down_scales (experts, ceil(inter/128), ceil(hidden/128)), float32.
    hidden and inter are multiples of 16, every tensor is contiguous.  The layer
    keeps the memory that the tensors have when it is made: changes in place are
    seen, a tensor that is given other memory (``.data = ``) afterwards is not.

    Calls share the layer's workspace, which is cleared on the stream that is
    current when the layer is made: making it and calling it run in the order of
    one stream, or with events between them.  Called on another stream than that,
    the layer has to live until the call's work has ended.

    There is no backward pass: where gradients are on, an x or weights that
    require one are refused, and an x with a tangent of forward mode always, as is
    a call within torch.jit.trace.
    """

    def __init__(self, router: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, topk: int,
                 max_tokens: int = 64, normalize: bool = True, gate_up_scales: Optional[torch.Tensor] = None,
                 down_scales: Optional[torch.Tensor] = None):
        if router.dim() != 2 or gate_up.dim() != 3 or down.dim() != 3 or router.dtype not in _DT:
            raise ValueError("MoELayer: router (experts, hidden) in float16 or bfloat16, gate_up and down of 3 dimensions")
        experts, hidden = router.shape
        inter = down.shape[2]
        if tuple(gate_up.shape) != (experts, 2 * inter, hidden) or tuple(down.shape) != (experts, hidden, inter):
            raise ValueError("MoELayer: gate_up is (experts, 2*inter, hidden) and down (experts, hidden, inter)")
        e8 = gate_up.dtype == torch.float8_e4m3fn
        if gate_up.dtype != down.dtype or not (e8 or gate_up.dtype == router.dtype):
            raise ValueError("MoELayer: expert weights are of the router's type or float8_e4m3fn")
        tensors = [router, gate_up, down]
        if e8:
            up = lambda n: -(-n // 128)   # noqa: E731
            for s, shape in ((gate_up_scales, (experts, up(hidden), up(2 * inter))),
                             (down_scales, (experts, up(inter), up(hidden)))):
                if s is None or s.dtype != torch.float32 or tuple(s.shape) != shape:
                    raise ValueError(f"MoELayer: 8-bit weights need float32 scales of shape {shape}")
            tensors += [gate_up_scales, down_scales]
        elif gate_up_scales is not None or down_scales is not None:
            raise ValueError("MoELayer: scales belong to 8-bit weights")
        self.device = router.device
        if any(t.device != self.device or not t.is_cuda or not t.is_contiguous() for t in tensors):
            raise ValueError("MoELayer: contiguous tensors on one GPU are needed")
        self.dtype, self.hidden, self.inter, self.experts, self.topk = router.dtype, hidden, inter, experts, int(topk)
        self.max_tokens = int(max_tokens)
        self._trained = any(t.requires_grad for t in tensors)
        self._keep = [t.detach() for t in tensors]       # the memory that the addresses below belong to
        dt = _DT[router.dtype]
        self._c = T.tlr_moe_layer(hidden, inter, experts, self.topk, dt, T.TLR_E4M3 if e8 else dt, 1 if normalize else 0,
                                  0, router.data_ptr(), gate_up.data_ptr(), down.data_ptr(),
                                  gate_up_scales.data_ptr() if e8 else None, down_scales.data_ptr() if e8 else None)
        self._ws = torch.empty(max(256, T.tlr_moe_workspace_bytes(self._c, self.max_tokens)), dtype=torch.uint8,
                               device=self.device)
        self._at, self._ws_at, self._ws_bytes = ctypes.addressof(self._c), self._ws.data_ptr(), self._ws.numel()
        with torch.cuda.device(self.device):
            T.tlr_moe_init(self._c, self._ws_at, self._ws_bytes, torch.cuda.current_stream().cuda_stream)

    # Calls use the addresses of these two: neither can be replaced, and the first is handed out as a copy.
    @property
    def c(self) -> T.tlr_moe_layer:
        """What the C ABI takes."""
        return T.tlr_moe_layer.from_buffer_copy(self._c)

    @property
    def ws(self) -> torch.Tensor:
        """The workspace."""
        return self._ws

    def __call__(self, x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(y, ids, weights) of x (tokens, hidden): the layer's output in x's
        type, the chosen experts (int32) and their probabilities (float32).  ids
        and weights are views of one allocation: keeping or saving either keeps or
        saves both."""
        if torch.is_grad_enabled() and (x.requires_grad or self._trained):
            raise RuntimeError("MoELayer has no backward pass: call it under torch.no_grad() or on detached tensors")
        if x.device != self.device:
            raise ValueError(f"MoELayer: x is on {self.device}")
        got = binding().moe(self._at, x, self.max_tokens, self._ws_at, self._ws_bytes)
        if type(got) is int:
            T._check(got, "tlr_moe")
        return got


class Order(NamedTuple):
    """Assignments of tokens to experts, sorted by expert.

    offsets  (experts + 1,) int32: expert e has rows offsets[e] .. offsets[e+1] - 1;
             rows from offsets[-1] on belong to none
    place    (tokens, topk) int32: the row of each assignment
    rows     (tokens * topk,) int32: the token of each row, -1 for rows of no expert
    """
    offsets: torch.Tensor
    place: torch.Tensor
    rows: torch.Tensor


def sort(ids: torch.Tensor, experts: int) -> Order:
    """A row for each assignment ids (tokens, topk), int32 or int64: by expert, those
    of one expert in the order of the tokens, those to no expert (an id that is none
    of 0 .. experts - 1: padding, experts elsewhere) last.  The results are views of
    one allocation.  Up to 1024 experts, topk up to 64, 2^24 assignments."""
    got = binding().sort(ids, experts)
    if type(got) is int:
        T._check(got, "tlr_expert_sort")
    return Order(*got)


def gather(x: torch.Tensor, order: Order) -> torch.Tensor:
    """Each token x (tokens, hidden) at the rows of its assignments, (tokens * topk,
    hidden); rows of no expert are zeros.  The gradient of a token is the sum of its
    rows', in float, rounded once, in the order of its assignments; rows of no expert
    add nothing.  No double backward, no forward mode: a tangent is refused."""
    got = binding().gather(x, order.place, order.offsets)
    if type(got) is int:
        T._check(got, "tlr_expert_gather")
    return got


def combine(y: torch.Tensor, weights: Optional[torch.Tensor], order: Order) -> torch.Tensor:
    """The rows y (tokens * topk, hidden) of each token's assignments added with its
    weights (tokens, topk), float32 (None: 1): (tokens, hidden) in y's type, sums in
    float in the order of the assignments.  Rows of no expert are not read.  Gradients
    of y (zeros for rows of no expert) and of the weights; y's memory is kept for the
    latter alone, though a change of y in place is always noticed.  No double backward, no
    forward mode: a tangent is refused."""
    got = binding().combine(y, weights, order.place, order.offsets)
    if type(got) is int:
        T._check(got, "tlr_expert_combine")
    return got


class Int8Experts:
    """Gated experts (silu) on 8-bit integers, for any number of tokens.

    gate_up  int8.RowScaled (experts, 2*inter, hidden): inter gate rows, then inter
             up rows, a scale for each
    down     int8.RowScaled (experts, hidden, inter)

    A call sorts the tokens by expert, quantizes them on the way to their rows,
    multiplies each expert's rows with its weights, and the same for the gated
    results; every product rounds to x's type.  No backward pass, no forward mode:
    where gradients are on, x or weights that require one are refused, and a tangent
    always.
    """

    def __init__(self, gate_up: int8.RowScaled, down: int8.RowScaled):
        if gate_up.codes.dim() != 3 or down.codes.dim() != 3:
            raise ValueError("Int8Experts: weights are (experts, rows, k)")
        experts, hidden, inter = gate_up.codes.shape[0], gate_up.k, down.k
        if gate_up.rows != 2 * inter or down.rows != hidden or down.codes.shape[0] != experts:
            raise ValueError("Int8Experts: gate_up is (experts, 2*inter, hidden) and down (experts, hidden, inter)")
        self.gate_up, self.down, self.experts, self.hidden = gate_up, down, experts, hidden

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        """The experts' outputs for x (tokens, hidden), added with the router's
        weights (tokens, topk), float32, for its choices ids; in x's type."""
        if torch.is_grad_enabled() and (x.requires_grad or weights.requires_grad):
            raise RuntimeError("Int8Experts has no backward pass: call it under torch.no_grad() or on detached tensors")
        for t in (x, weights):
            binding().no_tangent("Int8Experts", t)
        if x.dim() != 2 or x.shape[1] != self.hidden or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
            raise ValueError(f"Int8Experts: x is (tokens, {self.hidden}) and ids (tokens, topk)")
        dtype = _NAME.get(x.dtype)
        if dtype is None:
            raise ValueError("Int8Experts: x is float32, float16 or bfloat16")
        order = sort(ids, self.experts)
        h = gated(int8.gemm(self.gate_up, int8.quantize(x, rows=order.rows), offsets=order.offsets, dtype=dtype))
        return combine(int8.gemm(self.down, int8.quantize(h), offsets=order.offsets, dtype=dtype), weights, order)
