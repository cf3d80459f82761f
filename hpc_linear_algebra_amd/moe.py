"""A mixture-of-experts layer for a few tokens (torch plumbing around tlr_moe,
include/tlrgemm.h): router, softmax, top-k, gated experts (silu), weighted sum.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import tlrgemm as T
from .blocks import binding, quantize

MAX_TOKENS = 256
_DT = {torch.float16: T.TLR_F16, torch.bfloat16: T.TLR_BF16}


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
    require one are refused.
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
