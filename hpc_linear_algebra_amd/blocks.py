"""Block-scaled 8-bit floating point matrices and their products (torch plumbing
around tlr_block_quantize and tlr_block_gemm, include/tlrgemm.h).

    W8, W8t = blocks.quantize(W, block=128, transposed=True)    # a weight, once per update
    x8, x8t = blocks.quantize(x, transposed=True)               # activations, 1 x 128 blocks
    y = blocks.gemm(W8, x8, fast=True)                          # x W^T
    dy8, dy8t = blocks.quantize(dy, transposed=True)
    dx = blocks.gemm(W8t, dy8, fast=True)                       # dy W
    dW = blocks.gemm(x8t, dy8t, dtype="f32")                    # dy^T x

``linear`` wraps these three products as one differentiable function; ``gated``
is the activation between two of them, its input kept in 8 bits as well.  Every
call runs on torch's current stream of the operands' device.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import tlrgemm as T

BLOCK = 128
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_CODE = {torch.float8_e4m3fn: T.TLR_E4M3, torch.float8_e5m2: T.TLR_E5M2}
_DT = {torch.float32: T.TLR_F32, torch.float16: T.TLR_F16, torch.bfloat16: T.TLR_BF16}
_FMT = {"e4m3": T.TLR_E4M3, "e5m2": T.TLR_E5M2}
_NEW = {"f32": T.TLR_F32, "f16": T.TLR_F16, "bf16": T.TLR_BF16}


@functools.lru_cache(None)
def binding():
    """The extension module, calling the entries of the loaded library."""
    lib = T.lib()
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError("the extension module is not built: python -m hpc_linear_algebra_amd.build") from e
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value   # noqa: E731
    _binding.connect(*(address(getattr(lib, name)) for name in (
        "tlr_block_quantize", "tlr_block_gemm", "tlr_moe", "tlr_row_quantize", "tlr_row_gemm_workspace_bytes", "tlr_row_gemm",
        "tlr_row_linear_workspace_bytes", "tlr_row_linear", "tlr_expert_sort_workspace_bytes", "tlr_expert_sort",
        "tlr_expert_gather", "tlr_expert_combine", "tlr_expert_combine_grad", "tlr_gated", "tlr_gated_grad")))
    return _binding


@functools.lru_cache(4096)
def _gemm_workspace(m: int, n: int, k: int, flags: int) -> int:
    return int(T.tlr_block_gemm_plan(m, n, k, flags).workspace)


class BlockScaled:
    """A rows x k matrix of 8-bit codes with block scales.

    codes    (rows, ld) float8 tensor, rows contiguous, ld a multiple of 16
    scales   (ceil(k/128), row blocks) float32 tensor: the scale of row block r
             and column block q is scales[q, r]
    block    rows of a block: 1 or 128
    """

    __slots__ = ("codes", "scales", "rows", "k", "block")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, k: int, block: int):
        self.codes, self.scales, self.rows, self.k, self.block = codes, scales, rows, k, block
        self.c      # its checks

    @property
    def c(self) -> T.tlr_block_matrix:
        """What the C ABI takes, made anew from the tensors as they are: it points into them and does not keep them."""
        codes, scales, rows, k, block = self.codes, self.scales, self.rows, self.k, self.block
        if codes.dtype not in _CODE or codes.dim() != 2:
            raise ValueError("codes: a 2-d float8_e4m3fn or float8_e5m2 tensor is needed")
        if block not in (1, BLOCK):
            raise ValueError(f"blocks are 1 or {BLOCK} rows high, not {block}")
        if scales.dtype != torch.float32 or scales.dim() != 2 or scales.device != codes.device:
            raise ValueError("scales: a 2-d float32 tensor on the codes' device is needed")
        nq, nr = -(-k // BLOCK), rows if block == 1 else -(-rows // BLOCK)
        ld = codes.stride(0) if codes.shape[0] > 1 else max(codes.stride(0), codes.shape[1])
        lds = scales.stride(0) if scales.shape[0] > 1 else max(scales.stride(0), nr)
        if codes.shape[0] != rows or codes.shape[1] < k or (codes.shape[1] > 1 and codes.stride(1) != 1):
            raise ValueError(f"codes: {rows} contiguous rows of {k} entries are needed")
        if rows and k and codes.storage_offset() + (rows - 1) * ld + -(-k // 16) * 16 > codes.untyped_storage().nbytes():
            raise ValueError("codes: every row has to be readable up to a multiple of 16 entries")
        if tuple(scales.shape) != (nq, nr) or (nr > 1 and scales.stride(1) != 1):
            raise ValueError(f"scales: shape {(nq, nr)}, rows contiguous, is needed")
        return T.tlr_block_matrix(codes.data_ptr(), scales.data_ptr(), ld, lds, block, _CODE[codes.dtype])

    def dequantize(self) -> torch.Tensor:
        """The (rows, k) float32 matrix that the codes and scales stand for."""
        s = self.scales.t().repeat_interleave(BLOCK, dim=1)[:, :self.k]
        if self.block == BLOCK:
            s = s.repeat_interleave(BLOCK, dim=0)[:self.rows]
        return self.codes[:, :self.k].float() * s


def _made(codes: torch.Tensor, scales: torch.Tensor, rows: int, k: int, block: int) -> BlockScaled:
    q = BlockScaled.__new__(BlockScaled)        # right by construction: the checks cost more than the launch
    q.codes, q.scales, q.rows, q.k, q.block = codes, scales, rows, k, block
    return q


def quantize(x: torch.Tensor, block: int = 1, fmt: str = "e4m3", straight: bool = True,
             transposed: bool = False) -> Tuple[Optional[BlockScaled], Optional[BlockScaled]]:
    """(codes of x, codes of x^T), each None unless wanted, from one read of x.

    x is a 2-d float32, float16 or bfloat16 tensor whose rows are contiguous
    (any row stride).  block 1: a scale for every 128 entries of a row of the
    result; block 128: one for every 128 x 128 tile.  Codes and scales carry no
    gradient, whatever x does: linear is the differentiable function.  A result's
    codes and scales are views of one allocation, codes first: keeping or saving
    either keeps or saves both; ``clone()`` one to part them."""
    f8 = _FMT.get(fmt)
    if f8 is None or block not in (1, BLOCK) or not (straight or transposed):
        raise ValueError("quantize: fmt is e4m3 or e5m2, block 1 or 128, and a result has to be wanted")
    got = binding().quantize(x, f8, block, straight, transposed)
    if type(got) is int:
        T._check(got, "tlr_block_quantize")
    rows, k = x.shape
    return (_made(got[0], got[1], rows, k, block) if straight else None,
            _made(got[2], got[3], k, rows, block) if transposed else None)


def gemm(A: BlockScaled, B: BlockScaled, out: Optional[torch.Tensor] = None, alpha: float = 1.0, beta: float = 0.0,
         dtype: str = "bf16", fast: bool = False) -> torch.Tensor:
    """alpha B A^T + beta out, a (B.rows, A.rows) tensor: column-major A.rows x
    B.rows to the C ABI, x W^T to a linear layer with A = W and B = x.  Without
    ``out`` the result is a new tensor of type ``dtype`` (beta must be 0).  It has
    no gradient: where gradients are on, scales or an out that require one are
    refused.

    Sums are held in float.  ``fast`` sums within a block on the 8-bit matrix
    instructions, which cut every product below 2^-13 of the block's largest
    one: 1.4e-5 of the result on normally distributed data, 5e-5 to 7e-5 where
    one column of each block is ten to a hundred times the others on both sides,
    all of it where larger products cancel.  For results in 16 bits whose operands
    allow it."""
    if A.k != B.k:
        raise ValueError(f"gemm: contraction lengths differ ({A.k} and {B.k})")
    new = _NEW.get(dtype)
    if new is None:
        raise ValueError(f"gemm: dtype is f32, f16 or bf16, not {dtype!r}")
    device = A.codes.device
    if B.codes.device != device:
        raise ValueError("gemm: operands on different devices")
    m, n = A.rows, B.rows
    if out is None:
        if beta != 0.0:
            raise ValueError("gemm: beta needs an out to add to")
    elif tuple(out.shape) != (n, m) or out.dtype not in _DT or out.device != device or (m > 1 and out.stride(1) != 1):
        raise ValueError(f"gemm: out has to be a ({n}, {m}) float32, float16 or bfloat16 tensor with contiguous rows")
    flags = T.TLR_BLOCK_FAST if fast else 0
    got = binding().gemm(A.codes, A.scales, A.block, B.codes, B.scales, B.block, m, n, A.k, alpha, beta, out, new,
                         flags, _gemm_workspace(m, n, A.k, flags) if alpha != 0.0 else 0)
    if type(got) is int:
        T._check(got, "tlr_block_gemm")
    return got


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x as a matrix of contiguous rows, copied only where they are not."""
    x = x.reshape(x.shape[:-1].numel(), x.shape[-1])
    return x if x.stride(1) == 1 else x.contiguous()


def _parts(q: Optional[BlockScaled]) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    return (q.codes, q.scales) if q is not None else (None, None)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, grad_fmt, fast):
        x2 = _rows(x)
        need_x, need_w = ctx.needs_input_grad[:2]
        x8, x8t = quantize(x2, transposed=need_w)
        w8, w8t = quantize(_rows(w), block=BLOCK, transposed=need_x)
        ctx.save_for_backward(*_parts(x8t), *_parts(w8t))
        ctx.grad_fmt, ctx.fast = grad_fmt, fast
        ctx.shape, ctx.types = x.shape, (x.dtype, w.dtype)
        # no view of another tensor is returned: autograd refuses changes of one in place
        out = torch.empty((*x.shape[:-1], w.shape[0]), dtype=x.dtype, device=x.device)
        gemm(w8, x8, out=out.view(x2.shape[0], w.shape[0]), fast=fast and x.dtype != torch.float32)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad[:2]
        dx = dw = None
        x_codes, x_scales, w_codes, w_scales = ctx.saved_tensors
        if need_x or need_w:
            dy = _rows(dy)
            tokens, features = dy.shape
            width = ctx.shape[-1]
            d8, d8t = quantize(dy, fmt=ctx.grad_fmt, straight=need_x, transposed=need_w)
            if need_x:
                dx = torch.empty((tokens, width), dtype=ctx.types[0], device=dy.device)
                w8t = _made(w_codes, w_scales, width, features, BLOCK)
                dx = gemm(w8t, d8, out=dx, fast=ctx.fast and dx.dtype != torch.float32).reshape(ctx.shape)
            if need_w:
                dw = torch.empty((features, width), dtype=ctx.types[1], device=dy.device)
                x8t = _made(x_codes, x_scales, width, tokens, 1)
                gemm(x8t, d8t, out=dw, fast=ctx.fast and dw.dtype != torch.float32)
        return dx, dw, None, None


def linear(x: torch.Tensor, w: torch.Tensor, grad_fmt: str = "e4m3", fast: bool = False) -> torch.Tensor:
    """x W^T (x: (..., k), w: (features, k)) with both operands, and in the
    backward pass dy, quantized to block-scaled 8 bits: x and dy in 1 x 128
    blocks along each contraction, w in 128 x 128 blocks.  The forward pass
    saves the transposed codes, a byte an entry, in place of x and w.  Sums are
    held in float; ``fast`` sums those of the three results that have 16 bits on
    the 8-bit instructions (see gemm).  No double backward.  In a captured graph
    take torch.autograd.grad, or leaves that no live eager graph holds: their
    accumulation belongs to its stream."""
    if x.shape[-1:] != w.shape[1:] or w.dim() != 2:
        raise ValueError("linear: x is (..., k) and w (features, k)")
    if grad_fmt not in FORMATS:
        raise ValueError("linear: grad_fmt is e4m3 or e5m2")
    return _Linear.apply(x, w, grad_fmt, fast)


def gated_forward(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, codes, scales) of a 2-d x: y = silu(gate) * up, and x as int8 codes
    (rows, 2, inter rounded up to 16) with a float32 scale for every 128 of them
    (rows, 2, ceil(inter/128)), gate first.  The scale is the largest magnitude over
    127, codes behind the last entry are zeros.  Codes and scales are views of one
    allocation.  None of them carries a gradient, whatever x does, and a tangent of
    forward mode is refused: gated is the function for autograd."""
    got = binding().gated_forward(x)
    if type(got) is int:
        T._check(got, "tlr_gated")
    return got


def gated_backward(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """The gradient of gated_forward's x, in dy's type, taken at the values that
    the codes and scales stand for."""
    got = binding().gated_backward(dy, codes, scales)
    if type(got) is int:
        T._check(got, "tlr_gated_grad")
    return got


def gated(x: torch.Tensor) -> torch.Tensor:
    """silu(gate) * up for x (..., 2*inter) whose last dimension holds `inter`
    gate entries, then `inter` up entries: (..., inter), in x's type.

    Where x requires a gradient it is kept for the backward pass as int8 codes with
    one scale for every 128 entries, a byte an entry in place of x; the gradient is
    that at the values the codes stand for (off by at most the block's largest
    magnitude / 254).  A block that holds an infinity or a NaN has NaN gradients.
    No double backward, no forward mode: a tangent is refused, and a call within
    torch.jit.trace.  In a captured graph take torch.autograd.grad, or leaves that no
    live eager graph holds: their accumulation belongs to its stream."""
    got = binding().gated(x)
    if type(got) is int:
        T._check(got, "tlr_gated")
    return got
