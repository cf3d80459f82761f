"""Block-scaled 8-bit floating point matrices and their products (torch plumbing
around tlr_block_quantize and tlr_block_gemm, include/tlrgemm.h).

    W8, W8t = blocks.quantize(W, block=128, transposed=True)    # a weight, once per update
    x8, x8t = blocks.quantize(x, transposed=True)               # activations, 1 x 128 blocks
    y = blocks.gemm(W8, x8, fast=True)                          # x W^T
    dy8, dy8t = blocks.quantize(dy, transposed=True)
    dx = blocks.gemm(W8t, dy8, fast=True)                       # dy W
    dW = blocks.gemm(x8t, dy8t, dtype="f32")                    # dy^T x

``linear`` wraps these three products as one differentiable function.  Every
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
_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


_raw_stream = torch._C._cuda_getCurrentRawStream      # 0.1 us, the stream object's way 2.7
_device = torch._C._cuda_getDevice                    # what torch.cuda.current_device asks once torch is set up


def call(device: torch.device, f, *args) -> int:
    """f(*args, torch's current stream of the device) with that device current.
    A decode step is bound by what the host does between launches: the guard is
    entered only where it changes something."""
    index = device.index
    if _device() == index:
        return f(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return f(*args, _raw_stream(index))


_lib = functools.lru_cache(None)(T.lib)
_gemm_workspace = functools.lru_cache(4096)(T.tlr_block_gemm_workspace_bytes)      # of the sizes alone


class BlockScaled:
    """A rows x k matrix of 8-bit codes with block scales.

    codes    (rows, ld) float8 tensor, rows contiguous, ld a multiple of 16
    scales   (ceil(k/128), row blocks) float32 tensor: the scale of row block r
             and column block q is scales[q, r]
    block    rows of a block: 1 or 128
    """

    __slots__ = ("codes", "scales", "rows", "k", "block", "_c")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, k: int, block: int):
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
        self.codes, self.scales, self.rows, self.k, self.block = codes, scales, rows, k, block
        self._c = T.tlr_block_matrix(codes.data_ptr(), scales.data_ptr(), ld, lds, block, _CODE[codes.dtype])

    @property
    def c(self) -> T.tlr_block_matrix:
        """What the C ABI takes; made when a product first asks for it."""
        if self._c is None:
            codes, scales = self.codes, self.scales
            self._c = T.tlr_block_matrix(codes.data_ptr(), scales.data_ptr(), codes.shape[1], scales.shape[1], self.block,
                                         _CODE[codes.dtype])
        return self._c

    def dequantize(self) -> torch.Tensor:
        """The (rows, k) float32 matrix that the codes and scales stand for."""
        s = self.scales.t().repeat_interleave(BLOCK, dim=1)[:, :self.k]
        if self.block == BLOCK:
            s = s.repeat_interleave(BLOCK, dim=0)[:self.rows]
        return self.codes[:, :self.k].float() * s


def _empty(rows: int, k: int, block: int, dt: torch.dtype, device) -> BlockScaled:
    q = BlockScaled.__new__(BlockScaled)        # right by construction: the checks cost more than the launch
    nr = rows if block == 1 else -(-rows // BLOCK)
    q.codes = torch.empty((rows, -(-k // 16) * 16), dtype=dt, device=device)
    q.scales = torch.empty((-(-k // BLOCK), nr), dtype=torch.float32, device=device)
    q.rows, q.k, q.block, q._c = rows, k, block, None
    return q


def _result(q: Optional[BlockScaled]):
    """(codes, ld, scales, lds) of a result of _empty for the C ABI."""
    if q is None:
        return None, 0, None, 0
    codes, scales = q.codes, q.scales
    return codes.data_ptr() or None, codes.shape[1], scales.data_ptr() or None, scales.shape[1]


def quantize(x: torch.Tensor, block: int = 1, fmt: str = "e4m3", straight: bool = True,
             transposed: bool = False) -> Tuple[Optional[BlockScaled], Optional[BlockScaled]]:
    """(codes of x, codes of x^T), each None unless wanted, from one read of x.

    x is a 2-d float32, float16 or bfloat16 tensor whose rows are contiguous
    (any row stride).  block 1: a scale for every 128 entries of a row of the
    result; block 128: one for every 128 x 128 tile."""
    dt = _DT.get(x.dtype)
    if dt is None or x.dim() != 2 or not x.is_cuda:
        raise ValueError("quantize: a 2-d float32, float16 or bfloat16 tensor on a GPU is needed")
    f8 = FORMATS.get(fmt)
    if f8 is None or block not in (1, BLOCK) or not (straight or transposed):
        raise ValueError("quantize: fmt is e4m3 or e5m2, block 1 or 128, and a result has to be wanted")
    rows, k = x.shape
    ldx, step = x.stride()
    if k > 1 and step != 1:
        raise ValueError("quantize: the rows of x have to be contiguous")
    if rows <= 1:
        ldx = max(ldx, k, 1)
    device = x.device
    a = _empty(rows, k, block, f8, device) if straight else None
    b = _empty(k, rows, block, f8, device) if transposed else None
    st = call(device, _lib().tlr_block_quantize, dt, _FMT[fmt], block, rows, k, x.data_ptr() or None, ldx, *_result(a),
              *_result(b))
    if st:
        T._check(st, "tlr_block_quantize")
    return a, b


def gemm(A: BlockScaled, B: BlockScaled, out: Optional[torch.Tensor] = None, alpha: float = 1.0, beta: float = 0.0,
         dtype: str = "bf16", fast: bool = False) -> torch.Tensor:
    """alpha B A^T + beta out, a (B.rows, A.rows) tensor: column-major A.rows x
    B.rows to the C ABI, x W^T to a linear layer with A = W and B = x.  Without
    ``out`` the result is a new tensor of type ``dtype`` (beta must be 0).

    Sums are held in float.  ``fast`` sums within a block on the 8-bit matrix
    instructions, which cut every product below 2^-13 of the block's largest
    one: about 2e-5 of the result, for results in 16 bits."""
    if A.k != B.k:
        raise ValueError(f"gemm: contraction lengths differ ({A.k} and {B.k})")
    device = A.codes.device
    if B.codes.device != device:
        raise ValueError("gemm: operands on different devices")
    m, n = A.rows, B.rows
    if out is None:
        if beta != 0.0:
            raise ValueError("gemm: beta needs an out to add to")
        out = torch.empty((n, m), dtype=_TORCH[dtype], device=device)
    elif tuple(out.shape) != (n, m) or out.dtype not in _DT or out.device != device or (m > 1 and out.stride(1) != 1):
        raise ValueError(f"gemm: out has to be a ({n}, {m}) float32, float16 or bfloat16 tensor with contiguous rows")
    ldc = out.stride(0) if n > 1 else max(out.stride(0), m, 1)
    nws = _gemm_workspace(m, n, A.k)
    ws = torch.empty(nws, dtype=torch.uint8, device=device) if nws else None
    st = call(device, _lib().tlr_block_gemm, _DT[out.dtype], m, n, A.k, alpha, ctypes.byref(A.c), ctypes.byref(B.c),
              beta, out.data_ptr() or None, ldc, T.TLR_BLOCK_FAST if fast else 0, ws.data_ptr() if nws else None, nws)
    if st:
        T._check(st, "tlr_block_gemm")
    return out


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, grad_fmt):
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        need_x, need_w = ctx.needs_input_grad[:2]
        x8, x8t = quantize(x2, transposed=need_w)
        w8, w8t = quantize(w.contiguous(), block=BLOCK, transposed=need_x)
        ctx.x8t, ctx.w8t, ctx.grad_fmt = x8t, w8t, grad_fmt
        ctx.shape, ctx.types = x.shape, (x.dtype, w.dtype)
        out = torch.empty((x2.shape[0], w.shape[0]), dtype=x.dtype, device=x.device)
        return gemm(w8, x8, out=out, fast=x.dtype != torch.float32).reshape(*x.shape[:-1], w.shape[0])

    @staticmethod
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad[:2]
        dx = dw = None
        if need_x or need_w:
            dy = dy.reshape(-1, dy.shape[-1]).contiguous()
            d8, d8t = quantize(dy, fmt=ctx.grad_fmt, straight=need_x, transposed=need_w)
            if need_x:
                dx = torch.empty((dy.shape[0], ctx.shape[-1]), dtype=ctx.types[0], device=dy.device)
                dx = gemm(ctx.w8t, d8, out=dx, fast=dx.dtype != torch.float32).reshape(ctx.shape)
            if need_w:
                dw = torch.empty((dy.shape[1], ctx.shape[-1]), dtype=ctx.types[1], device=dy.device)
                gemm(ctx.x8t, d8t, out=dw, fast=dw.dtype != torch.float32)
        return dx, dw, None


def linear(x: torch.Tensor, w: torch.Tensor, grad_fmt: str = "e4m3") -> torch.Tensor:
    """x W^T (x: (..., k), w: (features, k)) with both operands, and in the
    backward pass dy, quantized to block-scaled 8 bits: x and dy in 1 x 128
    blocks along each contraction, w in 128 x 128 blocks.  The forward pass
    keeps the transposed codes, a byte an entry, in place of x and w.  Results
    in 16 bits are summed with ``fast`` (see gemm), float32 ones in float.  No
    double backward."""
    if x.shape[-1:] != w.shape[1:] or w.dim() != 2:
        raise ValueError("linear: x is (..., k) and w (features, k)")
    if grad_fmt not in FORMATS:
        raise ValueError("linear: grad_fmt is e4m3 or e5m2")
    return _Linear.apply(x, w, grad_fmt)
