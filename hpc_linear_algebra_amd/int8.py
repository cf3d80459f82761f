"""8-bit integer matrices with a scale for each row, and their products (torch
plumbing around tlr_row_quantize and tlr_row_gemm, include/tlrgemm.h).

    W8 = int8.quantize(W)                       # a weight, once: a scale for each output channel
    y = int8.linear(x, W8)                      # x W^T, x quantized in the call, a scale for each token
    x8 = int8.quantize(x)
    y = int8.gemm(W8, x8)                       # the same from codes
    E8 = int8.quantize(experts)                 # (experts, rows, k)
    order = moe.sort(ids, len(experts))
    y = int8.gemm(E8, int8.quantize(x, rows=order.rows), offsets=order.offsets)

For inference: nothing here has a gradient, and codes, being integers, pass none on.
A tangent of forward mode is refused by the products, and every call within
torch.jit.trace, which records torch's own operations alone.  Every call runs on
torch's current stream of the operands' device.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import tlrgemm as T
from .blocks import _NEW, _rows, binding


class RowScaled:
    """A matrix of 8-bit integers with a scale for each row, or one for each expert.

    codes    (rows, ld) or (experts, rows, ld) int8 tensor, rows contiguous, each
             readable up to k rounded up to 16, strides multiples of 16
    scales   (rows,) or (experts, rows) float32 tensor
    k        columns; codes behind the k-th are not used
    """

    __slots__ = ("codes", "scales", "k")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int):
        if codes.dtype != torch.int8 or codes.dim() not in (2, 3):
            raise ValueError("codes: an int8 tensor of 2 or 3 dimensions is needed")
        if codes.shape[-1] < k or k < 0 or (codes.shape[-1] > 1 and codes.stride(-1) != 1):
            raise ValueError(f"codes: contiguous rows of {k} entries are needed")
        if scales.dtype != torch.float32 or scales.shape != codes.shape[:-1] or scales.device != codes.device:
            raise ValueError(f"scales: a float32 tensor {tuple(codes.shape[:-1])} on the codes' device is needed")
        self.codes, self.scales, self.k = codes, scales, k

    @property
    def rows(self) -> int:
        return self.codes.shape[-2]

    def dequantize(self) -> torch.Tensor:
        """The float32 matrix that the codes and scales stand for."""
        return self.codes[..., :self.k].float() * self.scales.unsqueeze(-1)


def _made(codes: torch.Tensor, scales: torch.Tensor, k: int) -> RowScaled:
    q = RowScaled.__new__(RowScaled)        # right by construction
    q.codes, q.scales, q.k = codes, scales, k
    return q


def quantize(x: torch.Tensor, rows: Optional[torch.Tensor] = None) -> RowScaled:
    """Codes and scales of x (rows, k) or (experts, rows, k), float32, float16 or
    bfloat16: a row's scale is its largest magnitude over 127 (at least 2^-100), a
    code the integer nearest to the float quotient, ties to even.  A row that holds
    an infinity or a NaN gets a NaN scale.

    ``rows`` (int32, x of 2 dimensions): row r of the result is x[rows[r]], one of
    zeros where rows[r] is no row of x.  Codes and scales carry no gradient, whatever
    x does, and are views of one allocation: keeping either keeps both."""
    if rows is not None and x.dim() != 2:
        raise ValueError("quantize: rows are picked from an x of 2 dimensions")
    got = binding().row_quantize(x if x.dim() == 2 else _rows(x) if x.dim() == 3 else x, rows)
    if type(got) is int:
        T._check(got, "tlr_row_quantize")
    codes, scales = got
    if x.dim() == 3:
        codes, scales = codes.view(*x.shape[:2], codes.shape[1]), scales.view(x.shape[:2])
    return _made(codes, scales, x.shape[-1])


def gemm(A: RowScaled, B: RowScaled, offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
         dtype: str = "bf16") -> torch.Tensor:
    """B A^T, a (B.rows, A.rows) tensor: x W^T with A = W and B = x.  Without ``out``
    a new tensor of type ``dtype``.  Sums are exact (32-bit integers), scaled in
    float and rounded once; k is 131071 at most.

    ``offsets`` (groups + 1, int32, on the GPU, ascending): A has a matrix for each
    group (3 dimensions), and rows offsets[g] .. offsets[g+1] - 1 of B take the g-th.
    Rows of no group, before the first or behind the last, are zeros in a new result,
    and left as they are in a given one.

    It has no gradient: where gradients are on, scales or an out that require one are
    refused (codes made of an x that requires one are not: quantize has cut it)."""
    if A.k != B.k:
        raise ValueError(f"gemm: contraction lengths differ ({A.k} and {B.k})")
    new = _NEW.get(dtype)
    if new is None:
        raise ValueError(f"gemm: dtype is f32, f16 or bf16, not {dtype!r}")
    got = binding().row_gemm(A.codes, A.scales, B.codes, B.scales, A.k, offsets, out, new)
    if type(got) is int:
        T._check(got, "tlr_row_gemm")
    return got


def linear(x: torch.Tensor, w: RowScaled) -> torch.Tensor:
    """x W^T for x (..., k) in float32, float16 or bfloat16, quantized with a scale
    for each token, and a weight of 2 dimensions; in x's type.  There is no backward
    pass: where gradients are on, an x or scales that require one are refused."""
    got = binding().row_linear(x, w.codes, w.scales, w.k)
    if type(got) is int:
        T._check(got, "tlr_row_linear")
    return got
