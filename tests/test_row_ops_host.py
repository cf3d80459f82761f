"""Refusals of the 8-bit integer, expert sorting and gated entry points: every check comes before any launch, so they run
without a GPU (made-up addresses are never read)."""
import ctypes

import pytest
import torch

from hpc_linear_algebra_amd import blocks, int8, moe
from hpc_linear_algebra_amd import tlrgemm as T

A16 = 0x10000            # a 256-byte aligned address
BAD, NOT, SPACE, OK = T.TLR_ERR_INVALID_ARG, T.TLR_ERR_UNSUPPORTED, T.TLR_ERR_WORKSPACE, T.TLR_OK


def status(f, *a, **k):
    try:
        f(*a, **k)
    except T.TLRError as e:
        return e.status
    return T.TLR_OK


Q = dict(dtype="bf16", rows=8, k=40, X=A16, x_rows=8, ldx=40, index=0, codes=A16, ldq=48, scales=A16)


@pytest.mark.parametrize("change,want", [
    (dict(dtype="f64"), NOT), (dict(dtype="e4m3"), BAD), (dict(rows=-1), BAD), (dict(k=-1), BAD), (dict(x_rows=-1), BAD),
    (dict(rows=1 << 31, x_rows=1 << 31), BAD), (dict(k=(1 << 30) + 16, ldx=1 << 31, ldq=1 << 31), BAD), (dict(rows=9), BAD),
    (dict(ldx=39), BAD), (dict(X=0), BAD), (dict(X=A16 + 1), BAD), (dict(codes=0), BAD), (dict(codes=A16 + 8), BAD), (dict(ldq=40), BAD),
    (dict(ldq=32), BAD), (dict(scales=0), BAD), (dict(scales=A16 + 2), BAD), (dict(index=A16 + 2, rows=3), BAD),
    (dict(rows=0), OK), (dict(rows=0, x_rows=0, X=0, codes=0, scales=0), OK)])
def test_quantize_refusals(change, want):
    assert status(T.tlr_row_quantize, **dict(Q, **change)) == want


def matrix(**change):
    m = dict(codes=A16, scales=A16, ld=48)
    m.update(change)
    return T.tlr_row_matrix(**m)


def groups(**change):
    g = dict(offsets=A16, code_step=48 * 64, scale_step=64, count=4, clear=0)
    g.update(change)
    return T.tlr_row_groups(**g)


G = dict(dtype="bf16", m=64, n=8, k=40, A=matrix(), B=matrix(), C=A16, ldc=64)


@pytest.mark.parametrize("change,want", [
    (dict(dtype="f64"), NOT), (dict(dtype="e4m3"), BAD), (dict(m=-1), BAD), (dict(n=1 << 31), BAD), (dict(k=131072), NOT),
    (dict(ldc=63), BAD), (dict(C=0), BAD), (dict(C=A16 + 1), BAD), (dict(A=matrix(codes=0)), BAD), (dict(B=matrix(scales=0)), BAD),
    (dict(A=matrix(codes=A16 + 8)), BAD), (dict(B=matrix(ld=40)), BAD), (dict(B=matrix(ld=32)), BAD), (dict(A=matrix(ld=1 << 22)), BAD),
    (dict(A=matrix(scales=A16 + 1)), BAD), (dict(m=1 << 30, ldc=1 << 30, n=1 << 16), BAD),
    (dict(groups=groups(count=0)), BAD), (dict(groups=groups(count=1025)), BAD), (dict(groups=groups(offsets=0)), BAD),
    (dict(groups=groups(offsets=A16 + 2)), BAD), (dict(groups=groups(code_step=8)), BAD), (dict(groups=groups(code_step=-16)), BAD),
    (dict(groups=groups(scale_step=-1)), BAD), (dict(groups=groups(clear=2)), BAD),
    (dict(m=362, n=548, k=4009, ldc=362, A=matrix(ld=4016), B=matrix(ld=4016)), BAD),                              # in parts: no workspace
    (dict(m=362, n=548, k=4009, ldc=362, A=matrix(ld=4016), B=matrix(ld=4016), workspace=A16, workspace_bytes=64), SPACE),
    (dict(m=0), OK), (dict(n=0), OK), (dict(n=0, groups=groups()), OK)])
def test_product_refusals(change, want):
    assert status(T.tlr_row_gemm, **dict(G, **change)) == want


L = dict(dtype="bf16", m=64, n=40, k=40, A=matrix(), X=A16, ldx=40, C=A16, ldc=64, workspace=A16, workspace_bytes=1 << 20)


@pytest.mark.parametrize("change,want", [
    (dict(dtype="f64"), NOT), (dict(dtype="e5m2"), BAD), (dict(k=131072), NOT), (dict(ldx=39), BAD), (dict(ldc=63), BAD), (dict(X=0), BAD),
    (dict(X=A16 + 1), BAD), (dict(C=0), BAD), (dict(A=matrix(codes=0)), BAD), (dict(A=matrix(ld=40)), BAD), (dict(workspace=0), BAD),
    (dict(workspace=A16 + 16), BAD), (dict(workspace_bytes=100), SPACE), (dict(n=0), OK), (dict(m=0), OK)])
def test_linear_refusals(change, want):
    assert status(T.tlr_row_linear, **dict(L, **change)) == want


S = dict(id_bytes=4, tokens=6000, topk=2, experts=8, ids=A16, offsets=A16, place=A16, rows=A16, workspace=A16, workspace_bytes=1 << 20)


@pytest.mark.parametrize("change,want", [
    (dict(id_bytes=2), BAD), (dict(tokens=-1), BAD), (dict(tokens=(1 << 23) + 1), BAD), (dict(topk=0), BAD), (dict(topk=65), BAD),
    (dict(experts=0), BAD), (dict(experts=1025), BAD), (dict(ids=0), BAD), (dict(ids=A16 + 4, id_bytes=8), BAD), (dict(ids=A16 + 2), BAD),
    (dict(offsets=0), BAD), (dict(place=A16 + 1), BAD), (dict(rows=0), BAD), (dict(workspace=0), BAD), (dict(workspace_bytes=16), SPACE)])
def test_sort_refusals(change, want):
    assert status(T.tlr_expert_sort, **dict(S, **change)) == want


def test_sort_workspace():
    assert T.tlr_expert_sort_workspace_bytes(512, 8, 64) == 0
    assert T.tlr_expert_sort_workspace_bytes(513, 8, 64) == 4 * 65 * (5 + 1)
    assert T.tlr_expert_sort_workspace_bytes(1 << 23, 2, 1024) == 4 * 1025 * (4096 + 1)
    assert status(T.tlr_expert_sort_workspace_bytes, 1, 1, 1025) == BAD


R = dict(dtype="bf16", tokens=5, topk=2, hidden=40, place=A16, end=A16)
ROWS = [(dict(dtype="f64"), NOT), (dict(dtype="e4m3"), BAD), (dict(tokens=-1), BAD), (dict(topk=0), BAD), (dict(topk=65), BAD),
        (dict(tokens=(1 << 23) + 1), BAD), (dict(hidden=-1), BAD), (dict(hidden=(1 << 24) + 1), BAD), (dict(place=0), BAD), (dict(end=A16 + 2), BAD)]


@pytest.mark.parametrize("change,want", ROWS + [
    (dict(X=0), BAD), (dict(X=A16 + 1), BAD), (dict(ldx=39), BAD), (dict(Y=0), BAD), (dict(ldy=39), BAD), (dict(ldy=1 << 31), BAD),
    (dict(tokens=0), OK), (dict(hidden=0), OK)])
def test_gather_refusals(change, want):
    assert status(T.tlr_expert_gather, **dict(R, X=A16, ldx=40, Y=A16, ldy=40, **{}) | change) == want


@pytest.mark.parametrize("change,want", ROWS + [
    (dict(Y=0), BAD), (dict(ldy=39), BAD), (dict(out=A16 + 1), BAD), (dict(ldo=39), BAD), (dict(weights=A16 + 2), BAD), (dict(tokens=0), OK)])
def test_combine_refusals(change, want):
    assert status(T.tlr_expert_combine, **dict(R, Y=A16, ldy=40, weights=A16, out=A16, ldo=40) | change) == want


@pytest.mark.parametrize("change,want", ROWS + [
    (dict(dout=0), BAD), (dict(ldd=39), BAD), (dict(Y=0), BAD), (dict(ldy=39), BAD), (dict(dY=A16 + 1), BAD), (dict(lddy=39), BAD),
    (dict(weights=0), BAD), (dict(dweights=A16 + 2), BAD), (dict(tokens=0), OK), (dict(dY=0, dweights=0), OK)])
def test_combine_grad_refusals(change, want):
    assert status(T.tlr_expert_combine_grad, **dict(R, dout=A16, ldd=40, Y=A16, ldy=40, weights=A16, dY=A16, lddy=40, dweights=A16) | change) == want


F = dict(dtype="bf16", rows=5, inter=40, X=A16, ldx=80, Y=A16, ldy=40, codes=A16, ldq=48, scales=A16, lds=1)
COMMON = [(dict(dtype="f64"), NOT), (dict(dtype="e4m3"), BAD), (dict(rows=-1), BAD), (dict(inter=-1), BAD), (dict(rows=1 << 31), BAD),
          (dict(rows=(1 << 30), inter=300, ldq=304, lds=3), BAD), (dict(codes=A16 + 8), BAD), (dict(ldq=40), BAD), (dict(ldq=32), BAD),
          (dict(scales=0), BAD), (dict(scales=A16 + 2), BAD), (dict(lds=0), BAD), (dict(rows=0), OK), (dict(inter=0), OK)]


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(ldx=79), BAD), (dict(ldy=39), BAD), (dict(X=0), BAD), (dict(X=A16 + 1), BAD), (dict(Y=0), BAD), (dict(Y=A16 + 1), BAD)])
def test_gated_refusals(change, want):
    assert status(T.tlr_gated, **dict(F, **change)) == want


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(codes=0), BAD), (dict(lddx=79), BAD), (dict(lddy=39), BAD), (dict(dX=0), BAD), (dict(dY=A16 + 1), BAD)])
def test_gated_grad_refusals(change, want):
    base = {k: v for k, v in F.items() if k not in ("X", "ldx", "Y", "ldy")}
    assert status(T.tlr_gated_grad, **dict(base, dY=A16, lddy=40, dX=A16, lddx=80, **{}) | change) == want


def test_python_refusals():
    i8 = torch.int8
    c, s = torch.zeros(4, 48, dtype=i8), torch.zeros(4)
    W = int8.RowScaled(c, s, 40)
    assert W.rows == 4 and W.dequantize().shape == (4, 40)
    assert int8.RowScaled(torch.zeros(2, 4, 48, dtype=i8), torch.zeros(2, 4), 48).rows == 4
    for bad in ((c.float(), s, 40), (c, s.double(), 40), (c, s[:3], 40), (c, s, 49), (c, s, -1), (c[0], s[0], 40), (c.t().contiguous().t(), s, 40)):
        with pytest.raises(ValueError):
            int8.RowScaled(*bad)
    x = torch.zeros(3, 40)
    order = moe.Order(torch.zeros(5, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32), None)
    for call in (lambda: int8.quantize(x), lambda: int8.quantize(x, rows=torch.zeros(2, dtype=torch.int32)), lambda: int8.quantize(x[None, None]),
                 lambda: int8.quantize(x[None], rows=torch.zeros(2, dtype=torch.int32)), lambda: int8.gemm(W, W), lambda: int8.linear(x, W),
                 lambda: int8.gemm(W, int8.RowScaled(c, s, 39)), lambda: int8.gemm(W, W, dtype="f64"), lambda: int8.linear(x[:, :39], W),
                 lambda: moe.sort(torch.zeros(3, 2, dtype=torch.int64), 4), lambda: moe.sort(x, 4), lambda: moe.gather(x, order),
                 lambda: moe.combine(torch.zeros(6, 4), None, order), lambda: blocks.gated(x), lambda: blocks.gated(x[:, :39]),
                 lambda: blocks.gated_forward(x), lambda: blocks.gated_backward(x, c, s), lambda: moe.Int8Experts(W, W)):
        with pytest.raises(ValueError):
            call()                                   # on the host, or of the wrong shape: nothing is launched
    with pytest.raises(RuntimeError):
        int8.linear(x.requires_grad_(), W)
    E1, E2 = (int8.RowScaled(torch.zeros(2, r, 48, dtype=i8), torch.zeros(2, r), k) for r, k in ((64, 40), (40, 32)))
    layer = moe.Int8Experts(E1, E2)
    ids, w = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(RuntimeError):
        layer(x, ids, w)
    x = x.detach()
    for bad in ((x[:, :39], ids, w), (x, ids[:2], w), (x.double(), ids, w), (x, ids, w)):
        with pytest.raises(ValueError):
            layer(*bad)
    with pytest.raises(ValueError):
        moe.Int8Experts(E2, E1)
    assert ctypes.sizeof(T.tlr_row_matrix) == 24 and ctypes.sizeof(T.tlr_row_groups) == 32
