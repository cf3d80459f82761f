"""Refusals of the block-scaled and mixture-of-experts entry points: every check comes before any launch, so they run
without a GPU (made-up addresses are never read)."""
import ctypes

import pytest
import torch

from hpc_linear_algebra_amd import tlrgemm as T
from hpc_linear_algebra_amd import blocks, moe

A16 = 0x10000            # a 256-byte aligned address


def status(f, *a, **k):
    try:
        f(*a, **k)
    except T.TLRError as e:
        return e.status
    return T.TLR_OK


Q = dict(dtype="bf16", fmt="e4m3", block=1, rows=8, k=40, X=A16, ldx=40, codes=A16, ldq=48, scales=A16, lds=8,
         codes_t=0, ldq_t=0, scales_t=0, lds_t=0)


@pytest.mark.parametrize("change,want", [
    (dict(dtype="f64"), T.TLR_ERR_UNSUPPORTED), (dict(dtype="e4m3"), T.TLR_ERR_INVALID_ARG),
    (dict(fmt="bf16"), T.TLR_ERR_INVALID_ARG), (dict(block=64), T.TLR_ERR_INVALID_ARG),
    (dict(rows=-1), T.TLR_ERR_INVALID_ARG), (dict(k=-1), T.TLR_ERR_INVALID_ARG),
    (dict(rows=1 << 31), T.TLR_ERR_INVALID_ARG), (dict(rows=1 << 24, lds=1 << 24), T.TLR_ERR_INVALID_ARG),
    (dict(ldx=39), T.TLR_ERR_INVALID_ARG), (dict(X=0), T.TLR_ERR_INVALID_ARG), (dict(X=A16 + 1), T.TLR_ERR_INVALID_ARG),
    (dict(codes=0), T.TLR_ERR_INVALID_ARG), (dict(codes=A16 + 8), T.TLR_ERR_INVALID_ARG),
    (dict(ldq=40), T.TLR_ERR_INVALID_ARG), (dict(ldq=32), T.TLR_ERR_INVALID_ARG), (dict(scales=0), T.TLR_ERR_INVALID_ARG),
    (dict(scales=A16 + 2), T.TLR_ERR_INVALID_ARG), (dict(lds=7), T.TLR_ERR_INVALID_ARG),
    (dict(codes_t=A16), T.TLR_ERR_INVALID_ARG),
    (dict(codes_t=A16, ldq_t=16, scales_t=A16, lds_t=39), T.TLR_ERR_INVALID_ARG),
    (dict(rows=0), T.TLR_OK), (dict(k=0), T.TLR_OK)])
def test_quantize_refusals(change, want):
    assert status(T.tlr_block_quantize, **dict(Q, **change)) == want


def matrix(**change):
    m = dict(codes=A16, scales=A16, ld=48, lds=64, block=1, fmt=T.TLR_E4M3)
    m.update(change)
    return T.tlr_block_matrix(**m)


G = dict(dtype="bf16", m=64, n=8, k=40, alpha=1.0, A=matrix(), B=matrix(), beta=0.0, C=A16, ldc=64)


@pytest.mark.parametrize("change,want", [
    (dict(dtype="f64"), T.TLR_ERR_UNSUPPORTED), (dict(dtype="e4m3"), T.TLR_ERR_INVALID_ARG),
    (dict(m=-1), T.TLR_ERR_INVALID_ARG), (dict(n=1 << 31), T.TLR_ERR_INVALID_ARG), (dict(ldc=63), T.TLR_ERR_INVALID_ARG),
    (dict(C=0), T.TLR_ERR_INVALID_ARG), (dict(C=A16 + 1), T.TLR_ERR_INVALID_ARG), (dict(flags=2), T.TLR_ERR_INVALID_ARG),
    (dict(A=matrix(codes=0)), T.TLR_ERR_INVALID_ARG), (dict(B=matrix(scales=0)), T.TLR_ERR_INVALID_ARG),
    (dict(A=matrix(codes=A16 + 8)), T.TLR_ERR_INVALID_ARG), (dict(B=matrix(ld=40)), T.TLR_ERR_INVALID_ARG),
    (dict(B=matrix(ld=32)), T.TLR_ERR_INVALID_ARG), (dict(A=matrix(ld=1 << 22)), T.TLR_ERR_INVALID_ARG),
    (dict(A=matrix(lds=63)), T.TLR_ERR_INVALID_ARG), (dict(A=matrix(block=128, lds=0)), T.TLR_ERR_INVALID_ARG),
    (dict(A=matrix(block=2)), T.TLR_ERR_INVALID_ARG), (dict(B=matrix(fmt=T.TLR_F16)), T.TLR_ERR_INVALID_ARG),
    (dict(A=matrix(scales=A16 + 1)), T.TLR_ERR_INVALID_ARG),
    (dict(m=0), T.TLR_OK), (dict(n=0), T.TLR_OK), (dict(k=0, beta=1.0), T.TLR_OK)])
def test_product_refusals(change, want):
    assert status(T.tlr_block_gemm, **dict(G, **change)) == want


def layer(**change):
    v = dict(hidden=64, inter=32, experts=8, topk=2, dt=T.TLR_BF16, wdt=T.TLR_BF16, normalize=1, reserved=0, router=A16,
             gate_up=A16, down=A16, gate_up_scales=None, down_scales=None)
    v.update(change)
    return T.tlr_moe_layer(**v)


M = dict(layer=layer(), tokens=3, X=A16, ldx=64, Y=A16, ldy=64, ids=A16, weights=A16, workspace=A16,
         workspace_bytes=1 << 30)


@pytest.mark.parametrize("change,want", [
    (dict(layer=layer(dt=T.TLR_F32, wdt=T.TLR_F32)), T.TLR_ERR_UNSUPPORTED),
    (dict(layer=layer(dt=7)), T.TLR_ERR_INVALID_ARG), (dict(layer=layer(wdt=T.TLR_F16)), T.TLR_ERR_UNSUPPORTED),
    (dict(layer=layer(wdt=T.TLR_E5M2)), T.TLR_ERR_UNSUPPORTED), (dict(layer=layer(wdt=T.TLR_E4M3)), T.TLR_ERR_INVALID_ARG),
    (dict(layer=layer(hidden=72)), T.TLR_ERR_INVALID_ARG), (dict(layer=layer(inter=8)), T.TLR_ERR_INVALID_ARG),
    (dict(layer=layer(experts=513)), T.TLR_ERR_INVALID_ARG), (dict(layer=layer(topk=9)), T.TLR_ERR_INVALID_ARG),
    (dict(layer=layer(topk=0)), T.TLR_ERR_INVALID_ARG), (dict(layer=layer(experts=64, topk=17)), T.TLR_ERR_INVALID_ARG),
    (dict(layer=layer(normalize=2)), T.TLR_ERR_INVALID_ARG), (dict(layer=layer(reserved=1)), T.TLR_ERR_INVALID_ARG),
    (dict(layer=layer(router=None)), T.TLR_ERR_INVALID_ARG), (dict(layer=layer(down=A16 + 4)), T.TLR_ERR_INVALID_ARG),
    (dict(tokens=-1), T.TLR_ERR_INVALID_ARG), (dict(tokens=257), T.TLR_ERR_INVALID_ARG), (dict(X=0), T.TLR_ERR_INVALID_ARG),
    (dict(X=A16 + 2), T.TLR_ERR_INVALID_ARG), (dict(ldx=68), T.TLR_ERR_INVALID_ARG), (dict(ldx=56), T.TLR_ERR_INVALID_ARG),
    (dict(ldy=63), T.TLR_ERR_INVALID_ARG), (dict(ids=0), T.TLR_ERR_INVALID_ARG), (dict(weights=A16 + 1), T.TLR_ERR_INVALID_ARG),
    (dict(workspace=A16 + 16), T.TLR_ERR_INVALID_ARG), (dict(workspace_bytes=256), T.TLR_ERR_WORKSPACE),
    (dict(tokens=0), T.TLR_OK)])
def test_moe_refusals(change, want):
    assert status(T.tlr_moe, **dict(M, **change)) == want


def test_moe_workspace_grows_with_tokens():
    sizes = [T.tlr_moe_workspace_bytes(layer(), t) for t in (0, 1, 2, 64, 256)]
    assert sizes == sorted(sizes) and sizes[1] > 0
    assert status(T.tlr_moe_workspace_bytes, layer(), 257) == T.TLR_ERR_INVALID_ARG


def test_the_tlr_products_refuse_8_bit_types():
    import numpy as np
    s = T.Shape(8, 8, 4, np.zeros((2, 2), np.int32), True)
    for dt in ("e4m3", "e5m2"):
        assert status(T.tlr_gemm_analyze, dt, "N", s, "N", s, ldc=8) == T.TLR_ERR_INVALID_ARG
        assert status(T.tlr_dense_gemm, dt, "N", "N", 8, 8, 8, 1.0, A16, 8, A16, 8, 0.0, A16, 8) == T.TLR_ERR_INVALID_ARG
        assert status(T.tlr_expand, dt, 8, 8, 4, True, A16, T.buffers(A16, A16, A16), 1.0, 0.0, A16, 8, A16, 1024) != T.TLR_OK
        assert status(T.tlr_compress_workspace_bytes, dt, 64, 64, 32, 8) != T.TLR_OK


def test_python_refusals():
    e4 = torch.float8_e4m3fn
    c, s = torch.zeros(4, 48, dtype=e4), torch.zeros(1, 4)
    blocks.BlockScaled(c, s, 4, 40, 1)
    for bad in ((c.float(), s, 4, 40, 1), (c, s, 4, 40, 2), (c, s.double(), 4, 40, 1), (c, s, 5, 40, 1), (c, s, 4, 49, 1),
                (c, s.t(), 4, 40, 1), (c, torch.zeros(2, 4), 4, 40, 1), (c.t().contiguous().t(), s, 4, 40, 1)):
        with pytest.raises(ValueError):
            blocks.BlockScaled(*bad)
    with pytest.raises(ValueError):
        blocks.quantize(torch.zeros(4, 40))                      # not on a GPU
    a, b = blocks.BlockScaled(c, s, 4, 40, 1), blocks.BlockScaled(c, s, 4, 39, 1)
    with pytest.raises(ValueError):
        blocks.gemm(a, b)
    with pytest.raises(ValueError):
        blocks.gemm(a, a, beta=1.0)
    with pytest.raises(ValueError):
        blocks.linear(torch.zeros(3, 8), torch.zeros(4, 9))
    with pytest.raises(ValueError):
        moe.MoELayer(torch.zeros(4, 32), torch.zeros(4, 32, 32), torch.zeros(4, 32, 16), 2)
    with pytest.raises(ValueError):
        bf = torch.bfloat16
        moe.MoELayer(torch.zeros(4, 32, dtype=bf), torch.zeros(4, 30, 32, dtype=bf), torch.zeros(4, 32, 16, dtype=bf), 2)
    assert ctypes.sizeof(T.tlr_block_matrix) == 40 and ctypes.sizeof(T.tlr_moe_layer) == 72


def test_block_operators_refuse_host_tensors():
    """No pointer to host memory reaches a kernel."""
    import torch

    from hpc_linear_algebra_amd import blocks
    with pytest.raises(ValueError):
        blocks.quantize(torch.zeros(4, 32))
    with pytest.raises(ValueError):
        blocks.quantize("x")
    q = blocks.BlockScaled(torch.zeros(4, 32, dtype=torch.float8_e4m3fn), torch.ones(1, 4), 4, 32, 1)
    for out in (None, torch.zeros(4, 4)):
        with pytest.raises(ValueError):
            blocks.gemm(q, q, out=out, dtype="f32")
