"""Refusals of the serving operators: bad arguments are rejected on the host before anything
is launched (no GPU needed: no call below reaches the device)."""
import math
import os

import pytest

import block_scaled_fp8_dispatch_amd as moe

A = 0x10000          # aligned fake address


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.fail("libmoe.so is not built (run python -m block_scaled_fp8_dispatch_amd.build)")
    return moe.load_library()


def test_router_refusals():
    def call(idx=A, w=A, logits=A, ty=1, T=4, E=8, k=2, over=0, scale=1.0):
        return moe.gemm_call_raw("moe_topk_router", idx, w, logits, ty, T, E, k, over, scale, None)

    for bad in (dict(idx=None), dict(w=None), dict(logits=None)):
        assert call(**bad) == moe.MOE_ERR_NULL
    for bad in (dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=100, k=65), dict(ty=2), dict(ty=-1), dict(over=2),
                dict(scale=math.inf), dict(scale=math.nan), dict(T=2 ** 30)):
        assert call(**bad) == moe.MOE_ERR_SHAPE, bad
    assert call(T=-1) == moe.MOE_ERR_TOKENS
    for bad in (dict(idx=A + 4), dict(w=A + 8), dict(logits=A + 2)):
        assert call(**bad) == moe.MOE_ERR_ALIGN
    assert call(T=0) == moe.MOE_OK


def test_few_sizes_and_refusals():
    s = moe.make_shape(32, 7168, 2048, 8, 64)
    nb = moe.moe_few_workspace_bytes(s)
    assert nb >= 32 * 8 * 2048 + 32 * 8 * 16
    assert nb <= moe.moe_workspace_bytes(s)
    assert moe.moe_few_workspace_bytes(moe.make_shape(32, 7168, 2048, 8, 3)) < nb
    for shape in (moe.make_shape(4, 128, 128, 2, 1), moe.make_shape(1024, 256, 384, 64, 40), moe.make_shape(8, 640, 128, 1, 7)):
        assert 0 < moe.moe_few_workspace_bytes(shape) <= moe.moe_workspace_bytes(shape)
    assert moe.moe_few_workspace_bytes(moe.make_shape(4, 200, 128, 1, 1)) == 0

    def call(T=4, shape=s, wsb=nb, y=A, x=A, xsf=A, idx=A, w=A, packed=A, ws=A):
        import ctypes
        return moe.gemm_call_raw("moe_forward_few", y, x, xsf, idx, w, T,
                                 None if shape is None else ctypes.byref(shape), packed, ws, wsb, None)

    for name in ("y", "x", "xsf", "idx", "w", "packed", "ws", "shape"):
        assert call(**{name: None}) == moe.MOE_ERR_NULL, name
    for name in ("y", "x", "xsf", "idx", "w", "packed", "ws"):
        assert call(**{name: A + 8}) == moe.MOE_ERR_ALIGN, name
    assert call(wsb=nb - 1) == moe.MOE_ERR_WORKSPACE
    assert call(T=33) == moe.MOE_ERR_TOKENS            # more than a few
    assert call(T=-1) == moe.MOE_ERR_TOKENS
    assert call(T=4, shape=moe.make_shape(32, 7168, 2048, 8, 3)) == moe.MOE_ERR_TOKENS
    assert call(shape=moe.make_shape(32, 7000, 2048, 8, 64)) == moe.MOE_ERR_SHAPE
    wide = moe.make_shape(4, 2 ** 27, 128, 3, 1)       # more columns than one launch covers
    assert moe.moe_few_workspace_bytes(wide) == 0 and call(T=1, shape=wide, wsb=1 << 40) == moe.MOE_ERR_SHAPE
    assert call(T=0) == moe.MOE_OK


def test_fp8_gemm_refusals():
    call = moe.gemm_call_raw
    wsb = moe.moe_fp8_gemm_workspace_bytes(64, 1)
    assert wsb > 0 and moe.moe_fp8_gemm_workspace_bytes(-1, 1) == 0 and moe.moe_fp8_gemm_workspace_bytes(1, 0) == 0
    assert moe.moe_fp8_gemm_workspace_bytes(1, 1025) == 0

    def dense(d=A, ty=0, a=A, asf=A, m=64, n=33, k=256, b=A, bsf=A, ws=A, wb=wsb):
        return call("moe_fp8_gemm", d, ty, a, asf, m, n, k, b, bsf, ws, wb, None)

    for name in ("d", "a", "asf", "b", "bsf", "ws"):
        assert dense(**{name: None}) == moe.MOE_ERR_NULL, name
        assert dense(**{name: A + 4}) == moe.MOE_ERR_ALIGN, name
    for bad in (dict(n=0), dict(n=-5), dict(n=2 ** 30 + 1), dict(k=0), dict(k=64), dict(k=200), dict(k=2 ** 23), dict(ty=2), dict(ty=-1),
                dict(m=2 ** 23, n=2 ** 30, k=128, wb=1 << 40), dict(m=2 ** 15, n=2 ** 24, k=128, wb=1 << 40)):
        assert dense(**bad) == moe.MOE_ERR_SHAPE, bad
    assert dense(m=-1) == moe.MOE_ERR_TOKENS
    assert dense(m=2 ** 24, k=256) == moe.MOE_ERR_TOKENS
    assert dense(wb=wsb - 1) == moe.MOE_ERR_WORKSPACE
    assert dense(m=0) == moe.MOE_OK

    def contiguous(d=A, ty=1, a=A, asf=A, grp=A, m=64, g=3, n=33, k=256, b=A, bsf=A, ws=A, wb=None):
        wb = moe.moe_fp8_gemm_workspace_bytes(max(m, 0), max(g, 1)) if wb is None else wb
        return call("moe_m_grouped_fp8_gemm_contiguous", d, ty, a, asf, grp, m, g, n, k, b, bsf, ws, wb, None)

    for name in ("d", "a", "asf", "grp", "b", "bsf", "ws"):
        assert contiguous(**{name: None}) == moe.MOE_ERR_NULL, name
        assert contiguous(**{name: A + 4}) == moe.MOE_ERR_ALIGN, name
    assert contiguous(g=0) == moe.MOE_ERR_SHAPE and contiguous(n=0) == moe.MOE_ERR_SHAPE
    assert contiguous(m=-1) == moe.MOE_ERR_TOKENS
    assert contiguous(wb=moe.moe_fp8_gemm_workspace_bytes(64, 3) - 1) == moe.MOE_ERR_WORKSPACE
    assert contiguous(m=0) == moe.MOE_OK

    def masked(d=A, ty=1, a=A, asf=A, cnt=A, g=3, mm=16, n=33, k=256, b=A, bsf=A, ws=A, wb=None):
        wb = moe.moe_fp8_gemm_workspace_bytes(max(g * mm, 0), max(g, 1)) if wb is None else wb
        return call("moe_m_grouped_fp8_gemm_masked", d, ty, a, asf, cnt, g, mm, 8, n, k, b, bsf, ws, wb, None)

    for name in ("d", "a", "asf", "cnt", "b", "bsf", "ws"):
        assert masked(**{name: None}) == moe.MOE_ERR_NULL, name
        assert masked(**{name: A + 4}) == moe.MOE_ERR_ALIGN, name
    assert masked(g=1025, wb=1 << 30) == moe.MOE_ERR_SHAPE and masked(k=100) == moe.MOE_ERR_SHAPE
    assert masked(mm=-1, wb=1 << 30) == moe.MOE_ERR_TOKENS
    assert masked(wb=moe.moe_fp8_gemm_workspace_bytes(48, 3) - 1) == moe.MOE_ERR_WORKSPACE
    assert masked(mm=0) == moe.MOE_OK
