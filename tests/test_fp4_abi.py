"""Refusals of the norm with FP8 output, the 4-bit casts and the FP4 x FP4 GEMMs: bad arguments are rejected on the host
before anything is launched (no GPU needed: no call below reaches the device)."""
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


def test_rmsnorm_refusals():
    def call(q=A, sf=A, normed=A, out=A, x=A, res=A, w=A, ty=0, rows=4, cols=256, eps=1e-6):
        return moe.gemm_call_raw("moe_rmsnorm_to_fp8", q, sf, normed, out, x, res, w, ty, rows, cols, eps, None)

    for name in ("q", "sf", "x", "w"):
        assert call(**{name: None}) == moe.MOE_ERR_NULL, name
    for name in ("q", "sf", "normed", "out", "x", "res", "w"):
        assert call(**{name: A + 8}) == moe.MOE_ERR_ALIGN, name
    for bad in (dict(cols=0), dict(cols=64), dict(cols=200), dict(cols=-128), dict(ty=2), dict(ty=-1), dict(eps=0.0),
                dict(eps=-1e-6), dict(eps=math.inf), dict(eps=math.nan)):
        assert call(**bad) == moe.MOE_ERR_SHAPE, bad
    assert call(rows=-1) == moe.MOE_ERR_TOKENS
    assert call(rows=0) == moe.MOE_OK and call(rows=0, normed=None, out=None, res=None) == moe.MOE_OK


@pytest.mark.parametrize("back", [False, True])
def test_cast_refusals(back):
    def call(x=A, ty=0, rows=4, cols=64, q=A, sf=A):
        args = (q, sf, rows, cols, x, ty, None) if back else (x, ty, rows, cols, q, sf, None)
        return moe.gemm_call_raw("moe_cast_from_fp4" if back else "moe_cast_to_fp4", *args)

    for name in ("x", "q", "sf"):
        assert call(**{name: None}) == moe.MOE_ERR_NULL, name
        assert call(**{name: A + 4}) == moe.MOE_ERR_ALIGN, name
    for bad in (dict(cols=0), dict(cols=16), dict(cols=40), dict(cols=-32), dict(ty=2), dict(ty=-1)):
        assert call(**bad) == moe.MOE_ERR_SHAPE, bad
    assert call(rows=-1) == moe.MOE_ERR_TOKENS
    assert call(rows=0) == moe.MOE_OK


def test_fp4_gemm_refusals():
    call = moe.gemm_call_raw
    wsb = moe.moe_fp4_gemm_workspace_bytes(64, 1)
    assert 0 < wsb <= moe.moe_gemm_workspace_bytes(64, 1)
    assert [moe.moe_fp4_gemm_workspace_bytes(*v) for v in ((-1, 1), (1, 0), (1, 1025))] == [0, 0, 0]

    def dense(d=A, ty=0, a=A, asf=A, m=64, n=48, k=256, b=A, ws=A, wb=wsb):
        return call("moe_fp4_gemm", d, ty, a, asf, m, n, k, b, ws, wb, None)

    for name in ("d", "a", "asf", "b", "ws"):
        assert dense(**{name: None}) == moe.MOE_ERR_NULL, name
        assert dense(**{name: A + 4}) == moe.MOE_ERR_ALIGN, name
    for bad in (dict(n=0), dict(n=-16), dict(n=8), dict(n=40), dict(n=2 ** 30 + 16), dict(k=0), dict(k=64), dict(k=200), dict(k=2 ** 23),
                dict(ty=2), dict(ty=-1), dict(m=2 ** 23, n=2 ** 30, k=128, wb=1 << 40), dict(m=2 ** 15, n=2 ** 24, k=128, wb=1 << 40)):
        assert dense(**bad) == moe.MOE_ERR_SHAPE, bad
    assert dense(m=-1) == moe.MOE_ERR_TOKENS and dense(m=2 ** 24, k=256) == moe.MOE_ERR_TOKENS
    assert dense(wb=wsb - 1) == moe.MOE_ERR_WORKSPACE
    assert dense(m=0) == moe.MOE_OK

    def contiguous(d=A, ty=1, a=A, asf=A, grp=A, m=64, g=3, n=48, k=256, b=A, ws=A, wb=None):
        wb = moe.moe_fp4_gemm_workspace_bytes(max(m, 0), max(g, 1)) if wb is None else wb
        return call("moe_m_grouped_fp4_gemm_contiguous", d, ty, a, asf, grp, m, g, n, k, b, ws, wb, None)

    for name in ("d", "a", "asf", "grp", "b", "ws"):
        assert contiguous(**{name: None}) == moe.MOE_ERR_NULL, name
        assert contiguous(**{name: A + 4}) == moe.MOE_ERR_ALIGN, name
    assert contiguous(g=0) == moe.MOE_ERR_SHAPE and contiguous(n=24) == moe.MOE_ERR_SHAPE and contiguous(ty=5) == moe.MOE_ERR_SHAPE
    assert contiguous(m=-1) == moe.MOE_ERR_TOKENS
    assert contiguous(wb=moe.moe_fp4_gemm_workspace_bytes(64, 3) - 1) == moe.MOE_ERR_WORKSPACE
    assert contiguous(m=0) == moe.MOE_OK

    def masked(d=A, ty=1, a=A, asf=A, cnt=A, g=3, mm=16, n=48, k=256, b=A, ws=A, wb=None):
        wb = moe.moe_fp4_gemm_workspace_bytes(max(g * mm, 0), max(g, 1)) if wb is None else wb
        return call("moe_m_grouped_fp4_gemm_masked", d, ty, a, asf, cnt, g, mm, 8, n, k, b, ws, wb, None)

    for name in ("d", "a", "asf", "cnt", "b", "ws"):
        assert masked(**{name: None}) == moe.MOE_ERR_NULL, name
        assert masked(**{name: A + 4}) == moe.MOE_ERR_ALIGN, name
    assert masked(g=1025, wb=1 << 30) == moe.MOE_ERR_SHAPE and masked(k=100) == moe.MOE_ERR_SHAPE
    assert masked(mm=-1, wb=1 << 30) == moe.MOE_ERR_TOKENS
    assert masked(wb=moe.moe_fp4_gemm_workspace_bytes(48, 3) - 1) == moe.MOE_ERR_WORKSPACE
    assert masked(mm=0) == moe.MOE_OK
