"""FP8 x FP8 GEMMs over the whole range of UE8M0 scale bytes: products that are ordinary numbers although one
operand times its own scale passes FP32's range, scales that differ from row to row and from block
to block, and results at FP32's own ends.

Tolerance: the bounds of test_gpu_fp8_gemm.py. FP32 outputs near FP32's smallest numbers are sums of K
products, each of which (and each sum) may be rounded to a multiple of 2^-149: K - 1 sums and K products are
off by at most 2^-150 each, less than K * 2^-149 in all. bf16 outputs likewise, and their half step is
at most 2^-134 there. Where the exact result is within the bound of FP32's (bf16's) largest number it may be
infinite or not; codes of one sign keep every partial sum below the whole."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402
from test_gpu_fp8_gemm import Problem  # noqa: E402

# both ends of the byte's range and the borders at which an e4m3 code's product with its scale leaves
# bf16's: 448 * 2^119 and 2^-9 * 2^-124 are the last that it holds
ENDS = [0, 1, 2, 3, 4, 9, 10, 11, 117, 127, 137, 243, 244, 245, 246, 247, 248, 250, 251, 252, 253, 254]

# (rows, columns, K): from the smallest tiles to the largest of both output types
SHAPES = [(5, 40, 640), (48, 96, 1024), (130, 511, 1152), (300, 640, 2176), (1000, 2000, 1024), (1100, 2600, 640)]


def set_scales(p, a_sf, b_sf):
    nb = p.K // 128
    p.a_sf[:, :nb], p.b_sf[:, :, :nb] = a_sf, b_sf
    p.dev[1], p.dev[3] = torch.from_numpy(p.a_sf).cuda(), torch.from_numpy(p.b_sf).cuda()


def cancelling(p, seed):
    """B's scale bytes from ENDS by block; A's so that every product's scale is about 1."""
    rng = np.random.default_rng(seed)
    nb = p.K // 128
    base = rng.choice(ENDS, nb)
    b_sf = np.clip(base + rng.integers(-1, 2, (p.G, p.b_sf.shape[1], nb)), 0, 254)
    a_sf = np.clip(254 - base + rng.integers(-4, 5, (p.rows, nb)), 0, 254)
    set_scales(p, a_sf, b_sf)


def close(p, got, rows, g=0):
    ref = oracle.fp8_gemm(p.a[rows], p.a_sf[rows], p.b[g], p.b_sf[g], p.K)
    exact, tiny = ref["exact"], p.K * 2.0 ** -149
    if p.d_type == moe.MOE_F32:
        got = got[rows].view(np.float32).astype(np.float64)
        bound = ref["bound"] + 2.0 ** -24 * (np.abs(exact) + ref["bound"]) + tiny
        largest = float(np.finfo(np.float32).max)
    else:
        got = (got[rows].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        bound = ref["bound"] + p.alignment(rows, g)
        bound = bound + 2.0 ** -8 * (np.abs(exact) + bound) + tiny + 2.0 ** -134
        largest = (2 - 2.0 ** -7) * 2.0 ** 127
    over, border = np.abs(exact) > largest + bound, np.abs(np.abs(exact) - largest) <= bound
    with np.errstate(invalid="ignore"):
        ok = np.where(over, np.isinf(got), (np.abs(got - exact) <= bound) | (border & np.isinf(got)))
    assert ok.all(), f"{(~ok).sum()} of {ok.size} off, first at {np.argwhere(~ok)[0]}"


def some(M):
    return np.unique(np.r_[0:min(M, 70), M // 2, M - 1 - np.arange(min(M, 40))])


@pytest.mark.parametrize("d_type", [moe.MOE_BF16, moe.MOE_F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_that_cancel(M, N, K, d_type):
    print(f"[fp8] range, dense {M} {N} {K} {d_type}", flush=True)
    p = Problem(M, N, K, 1, d_type, seed=M)
    for seed in (1, 2):
        cancelling(p, seed)
        close(p, p.dense(), some(M))


@pytest.mark.parametrize("d_type", [moe.MOE_BF16, moe.MOE_F32])
@pytest.mark.parametrize("M,N", [(510, 900), (260, 2100), (40, 300)])
def test_every_pair_of_ends(M, N, d_type):
    """One block along K: row r has byte r mod 255, the 128-column blocks bytes from ENDS, so that results range from
    zero to infinity; codes are not negative."""
    print(f"[fp8] pairs, dense {M} {N} {d_type}", flush=True)
    p = Problem(M, N, 128, 1, d_type, seed=N)
    p.a &= 0x7F
    p.b &= 0x7F
    p.dev[0], p.dev[2] = torch.from_numpy(p.a).cuda(), torch.from_numpy(p.b).cuda()
    rng = np.random.default_rng(M)
    for _ in range(3):
        set_scales(p, (np.arange(M)[:, None] * 7) % 255, rng.choice(ENDS, (1, p.b_sf.shape[1], 1)))
        close(p, p.dense(), np.arange(M))


@pytest.mark.parametrize("d_type", [moe.MOE_BF16, moe.MOE_F32])
def test_grouped(d_type):
    G, M, N, K = 5, 900, 392, 768
    p = Problem(M, N, K, G, d_type, seed=3)
    grp = np.random.default_rng(3).integers(-1, G, size=M).astype(np.int32)
    cancelling(p, 3)
    d = p.contiguous(grp)
    for g in range(G):
        close(p, d, np.nonzero(grp == g)[0], g)
    max_m = M // G
    cnt = np.array([max_m, 0, 7, 65, 128], dtype=np.int32)
    for expected in (1, 64, 400):
        d = p.masked(cnt, max_m, expected)
        for g in range(G):
            if cnt[g]:
                close(p, d, g * max_m + np.arange(cnt[g]), g)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_other_rows_keep_their_bytes(M, N, K):
    """A row whose scales are at the ends of their range changes no bit of the other rows."""
    p = Problem(M, N, K, 1, moe.MOE_F32, seed=M + 1)
    clean = p.dense()
    rng = np.random.default_rng(M)
    rows = rng.choice(M, max(1, M // 9), replace=False)
    a_sf = p.a_sf[:, : K // 128].copy()
    a_sf[rows] = rng.choice([0, 1, 2, 247, 254, 255], (len(rows), K // 128))
    set_scales(p, a_sf, p.b_sf[:, :, : K // 128])
    d = p.dense()
    others = np.setdiff1d(np.arange(M), rows)
    assert np.array_equal(d[others], clean[others])
    assert not np.array_equal(d[rows], clean[rows])


@pytest.mark.parametrize("d_type", [moe.MOE_BF16, moe.MOE_F32])
def test_nan_codes_and_scales_next_to_the_ends(d_type):
    """Byte 255 and a NaN code give NaN next to scales at the ends of their range, in their row or columns only."""
    M, N, K = 200, 300, 512
    p = Problem(M, N, K, 1, d_type, seed=8)
    a_sf = np.full((M, 4), 254)
    b_sf = np.zeros((1, 3, 4), dtype=np.int64)
    a_sf[3, 1], b_sf[0, 2, 3] = 255, 255
    set_scales(p, a_sf, b_sf)
    p.dev[0][4, 100] = 0x7F
    p.dev[2][0, 17, 300] = 0xFF
    d = p.dense()
    v = d.view(np.float32) if d_type == moe.MOE_F32 else (d.astype(np.uint32) << 16).view(np.float32)
    bad = np.zeros((M, N), dtype=bool)
    bad[[3, 4]] = True
    bad[:, 17] = True
    bad[:, 256:] = True
    assert np.isnan(v[bad]).all() and np.isfinite(v[~bad]).all()
