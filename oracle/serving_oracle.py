"""Plain fp64 CPU oracle of the serving operators (numpy): the top-k router and the FP8 x FP8
GEMM with one scale per block of 128. The few-token forward has the forward's own oracle
(moe_oracle.forward).

TEST INFRASTRUCTURE: shares no code with the HIP path and imports nothing from it.

Sources: chenxutan.com/d/1930 sections 9.2 (top-k, then a softmax over the chosen logits),
11.1 (a scale per block), 4.2 (FP32 accumulation); zevenfang.github.io 2026/04/23 section 二
(the GEMM family). Readings: equal logits go to the lowest expert; -inf and NaN logits are
never chosen; B's scales are UE8M0 per 128x128 block.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import bf16_rne_bits, decode_e4m3, decode_ue8m0, dequant_fp8_rows

_U32 = 2.0 ** -24


def topk_router(logits: np.ndarray, k: int, over_all: bool, scale: float = 1.0):
    """logits fp64 [T, E] -> (idx i32 [T, k], weights fp64 [T, k]); see moe_serving.h."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    T, E = x.shape
    idx = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))[:k]
        if not order:
            continue
        m = x[t, order[0]]

        def ex(v):
            return 1.0 if v == m else float(np.exp(v - m))
        over = range(E) if over_all else order
        den = sum(ex(x[t, e]) for e in over if x[t, e] > -np.inf)
        for j, e in enumerate(order):
            idx[t, j] = e
            w[t, j] = scale * ex(x[t, e]) / den
    return idx, w


def dequant_fp8_blocks(codes: np.ndarray, sf: np.ndarray, K: int) -> np.ndarray:
    """b[n, c] = e4m3(codes[n, c]) * 2^(sf[n // 128, c // 128] - 127)."""
    N = codes.shape[0]
    scale = decode_ue8m0(np.asarray(sf)[:, : K // 128])
    rows = np.repeat(np.repeat(scale, 128, axis=0)[:N], 128, axis=1)
    return decode_e4m3(codes) * rows


def fp8_gemm(a, a_sf, b, b_sf, K: int):
    """D = A . B^T (a u8 [M, K], b u8 [N, K]). Returns exact (fp64), bits (bf16 RNE of exact)
    and bound (gamma_{K-1} * sum |a b|, how far any FP32 summation order can land)."""
    A = dequant_fp8_rows(np.asarray(a), np.asarray(a_sf), K)
    B = dequant_fp8_blocks(np.asarray(b), np.asarray(b_sf), K)
    exact = A @ B.T
    gamma = (K - 1) * _U32 / (1.0 - (K - 1) * _U32)
    return {"exact": exact, "bits": bf16_rne_bits(exact), "bound": gamma * (np.abs(A) @ np.abs(B).T)}


def gemm_f32_within_bound(d: np.ndarray, exact: np.ndarray, bound: np.ndarray) -> np.ndarray:
    """Per element: |d - exact| within the FP32 accumulation bound and one FP32 rounding."""
    return np.abs(np.asarray(d, dtype=np.float64) - exact) <= bound + _U32 * (np.abs(exact) + bound) + 2.0 ** -149
