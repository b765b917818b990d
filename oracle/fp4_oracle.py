"""Plain fp64 CPU oracle of the 4-bit casts, the FP4 x FP4 GEMM and the norm with FP8 output (numpy).

TEST INFRASTRUCTURE: shares no code with the HIP path and imports nothing from it.

Sources: chenxutan.com/d/1930 sections 4.1-4.2 (E2M1, UE8M0, FP32 accumulation), 11.1 (a scale per block), 9.2 (the
activation as FP8 codes and scales before the MoE call). Readings: E2M1 rounds to nearest, ties to the even code, and keeps
the sign of what rounds to 0; a block with an infinity or a NaN has the scale byte 255.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import bf16_rne_bits, dequant_fp4_rows

_U32 = 2.0 ** -24
E2M1_MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode_e2m1_rne(v: np.ndarray) -> np.ndarray:
    """E2M1 codes u8 of fp64 values within [-6, 6]: the nearest magnitude, a tie to the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)[..., None]
    far = np.abs(a - E2M1_MAGNITUDES)
    nearest = far == far.min(-1, keepdims=True)
    # of two nearest, the even code
    even = np.arange(8) % 2 == 0
    pick = np.where(nearest.sum(-1, keepdims=True) > 1, nearest & even, nearest)
    return (pick.argmax(-1) | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def fp4_exponent(amax: np.ndarray) -> np.ndarray:
    """The least integer s >= -127 with amax <= 6 * 2^s; 0 for amax 0."""
    amax = np.asarray(amax, dtype=np.float64)
    s = np.full(amax.shape, -127, dtype=np.int64)
    for e in range(-127, 128):
        s += (amax > 6.0 * 2.0 ** e).astype(np.int64)
    return np.where(amax == 0, 0, s)


def cast_to_fp4(x: np.ndarray):
    """fp64 rows [R, C] (the exact values of the bf16 or FP32 input) -> packed codes u8 [R, C/2], scale bytes u8 [R, C/32]."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    b = x.reshape(R, C // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    s = fp4_exponent(np.abs(b).max(-1))
    code = encode_e2m1_rne(b * 2.0 ** -s[..., None].astype(np.float64))
    code[bad] = 0
    code = code.reshape(R, C)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, s + 127).astype(np.uint8)


def cast_from_fp4(q: np.ndarray, sf: np.ndarray) -> np.ndarray:
    """fp64 values [R, C] of the codes (NaN for a scale byte of 255)."""
    q = np.asarray(q)
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1)
    v = np.where(code >= 8, -1.0, 1.0) * E2M1_MAGNITUDES[code & 7]
    scale = np.where(sf == 255, np.nan, 2.0 ** (np.asarray(sf, dtype=np.float64) - 127))
    return v * np.repeat(scale, 32, axis=1)


def fp4_gemm(a: np.ndarray, a_sf: np.ndarray, b: np.ndarray, b_sf: np.ndarray, K: int):
    """D = A . B^T (a u8 [M, K/2], b u8 [N, K/2]). Returns exact (fp64), bits (bf16 RNE of exact) and bound
    (gamma_{K-1} * sum |a b|, how far any FP32 summation order can land)."""
    A = dequant_fp4_rows(np.asarray(a), np.asarray(a_sf), K)
    B = dequant_fp4_rows(np.asarray(b), np.asarray(b_sf), K)
    exact = A @ B.T
    gamma = (K - 1) * _U32 / (1.0 - (K - 1) * _U32)
    return {"exact": exact, "bits": bf16_rne_bits(exact), "bound": gamma * (np.abs(A) @ np.abs(B).T)}


def rmsnorm(x: np.ndarray, residual, weight: np.ndarray, eps: float):
    """fp64 (h, n) of fp64 rows: h = x + residual rounded to FP32 as the operator's sum is, n = h * weight / sqrt(mean(h^2)
    + eps)."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = (h.astype(np.float32) + np.asarray(residual, dtype=np.float32)).astype(np.float64)
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    return h, h * r * np.asarray(weight, dtype=np.float64)
