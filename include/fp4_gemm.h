/*
 * fp4_gemm.h -- C ABI of the 4-bit casts and of the FP4 x FP4 GEMMs, in the same library as the MoE forward (libmoe.so,
 * MI355X / gfx950):
 *   moe_cast_to_fp4     bf16 or FP32 rows -> E2M1 codes with one UE8M0 scale per 1x32 block: the format of the expert
 *                       weights that moe_prepare_weights packs, of B of moe_gemm_prepare_b, and of A below
 *   moe_cast_from_fp4   the numbers that such codes stand for
 *   moe_fp4_gemm, moe_m_grouped_fp4_gemm_contiguous, moe_m_grouped_fp4_gemm_masked
 *                       the GEMMs of fp8_fp4_gemm.h (zevenfang.github.io 2026/04/23 section 二: the dense, M-grouped
 *                       contiguous and M-grouped masked families) with FP4 activations too. B is packed as there: one
 *                       packed buffer serves both.
 *
 *   D[m, n] = sum over k of  A[m, k] * 2^(a_sf[m, k/32] - 127) * B[n, k] * 2^(b_sf[n, k/32] - 127)
 *
 * Formats: E2M1, two per byte, element 2i in the low nibble, rows of K/2 bytes; UE8M0 bytes (2^(b-127), 255: NaN) per
 * 1x32 block along K, rows of K/32 bytes. D is bf16 or FP32, as d_type (MOE_BF16, MOE_F32 of moe_serving.h) says.
 *
 * Sums: FP32 sums of the exact products, in no promised order, rounded once to nearest even for bf16 outputs. Every scale
 * byte from 0 to 254 counts as written; a byte of 255 makes NaN of what it scales, whatever the codes.
 *
 * GEMM shapes: K a positive multiple of 128, at most 2^22; N a multiple of 16 from 16 to 2^30; G (groups) in
 * [1, MOE_MAX_EXPERTS]; the rows of A times K below 2^32 (MOE_ERR_TOKENS); fewer than 2^24 tiles of 128 x 256 in D,
 * counting one part tile per group (MOE_ERR_SHAPE).
 *
 * Memory, errors and streams as in moe.h: device pointers, 16-byte aligned, owned by the caller; host-detectable problems
 * return a negative MOE_ERR_* status before any launch; every call is asynchronous on `stream`, and the buffers belong to
 * the current device, as `stream` does. Calls that share a workspace must not overlap.
 * Results are deterministic.
 */
#ifndef MOE_FP4_GEMM_H
#define MOE_FP4_GEMM_H

#include "moe.h"
#include "moe_serving.h"
#include "fp8_fp4_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* FP4 cast: x [rows][cols] of x_type (MOE_BF16 or MOE_F32), cols a positive multiple of 32 ->
 *   x_fp4  u8 [rows][cols/2] E2M1 pairs, x_sf  u8 [rows][cols/32] UE8M0,
 * per 1x32 block: byte = max(s + 127, 0) with s the least integer such that amax <= 6 * 2^s (s = 0 for an all-zero block),
 * code = E2M1 round-to-nearest-even of x * 2^-(byte - 127), with x's sign also where it rounds to 0. A block that holds an
 * infinity or a NaN gets the byte 255 (NaN) and codes of 0. rows = 0 launches nothing. MOE_ERR_SHAPE: cols, or an unknown
 * x_type; MOE_ERR_TOKENS: rows < 0. */
int moe_cast_to_fp4(const void* x, int32_t x_type, int32_t rows, int32_t cols, uint8_t* x_fp4, uint8_t* x_sf,
                    hipStream_t stream);

/* The cast back: x [rows][cols] = E2M1 * 2^(byte - 127), in x_type. Exact but for infinities above the type's range
 * (bytes of 253 and 254 can reach it) and NaN for a byte of 255. Arguments as moe_cast_to_fp4's. */
int moe_cast_from_fp4(const uint8_t* x_fp4, const uint8_t* x_sf, int32_t rows, int32_t cols, void* x, int32_t x_type,
                      hipStream_t stream);

/* Workspace bytes of a GEMM call whose A has up to `max_rows` rows in `groups` groups (dense: m rows, 1 group; contiguous:
 * m rows; masked: groups * max_m rows). A workspace of moe_gemm_workspace_bytes for the same rows and groups serves as
 * well. Contents need no initialisation. 0 if unsupported. */
size_t moe_fp4_gemm_workspace_bytes(int32_t max_rows, int32_t groups);

/* Dense: d [m][n] = A [m][k] . B^T, B = group 0 of packed_b (moe_gemm_prepare_b). m = 0 launches nothing.
 *   a  u8 [m][k/2]; a_sf  u8 [m][k/32] */
int moe_fp4_gemm(void* d, int32_t d_type, const uint8_t* a, const uint8_t* a_sf, int32_t m, int32_t n, int32_t k,
                 const void* packed_b, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* M-grouped, contiguous layout: row r of A is multiplied by B[group_of_row[r]].
 *   group_of_row  i32 [m] device; rows whose id is outside [0, groups) are skipped, their D rows not written. Rows of one
 *                 group need not be adjacent or aligned. */
int moe_m_grouped_fp4_gemm_contiguous(void* d, int32_t d_type, const uint8_t* a, const uint8_t* a_sf,
                                      const int32_t* group_of_row, int32_t m, int32_t groups, int32_t n, int32_t k,
                                      const void* packed_b, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* M-grouped, masked layout: for each group g and i < clamp(masked_m[g], 0, max_m), d[g, i, :] = A[g, i, :] . B[g]^T;
 * other rows of d are not written.
 *   a u8 [groups][max_m][k/2], a_sf u8 [groups][max_m][k/32], d [groups][max_m][n]
 *   masked_m  i32 [groups] device (read on the device: the call never synchronises)
 *   expected_m  the expected rows per group, a hint that picks the row-tile size. */
int moe_m_grouped_fp4_gemm_masked(void* d, int32_t d_type, const uint8_t* a, const uint8_t* a_sf, const int32_t* masked_m,
                                  int32_t groups, int32_t max_m, int32_t expected_m, int32_t n, int32_t k,
                                  const void* packed_b, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP4_GEMM_H */
