/*
 * fp8_gemm.h -- C ABI of the FP8 x FP8 GEMMs with one scale per block of 128, in the same
 * library as the MoE forward (libmoe.so, MI355X / gfx950): the FP8-weight counterparts of the
 * FP8 x FP4 GEMMs of fp8_fp4_gemm.h (zevenfang.github.io 2026/04/23 section 二: the dense,
 * M-grouped contiguous and M-grouped masked families; chenxutan.com/d/1930 section 11.1: a
 * scale per block; section 4.2: FP32 accumulation).
 *
 *   D[m, n] = sum over k of  A[m, k] * 2^(a_sf[m, k/128] - 127)
 *                          * B[n, k] * 2^(b_sf[n/128, k/128] - 127)
 *
 * Formats: A is OCP e4m3fn, rows of K bytes, with UE8M0 bytes per 1x128 block along K,
 * 4*ceil(K/512) bytes per row, as moe_cast_to_fp8 writes them. B is e4m3fn [G][N][K], read as
 * it is (no packing), with one UE8M0 byte per 128x128 block, [G][ceil(N/128)][4*ceil(K/512)]
 * (byte j of a row = block j along K; bytes past K/128 are ignored). D is bf16 or FP32, as d_type
 * (MOE_BF16, MOE_F32 of moe_serving.h) says.
 *
 * Sums: FP32 outputs are FP32 sums of the exact products (in no promised order). bf16 outputs are
 * sums on the FP8 matrix unit, rounded once to nearest even: within each 8 consecutive K the unit
 * aligns the products to the largest and drops what lies more than 13 bits below it, and adds the
 * groups of 8 in FP32. Beside the error of an FP32 sum that is at most 2^-10 times the sum over the
 * groups of max|a| max|b| (operands with their scales): about 1.5e-5 of D's norm on normal data, 5e-5
 * on codes of every magnitude alike, where bf16's own rounding is 1.7e-3. Where products cancel to
 * well below their size it can be many bf16 steps of the result: take FP32 outputs there.
 *
 * Every scale byte from 0 to 254 counts as written (255: NaN). With FP32 outputs, rows for which
 * one of A's or B's bytes lies outside 3 .. 246 are multiplied a second time in a slower way; their
 * tiles take a few times as long. The other rows' bits do not depend on it.
 *
 * Shapes: K a positive multiple of 128, at most 2^22; N any number from 1 to 2^30; G (groups) in
 * [1, MOE_MAX_EXPERTS]; the rows of A times K below 2^32 (MOE_ERR_TOKENS); fewer than 2^24 tiles
 * of 128 x 256 in D, counting one part tile per group (MOE_ERR_SHAPE); B of any size.
 *
 * Memory, errors and streams as in moe.h: device pointers, 16-byte aligned, owned by the
 * caller; host-detectable problems return a negative MOE_ERR_* status before any launch;
 * every call is asynchronous on `stream`, and the buffers belong to the current device, as
 * `stream` does. Calls that share a workspace must not overlap.
 * Results are deterministic.
 */
#ifndef MOE_FP8_GEMM_H
#define MOE_FP8_GEMM_H

#include "moe.h"
#include "moe_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of a call whose A has up to `max_rows` rows in `groups` groups (dense: m
 * rows, 1 group; contiguous: m rows; masked: groups * max_m rows): the row and tile lists. A
 * workspace of moe_gemm_workspace_bytes for the same rows and groups serves as well. Contents
 * need no initialisation. 0 if unsupported. */
size_t moe_fp8_gemm_workspace_bytes(int32_t max_rows, int32_t groups);

/* Dense: d [m][n] = A [m][k] . B [n][k]^T. m = 0 launches nothing. */
int moe_fp8_gemm(void* d, int32_t d_type, const uint8_t* a, const uint8_t* a_sf, int32_t m,
                 int32_t n, int32_t k, const uint8_t* b, const uint8_t* b_sf, void* workspace,
                 size_t workspace_bytes, hipStream_t stream);

/* M-grouped, contiguous layout: row r of A is multiplied by B[group_of_row[r]].
 *   group_of_row  i32 [m] device; rows whose id is outside [0, groups) are skipped, their D
 *                 rows not written. Rows of one group need not be adjacent or aligned. */
int moe_m_grouped_fp8_gemm_contiguous(void* d, int32_t d_type, const uint8_t* a,
                                      const uint8_t* a_sf, const int32_t* group_of_row,
                                      int32_t m, int32_t groups, int32_t n, int32_t k,
                                      const uint8_t* b, const uint8_t* b_sf, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/* M-grouped, masked layout: for each group g and i < clamp(masked_m[g], 0, max_m),
 * d[g, i, :] = A[g, i, :] . B[g]^T; other rows of d are not written.
 *   a u8 [groups][max_m][k], a_sf u8 [groups][max_m][4*ceil(k/512)], d [groups][max_m][n]
 *   masked_m  i32 [groups] device (read on the device: the call never synchronises)
 *   expected_m  the expected rows per group, a hint that picks the row-tile size. */
int moe_m_grouped_fp8_gemm_masked(void* d, int32_t d_type, const uint8_t* a, const uint8_t* a_sf,
                                  const int32_t* masked_m, int32_t groups, int32_t max_m,
                                  int32_t expected_m, int32_t n, int32_t k, const uint8_t* b,
                                  const uint8_t* b_sf, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_GEMM_H */
