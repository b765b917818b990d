/*
 * moe_serving.h -- C ABI of the operators around the MoE forward that a decoding loop needs,
 * in the same library (libmoe.so, MI355X / gfx950):
 *   moe_topk_router   router logits -> the topk_idx / topk_weights that moe_forward reads
 *                     (chenxutan.com/d/1930 section 9.2: top-k, then softmax over the chosen
 *                     logits)
 *   moe_forward_few   moe_forward for at most MOE_FEW_MAX_TOKENS tokens, in two kernels
 *
 * Formats, memory, errors and streams as in moe.h: device pointers, 16-byte aligned, owned by
 * the caller (the library allocates nothing); host-detectable problems return a negative
 * MOE_ERR_* status before any launch; every call is asynchronous on `stream` and may be
 * captured into a graph. The buffers belong to the current device, and `stream` to it too.
 */
#ifndef MOE_SERVING_H
#define MOE_SERVING_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of logits and of GEMM outputs. */
enum { MOE_BF16 = 0, MOE_F32 = 1 };

/* Which logits the router's softmax runs over. */
enum {
    MOE_ROUTER_SOFTMAX_CHOSEN = 0, /* the chosen ones: a token's weights add up to weight_scale */
    MOE_ROUTER_SOFTMAX_ALL = 1     /* all experts': the chosen probabilities, not renormalised */
};

/* Router: for each token the num_topk experts with the largest logits, in descending order,
 * equal logits in ascending expert order, and their softmax weights times weight_scale.
 *   topk_idx      i32 [T, k] out    topk_weights  f32 [T, k] out, both fully overwritten
 *   logits        [T, E] of logits_type (MOE_BF16 or MOE_F32)
 * An expert whose logit is -inf or NaN is never chosen and adds nothing to the softmax; where
 * fewer than k experts are left, the remaining slots get id -1 (moe_forward's unused slot) and
 * weight 0. Experts at +inf share the weight equally. The softmax is computed in FP32.
 * 1 <= E <= MOE_MAX_EXPERTS, 1 <= k <= min(MOE_MAX_TOPK, E), else MOE_ERR_SHAPE (also for an
 * unknown logits_type or softmax_over, a weight_scale that is not finite, or T * k >= 2^31).
 * num_tokens < 0 is MOE_ERR_TOKENS; num_tokens = 0 launches nothing. */
int moe_topk_router(int32_t* topk_idx, float* topk_weights, const void* logits,
                    int32_t logits_type, int32_t num_tokens, int32_t num_experts,
                    int32_t num_topk, int32_t softmax_over, float weight_scale,
                    hipStream_t stream);

/* Most tokens of one moe_forward_few call. */
#define MOE_FEW_MAX_TOKENS 32

/* Bytes of the workspace moe_forward_few needs for up to min(shape->max_tokens,
 * MOE_FEW_MAX_TOKENS) tokens; a moe_forward workspace of the same shape is always large
 * enough for it. 0 if the shape is unsupported (as moe_forward's, and hidden below 2^27). */
size_t moe_few_workspace_bytes(const moe_shape_t* shape);

/* The forward for a few tokens: moe_forward's arguments, formats and packed weights, with
 * 0 <= num_tokens <= min(max_tokens, MOE_FEW_MAX_TOKENS) (else MOE_ERR_TOKENS). Two kernels:
 * Linear1 with SwiGLU and the FP8 requantisation, then Linear2 with the weighted sum over the
 * token's experts; the weights of the chosen experts are read once each, whatever their number
 * of tokens.
 * Both products run on the FP8 matrix unit, as moe_forward's: FP32 sums of groups of 8 consecutive
 * K, within which what lies more than 13 bits below the largest product is dropped (fp8_gemm.h
 * gives the bound).
 * The result differs from moe_forward's by rounding only: the sum over a token's experts runs
 * in FP32 in ascending expert order (moe_forward rounds each slot's output to bf16 first), and
 * a token that names an expert in several slots has their weights added up. Slots whose id is
 * outside [0, E) add nothing (they are not counted); a token without a valid slot gets zeros.
 * Results do not depend on scheduling (no floating-point atomics).
 *   workspace     >= moe_few_workspace_bytes(shape) bytes, uninitialised; the call writes
 *                 nothing past that many bytes. Calls sharing one must be ordered. It is left
 *                 with the requantised intermediate (for tests and tools): with S =
 *                 min(max_tokens, MOE_FEW_MAX_TOKENS) * k, codes u8 [S][I], then from the next
 *                 multiple of 256 bytes UE8M0 bytes [S][4*ceil(I/512)]; the row of a (token,
 *                 expert) pair is the token's first slot t*k + j that names the expert. */
int moe_forward_few(uint16_t* y_bf16,
                    const uint8_t* x_fp8, const uint8_t* x_sf,
                    const int32_t* topk_idx, const float* topk_weights,
                    int32_t num_tokens, const moe_shape_t* shape, const void* packed,
                    void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_SERVING_H */
