// C ABI of the router, of the norm with FP8 output and of the few-token forward (include/moe_serving.h): argument checks
// and launches. Host code only.
#include <cmath>

#include "moe_serving.h"
#include "moe_internal.h"

namespace {
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// 512 threads per 32 columns of the output have to stay below a launch's 2^32
bool few_shape_ok(const moe_shape_t* s) { return moe::shape_ok(s) && s->hidden < (1 << 27); }
}  // namespace

using namespace moe;

extern "C" {

int moe_topk_router(int32_t* topk_idx, float* topk_weights, const void* logits, int32_t logits_type,
                    int32_t num_tokens, int32_t num_experts, int32_t num_topk, int32_t softmax_over,
                    float weight_scale, hipStream_t stream) {
    if (!topk_idx || !topk_weights || !logits) return MOE_ERR_NULL;
    if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS) return MOE_ERR_SHAPE;
    if (num_topk < 1 || num_topk > MOE_MAX_TOPK || num_topk > num_experts) return MOE_ERR_SHAPE;
    if (logits_type != MOE_BF16 && logits_type != MOE_F32) return MOE_ERR_SHAPE;
    if (softmax_over != MOE_ROUTER_SOFTMAX_CHOSEN && softmax_over != MOE_ROUTER_SOFTMAX_ALL) return MOE_ERR_SHAPE;
    if (!std::isfinite(weight_scale)) return MOE_ERR_SHAPE;
    if (num_tokens < 0) return MOE_ERR_TOKENS;
    if ((uint64_t)num_tokens * (uint64_t)num_topk >= (1ull << 31)) return MOE_ERR_SHAPE;
    if (!aligned16(topk_idx) || !aligned16(topk_weights) || !aligned16(logits)) return MOE_ERR_ALIGN;
    if (num_tokens == 0) return MOE_OK;
    if (launch_router(logits, logits_type, num_tokens, num_experts, num_topk,
                      softmax_over == MOE_ROUTER_SOFTMAX_ALL, weight_scale, topk_idx, topk_weights,
                      stream) != hipSuccess)
        return MOE_ERR_HIP;
    return MOE_OK;
}

int moe_rmsnorm_to_fp8(uint8_t* x_fp8, uint8_t* x_sf, uint16_t* normed, uint16_t* residual_out, const uint16_t* x,
                       const uint16_t* residual, const void* weight, int32_t weight_type, int32_t rows, int32_t cols, float eps,
                       hipStream_t stream) {
    if (!x_fp8 || !x_sf || !x || !weight) return MOE_ERR_NULL;
    if (cols < 128 || cols % 128 != 0 || (weight_type != MOE_BF16 && weight_type != MOE_F32)) return MOE_ERR_SHAPE;
    if (!std::isfinite(eps) || eps <= 0.0f) return MOE_ERR_SHAPE;
    if (rows < 0) return MOE_ERR_TOKENS;
    if (!aligned16(x_fp8) || !aligned16(x_sf) || !aligned16(normed) || !aligned16(residual_out) || !aligned16(x) ||
        !aligned16(residual) || !aligned16(weight))
        return MOE_ERR_ALIGN;
    if (rows == 0) return MOE_OK;
    if (launch_rmsnorm(x, residual, weight, weight_type, rows, cols, eps, x_fp8, x_sf, normed, residual_out, stream) != hipSuccess)
        return MOE_ERR_HIP;
    return MOE_OK;
}

size_t moe_few_workspace_bytes(const moe_shape_t* shape) {
    if (!few_shape_ok(shape)) return 0;
    return few_layout(*shape).total;
}

int moe_forward_few(uint16_t* y_bf16, const uint8_t* x_fp8, const uint8_t* x_sf, const int32_t* topk_idx,
                    const float* topk_weights, int32_t num_tokens, const moe_shape_t* shape, const void* packed,
                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!shape) return MOE_ERR_NULL;
    if (!few_shape_ok(shape)) return MOE_ERR_SHAPE;
    if (num_tokens < 0 || num_tokens > shape->max_tokens || num_tokens > MOE_FEW_MAX_TOKENS) return MOE_ERR_TOKENS;
    if (!y_bf16 || !x_fp8 || !x_sf || !topk_idx || !topk_weights || !packed || !workspace) return MOE_ERR_NULL;
    if (!aligned16(y_bf16) || !aligned16(x_fp8) || !aligned16(x_sf) || !aligned16(topk_idx) ||
        !aligned16(topk_weights) || !aligned16(packed) || !aligned16(workspace))
        return MOE_ERR_ALIGN;
    if (workspace_bytes < few_layout(*shape).total) return MOE_ERR_WORKSPACE;
    if (num_tokens == 0) return MOE_OK;
    if (launch_few(*shape, packed_layout(*shape), x_fp8, x_sf, topk_idx, topk_weights, num_tokens,
                   static_cast<const uint8_t*>(packed), static_cast<uint8_t*>(workspace), y_bf16,
                   stream) != hipSuccess)
        return MOE_ERR_HIP;
    return MOE_OK;
}

}  // extern "C"
