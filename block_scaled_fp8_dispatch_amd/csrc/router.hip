// Top-k router (chenxutan.com/d/1930 section 9.2: topk of the router logits, then a softmax
// over the chosen ones): per token the k largest of E logits in descending order, ties to the
// lowest expert, and their softmax weights.
//
// One wave per token; lane l holds the logits of experts l, 64 + l, .... Each logit becomes an
// unsigned key that orders like the value (0 for -inf and NaN, which are never chosen; -0 and
// +0 share a key, as they compare equal). k rounds: the wave's largest key (DPP maximum), the
// lowest expert that holds it (ballots in ascending expert order), which then drops out. Lane
// j keeps round j's choice, so the softmax over the chosen and the stores are one pass over
// the lanes (k <= 64).
#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

constexpr int kRouterThreads = 256;

__device__ inline uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);                  // -0 -> +0
    if ((b & 0x7fffffffu) > 0x7f800000u || b == 0xff800000u) return 0u;
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ inline float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ inline uint32_t wave_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)m);
}

__device__ inline float wave_sum(float v) {
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// exp(x - m) for x <= m, 1 at x == m (also where both are +inf)
__device__ inline float exp_below(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// V: experts per lane (E <= 64 * V)
template <int V, bool BF16>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(const void* __restrict__ logits, int T, int E, int k,
                                                                int over_all, float scale,
                                                                int32_t* __restrict__ topk_idx,
                                                                float* __restrict__ topk_weights) {
    const int t = (int)(blockIdx.x * (kRouterThreads / 64) + (threadIdx.x >> 6));
    if (t >= T) return;
    const int lane = threadIdx.x & 63;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 64 + lane;
        float x = -INFINITY;
        if (e < E) {
            if constexpr (BF16)
                x = __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[(size_t)t * E + e] << 16);
            else
                x = static_cast<const float*>(logits)[(size_t)t * E + e];
        }
        key[i] = order_key(x);
    }
    uint32_t first = 0;
    float denom = 0.f;
    int my_idx = -1;
    uint32_t my_key = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = max(m, key[i]);
        m = wave_max(m);
        if (m == 0) break;                                  // uniform: nothing left to choose
        if (j == 0) {
            first = m;
            if (over_all) {
                const float top = key_value(m);
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) s += key[i] ? exp_below(key_value(key[i]), top) : 0.f;
                denom = wave_sum(s);
            }
        }
        bool found = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t b = found ? 0ull : __ballot(key[i] == m);
            if (b) {
                found = true;
                const int l = __ffsll((unsigned long long)b) - 1;
                if (lane == l) key[i] = 0;
                if (lane == j) {
                    my_idx = i * 64 + l;
                    my_key = m;
                }
            }
        }
    }
    const float e = my_idx >= 0 ? exp_below(key_value(my_key), key_value(first)) : 0.f;
    if (!over_all) denom = wave_sum(e);
    if (lane < k) {
        topk_idx[(size_t)t * k + lane] = my_idx;
        topk_weights[(size_t)t * k + lane] = my_idx >= 0 ? e / denom * scale : 0.f;
    }
}

template <bool BF16>
void launch(const void* logits, int T, int E, int k, int over_all, float scale, int32_t* idx, float* w,
            hipStream_t stream) {
    const unsigned grid = (unsigned)((T + kRouterThreads / 64 - 1) / (kRouterThreads / 64));
    if (E <= 64)
        router_kernel<1, BF16><<<grid, kRouterThreads, 0, stream>>>(logits, T, E, k, over_all, scale, idx, w);
    else if (E <= 128)
        router_kernel<2, BF16><<<grid, kRouterThreads, 0, stream>>>(logits, T, E, k, over_all, scale, idx, w);
    else if (E <= 256)
        router_kernel<4, BF16><<<grid, kRouterThreads, 0, stream>>>(logits, T, E, k, over_all, scale, idx, w);
    else if (E <= 512)
        router_kernel<8, BF16><<<grid, kRouterThreads, 0, stream>>>(logits, T, E, k, over_all, scale, idx, w);
    else
        router_kernel<16, BF16><<<grid, kRouterThreads, 0, stream>>>(logits, T, E, k, over_all, scale, idx, w);
}

}  // namespace

hipError_t launch_router(const void* logits, int logits_type, int T, int E, int k, int over_all, float scale,
                         int32_t* idx, float* w, hipStream_t stream) {
    if (logits_type == MOE_BF16)
        launch<true>(logits, T, E, k, over_all, scale, idx, w, stream);
    else
        launch<false>(logits, T, E, k, over_all, scale, idx, w, stream);
    return hipGetLastError();
}

}  // namespace moe
