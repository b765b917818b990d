// Top-k router (chenxutan.com/d/1930 section 9.2: topk of the router logits, then a softmax
// over the chosen ones): per token the k largest of E logits in descending order, ties to the
// lowest expert, and their softmax weights.
//
// Each logit becomes an integer key that orders like the value (-inf and NaN below all, never
// chosen; -0 and +0 share a key, as they compare equal).
//
// router_kernel (k <= 16): 16 lanes per token up to E = 256 (32 or 64 beyond), at most 16 experts
// per lane, as up to four lists in descending order. A key keeps its upper bits and carries its
// expert in the lower ones (16 bits for bf16 logits, which lose nothing; log2 of the experts held
// for FP32), so a round is one maximum over the heads and the token's lanes (DPP), and the list
// whose head it was moves up; the expert comes out of the key. For FP32 logits with bits below the
// kept ones, where neighbours in the resulting order (the best one left over included) agree in
// the kept bits, the wave chooses again by whole keys; elsewhere the order is that of the whole
// keys. A wave takes several passes, the next one's logits loading while it chooses.
//
// router_wave_kernel (k > 16): one wave per token, lane l holding experts l, 64 + l, ...: k rounds
// of the wave's largest key and the lowest expert that holds it.
//
// 32768 x 256 FP32 logits, top-8: 12.0 us a call among others (2.8 TB/s of logits; a copy of the kernel that only
// loads them takes 7.2), 12.9 where calls follow one another in a graph, bound by the vector instructions of the key sorts and of the rounds. 128 x 256: 5.2 us,
// a launch and one chain of dependent rounds. One wave per token takes 22 us for the first.
#include <algorithm>

#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

constexpr int kRouterThreads = 256;
constexpr unsigned kRouterGroups = 2048;
constexpr unsigned kWaveGroups = 1u << 20;

__device__ inline uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);                  // -0 -> +0
    if ((b & 0x7fffffffu) > 0x7f800000u || b == 0xff800000u) return 0u;
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ inline float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// One DPP step: v, combined by the caller, of the lane that CTRL names; lanes without one (or
// in rows outside ROWS) get `old`
template <int CTRL, int ROWS = 0xF>
__device__ inline uint32_t dpp(uint32_t old, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xF, false);
}

// Largest of the 64 lanes' values, uniform: neighbours, pairs, half rows and rows mirrored, then
// lane 15 of each row into the next and lane 31 into the upper half
__device__ inline uint32_t wave_max(uint32_t m) {
    m = max(m, dpp<0xB1>(0, m));
    m = max(m, dpp<0x4E>(0, m));
    m = max(m, dpp<0x141>(0, m));
    m = max(m, dpp<0x140>(0, m));
    m = max(m, dpp<0x142, 0xA>(0, m));
    m = max(m, dpp<0x143, 0xC>(0, m));
    return (uint32_t)__builtin_amdgcn_readlane((int)m, 63);
}

// Sum of the 64 lanes' values, uniform, by the same steps
__device__ inline float wave_sum(float v) {
    const auto add = [](float x, uint32_t y) __attribute__((always_inline)) { return x + __uint_as_float(y); };
    v = add(v, dpp<0xB1>(0, __float_as_uint(v)));
    v = add(v, dpp<0x4E>(0, __float_as_uint(v)));
    v = add(v, dpp<0x141>(0, __float_as_uint(v)));
    v = add(v, dpp<0x140>(0, __float_as_uint(v)));
    v = add(v, dpp<0x142, 0xA>(0, __float_as_uint(v)));
    v = add(v, dpp<0x143, 0xC>(0, __float_as_uint(v)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// A signed key that orders like the value: negative values' magnitude bits inverted, -0 as +0
__device__ inline int signed_key(float x) {
    const int bits = __float_as_int(x + 0.0f);
    return bits ^ (int)((uint32_t)(bits >> 31) >> 1);
}

// exp(x - m) for x <= m, 1 at x == m (also where both are +inf)
__device__ inline float exp_below(float x, float m) { return x == m ? 1.0f : expf(x - m); }

template <bool BF16>
__device__ inline float load_logit(const void* logits, size_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[i] << 16);
    else return static_cast<const float*>(logits)[i];
}

// One token by the whole wave. V: experts per lane (E <= 64 * V)
template <int V, bool BF16>
__device__ inline void route_token(const void* __restrict__ logits, int t, int E, int k, int over_all, float scale, int lane,
                                   int32_t* __restrict__ topk_idx, float* __restrict__ topk_weights) {
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 64 + lane;
        key[i] = order_key(e < E ? load_logit<BF16>(logits, (size_t)t * E + e) : -INFINITY);
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
        // the first i, then the lowest lane, that holds m
        uint64_t hit = __ballot(key[0] == m);
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i) {
            const uint64_t h = __ballot(key[i] == m);
            if (!hit) {
                hit = h;
                at = i;
            }
        }
        const int l = __ffsll((unsigned long long)hit) - 1;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (at == i) key[i] = lane == l ? 0 : key[i];         // uniform branch
        my_idx = lane == j ? at * 64 + l : my_idx;
        my_key = lane == j ? m : my_key;
    }
    const float e = my_idx >= 0 ? exp_below(key_value(my_key), key_value(first)) : 0.f;
    if (!over_all) denom = wave_sum(e);
    if (lane < k) {
        topk_idx[(size_t)t * k + lane] = my_idx;
        topk_weights[(size_t)t * k + lane] = my_idx >= 0 ? e / denom * scale : 0.f;
    }
}

template <int V, bool BF16>
__global__ __launch_bounds__(kRouterThreads) void router_wave_kernel(const void* __restrict__ logits, int T, int E, int k,
                                                                     int over_all, float scale,
                                                                     int32_t* __restrict__ topk_idx,
                                                                     float* __restrict__ topk_weights) {
    const uint32_t stride = gridDim.x * (kRouterThreads / 64);
    for (uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)(blockIdx.x * (kRouterThreads / 64) + (threadIdx.x >> 6)));
         t < (uint32_t)T; t += stride)
        route_token<V, BF16>(logits, (int)t, E, k, over_all, scale, threadIdx.x & 63, topk_idx, topk_weights);
}

// The largest (sum) of a token's L lanes, in each of them: within rows of 16 by DPP, across rows
// by swapping the odd rows, then the halves
template <int L>
__device__ inline int lanes_max(int m) {
    m = max(m, (int)dpp<0xB1>(0, (uint32_t)m));
    m = max(m, (int)dpp<0x4E>(0, (uint32_t)m));
    m = max(m, (int)dpp<0x141>(0, (uint32_t)m));
    m = max(m, (int)dpp<0x140>(0, (uint32_t)m));
    if constexpr (L >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap((uint32_t)m, (uint32_t)m, false, false);
        m = max((int)p[0], (int)p[1]);
    }
    if constexpr (L >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap((uint32_t)m, (uint32_t)m, false, false);
        m = max((int)p[0], (int)p[1]);
    }
    return m;
}

template <int L>
__device__ inline float lanes_sum(float v) {
    v += __uint_as_float(dpp<0xB1>(0, __float_as_uint(v)));
    v += __uint_as_float(dpp<0x4E>(0, __float_as_uint(v)));
    v += __uint_as_float(dpp<0x141>(0, __float_as_uint(v)));
    v += __uint_as_float(dpp<0x140>(0, __float_as_uint(v)));
    if constexpr (L >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if constexpr (L >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return v;
}

// 64/L tokens per wave, V experts per lane (E <= L * V), k <= 16. Q: experts of a lane that are
// adjacent and loaded at once (4: E % 4 == 0)
template <int L, int V, bool BF16, int Q>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(const void* __restrict__ logits, int T, int E, int k,
                                                                int over_all, float scale,
                                                                int32_t* __restrict__ topk_idx,
                                                                float* __restrict__ topk_weights) {
    // gfx950 buffer descriptors are a device-only type: the host pass sees an empty kernel
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int kTokens = 64 / L;                        // per wave
    constexpr int LISTS = V < 4 ? V : 4, D = V / LISTS;
    constexpr int kNone = -0x7fffffff - 1;                 // below every key: nothing (left)
    constexpr uint32_t IDX = BF16 ? 0xffffu : L * V - 1;   // bits of the packed key that hold the expert
    static_assert((IDX & (IDX + 1)) == 0 && (int)IDX + 1 >= L * V, "");
    const int lane = threadIdx.x & 63, l = lane & (L - 1);
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(blockIdx.x * (kRouterThreads / 64) + (threadIdx.x >> 6)));
    const uint32_t tokens = (uint32_t)T, stride = gridDim.x * (kRouterThreads / 64) * kTokens;
    // The logits of a pass, one pass ahead: buffer loads from the pass's first row on, so that one
    // offset register serves them all. What lies past a row's end is never looked at; past the
    // last row the loads return 0.
    constexpr int kBytes = BF16 ? 2 : 4;
    const uint32_t offset = (uint32_t)(lane / L * E + l * Q) * kBytes;
    // expert i of a lane, less the lane's own part
    auto base = [](int i) __attribute__((always_inline)) -> int { return i / Q * (Q * L) + i % Q; };
    float ahead[V];
    auto load = [&](uint32_t t0) __attribute__((always_inline)) {
        const size_t rest = (size_t)(tokens - t0) * E * kBytes;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(static_cast<const uint8_t*>(logits) + (size_t)t0 * E * kBytes), 0,
            (int)(uint32_t)(rest < 0xffffffffu ? rest : 0xffffffffu), 0x00020000);
#pragma unroll
        for (int i = 0; i < V; i += Q) {
            if constexpr (Q == 4 && BF16) {
                typedef uint32_t v2u __attribute__((ext_vector_type(2)));
                const v2u x = __builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(rs, offset + i * L * kBytes, 0, 0));
#pragma unroll
                for (int q = 0; q < 4; ++q) ahead[i + q] = __uint_as_float(q % 2 ? x[q / 2] & 0xffff0000u : x[q / 2] << 16);
            } else if constexpr (Q == 4) {
                typedef float v4f __attribute__((ext_vector_type(4)));
                const v4f x = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, offset + i * L * kBytes, 0, 0));
#pragma unroll
                for (int q = 0; q < 4; ++q) ahead[i + q] = x[q];
            } else if constexpr (BF16)
                ahead[i] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rs, offset + i * L * kBytes, 0, 0) << 16);
            else
                ahead[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, offset + i * L * kBytes, 0, 0));
        }
    };
    uint32_t t0 = wave * kTokens;
    if (t0 >= tokens) return;
    load(t0);
    for (; t0 < tokens; t0 += stride) {
    const uint32_t t = t0 + lane / L;
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = ahead[i];
    if (t0 + stride < tokens) load(t0 + stride);
    // whether x[i] may be chosen (false for a NaN)
    auto valid = [&](int i) __attribute__((always_inline)) -> bool { return x[i] > -INFINITY && l * Q < E - i / Q * (Q * L); };
    int h[LISTS][D];
    uint32_t low = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        low |= __float_as_uint(x[i]);
        h[i / D][i % D] = valid(i) ? (int)(((uint32_t)signed_key(x[i]) & ~IDX) | (IDX - (uint32_t)(base(i) + l * Q))) : kNone;
    }
    // every list in descending order
    auto order = [&](int& a, int& b) __attribute__((always_inline)) {
        const int hi = max(a, b);
        b = min(a, b);
        a = hi;
    };
#pragma unroll
    for (int s = 0; s < LISTS; ++s) {
        if constexpr (D == 2) order(h[s][0], h[s][1]);
        if constexpr (D == 4) {
            order(h[s][0], h[s][1]);
            order(h[s][2], h[s][3]);
            order(h[s][0], h[s][2]);
            order(h[s][1], h[s][3]);
            order(h[s][1], h[s][2]);
        }
    }
    auto head = [&]() __attribute__((always_inline)) -> int {
        int m = h[0][0];
#pragma unroll
        for (int s = 1; s < LISTS; ++s) m = max(m, h[s][0]);
        return lanes_max<L>(m);
    };
    int mine = kNone;
    for (int j = 0; j < k; ++j) {
        const int m = head();
#pragma unroll
        for (int s = 0; s < LISTS; ++s) {
            const bool hit = h[s][0] == m;
#pragma unroll
            for (int d = 0; d < D; ++d) h[s][d] = hit ? (d + 1 < D ? h[s][d + 1] : kNone) : h[s][d];
        }
        mine = l == j ? m : mine;
    }
    int idx = mine != kNone ? (int)(IDX - ((uint32_t)mine & IDX)) : -1;
    // Where a logit has bits below the packed ones, two neighbours in the order that agree in the
    // bits kept may be in the wrong order: the wave then chooses again by whole keys.
    if (!BF16 && __ballot((low & IDX) != 0)) {
        const int left = head(), right = (int)dpp<0x101>((uint32_t)kNone, (uint32_t)mine);   // best left over, next lane's
        const int next = l == k - 1 ? left : right;
        if (__ballot(l < k && mine != kNone && next != kNone && ((uint32_t)(mine ^ next) & ~IDX) == 0)) {
            int key[V];
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = valid(i) ? signed_key(x[i]) : kNone;
            idx = -1;
            for (int j = 0; j < k; ++j) {
                int m = key[0];
#pragma unroll
                for (int i = 1; i < V; ++i) m = max(m, key[i]);
                m = lanes_max<L>(m);
                int lowest = 0x7fffffff;           // expert among those that hold m
#pragma unroll
                for (int i = 0; i < V; ++i) lowest = min(lowest, key[i] == m ? base(i) + l * Q : 0x7fffffff);
                lowest = -lanes_max<L>(-lowest);
#pragma unroll
                for (int i = 0; i < V; ++i) key[i] = base(i) + l * Q == lowest ? kNone : key[i];
                if (l == j && m != kNone) idx = lowest;
            }
        }
    }
    const float v = idx >= 0 && t < tokens ? load_logit<BF16>(logits, (size_t)t * E + idx) : -INFINITY;
    const float top = __shfl(v, lane & ~(L - 1), 64);
    const float e = idx >= 0 ? exp_below(v, top) : 0.f;
    float denom;
    if (over_all) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += valid(i) ? exp_below(x[i], top) : 0.f;
        denom = lanes_sum<L>(s);
    } else {
        denom = lanes_sum<16>(e);                  // the chosen sit in the token's first 16 lanes
    }
    if (l < k && t < tokens) {
        topk_idx[(size_t)t * k + l] = idx;
        topk_weights[(size_t)t * k + l] = idx >= 0 ? e / denom * scale : 0.f;
    }
    }
#endif
}

template <bool BF16>
void launch(const void* logits, int T, int E, int k, int over_all, float scale, int32_t* idx, float* w,
            hipStream_t stream) {
    auto grid = [&](int tokens) { return (unsigned)(((long long)T + 4 * tokens - 1) / (4 * tokens)); };
    // passes: at most 8 waves per SIMD, whose next logits arrive while they choose. A wave a token: as many
    // waves as tokens, below the 2^32 threads of a launch (8 per SIMD in passes: 32768 x 256, top-20, 54 us
    // instead of 47, since nothing is loaded ahead)
    auto run = [&](auto kernel, int tokens, unsigned most = kRouterGroups) {
        kernel<<<std::min(grid(tokens), most), kRouterThreads, 0, stream>>>(logits, T, E, k, over_all, scale, idx, w);
    };
    if (k <= 16) {
        // 32768 x 256, top-8, in a graph: FP32 13.8 us with single loads, 12.9 with fours; bf16 10.1 and 9.3
        const bool quads = E % 4 == 0;
        if (E <= 32) run(router_kernel<16, 2, BF16, 1>, 4);
        else if (E <= 64) quads ? run(router_kernel<16, 4, BF16, 4>, 4) : run(router_kernel<16, 4, BF16, 1>, 4);
        else if (E <= 128) quads ? run(router_kernel<16, 8, BF16, 4>, 4) : run(router_kernel<16, 8, BF16, 1>, 4);
        else if (E <= 256) quads ? run(router_kernel<16, 16, BF16, 4>, 4) : run(router_kernel<16, 16, BF16, 1>, 4);
        else if (E <= 512) quads ? run(router_kernel<32, 16, BF16, 4>, 2) : run(router_kernel<32, 16, BF16, 1>, 2);
        else quads ? run(router_kernel<64, 16, BF16, 4>, 1) : run(router_kernel<64, 16, BF16, 1>, 1);
    } else {
        if (E <= 64) run(router_wave_kernel<1, BF16>, 1, kWaveGroups);
        else if (E <= 128) run(router_wave_kernel<2, BF16>, 1, kWaveGroups);
        else if (E <= 256) run(router_wave_kernel<4, BF16>, 1, kWaveGroups);
        else if (E <= 512) run(router_wave_kernel<8, BF16>, 1, kWaveGroups);
        else run(router_wave_kernel<16, BF16>, 1, kWaveGroups);
    }
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
