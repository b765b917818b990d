// FP4 cast of bf16 or FP32 rows and the cast back: E2M1 codes with one UE8M0 scale per 1x32 block, the format of the expert
// weights and of the 4-bit operands (chenxutan.com/d/1930 sections 4.1-4.2: E2M1 and UE8M0; 11.1: a block's scale follows
// its largest magnitude).
//
// Per block: s = the least integer with amax <= 6 * 2^s (amax = 0: s = 0), byte = max(s + 127, 0), code = E2M1 of
// x * 2^-(byte - 127), round to nearest even. Nothing rounds before that decision: the conversion instruction takes FP32
// and a scale of which it reads the exponent (checked against the definition on 2^20 numbers, all midpoints and both
// signs of zero among them). Rows are whole blocks, so rows and blocks are one flat list.
//
// Memory-bound: 8 elements per lane and group, 4 lanes a block, whose largest magnitude is two steps within the quad; the
// way back reads the codes' words and stores 16 bytes a lane. Both move 5.75 to 5.9 TB/s of large tensors (8192 x 7168 bf16 25.1
// us there, 25.8 back), where a copy moves 5.1.
#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr size_t kLaunchThreads = size_t(1) << 31;   // of one launch: from 2^32 on it wraps without an error

// UE8M0 byte of a block whose largest magnitude has FP32 bit pattern `bits` (sign clear): 6 = 1.5 * 2^2
__device__ inline uint32_t fp4_scale_byte(uint32_t bits) {
    if (bits == 0) return 127u;
    if (bits >= 0x7f800000u) return 255u;             // an infinity or a NaN in the block
    const int b = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);
    return b < 0 ? 0u : (uint32_t)b;                  // a subnormal amax: s <= -128
}

// 2^(byte - 127); byte 0 is subnormal
__device__ inline float ue8m0(uint32_t byte) { return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23); }

__device__ inline uint32_t max_of_quad(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
}

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));

// From 3 * 2^20 elements on loads and stores go past the caches (NT), and a thread has several groups in flight; below, one. FP32
// 36864 x 7168 to FP4 208 us with one group, 208 with two and NT; bf16 8192 x 7168 27.2 and 25.1; back 294 us with one, 207 with four,
// 36.2 and 25.8. 1000 x 7168 to FP4 5.6 and 4.9, back 6.4 and 5.0, from FP32 7.9 and 7.8, back 11.3 and 7.8; 256 x 7168, below,
// 3.1 and 3.2, back 2.8 and 3.4, FP32 3.5 and 3.8, 3.6 and 4.3; behind the kernel that wrote the rows, 1000 x 4096 there and back gains
// 3 us of 24, 400 x 7168 loses 1.4 of 18.
constexpr size_t kPastCaches = size_t(3) << 20;
template <bool NT>
constexpr int kUnitsTo = NT ? 2 : 1;
template <bool NT>
constexpr int kUnitsFrom = NT ? 4 : 1;

// NT: past the caches
template <bool NT, class V>
__device__ inline V get(const V* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool NT, class V>
__device__ inline void put(V* p, const V& v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// 8 elements: FP32 as two words of 4, bf16 as one
template <bool F32>
struct Eight;
template <>
struct Eight<true> {
    v4f v[2];
    template <bool NT>
    __device__ static Eight load(const void* x, size_t i) {
        return {{get<NT>(static_cast<const v4f*>(x) + 2 * i), get<NT>(static_cast<const v4f*>(x) + 2 * i + 1)}};
    }
    __device__ float at(int j) const { return v[j >> 2][j & 3]; }
};
template <>
struct Eight<false> {
    v4u v;
    template <bool NT>
    __device__ static Eight load(const void* x, size_t i) {
        return {get<NT>(static_cast<const v4u*>(x) + i)};
    }
    __device__ float at(int j) const { return __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16); }
};

// Group i: elements 8i .. 8i+7 (n groups, a multiple of 4, so quads are whole)
template <bool F32, bool NT>
__global__ __launch_bounds__(kThreads) void cast_to_fp4_kernel(size_t first, const void* __restrict__ x, uint32_t* __restrict__ q,
                                                               uint8_t* __restrict__ sf, size_t n) {
    constexpr int U = kUnitsTo<NT>;
    const size_t i0 = first + blockIdx.x * (size_t)(U * kThreads) + threadIdx.x;
    Eight<F32> e[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (i0 + u * kThreads < n) e[u] = Eight<F32>::template load<NT>(x, i0 + u * kThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t i = i0 + u * kThreads;
        if (i >= n) return;
        float f[8];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = e[u].at(j);
            m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
        }
        const uint32_t byte = fp4_scale_byte(max_of_quad(m));
        const float scale = ue8m0(byte);
        uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0], f[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
        put<NT>(q + i, byte == 255u ? 0u : c);
        if ((i & 3) == 0) sf[i >> 2] = (uint8_t)byte;
    }
}

// Group i: elements 8i .. 8i+7, or 4i .. 4i+3 in FP32, so that a wave's 16-byte stores are adjacent
template <bool F32, bool NT>
__global__ __launch_bounds__(kThreads) void cast_from_fp4_kernel(size_t first, const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ sf, void* __restrict__ x, size_t n) {
    constexpr int U = kUnitsFrom<NT>;
    const size_t i0 = first + blockIdx.x * (size_t)(U * kThreads) + threadIdx.x;
    uint32_t c[U], byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t i = i0 + u * kThreads;
        if (i >= n) continue;
        if constexpr (F32) c[u] = get<NT>(reinterpret_cast<const uint16_t*>(q) + i);
        else c[u] = get<NT>(reinterpret_cast<const uint32_t*>(q) + i);
        byte[u] = sf[i >> (F32 ? 3 : 2)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t i = i0 + u * kThreads;
        if (i >= n) return;
        const float scale = ue8m0(byte[u]);
        const bool nan = byte[u] == 255u;
        if constexpr (F32) {
            const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 1);
            const float none = __uint_as_float(0x7fc00000u);
            put<NT>(static_cast<v4f*>(x) + i, nan ? (v4f){none, none, none, none} : (v4f){a.x, a.y, b.x, b.y});
        } else {
            v4u w;
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], scale, 0));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], scale, 1));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], scale, 2));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], scale, 3));
            put<NT>(static_cast<v4u*>(x) + i, nan ? (v4u){0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u} : w);
        }
    }
}

template <class... P, class... A>
hipError_t launch_flat(void (*kernel)(size_t, P...), int units, size_t n, hipStream_t stream, A... args) {
    const size_t each = (size_t)units * kThreads, most = kLaunchThreads * units;   // groups of a workgroup, of a launch
    for (size_t first = 0; first < n; first += most) {
        const size_t m = n - first < most ? n - first : most;
        kernel<<<(unsigned)((m + each - 1) / each), kThreads, 0, stream>>>(first, args..., n);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cast_to_fp4(const void* x, int x_type, int rows, int cols, uint8_t* q, uint8_t* sf, hipStream_t stream) {
    const size_t n = (size_t)rows * cols;
    uint32_t* words = reinterpret_cast<uint32_t*>(q);
    if (x_type == MOE_F32)
        return n > kPastCaches ? launch_flat(cast_to_fp4_kernel<true, true>, kUnitsTo<true>, n / 8, stream, x, words, sf)
                      : launch_flat(cast_to_fp4_kernel<true, false>, kUnitsTo<false>, n / 8, stream, x, words, sf);
    return n > kPastCaches ? launch_flat(cast_to_fp4_kernel<false, true>, kUnitsTo<true>, n / 8, stream, x, words, sf)
                  : launch_flat(cast_to_fp4_kernel<false, false>, kUnitsTo<false>, n / 8, stream, x, words, sf);
}

hipError_t launch_cast_from_fp4(const uint8_t* q, const uint8_t* sf, int rows, int cols, void* x, int x_type, hipStream_t stream) {
    const size_t n = (size_t)rows * cols;
    if (x_type == MOE_F32)
        return n > kPastCaches ? launch_flat(cast_from_fp4_kernel<true, true>, kUnitsFrom<true>, n / 4, stream, q, sf, x)
                      : launch_flat(cast_from_fp4_kernel<true, false>, kUnitsFrom<false>, n / 4, stream, q, sf, x);
    return n > kPastCaches ? launch_flat(cast_from_fp4_kernel<false, true>, kUnitsFrom<true>, n / 8, stream, q, sf, x)
                  : launch_flat(cast_from_fp4_kernel<false, false>, kUnitsFrom<false>, n / 8, stream, q, sf, x);
}

}  // namespace moe
