// FP4 cast of bf16 or FP32 rows and the cast back: E2M1 codes with one UE8M0 scale per 1x32 block, the format of the expert
// weights and of the 4-bit operands (chenxutan.com/d/1930 sections 4.1-4.2: E2M1 and UE8M0; 11.1: a block's scale follows
// its largest magnitude).
//
// Per block: s = the least integer with amax <= 6 * 2^s (amax = 0: s = 0), byte = max(s + 127, 0), code = E2M1 of
// x * 2^-(byte - 127), round to nearest even. Nothing rounds before that decision: the conversion instruction takes FP32
// and a scale of which it reads the exponent (checked against the definition on 2^20 numbers, all midpoints and both
// signs of zero among them). Rows are whole blocks, so rows and blocks are one flat list.
//
// Memory-bound: 8 elements per lane, 4 lanes a block, whose largest magnitude is two steps within the quad.
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

template <bool F32>
__device__ inline void load8(const void* x, size_t i, float (&f)[8]) {
    if constexpr (F32) {
        const float4 a = static_cast<const float4*>(x)[2 * i], b = static_cast<const float4*>(x)[2 * i + 1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4 v = static_cast<const uint4*>(x)[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}

// Thread i: elements 8i .. 8i+7 (n: elements / 8, a multiple of 4, so quads are whole)
template <bool F32>
__global__ __launch_bounds__(kThreads) void cast_to_fp4_kernel(size_t first, const void* __restrict__ x, uint32_t* __restrict__ q,
                                                               uint8_t* __restrict__ sf, size_t n) {
    const size_t i = first + blockIdx.x * (size_t)kThreads + threadIdx.x;
    if (i >= n) return;
    float f[8];
    load8<F32>(x, i, f);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    const uint32_t byte = fp4_scale_byte(max_of_quad(m));
    const float scale = ue8m0(byte);
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0], f[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
    q[i] = byte == 255u ? 0u : c;
    if ((i & 3) == 0) sf[i >> 2] = (uint8_t)byte;
}

// E2M1 code as FP32: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives
__device__ inline float e2m1(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, man = c & 1u;
    const uint32_t mag = e == 0 ? (man ? 0x3f000000u : 0u) : ((126u + e) << 23) | (man << 22);
    return __uint_as_float(mag | (c & 8u) << 28);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void cast_from_fp4_kernel(size_t first, const uint32_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ sf, void* __restrict__ x, size_t n) {
    const size_t i = first + blockIdx.x * (size_t)kThreads + threadIdx.x;
    if (i >= n) return;
    const uint32_t c = q[i], byte = sf[i >> 2];
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = byte == 255u ? __uint_as_float(0x7fc00000u) : __builtin_ldexpf(e2m1((c >> (4 * j)) & 15u), (int)byte - 127);
    if constexpr (F32) {
        static_cast<float4*>(x)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4*>(x)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        typedef float v8f __attribute__((ext_vector_type(8)));
        typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
        const v8f v = {f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
        static_cast<uint4*>(x)[i] = __builtin_bit_cast(uint4, __builtin_convertvector(v, v8bf));
    }
}

template <class... P, class... A>
hipError_t launch_flat(void (*kernel)(size_t, P...), size_t n, hipStream_t stream, A... args) {
    for (size_t first = 0; first < n; first += kLaunchThreads) {
        const size_t m = n - first < kLaunchThreads ? n - first : kLaunchThreads;
        kernel<<<(unsigned)((m + kThreads - 1) / kThreads), kThreads, 0, stream>>>(first, args..., n);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cast_to_fp4(const void* x, int x_type, int rows, int cols, uint8_t* q, uint8_t* sf, hipStream_t stream) {
    const size_t n = (size_t)rows * cols / 8;
    uint32_t* words = reinterpret_cast<uint32_t*>(q);
    return x_type == MOE_F32 ? launch_flat(cast_to_fp4_kernel<true>, n, stream, x, words, sf)
                             : launch_flat(cast_to_fp4_kernel<false>, n, stream, x, words, sf);
}

hipError_t launch_cast_from_fp4(const uint8_t* q, const uint8_t* sf, int rows, int cols, void* x, int x_type, hipStream_t stream) {
    const size_t n = (size_t)rows * cols / 8;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(q);
    return x_type == MOE_F32 ? launch_flat(cast_from_fp4_kernel<true>, n, stream, words, sf, x)
                             : launch_flat(cast_from_fp4_kernel<false>, n, stream, words, sf, x);
}

}  // namespace moe
