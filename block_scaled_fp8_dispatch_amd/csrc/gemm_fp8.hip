// FP8 x FP8 GEMMs with one UE8M0 scale per 1x128 block of A and per 128x128 block of B, on
// v_mfma_scale_f32_16x16x128_f8f6f4: one instruction spans exactly one block along K, so both
// scales go into it (every lane's scale byte is its row's, or its 128-column block's) and the
// sum over K stays in the FP32 accumulators. That instruction adds the products of 8
// consecutive K after aligning them to the largest of the 8 and drops what lies more than 13
// bits below it (measured on gfx950: 2^16 + 270 within 8 gives 2^16 + 264; across groups of 8 the
// sum is FP32's), about 1.5e-5 of the result's norm on normal data: far below a bf16 output's
// rounding (1.7e-3), but not FP32. FP32 outputs therefore go through v_mfma_f32_16x16x32_bf16,
// at half its rate: an e4m3 value times its block's power of two is exact in bf16 (3 mantissa
// bits of 7, the exponent range of FP32), and that instruction's sums are FP32's.
//
// A workgroup of 4 waves owns 64 rows x 64 columns, wave w rows 16w .. 16w+15. Operands go
// from memory straight to registers in the instruction's layout: lane 16g + i holds bytes
// [16g, 16g+16) and [64+16g, 64+16g+16) of row (column) i's 128.
#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ inline v8i load_frag(const uint8_t* p) {
    const v4i lo = *reinterpret_cast<const v4i*>(p);
    const v4i hi = *reinterpret_cast<const v4i*>(p + 64);
    return (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// 2^(byte - 127) as the operand of the scaled conversions, which read its exponent field (byte
// 255: NaN)
__device__ inline float scale_f32(int byte) { return __uint_as_float(byte == 255 ? 0x7fc00000u : (uint32_t)byte << 23); }

// two words of e4m3 codes (8 values) times 2^(byte - 127), exact in bf16
__device__ inline v8bf to_bf16(int w0, int w1, float scale) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
    return (v8bf){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <bool F32>
__global__ __launch_bounds__(256) void gemm_fp8_simple(GemmFp8Args p) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l = lane & 15;
    const int NT = (p.N + 63) / 64;
    const int mt = (int)(blockIdx.x / NT), nt = (int)(blockIdx.x % NT);
    const bool dense = p.dense_rows > 0;
    if (!dense && mt >= min(p.meta[0], p.max_tiles)) return;
    const int group = dense ? 0 : p.tile_expert[mt];
    const int row0 = dense ? mt * 64 : p.tile_row0[mt];
    auto d_row = [&](int r) { return dense ? (row0 + r < p.dense_rows ? row0 + r : -1) : p.perm[row0 + r]; };
    const int ar = d_row(16 * wave + l);
    const size_t arow = ar < 0 ? 0 : (size_t)ar;      // padding rows read row 0 and are not stored
    const uint8_t* a = p.a + arow * p.K + 16 * g;
    const uint8_t* sa = p.a_sf + arow * p.sf_stride;
    const uint8_t *b[4], *sb[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const int n = min(nt * 64 + 16 * f + l, p.N - 1);
        b[f] = p.b + ((size_t)group * p.N + n) * p.K + 16 * g;
        sb[f] = p.b_sf + ((size_t)group * ((p.N + 127) / 128) + n / 128) * p.sf_stride;
    }
    v4f acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = (v4f){0.f, 0.f, 0.f, 0.f};
    for (int ks = 0; ks < p.K / 128; ++ks) {
        const v8i av = load_frag(a + ks * 128);
        const int s = sa[ks];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const v8i bv = load_frag(b[f] + ks * 128);
            if constexpr (F32) {
                // the same 8 consecutive codes of a lane on both sides: any order of K will do
#pragma unroll
                for (int q = 0; q < 8; q += 2)
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16(av[q], av[q + 1], scale_f32(s)),
                                                                     to_bf16(bv[q], bv[q + 1], scale_f32(sb[f][ks])), acc[f],
                                                                     0, 0, 0);
            } else {
                acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[f], 0, 0, 0, s, 0, (int)sb[f][ks]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = d_row(16 * wave + 4 * g + r);
        if (row < 0) continue;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int n = nt * 64 + 16 * f + l;
            if (n >= p.N) continue;
            if constexpr (F32)
                static_cast<float*>(p.d)[(size_t)row * p.N + n] = acc[f][r];
            else
                static_cast<uint16_t*>(p.d)[(size_t)row * p.N + n] = __builtin_bit_cast(uint16_t, (__bf16)acc[f][r]);
        }
    }
}

}  // namespace

hipError_t launch_gemm_fp8(int block_m, const GemmFp8Args& a, hipStream_t stream) {
    const size_t mt = a.dense_rows > 0 ? cdiv(a.dense_rows, 64) : a.max_tiles;
    const size_t grid = mt * (size_t)cdiv(a.N, 64);
    if (grid == 0) return hipSuccess;
    if (a.out_f32)
        gemm_fp8_simple<true><<<(unsigned)grid, 256, 0, stream>>>(a);
    else
        gemm_fp8_simple<false><<<(unsigned)grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
