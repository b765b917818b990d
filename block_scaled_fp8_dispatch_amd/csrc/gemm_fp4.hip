// FP4 x FP4 GEMMs with one UE8M0 scale per 1x32 block of both operands, on v_mfma_scale_f32_16x16x128_f8f6f4: lane 16g + i
// of an operand holds the 32 codes of row (column) i and K block g as 16 bytes, and their scale as a byte. E2M1 products are
// multiples of 1/4 below 2^6 times a power of two, and the unit adds them as FP32 sums do (measured: 128 products of scales
// 2^-27 to 2^22 apart within 1.5 * 2^-24 of the sum of their magnitudes; every scale byte from 0 to 254 counts, subnormal
// results included, 255 makes NaN), so FP32 outputs take the same products as bf16 ones.
//
// B is packed (pack.hip): a 16-column x 128-K fragment is one 1 KB read in lane order, its scales one 32-bit word per lane
// and four K steps. A is read as it is: a lane's 16 bytes of a K step, and its scale byte.
//
// Skinny kernel. A workgroup owns a tile of BM rows x FN fragments and its 8 waves share K, wave w taking the pairs of K
// steps w, w + 8, ... with sums of its own, which meet in LDS at the end. Operands go from memory straight into the
// registers of the wave that multiplies them: 16 bytes a lane are a whole operand, and the two steps of a pair use whole
// 128-byte lines of A's rows.
#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kGroupM = 4;
constexpr int kRsrcWord3 = 0x00020000;   // raw buffer descriptor: byte offsets, no swizzle
constexpr int kAllRecords = -1;
constexpr int kFp4 = 4;                  // the instruction's format code of E2M1

// Workgroups go round-robin to the XCDs: tile id of workgroup `block` with each XCD (workgroup id mod 8) owning a
// contiguous range of ids. -1: none left.
__device__ inline int xcd_tile(int total, unsigned block) {
    const int xcd = block & 7, li = block >> 3;
    const int per = total >> 3, rem = total & 7;
    if (li >= per + (xcd < rem ? 1 : 0)) return -1;
    return xcd * per + (xcd < rem ? xcd : rem) + li;
}

constexpr int kSkinnyWaves = 8;

template <int FM, int FN, bool F32>
__global__ __launch_bounds__(kSkinnyWaves * 64) void gemm_fp4_skinny(GemmFp4Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int BM = 16 * FM, SUB = 64 / BM, WAVES = kSkinnyWaves, PITCH = 16 * FN + 4;
    __shared__ __attribute__((aligned(16))) float sums[WAVES / 2 * BM * PITCH];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l = lane & 15;
    const bool dense = p.dense_rows > 0;
    // units of BM rows: of a dense product's rows, or of the 64-row tiles in the list
    const int units = dense ? (p.dense_rows + BM - 1) / BM : min(__builtin_amdgcn_readfirstlane(p.meta[0]), p.max_tiles) * SUB;
    // column units of FN fragments; a 128-column half tile is 8 fragments, whose columns interleave
    const int NT = (p.N + 127) / 128 * (8 / FN);
    const int v = xcd_tile(units * NT, blockIdx.x);
    if (v < 0) return;
    // groups of 4 row tiles across all column units: their rows of A stay in the XCD's L2
    constexpr int kSet = kGroupM * SUB;
    const int set = v / (kSet * NT), u0 = set * kSet, gu = min(kSet, units - u0), vin = v - set * kSet * NT;
    const int unit = u0 + vin % gu, nt = vin / gu;
    const int mt = unit / SUB;
    const int group = dense ? 0 : __builtin_amdgcn_readfirstlane(p.tile_expert[mt]);
    const int row0 = dense ? unit * BM : __builtin_amdgcn_readfirstlane(p.tile_row0[mt]) + unit % SUB * BM;
    auto d_row = [&](int r) __attribute__((always_inline)) -> int {
        if (dense) return row0 + r < p.dense_rows ? row0 + r : -1;
        return p.perm[row0 + r];
    };
    // padding comes last in a row tile: nothing but padding here
    if (__builtin_amdgcn_readfirstlane(d_row(0)) < 0) return;

    const int f0 = nt * FN, tile = f0 >> 4, frag = f0 & 15;      // fragments frag .. frag + FN - 1 of a 256-column tile
    uint32_t a_off[FM], sa_off[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int d = d_row(f * 16 + l);
        const uint32_t row = d < 0 ? 0u : (uint32_t)d;           // padding rows read row 0 and are never stored
        a_off[f] = row * (uint32_t)(p.K / 2) + 16u * g;
        sa_off[f] = row * (uint32_t)(p.K / 32) + (uint32_t)g;
    }
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)p.a, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_asf = __builtin_amdgcn_make_buffer_rsrc((void*)p.a_sf, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.b + (size_t)group * p.b_group + (size_t)tile * p.b_ntile + frag * kFragBytes), 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_bsf = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.b_sf + (size_t)group * p.bs_group + (size_t)tile * p.bs_ntile + frag * 256), 0, kAllRecords, kRsrcWord3);

    v4f acc[FM][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[f][n] = (v4f){0.f, 0.f, 0.f, 0.f};
    const int nks = p.K / kBK;
    for (int k0 = 2 * wave; k0 < nks; k0 += 2 * WAVES) {
        // step 2 of the last pair may lie past K: its loads repeat the first's and it is not multiplied
        const bool both = k0 + 1 < nks;
        v4i a[2][FM], b[2][FN];
        uint32_t sa[2][FM], sb[2][FN];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int ks = s && both ? k0 + 1 : k0;
#pragma unroll
            for (int n = 0; n < FN; ++n) {
                b[s][n] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_b, lane * 16 + n * kFragBytes, ks * kBTileBytes, 0));
                sb[s][n] = __builtin_amdgcn_raw_buffer_load_b8(rs_bsf, lane * 4 + n * 256, (ks >> 2) * kBScaleBlockBytes + (ks & 3), 0);
            }
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                a[s][f] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_a, a_off[f], ks * (kBK / 2), 0));
                sa[s][f] = __builtin_amdgcn_raw_buffer_load_b8(rs_asf, sa_off[f], ks * 4, 0);
            }
        }
        auto multiply = [&](int s) __attribute__((always_inline)) {
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const v8i x = {a[s][f].x, a[s][f].y, a[s][f].z, a[s][f].w, 0, 0, 0, 0};
#pragma unroll
                for (int n = 0; n < FN; ++n) {
                    const v8i y = {b[s][n].x, b[s][n].y, b[s][n].z, b[s][n].w, 0, 0, 0, 0};
                    acc[f][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[f][n], kFp4, kFp4, 0, (int)sa[s][f], 0, (int)sb[s][n]);
                }
            }
        };
        multiply(0);
        if (both) multiply(1);
    }
    // sums at column 16 * fragment + lane column, row of the tile
    auto at = [&](int w, int r, int n) __attribute__((always_inline)) -> float& { return sums[(w * BM + r) * PITCH + n]; };
    if (wave >= WAVES / 2) {
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) at(wave - WAVES / 2, f * 16 + 4 * g + r, n * 16 + l) = acc[f][n][r];
    }
    __syncthreads();
    if (wave < WAVES / 2) {
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) at(wave, f * 16 + 4 * g + r, n * 16 + l) += acc[f][n][r];
    }
    __syncthreads();
    // lane column j of fragment f is column 128 * (f / 8) + 8j + f % 8 of its tile: FN adjacent columns of D per thread
    for (int i = tid; i < BM * 16; i += WAVES * 64) {
        const int r = i >> 4, j = i & 15;
        const int row = d_row(r), col = tile * kBN + 128 * (frag >> 3) + 8 * j + (frag & 7);
        if (row < 0 || col >= p.N) continue;                     // (N is a multiple of 16: all FN columns or none)
        float x[FN];
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            x[n] = at(0, r, n * 16 + j);
#pragma unroll
            for (int w = 1; w < WAVES / 2; ++w) x[n] += at(w, r, n * 16 + j);
        }
        const size_t to = (size_t)row * p.N + col;
        if constexpr (F32) {
            float* d = static_cast<float*>(p.d) + to;
            if constexpr (FN == 4) *reinterpret_cast<v4f*>(d) = (v4f){x[0], x[1], x[2], x[3]};
            else
#pragma unroll
                for (int n = 0; n < FN; ++n) d[n] = x[n];
        } else {
            uint16_t* d = static_cast<uint16_t*>(p.d) + to;
            const v2bf lo = __builtin_convertvector(((v2f){x[0], x[FN > 1 ? 1 : 0]}), v2bf);
            const uint32_t w0 = __builtin_bit_cast(uint32_t, lo);
            if constexpr (FN == 1) *d = (uint16_t)w0;
            else if constexpr (FN == 2) *reinterpret_cast<uint32_t*>(d) = w0;
            else
                *reinterpret_cast<uint2*>(d) = make_uint2(w0, __builtin_bit_cast(uint32_t, __builtin_convertvector(((v2f){x[2], x[3]}), v2bf)));
        }
    }
#endif
}

template <int FM, int FN>
hipError_t launch_skinny(const GemmFp4Args& a, hipStream_t stream) {
    const size_t units = a.dense_rows > 0 ? cdiv(a.dense_rows, 16 * FM) : (size_t)a.max_tiles * (4 / FM);
    const size_t tiles = units * (size_t)(cdiv(a.N, 128) * (8 / FN));
    if (tiles >= (size_t(1) << 32) / (kSkinnyWaves * 64)) return hipErrorInvalidConfiguration;   // a launch wraps there
    const unsigned grid = (unsigned)tiles;
    if (a.out_f32) gemm_fp4_skinny<FM, FN, true><<<grid, kSkinnyWaves * 64, 0, stream>>>(a);
    else gemm_fp4_skinny<FM, FN, false><<<grid, kSkinnyWaves * 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_fp4(const GemmFp4Args& a, hipStream_t stream) {
    return launch_skinny<4, 4>(a, stream);
}

}  // namespace moe
