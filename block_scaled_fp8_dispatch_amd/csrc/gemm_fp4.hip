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
constexpr int kCus = 256;                 // compute units of an MI355X
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
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)p.a, 0, (int)(p.rows * (uint32_t)(p.K / 2)), kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_asf = __builtin_amdgcn_make_buffer_rsrc((void*)p.a_sf, 0, (int)(p.rows * (uint32_t)(p.K / 32)), kRsrcWord3);
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

// acc += A x B, both E2M1, scales from byte OPS of their words. As asm so that the accumulators stay in their registers; the
// operands are written by LDS or buffer loads, A's scale words a row of products ahead of their use, and the kernel separates
// the accumulators' other accesses by s_nop, so no hazard needs padding.
template <int OPS>
__device__ inline void mfma_scaled(v4f& acc, const v4i& a, const v4i& b, uint32_t sa, uint32_t sb) {
    if constexpr (OPS == 0)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else if constexpr (OPS == 1)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else if constexpr (OPS == 2)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[1,1,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
}

template <int N>
struct IntC {
    static constexpr int value = N;
};

#define MOE_LPTR(p) ((__attribute__((address_space(3))) void*)(p))

// A's scale words. A row's 16 scale bytes of four K steps lie together, 4 a step; lane 16g + i loads step g's word of row i, and
// needs byte g of each of the four. That is a 4 x 4 transpose of bytes over the lanes i, 16 + i, 32 + i, 48 + i: the words of the
// lane 32 away, then of the one 16 away, and two byte selections (for the lane: sel0, sel1).
struct ByteSelect {
    uint32_t first, second;
};
__device__ inline ByteSelect byte_select(int g) {
    const uint32_t h = 2u * (g >> 1), o = g & 1;
    return {h | (h + 1) << 8 | (h + 4) << 16 | (h + 5) << 24, o | (o + 4) << 8 | (o + 2) << 16 | (o + 6) << 24};
}
__device__ inline uint32_t transpose_bytes(uint32_t x, const ByteSelect& sel) {
    const auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const uint32_t z = __builtin_amdgcn_perm(p[1], p[0], sel.first);
    const auto q = __builtin_amdgcn_permlane16_swap(z, z, false, false);
    return __builtin_amdgcn_perm(q[1], q[0], sel.second);
}

// Bytes of a step (256 of K) of A's row and of a B tile
constexpr int kStep = 2 * kBK;
constexpr int kARow = kStep / 2;
constexpr int kBStep = 2 * kBTileBytes;

template <int BM, int WAVES_M, int WAVES_N>
struct Fp4Cfg {
    static constexpr int WM = BM / WAVES_M, WN = kBN / WAVES_N;
    static constexpr int FM = WM / 16, FN = WN / 16;
    static constexpr int A_BYTES = BM * kARow;
    // ring slots: 160 KB with 256 rows, 160 with 128, 128 with 64
    static constexpr int DB = BM == 256 ? 2 : 3, DA = DB + 1;
    static constexpr int LDS_BYTES = DA * A_BYTES + DB * kBStep;
    static constexpr int A_DMA = A_BYTES / 1024 / 4, B_DMA = kBStep / 1024 / 4;   // 1 KB loads per wave and step
    static_assert(WAVES_M * WAVES_N == 4 && LDS_BYTES <= 160 * 1024, "");
};

// Part `part` (of BM rows) of tile v. Tile ids walk groups of 4 row tiles (of args.block_m rows) across all column tiles.
template <int BM, int WAVES_M, int WAVES_N, bool F32>
__device__ inline __attribute__((always_inline)) void tiled_part(const GemmFp4Args& args, uint8_t* smem, int num_mt, int v, int part) {
    // gfx950 buffer descriptors are a device-only type: the host pass sees an empty function
#if defined(__HIP_DEVICE_COMPILE__)
    using C = Fp4Cfg<BM, WAVES_M, WAVES_N>;
    constexpr int WM = C::WM, FM = C::FM, FN = C::FN, DA = C::DA, DB = C::DB, A_DMA = C::A_DMA, B_DMA = C::B_DMA;
    uint8_t* const bring = smem + DA * C::A_BYTES;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int g = lane >> 4, l = lane & 15;
    const bool dense = args.dense_rows > 0;
    const int NT = (args.N + kBN - 1) / kBN;
    const int grp = v / (kGroupM * NT), mt0 = grp * kGroupM;
    const int gm = min(kGroupM, num_mt - mt0), vin = v - grp * kGroupM * NT;
    const int mt = mt0 + vin % gm, nt = vin / gm;
    const int group = dense ? 0 : __builtin_amdgcn_readfirstlane(args.tile_expert[mt]);
    const int row0 = (dense ? mt * args.block_m : __builtin_amdgcn_readfirstlane(args.tile_row0[mt])) + part * BM;
    const int nks = args.K / kBK, nst = (nks + 1) >> 1;   // K steps of 128 and steps of 256
    // A and D row of tile row r, -1 on padding
    auto d_row = [&](int r) __attribute__((always_inline)) -> int {
        if (dense) return row0 + r < args.dense_rows ? row0 + r : -1;
        return args.perm[row0 + r];
    };
    auto a_row = [&](int r) __attribute__((always_inline)) -> uint32_t {
        const int d = d_row(r);
        return d < 0 ? 0u : (uint32_t)d;      // padding rows read row 0 and are never stored
    };
    // padding comes last in a row tile: nothing but padding here
    if (part > 0 && __builtin_amdgcn_readfirstlane(d_row(0)) < 0) return;

    // ---- per-lane offsets --------------------------------------------------------------------
    // Load j of wave w fills LDS rows 8*(w*A_DMA + j) .. +7 of A's tile; lane l lands at row + l/8, physical 16-byte chunk
    // l%8, which holds logical chunk (l%8) ^ (row%8): chunk c < 4 is K block c of the step's first 128, 4 + c of its second.
    const int chunk = (lane & 7) ^ (lane >> 3);
    uint32_t a_off[A_DMA];
#pragma unroll
    for (int j = 0; j < A_DMA; ++j) a_off[j] = a_row(8 * (wave * A_DMA + j) + (lane >> 3)) * (uint32_t)(args.K / 2) + chunk * 16;
    // With an odd number of K steps the last step's second half lies past the rows. Its loads repeat the first half's, and its
    // products vanish by their scales: byte 0 on both sides, 2^-254 (A's by scale_words, B's as packed)
    const uint32_t past = (nks & 1) && chunk >= 4 ? 64u : 0u;
    // (the words of a last block's missing K steps repeat the last one's)
    const int last_kb = (nks - 1) >> 2;
    const uint32_t past_sf = 4u * max(0, 4 * last_kb + g - (nks - 1));
    uint32_t sa_off[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) sa_off[f] = a_row(wm * WM + f * 16 + l) * (uint32_t)(args.K / 32) + 4u * g;
    const ByteSelect sel = byte_select(g);
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)args.a, 0, (int)(args.rows * (uint32_t)(args.K / 2)), kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_asf = __builtin_amdgcn_make_buffer_rsrc((void*)args.a_sf, 0, (int)(args.rows * (uint32_t)(args.K / 32)), kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(args.b + (size_t)group * args.b_group + (size_t)nt * args.b_ntile), 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_bsf = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(args.b_sf + (size_t)group * args.bs_group + (size_t)nt * args.bs_ntile), 0, kAllRecords, kRsrcWord3);

    auto load_a = [&](int ks, int j) __attribute__((always_inline)) {
        const int kc = min(ks, nst - 1);      // steps past the last reload it into a free slot
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, MOE_LPTR(smem + (ks % DA) * C::A_BYTES + (wave * A_DMA + j) * 1024), 16,
                                                 a_off[j] - (kc == nst - 1 ? past : 0u), kc * kARow, 0, 0);
    };
    auto load_b = [&](int ks, int j) __attribute__((always_inline)) {
        const int i = wave * B_DMA + j;       // fragment i % 16 of the step's half i / 16
        const int kc = min(2 * ks + (i >> 4), nks - 1);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, MOE_LPTR(bring + (ks % DB) * kBStep + i * 1024), 16, lane * 16,
                                                 kc * kBTileBytes + (i & 15) * kFragBytes, 0, 0);
    };
    // scale words of a block of two steps: A's as loaded, and by byte of the K step in the block as the products take them
    uint32_t raw[FM], sa[2][FM], sb[2][FN];
    auto load_scale = [&](int kb, int i, int set) __attribute__((always_inline)) {
        if (i < FM) raw[i] = __builtin_amdgcn_raw_buffer_load_b32(rs_asf, sa_off[i] - (kb == last_kb ? past_sf : 0u), kb * 16, 0);
        else sb[set][i - FM] = __builtin_amdgcn_raw_buffer_load_b32(rs_bsf, lane * 4 + (wn * FN + i - FM) * 256, kb * kBScaleBlockBytes, 0);
    };
    // (bytes of K steps past the last: 0)
    auto scale_words = [&](int kb, int f) __attribute__((always_inline)) -> uint32_t {
        const uint32_t keep = kb == last_kb && (nks & 3) ? (1u << (8 * (nks & 3))) - 1u : ~0u;
        return transpose_bytes(raw[f], sel) & keep;
    };
    const uint32_t rd_lo = (uint32_t)(l * kARow + ((g ^ (l & 7)) << 4));
    const uint32_t rd_hi = (uint32_t)(l * kARow + (((g + 4) ^ (l & 7)) << 4));
    struct Pair {
        v4i half[2];
    };
    auto read_a = [&](int ks, int f) __attribute__((always_inline)) -> Pair {
        const uint8_t* p = smem + (ks % DA) * C::A_BYTES + (wm * FM + f) * 16 * kARow;
        return {{*reinterpret_cast<const v4i*>(p + rd_lo), *reinterpret_cast<const v4i*>(p + rd_hi)}};
    };
    auto read_b = [&](int ks, int h, int f) __attribute__((always_inline)) -> v4i {
        return *reinterpret_cast<const v4i*>(bring + (ks % DB) * kBStep + h * kBTileBytes + (wn * FN + f) * kFragBytes + lane * 16);
    };

    v4f acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
            acc[fm][fn] = (v4f){0.f, 0.f, 0.f, 0.f};
            asm volatile("" : "+a"(acc[fm][fn]));
        }
    asm volatile("s_nop 7" ::: "memory");   // accumulator writes -> first MFMA

    // A step's window of loads starts behind its barrier and ends before the next step's: B of DB steps ahead, A of DA, and
    // after even steps the next block's scale words, which have landed at the next step's barrier (DB = 2: behind B, which
    // has to land there as well; DB = 3: in front, so that B need not)
    constexpr int NS = FM + FN, TILE_OPS = A_DMA + B_DMA;
    constexpr bool kScalesFirst = DB > 2;
    constexpr int ROW = 2 * FN;             // MFMAs per fragment row
    constexpr int SPACE = (FM - 1) * ROW / (NS + TILE_OPS) > 3 ? 3 : (FM - 1) * ROW / (NS + TILE_OPS);   // MFMAs per load
    static_assert(SPACE >= 1, "a step's loads fit between its barriers");
    auto issue = [&](int kp, bool scales, int set, int op) __attribute__((always_inline)) {
        const int ns = scales ? NS : 0;
        const int s0 = kScalesFirst ? 0 : B_DMA;
        if (op >= s0 && op < s0 + ns) {
            load_scale(min((kp >> 1) + 1, last_kb), op - s0, set);
            return;
        }
        if (op >= s0 + ns) op -= ns;
        if (op < B_DMA) load_b(kp + DB, op);
        else if (op < TILE_OPS) load_a(kp + DA, op - B_DMA);
    };
    // the loads that the steps before step 0 would have issued
#pragma unroll
    for (int i = 0; i < NS; ++i) load_scale(0, i, 0);
#pragma unroll
    for (int j = 0; j < A_DMA; ++j) load_a(0, j);
#pragma unroll
    for (int s = 0; s < DB - 1; ++s) {
#pragma unroll
        for (int j = 0; j < B_DMA; ++j) load_b(s, j);
#pragma unroll
        for (int j = 0; j < A_DMA; ++j) load_a(s + 1, j);
    }
    // of the step before step 0 only what goes out in its last row; step 0 issues the rest
    constexpr int EARLY = (ROW + SPACE - 1) / SPACE < TILE_OPS ? (ROW + SPACE - 1) / SPACE : TILE_OPS;
#pragma unroll
    for (int op = 0; op < EARLY; ++op) issue(-1, false, 0, op);
    // everything after A and B of step 0
    constexpr int WAIT0 = EARLY + A_DMA + (DB - 2) * TILE_OPS;
    static_assert(WAIT0 < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (WAIT0 & 15) | (((WAIT0 >> 4) & 3) << 14));
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"(WAIT0) : "memory");
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[0][f] = scale_words(0, f);
    Pair a_cur, a_nx;
    v4i bq[2][FN];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < FN; ++f) bq[h][f] = read_b(0, h, f);
    a_nx = read_a(0, 0);
#pragma unroll
    for (int f = 0; f < FM; ++f) asm volatile("" : "+v"(sa[0][f]));
    asm volatile("s_nop 1" ::: "memory");   // scale words -> first MFMA

    // One step: 256 of K, FM rows of 2 x FN MFMAs. Its barrier stands before the last row: this wave's loads of step ks+1 have
    // landed, its LDS reads of step ks are done. Behind it each B fragment's registers take the next step's right after their
    // last use, and the step's window of loads begins.
    auto step = [&](int ks, auto odd_c, auto set_c) __attribute__((always_inline)) {
        constexpr int ODD = decltype(odd_c)::value, SET = decltype(set_c)::value;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            if (fm == FM - 1) {
                // in flight may be what was issued behind B of step ks+1 and (odd steps) the scale words
                constexpr int WN_ = DB == 2 ? A_DMA : ODD ? TILE_OPS : A_DMA + TILE_OPS;
                __builtin_amdgcn_s_waitcnt(0x0070 | (WN_ & 15) | (((WN_ >> 4) & 3) << 14));
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(WN_) : "memory");
                if constexpr (ODD) {
                    // the next block's scale words have landed: no wait of the compiler's own for them
#pragma unroll
                    for (int f = 0; f < FM; ++f) asm volatile("" : "+v"(raw[f]));
#pragma unroll
                    for (int f = 0; f < FN; ++f) asm volatile("" : "+v"(sb[SET ^ 1][f]));
                }
            }
            a_cur = a_nx;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int fn = 0; fn < FN; ++fn) {
                    if (h == 0) mfma_scaled<2 * ODD>(acc[fm][fn], a_cur.half[0], bq[0][fn], sa[SET][fm], sb[SET][fn]);
                    else mfma_scaled<2 * ODD + 1>(acc[fm][fn], a_cur.half[1], bq[1][fn], sa[SET][fm], sb[SET][fn]);
                    const int t = h * FN + fn;
                    if (t == 0) a_nx = fm + 1 < FM ? read_a(ks, fm + 1) : read_a(ks + 1, 0);
                    if (fm == FM - 1) {
                        bq[h][fn] = read_b(ks + 1, h, fn);
                        if (ODD && t % (ROW / FM) == 0) {
                            sa[SET ^ 1][t / (ROW / FM)] = scale_words((ks >> 1) + 1, t / (ROW / FM));
                            asm volatile("" : "+v"(sa[SET ^ 1][t / (ROW / FM)]));
                        }
                        if (t % SPACE == 0) issue(ks, !ODD, SET ^ 1, t / SPACE);
                    } else if ((ROW + fm * ROW + t) % SPACE == 0) {
                        issue(ks - 1, ODD, SET ^ 1, (ROW + fm * ROW + t) / SPACE);
                    }
                    __builtin_amdgcn_sched_barrier(0x7);
                }
            }
        }
    };

    // 4 steps per iteration: two blocks of scale words, one per set
    int ks0 = 0;
    for (; ks0 + 4 <= nst; ks0 += 4) {
        step(ks0, IntC<0>{}, IntC<0>{});
        step(ks0 + 1, IntC<1>{}, IntC<0>{});
        step(ks0 + 2, IntC<0>{}, IntC<1>{});
        step(ks0 + 3, IntC<1>{}, IntC<1>{});
    }
    if (ks0 < nst) step(ks0, IntC<0>{}, IntC<0>{});
    if (ks0 + 1 < nst) step(ks0 + 1, IntC<1>{}, IntC<0>{});
    if (ks0 + 2 < nst) step(ks0 + 2, IntC<0>{}, IntC<1>{});
    // the last steps' reloads must land before the workgroup's LDS is given back
    __builtin_amdgcn_s_waitcnt(0x0F70);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    // the accumulators' reads stay behind the wait states that the last MFMA's result needs
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) asm volatile("" : "+a"(acc[fm][fn]));

    // ---- epilogue: rows 16*fm + 4g + r, FN adjacent columns from col0 (all or none: N is a multiple of 16) -------------
    const int fw = wn * FN;
    const int col0 = nt * kBN + 128 * (fw >> 3) + 8 * l + (fw & 7);
    if (col0 >= args.N) return;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = d_row(wm * WM + fm * 16 + 4 * g + r);
            if (row < 0) continue;
            const size_t to = (size_t)row * args.N + col0;
            if constexpr (F32) {
                float* dst = static_cast<float*>(args.d) + to;
#pragma unroll
                for (int q = 0; q < FN; q += 4)
                    *reinterpret_cast<v4f*>(dst + q) = (v4f){acc[fm][q][r], acc[fm][q + 1][r], acc[fm][q + 2][r], acc[fm][q + 3][r]};
            } else {
                uint32_t pk[FN / 2];
#pragma unroll
                for (int q = 0; q < FN; q += 2) {
                    const v2f x = {acc[fm][q][r], acc[fm][q + 1][r]};
                    pk[q / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2bf));
                }
                uint16_t* dst = static_cast<uint16_t*>(args.d) + to;
                if constexpr (FN == 8) *reinterpret_cast<v4i*>(dst) = (v4i){(int)pk[0], (int)pk[1], (int)pk[2], (int)pk[3]};
                else *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
            }
        }
    }
#endif
}

// The row tiles in use: their number lies on the device unless the product is dense
__device__ inline int row_tiles(const GemmFp4Args& args, int bm) {
    const int n = args.dense_rows > 0 ? (args.dense_rows + bm - 1) / bm : __builtin_amdgcn_readfirstlane(args.meta[0]);
    return min(n, args.max_tiles);
}

template <int BM, int WAVES_M, int WAVES_N, bool F32>
__global__ __launch_bounds__(256, 1) void gemm_fp4_tiled(GemmFp4Args args) {
    using C = Fp4Cfg<BM, WAVES_M, WAVES_N>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS_BYTES];
    const int num_mt = row_tiles(args, BM);
    const int v = xcd_tile(num_mt * ((args.N + kBN - 1) / kBN), blockIdx.x);
    if (v < 0) return;
    tiled_part<BM, WAVES_M, WAVES_N, F32>(args, smem, num_mt, v, 0);
}

// 256 x 256 tiles in rounds of one per CU; a last round at most half full runs as parts of 64 rows where those are no more than
// the CUs, else of 128 rows, so that more of them work, and each starts when a CU is through with the rounds before.
template <bool F32>
__global__ __launch_bounds__(256, 1) void gemm_fp4_rounds(GemmFp4Args args) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[160 * 1024];
    const int num_mt = row_tiles(args, 256), total = num_mt * ((args.N + kBN - 1) / kBN);
    const int rem = total % kCus, full = rem <= kCus / 2 ? total - rem : total;
    if ((int)blockIdx.x < full) {
        tiled_part<256, 2, 2, F32>(args, smem, num_mt, xcd_tile(full, blockIdx.x), 0);
        return;
    }
    const int parts = rem <= kCus / 4 ? 4 : 2;
    const int u = xcd_tile((total - full) * parts, blockIdx.x - full);
    if (u < 0) return;
    if (parts == 4) tiled_part<64, 1, 4, F32>(args, smem, num_mt, full + u / 4, u % 4);
    else tiled_part<128, 2, 2, F32>(args, smem, num_mt, full + u / 2, u % 2);
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

hipError_t launch_gemm_fp4(const Fp4Plan& plan, const GemmFp4Args& a, hipStream_t stream) {
    const size_t mt = a.dense_rows > 0 ? cdiv(a.dense_rows, plan.block_m) : a.max_tiles;
    // one workgroup per possible tile; those past the tiles in use return at once
    const size_t grid = mt * (size_t)cdiv(a.N, kBN);
    switch (plan.kernel) {
        case Fp4Kernel::kTiled256: {
            // the parts are at most 256
            const unsigned blocks = (unsigned)(a.dense_rows > 0 ? (grid % kCus == 0 || grid % kCus > kCus / 2 ? grid : grid - grid % kCus + kCus) : grid + kCus);
            if (a.out_f32) gemm_fp4_rounds<true><<<blocks, 256, 0, stream>>>(a);
            else gemm_fp4_rounds<false><<<blocks, 256, 0, stream>>>(a);
            break;
        }
        case Fp4Kernel::kTiled128:
            if (a.out_f32) gemm_fp4_tiled<128, 2, 2, true><<<(unsigned)grid, 256, 0, stream>>>(a);
            else gemm_fp4_tiled<128, 2, 2, false><<<(unsigned)grid, 256, 0, stream>>>(a);
            break;
        case Fp4Kernel::kSkinny64: return launch_skinny<4, 4>(a, stream);
    }
    return hipGetLastError();
}

Fp4Plan fp4_plan(int groups, double rows_per_group, int max_rows, bool ragged, int N, int K) {
    if (rows_per_group > 256) return {Fp4Kernel::kTiled256, 256};
    if (rows_per_group > 64) return {Fp4Kernel::kTiled128, 128};
    return {Fp4Kernel::kSkinny64, 64};
}

}  // namespace moe
