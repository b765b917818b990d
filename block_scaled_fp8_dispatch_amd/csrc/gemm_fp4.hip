// FP4 x FP4 GEMMs with one UE8M0 scale per 1x32 block of both operands, on v_mfma_scale_f32_16x16x128_f8f6f4: lane 16g + i
// of an operand holds the 32 codes of row (column) i and K block g as 16 bytes, and their scale as a byte. E2M1 products are
// multiples of 1/4 below 2^6 times a power of two, and the unit adds them as FP32 sums do (measured: 128 products of scales
// 2^-27 to 2^22 apart within 1.5 * 2^-24 of the sum of their magnitudes; every scale byte from 0 to 254 counts, subnormal
// results included, 255 makes NaN), so FP32 outputs take the same products as bf16 ones.
//
// B is packed (pack.hip): a 16-column x 128-K fragment is one 1 KB read in lane order, its scales one 32-bit word per lane
// and four K steps. A is read as it is: a lane's 16 bytes of a K step, and its scale byte.
//
// Skinny kernel. Operands go from memory straight into the registers of the wave that multiplies them: 16 bytes a lane are a
// whole operand, and the two K steps of a pair use whole 128-byte lines of A's rows. A workgroup owns a tile of BM rows x FN
// fragments of columns, and its WAVES waves share K, taking a pair in turn and keeping sums of their own, which meet in LDS at
// the end. A wave keeps DEPTH pairs in flight. Bound by latency and, with more of them on a CU, by its loads (64 x 4096 x 4096 7.0 us,
// 33 x 7168 x 2048 6.1, 1 x 7168 x 18432 13.6: 5.2 TB/s of weights).
//
// Tiled kernel. Tiles of 256, 128 or 64 rows x 256 columns in four waves, steps of 256 of K through rings in LDS that are filled
// past the registers. A step has two barriers: behind the first row of products, by when every wave has B of the step in
// registers, so that B of a later step may land in its slot, and before the last row, when the next step's data is there. Waits
// count loads in flight and never drain them. A's scale words go through LDS too (128 rows and more) or straight to registers
// (64 rows, whose two workgroups fill a CU's LDS with operands), and a 4 x 4 transpose of bytes over lanes turns a row's words
// into the lanes' bytes.
// 4096 x 7168 x 18432 takes 233 us, 8192^3 236 (bf16), 275 (FP32): 4.65 PFLOP/s (another card 245 and 4.4). The chip holds 1.96 GHz
// of its 2.4 under it and the matrix units are busy in 53 % of the cycles; products of registers alone, nothing loaded, reach 7.1
// PFLOP/s on the same operands and 9.5 on zeros, and the whole kernel a quarter more on zeros: power is what bounds it, then LDS
// reads and loads.
// Few rows of many weights stream: 32 groups of about 32 rows x 4096 x 7168 83 us, 6.0 TB/s.
#include <algorithm>
#include <cmath>

#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
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

template <int N>
struct IntC {
    static constexpr int value = N;
};

// Row tiles of p.block_m rows. Dense: rows 0 .. dense_rows-1. Masked with at most 64 groups: every wave derives them from the
// counts, a group per lane. Otherwise the lists that a launch before has made.
struct RowTiles {
    int total;
    int tiles, upto, count;    // masked: lane g's row tiles, those of groups 0 .. g, its rows
};
// A row tile: of group `group`, rows row0 .. row0+count-1 of A and D, or, with a list, perm[row0 + r] (-1: padding, which
// comes last)
struct RowTile {
    int group, row0, count;
};

__device__ inline RowTiles row_tiles(const GemmFp4Args& p, int bm) {
    RowTiles t{};
    if (p.dense_rows > 0) {
        t.total = (p.dense_rows + bm - 1) / bm;
    } else if (p.masked_m) {
        const int lane = threadIdx.x & 63;
        t.count = lane < p.groups ? min(max(p.masked_m[lane], 0), p.max_m) : 0;
        t.tiles = (t.count + bm - 1) / bm;
        // inclusive sums: within 16 lanes, then the rows of 16 before
        int x = t.tiles;
        x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
        t.upto = x;
        t.total = __builtin_amdgcn_readlane(x, 63);
    } else {
        t.total = min(__builtin_amdgcn_readfirstlane(p.meta[0]), p.max_tiles);
    }
    return t;
}

__device__ inline RowTile row_tile(const GemmFp4Args& p, const RowTiles& t, int bm, int mt) {
    if (p.dense_rows > 0) return {0, mt * bm, p.dense_rows - mt * bm};
    if (p.masked_m) {
        const int g = __builtin_ctzll(__ballot(t.upto > mt));
        const int first = (mt - __builtin_amdgcn_readlane(t.upto, g) + __builtin_amdgcn_readlane(t.tiles, g)) * bm;
        return {g, g * p.max_m + first, __builtin_amdgcn_readlane(t.count, g) - first};
    }
    return {__builtin_amdgcn_readfirstlane(p.tile_expert[mt]), __builtin_amdgcn_readfirstlane(p.tile_row0[mt]), 0};
}

// NT: B through non-temporal loads (one row tile reads it)
template <int FM, int FN, int WAVES, int DEPTH, bool F32, bool NT>
__global__ __launch_bounds__(WAVES * 64) void gemm_fp4_skinny(GemmFp4Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int BM = 16 * FM, SUB = 64 / BM, kBAux = NT ? 2 : 0;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l = lane & 15;
    // units of BM rows of the row tiles (dense: of BM rows themselves)
    const bool dense = p.dense_rows > 0, list = p.perm != nullptr;
    const int bm = dense ? BM : 64, sub = dense ? 1 : SUB;
    const RowTiles rt = row_tiles(p, bm);
    const int units = rt.total * sub;
    // column units of FN fragments; the 8 fragments of 128 columns interleave their columns
    const int units_n = (p.N + 127) / 128 * (8 / FN);
    const int v = xcd_tile(units * units_n, blockIdx.x);
    if (v < 0) return;
    // groups of 4 row tiles across all column units: their rows of A stay in the XCD's L2
    const int set_units = kGroupM * SUB;
    const int set = v / (set_units * units_n), u0 = set * set_units, gu = min(set_units, units - u0), vin = v - set * set_units * units_n;
    const int unit = u0 + vin % gu;
    const RowTile at0 = row_tile(p, rt, bm, unit / sub);
    const int group = at0.group, row0 = at0.row0 + unit % sub * BM, count = at0.count - unit % sub * BM;
    // A and D row of row r of the unit, -1 on padding
    auto d_row = [&](int r) __attribute__((always_inline)) -> int {
        if (list) return p.perm[row0 + r];
        return r < count ? row0 + r : -1;
    };
    // padding comes last in a row tile: nothing but padding here
    if (__builtin_amdgcn_readfirstlane(d_row(0)) < 0) return;

    const int f0 = vin / gu * FN, tile = f0 >> 4, frag = f0 & 15;   // fragments frag .. frag + FN-1 of a 256-column tile
    const int nks = p.K / kBK;

    auto a_row = [&](int r) __attribute__((always_inline)) -> uint32_t {
        const int d = d_row(r);
        return d < 0 ? 0u : (uint32_t)d;                         // padding rows read row 0 and are never stored
    };
    uint32_t a_off[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) a_off[f] = a_row(f * 16 + l) * (uint32_t)(p.K / 2) + 16u * g;
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)p.a, 0, (int)(p.rows * (uint32_t)(p.K / 2)), kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_asf = __builtin_amdgcn_make_buffer_rsrc((void*)p.a_sf, 0, (int)(p.rows * (uint32_t)(p.K / 32)), kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.b + (size_t)group * p.b_group + (size_t)tile * p.b_ntile), 0, nks * kBTileBytes, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_bsf = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.b_sf + (size_t)group * p.bs_group + (size_t)tile * p.bs_ntile), 0, (nks + 3) / 4 * kBScaleBlockBytes, kRsrcWord3);
    const uint32_t b_off = frag * kFragBytes + lane * 16, sb_off = frag * 256 + lane * 4;

    v4f acc[FM][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[f][n] = (v4f){0.f, 0.f, 0.f, 0.f};
    struct Stage {
        v4i a[2][FM], b[2][FN];
        uint32_t sa[FM], sb[FN];
    } st[DEPTH];
    // A's scales, 4 bytes a row and K step. A load costs by the lines it touches, and the words of 16 rows lie in 16. With few
    // rows lane 16g + i loads row i's word of the pair's step g % 2 and takes the other step's from the lane 16 away. With 64 rows
    // (SHARED) the workgroup brings the words of 256 K steps into LDS, 16 of a row by 16 lanes, rows two banks apart, and a lane
    // reads both steps' from there (192 x 4096 x 7168 16.3 -> 14.2 us, 64 x 7168 x 18432 40 -> 33.4; the kernel of 32 x 64 28 ->
    // 25.5 there, but 5.6 -> 6.4 at 16 x 7168 x 2048 by the barrier). Of both words it picks byte g.
    constexpr bool SHARED = FM == 4;
    constexpr int kWords = 256, kRowWords = kWords + 2;
    constexpr int GROUPS = WAVES * 4, RG = BM < GROUPS ? BM : GROUPS, ROWS = BM / RG, BATCH = 4;   // of 16 lanes; rows at once, in turn
    static_assert(!SHARED || RG == GROUPS, "every group of lanes has rows of its own");
    __shared__ __attribute__((aligned(16))) uint32_t a_scales[SHARED ? BM * kRowWords : 1];
    const uint32_t sel = (uint32_t)g | (uint32_t)(g + 4) << 8 | 0x0c0c0000u;
    constexpr int NSA = SHARED ? ROWS : FM;
    uint32_t sa_off[NSA];
#pragma unroll
    for (int r = 0; r < NSA; ++r) sa_off[r] = a_row(SHARED ? (tid >> 4) + r * RG : r * 16 + l) * (uint32_t)(p.K / 32);
    auto stage_scales = [&](int first) __attribute__((always_inline)) {
        const int words = min(kWords, nks - first);
        for (int base = 0; base < words; base += 16 * BATCH) {
            uint32_t x[BATCH][ROWS];
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const int w = base + 16 * b + l;
                    if (w < words) x[b][r] = __builtin_amdgcn_raw_buffer_load_b32(rs_asf, sa_off[r] + 4u * (first + w), 0, 0);
                }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const int w = base + 16 * b + l;
                    if (w < words) a_scales[((tid >> 4) + r * RG) * kRowWords + w] = x[b][r];
                }
        }
    };
    // Pair `i` of this wave. The second step of the last pair may lie past K: its loads repeat the first's, and its scales are 0
    // on both sides (B's as packed), 2^-254, by which its products vanish
    auto load = [&](Stage& s, int i) __attribute__((always_inline)) {
        const int ks = 2 * (i * WAVES + wave);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = min(ks + h, nks - 1);
#pragma unroll
            for (int n = 0; n < FN; ++n)
                s.b[h][n] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_b, b_off + n * kFragBytes, at * kBTileBytes, kBAux));
#pragma unroll
            for (int f = 0; f < FM; ++f)
                s.a[h][f] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_a, a_off[f], at * (kBK / 2), 0));
        }
        if constexpr (!SHARED) {
            const uint32_t at = 4u * (uint32_t)min(ks + (g & 1), nks - 1);
#pragma unroll
            for (int f = 0; f < FM; ++f) s.sa[f] = __builtin_amdgcn_raw_buffer_load_b32(rs_asf, sa_off[f] + at, 0, 0);
        }
        // both steps' bytes of a fragment lie together
#pragma unroll
        for (int n = 0; n < FN; ++n)
            s.sb[n] = __builtin_amdgcn_raw_buffer_load_b16(rs_bsf, sb_off + n * 256, (ks >> 2) * kBScaleBlockBytes + (ks & 3), kBAux);
    };
    auto multiply = [&](const Stage& s, int i) __attribute__((always_inline)) {
        const uint32_t keep = 2 * (i * WAVES + wave) + 1 < nks ? ~0u : 0xffu;
        uint32_t sa[FM];
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            if constexpr (SHARED) {
                const uint2 w = *reinterpret_cast<const uint2*>(a_scales + (f * 16 + l) * kRowWords + (2 * (i * WAVES + wave) & (kWords - 1)));
                sa[f] = __builtin_amdgcn_perm(w.y, w.x, sel) & keep;
            } else {
                const auto q = __builtin_amdgcn_permlane16_swap(s.sa[f], s.sa[f], false, false);
                sa[f] = __builtin_amdgcn_perm(q[1], q[0], sel) & keep;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const v8i x = {s.a[h][f].x, s.a[h][f].y, s.a[h][f].z, s.a[h][f].w, 0, 0, 0, 0};
#pragma unroll
                for (int n = 0; n < FN; ++n) {
                    const v8i y = {s.b[h][n].x, s.b[h][n].y, s.b[h][n].z, s.b[h][n].w, 0, 0, 0, 0};
                    acc[f][n] = h == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[f][n], kFp4, kFp4, 0, (int)sa[f], 0, (int)s.sb[n])
                                       : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[f][n], kFp4, kFp4, 1, (int)sa[f], 1, (int)s.sb[n]);
                }
            }
    };
    // All pairs (SHARED: those whose scales LDS holds) at a time, this wave's i0 to n-1: DEPTH in flight, then each multiplied and
    // its registers loaded again while there are more
    const int pairs = (nks + 1) >> 1, chunk = SHARED ? kWords / 2 : pairs;
    for (int first = 0; first < pairs; first += chunk) {
        const int i0 = first / WAVES, n = (min(pairs, first + chunk) - wave + WAVES - 1) / WAVES;
        if constexpr (SHARED) {
            if (first > 0) __syncthreads();                     // every wave is through with the words before
            stage_scales(2 * first);
        }
        if (n - i0 < DEPTH) {
#pragma unroll
            for (int i = 0; i < DEPTH - 1; ++i)
                if (i0 + i < n) load(st[i], i0 + i);
            if constexpr (SHARED) __syncthreads();
#pragma unroll
            for (int i = 0; i < DEPTH - 1; ++i)
                if (i0 + i < n) multiply(st[i], i0 + i);
            continue;
        }
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) load(st[i], i0 + i);
        if constexpr (SHARED) __syncthreads();
        int i = i0;
        // the last DEPTH pairs, the first of them in stage S
        auto rest = [&](auto first) __attribute__((always_inline)) {
            constexpr int S = decltype(first)::value;
#pragma unroll
            for (int j = 0; j < DEPTH; ++j) multiply(st[(S + j) % DEPTH], i + j);
        };
        auto turn = [&](auto stage) __attribute__((always_inline)) -> bool {
            constexpr int S = decltype(stage)::value;
            if (i + DEPTH >= n) {
                rest(stage);
                return true;
            }
            multiply(st[S], i);
            load(st[S], i + DEPTH);
            ++i;
            return false;
        };
        for (;;) {
            if (turn(IntC<0>{})) break;
            if constexpr (DEPTH > 1)
                if (turn(IntC<1 % DEPTH>{})) break;
        }
    }
    static_assert(DEPTH <= 2, "");

    // Row of the tile and column of D of a lane's sums: rows 16f + 4g + r, columns col .. col + FN-1 (lane column j of fragment
    // f is column 128 * (f / 8) + 8j + f % 8 of its tile; all FN or none: N is a multiple of 16)
    auto store = [&](int r, int col, const float (&x)[FN]) __attribute__((always_inline)) {
        const int row = d_row(r);
        if (row < 0 || col >= p.N) return;
        const size_t to = (size_t)row * p.N + col;
        if constexpr (F32) {
            float* d = static_cast<float*>(p.d) + to;
            if constexpr (FN == 4) *reinterpret_cast<v4f*>(d) = (v4f){x[0], x[1], x[2], x[3]};
            else
#pragma unroll
                for (int n = 0; n < FN; ++n) d[n] = x[n];
        } else {
            uint16_t* d = static_cast<uint16_t*>(p.d) + to;
            const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector(((v2f){x[0], x[FN > 1 ? 1 : 0]}), v2bf));
            if constexpr (FN == 1) *d = (uint16_t)w0;
            else if constexpr (FN == 2) *reinterpret_cast<uint32_t*>(d) = w0;
            else *reinterpret_cast<uint2*>(d) = make_uint2(w0, __builtin_bit_cast(uint32_t, __builtin_convertvector(((v2f){x[2], x[3]}), v2bf)));
        }
    };
    const int col0 = tile * kBN + 128 * (frag >> 3) + (frag & 7);
    // the waves' sums as the lanes hold them, then thread t of a fragment row adds lane t / 4's row t % 4 over the waves
    constexpr int HALF = WAVES * FM * FN > 64 ? WAVES / 2 : WAVES;    // of the waves at a time: at most 64 KB
    __shared__ __attribute__((aligned(16))) float sums[HALF * FM * FN * 256];
    auto at = [&](int w, int f, int n) __attribute__((always_inline)) -> float* { return sums + ((w * FM + f) * FN + n) * 256; };
    if (HALF < WAVES) {
        if (wave >= HALF) {
#pragma unroll
            for (int f = 0; f < FM; ++f)
#pragma unroll
                for (int n = 0; n < FN; ++n) *reinterpret_cast<v4f*>(at(wave - HALF, f, n) + lane * 4) = acc[f][n];
        }
        __syncthreads();
        if (wave < HALF) {
#pragma unroll
            for (int f = 0; f < FM; ++f)
#pragma unroll
                for (int n = 0; n < FN; ++n) acc[f][n] += *reinterpret_cast<const v4f*>(at(wave, f, n) + lane * 4);
        }
        __syncthreads();
    }
    if (wave < HALF) {
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int n = 0; n < FN; ++n) *reinterpret_cast<v4f*>(at(wave, f, n) + lane * 4) = acc[f][n];
    }
    __syncthreads();
    for (int i = tid; i < FM * 256; i += WAVES * 64) {
        const int f = i >> 8, t = i & 255;
        float x[FN];
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            x[n] = at(0, f, n)[t];
#pragma unroll
            for (int w = 1; w < HALF; ++w) x[n] += at(w, f, n)[t];
        }
        store(f * 16 + 4 * (t >> 6) + (t & 3), col0 + 8 * ((t >> 2) & 15), x);
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
// Bytes of a chunk (4 steps) of a row's scales
constexpr int kChunkRow = 4 * kStep / 32;

// A's scale words: through LDS where there is room, or straight into registers (64 rows with two workgroups on a CU, whose
// operands fill its LDS). There kQuads loads a block's 16 bytes a lane and four blocks an instruction, kWords 4 bytes and one
// block: a load costs by the lines it touches, 16 rows' in either form. kQuads needs rows of whole blocks, K a multiple of 512
// (8192 x 256 x 7168 29.5 -> 24.5 us, 2048 x 2048 x 18432 68 -> 59, 300 x 7168 x 7168 24 -> 21).
enum class AScales { kStaged, kQuads, kWords };

template <int BM, int WAVES_M, int WAVES_N, AScales S>
struct Fp4Cfg {
    static constexpr int WM = BM / WAVES_M, WN = kBN / WAVES_N;
    static constexpr int FM = WM / 16, FN = WN / 16;
    static constexpr int A_BYTES = BM * kARow;
    static constexpr bool STAGED = S == AScales::kStaged, QUADS = S == AScales::kQuads;
    static_assert(STAGED || BM == 64, "");
    static constexpr int S_BYTES = STAGED ? BM * kChunkRow : 0;
    // ring slots: 144 KB with 256 rows, 152 with 128, 80 with 64 (84 staged)
    static constexpr int DA = BM == 128 ? 3 : 2, DB = BM == 128 ? 3 : 2;
    static constexpr int LDS_BYTES = DA * A_BYTES + DB * kBStep + 2 * S_BYTES;
    static constexpr int A_DMA = A_BYTES / 1024 / 4, B_DMA = kBStep / 1024 / 4;   // 1 KB loads per wave and step
    static constexpr int S_DMA = S_BYTES / 256 / 4;                                // 256-byte loads per wave and chunk
    static_assert(WAVES_M * WAVES_N == 4 && LDS_BYTES <= 160 * 1024 && DA >= 2 && DB >= 2, "");

    // A wave's loads go out in the order X(k), Y(k), X(k+1), ...; X(k): scale words, then B of step k+DB; Y(k): A of step k+DA.
    // Scale words of X(k), u = k % 4: A's of the next chunk in steps 0, 1 and, with DB = 2, 2 (into LDS), or of the next block in
    // even steps or (QUADS) of the next four blocks in step 0 (into registers); B's of the next block in even steps
    static constexpr int S_STEPS = DB == 2 ? 3 : 2;                                 // so that they are there in step 3
    static constexpr int S_EACH = (S_DMA + S_STEPS - 1) / S_STEPS;
    static constexpr int staged(int u) { return u >= S_STEPS ? 0 : u == S_STEPS - 1 ? S_DMA - u * S_EACH : S_EACH; }
    static constexpr int direct(int u) { return STAGED || u % 2 || (QUADS && u) ? 0 : FM; }
    static constexpr int scales(int u) { return staged(u) + direct(u) + (u % 2 ? 0 : FN); }
    // How many loads may be in flight at the second barrier of step k, when A and B of step k+1 and, in odd steps, the scale words
    // of X(k-1) have to be there: those behind the last one needed.
    static constexpr int in_flight(int u) {
        int n = 0;
        for (int d = 0;; ++d) {                        // X(k-d), then Y(k-d-1)
            if (DB <= d + 1) return n;                 // B of step k-d+DB
            n += B_DMA;
            if (u % 2 && d == 1) return n;             // (QUADS: needed in step 3, asked for in step 0)
            n += scales((u - d + 8) % 4);
            if (DA <= d + 2) return n;                 // A of step k-d-1+DA
            n += A_DMA;
        }
    }
};

// NT: B through non-temporal loads (one row tile reads it).
template <int BM, int WAVES_M, int WAVES_N, bool F32, bool NT, AScales S = AScales::kStaged>
__device__ inline __attribute__((always_inline)) void tiled_part(const GemmFp4Args& args, uint8_t* smem, const RowTiles& rt, int v, int part) {
    // gfx950 buffer descriptors are a device-only type: the host pass sees an empty function
#if defined(__HIP_DEVICE_COMPILE__)
    using C = Fp4Cfg<BM, WAVES_M, WAVES_N, S>;
    constexpr bool QUADS = C::QUADS;
    constexpr int WM = C::WM, FM = C::FM, FN = C::FN, DA = C::DA, DB = C::DB, A_DMA = C::A_DMA, B_DMA = C::B_DMA;
    constexpr int kBAux = NT ? 2 : 0;
    uint8_t* const bring = smem + DA * C::A_BYTES;
    uint8_t* const sring = bring + DB * kBStep;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int g = lane >> 4, l = lane & 15;
    const int tiles_n = (args.N + kBN - 1) / kBN;
    const int grp = v / (kGroupM * tiles_n), mt0 = grp * kGroupM;
    const int gm = min(kGroupM, rt.total - mt0), vin = v - grp * kGroupM * tiles_n;
    const int nt = vin / gm;
    const RowTile at0 = row_tile(args, rt, args.block_m, mt0 + vin % gm);
    const int group = at0.group, row0 = at0.row0 + part * BM, count = at0.count - part * BM;
    const bool list = args.perm != nullptr;
    const int nks = args.K / kBK, nst = (nks + 1) >> 1;   // K steps of 128 and steps of 256
    // A and D row of row r, -1 on padding
    auto d_row = [&](int r) __attribute__((always_inline)) -> int {
        if (list) return args.perm[row0 + r];
        return r < count ? row0 + r : -1;
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
    // A's scale words (4 bytes, a K step's): lane 16g + i takes step g's of row i, per fragment and block of 4 K steps, in
    // registers, or, staged, row r's 8 of a chunk lie in LDS as 8-row groups of 256 bytes: word 32 * (half ^ group % 2) + 4 *
    // (r % 8) + step in its half, so that a fragment's words lie in different banks. Words of K steps past the last repeat it.
    const int last_kb = (nks - 1) >> 2, last_kc = (nks - 1) >> 3;
    constexpr int NSA = C::STAGED ? C::S_DMA : FM;
    uint32_t sa_off[NSA], past_sf[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int step = C::STAGED ? 8 * last_kc + 4 * ((lane >> 5) ^ h) + (lane & 3) : 4 * last_kb + g;
        past_sf[h] = QUADS ? 16u * max(0, (last_kb & ~3) + g - last_kb) : 4u * max(0, step - (nks - 1));
    }
#pragma unroll
    for (int f = 0; f < NSA; ++f) {
        if constexpr (C::STAGED)
            sa_off[f] = a_row(8 * (wave * NSA + f) + ((lane >> 2) & 7)) * (uint32_t)(args.K / 32) + 16u * ((lane >> 5) ^ (f & 1)) + 4u * (lane & 3);
        else
            sa_off[f] = a_row(wm * WM + f * 16 + l) * (uint32_t)(args.K / 32) + (QUADS ? 16u : 4u) * g;
    }
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
                                                 kc * kBTileBytes + (i & 15) * kFragBytes, 0, kBAux);
    };
    // scale words of a block of two steps: A's as loaded, and by byte of the K step in the block as the products take them
    uint32_t raw[FM], sa[2][FM], sb[2][FN], next[FM];
    v4i quad[FM];
    auto load_sa = [&](int kb, int f) __attribute__((always_inline)) {
        raw[f] = __builtin_amdgcn_raw_buffer_load_b32(rs_asf, sa_off[f] - (kb == last_kb ? past_sf[0] : 0u), kb * 16, 0);
    };
    // QUADS: lane 16b + i has row i's 16 bytes of block 4 kq + b (blocks past the last: its)
    const int last_kq = last_kb >> 2;
    auto load_quad = [&](int kq, int f) __attribute__((always_inline)) {
        const int q = min(kq, last_kq);
        quad[f] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_asf, sa_off[f] - (q == last_kq ? past_sf[0] : 0u), q * 64, 0));
    };
    // the words of blocks 2 * pair and 2 * pair + 1, of the four in quad: bytes by block of 32 within the lane, then lane row and
    // word changed places
    auto take_quad = [&](int pair, int f) __attribute__((always_inline)) {
        const uint32_t d0 = quad[f].x, d1 = quad[f].y, d2 = quad[f].z, d3 = quad[f].w;
        const uint32_t a = __builtin_amdgcn_perm(d1, d0, 0x05010400u), b = __builtin_amdgcn_perm(d1, d0, 0x07030602u);
        const uint32_t c = __builtin_amdgcn_perm(d3, d2, 0x05010400u), d = __builtin_amdgcn_perm(d3, d2, 0x07030602u);
        const uint32_t w0 = __builtin_amdgcn_perm(c, a, 0x05040100u), w1 = __builtin_amdgcn_perm(c, a, 0x07060302u);
        const uint32_t w2 = __builtin_amdgcn_perm(d, b, 0x05040100u), w3 = __builtin_amdgcn_perm(d, b, 0x07060302u);
        const auto p02 = __builtin_amdgcn_permlane32_swap(w0, w2, false, false), p13 = __builtin_amdgcn_permlane32_swap(w1, w3, false, false);
        const bool second = pair & 1;
        const auto y = __builtin_amdgcn_permlane16_swap(second ? p02[1] : p02[0], second ? p13[1] : p13[0], false, false);
        sa[0][f] = y[0];
        next[f] = y[1];
    };
    auto load_sb = [&](int kb, int f, int set) __attribute__((always_inline)) {
        sb[set][f] = __builtin_amdgcn_raw_buffer_load_b32(rs_bsf, lane * 4 + (wn * FN + f) * 256, kb * kBScaleBlockBytes, kBAux);
    };
    auto stage_sa = [&](int kc, int j) __attribute__((always_inline)) {
        const int c = min(kc, last_kc);       // chunks past the last reload it into a free slot
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_asf, MOE_LPTR(sring + (kc & 1) * C::S_BYTES + (wave * NSA + j) * 256), 4,
                                                 sa_off[j] - (c == last_kc ? past_sf[j & 1] : 0u), c * kChunkRow, 0, 0);
    };
    uint32_t rd_sa[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        rd_sa[h] = (uint32_t)((wm * WM / 8 + (l >> 3)) * 256 + 128 * (h ^ (l >> 3)) + 16 * (l & 7) + 4 * g);
    auto read_sa = [&](int kb, int f) __attribute__((always_inline)) {
        raw[f] = *reinterpret_cast<const uint32_t*>(sring + ((kb >> 1) & 1) * C::S_BYTES + f * 512 + rd_sa[kb & 1]);
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

    // Loads of a step: scale words and B of DB steps ahead from its first barrier on, which every wave passes with B of this step
    // in registers; A of DA steps ahead from its second barrier on, which every wave passes with A of this step read
    constexpr int ROW = 2 * FN;             // MFMAs per fragment row
    constexpr int X_OPS = C::scales(0) + B_DMA, X_ROOM = (FM - 2) * ROW, X_SPACE = X_ROOM / X_OPS > 3 ? 3 : X_ROOM / X_OPS;   // MFMAs per load
    constexpr int Y_SPACE = ROW / A_DMA;
    static_assert(X_SPACE >= 1 && Y_SPACE >= 1 && C::scales(2) <= C::scales(0), "a step's loads fit between its barriers");
    auto issue_x = [&](int ks, int u, int set, int op) __attribute__((always_inline)) {
        if (op < C::staged(u)) {
            stage_sa((ks >> 2) + 1, u * C::S_EACH + op);
            return;
        }
        op -= C::staged(u);
        if (u % 2 == 0) {
            const int kb = min((ks >> 1) + 1, last_kb);
            if (op < C::direct(u)) {
                if constexpr (QUADS) load_quad((ks >> 3) + ((ks >> 2) & 1), op);     // (every second time again: no branch)
                else load_sa(kb, op);
                return;
            }
            op -= C::direct(u);
            if (op < FN) {
                load_sb(kb, op, set);
                return;
            }
            op -= FN;
        }
        if (op < B_DMA) load_b(ks + DB, op);
    };
    // the loads that the steps before step 0 would have issued
#pragma unroll
    for (int i = 0; i < NSA; ++i) {
        if constexpr (C::STAGED) stage_sa(0, i);
        else if constexpr (QUADS) load_quad(0, i);
        else load_sa(0, i);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) load_sb(0, f, 0);
#pragma unroll
    for (int k = DA > DB ? -DA : -DB; k < 0; ++k) {
#pragma unroll
        for (int j = 0; j < B_DMA; ++j)
            if (k + DB >= 0) load_b(k + DB, j);
#pragma unroll
        for (int j = 0; j < A_DMA; ++j)
            if (k + DA >= 0) load_a(k + DA, j);
    }
    // everything after A and B of step 0
    constexpr int WAIT0 = DA > DB ? (DB - 1) * B_DMA + DB * A_DMA : (DB - 1) * (B_DMA + A_DMA);
    static_assert(DA == DB || DA == DB + 1, "order of the first loads");
    static_assert(WAIT0 < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (WAIT0 & 15) | (((WAIT0 >> 4) & 3) << 14));
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"(WAIT0) : "memory");
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        if constexpr (C::STAGED) read_sa(0, f);
        if constexpr (QUADS) take_quad(0, f);
        else sa[0][f] = scale_words(0, f);
    }
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

    // One step: 256 of K, FM rows of 2 x FN MFMAs. Its first barrier stands behind the first row, where every wave holds B of the
    // step in registers. At the second, before the last row, this wave's loads of step ks+1 have landed and its LDS reads of A
    // are done; behind it each B fragment's registers take the next step's right after their last use.
    auto step = [&](int ks, auto u_c) __attribute__((always_inline)) {
        constexpr int U = decltype(u_c)::value, ODD = U & 1, SET = U >> 1;   // U: ks % 4
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            if (fm == 1) asm volatile("s_barrier" ::: "memory");
            if (fm == FM - 1) {
                // in flight may be what was issued behind B of step ks+1 and (odd steps) the scale words
                constexpr int WN_ = C::in_flight(U);
                static_assert(WN_ < 64, "vmcnt range");
                __builtin_amdgcn_s_waitcnt(0x0070 | (WN_ & 15) | (((WN_ >> 4) & 3) << 14));
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(WN_) : "memory");
                if constexpr (ODD) {
                    // the next block's scale words have landed: no wait of the compiler's own for them
                    // (QUADS: needed in step 3 only; a use in step 1 keeps the loads, which the waits count, in the steps behind the
                    // loop too)
                    if constexpr (QUADS) {
#pragma unroll
                        for (int f = 0; f < FM; ++f) asm volatile("" : "+v"(quad[f]));
                    } else if constexpr (!C::STAGED) {
#pragma unroll
                        for (int f = 0; f < FM; ++f) asm volatile("" : "+v"(raw[f]));
                    }
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
                        // the next block's words of A: read from LDS, half a row of products later put in order
                        if (ODD && C::STAGED && t < FM) read_sa((ks >> 1) + 1, t);
                        constexpr int LATE = ROW - FM;
                        if (ODD && t >= LATE) {
                            if constexpr (!QUADS) sa[SET ^ 1][t - LATE] = scale_words((ks >> 1) + 1, t - LATE);
                            else if (U == 3) take_quad((ks >> 2) + 1, t - LATE);
                            else sa[1][t - LATE] = next[t - LATE];
                            asm volatile("" : "+v"(sa[SET ^ 1][t - LATE]));
                            if (QUADS && U == 3) asm volatile("" : "+v"(next[t - LATE]));
                        }
                        if (t % Y_SPACE == 0 && t / Y_SPACE < A_DMA) load_a(ks + DA, t / Y_SPACE);
                    } else if (fm > 0 && ((fm - 1) * ROW + t) % X_SPACE == 0) {
                        issue_x(ks, U, SET ^ 1, ((fm - 1) * ROW + t) / X_SPACE);
                    }
                    __builtin_amdgcn_sched_barrier(0x7);
                }
            }
        }
    };

    // 4 steps per iteration: two blocks of scale words, one per set
    int ks0 = 0;
    for (; ks0 + 4 <= nst; ks0 += 4) {
        step(ks0, IntC<0>{});
        step(ks0 + 1, IntC<1>{});
        step(ks0 + 2, IntC<2>{});
        step(ks0 + 3, IntC<3>{});
    }
    if (ks0 < nst) step(ks0, IntC<0>{});
    if (ks0 + 1 < nst) step(ks0 + 1, IntC<1>{});
    if (ks0 + 2 < nst) step(ks0 + 2, IntC<2>{});
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
    // bf16 goes past the caches: all CUs store at once (4096 x 7168 x 18432 249 -> 244 us, 8192^3 258 -> 250, 1024 x 7168 x 2048 15.7
    // -> 14.6, 2048^3 10.5 -> 10.1; 3100 x 368 x 640, whose rows end within a line, 6.0 -> 6.2). FP32's 16-byte stores leave half a
    // line each, which the caches put together (8192^3 past them 271 -> 361 us, 2048^3 13.1 -> 16.1)
    auto put = [&](auto* to, const auto& x) __attribute__((always_inline)) {
        if constexpr (!F32) __builtin_nontemporal_store(x, to);
        else *to = x;
    };
    auto store = [&](int fm, int r, size_t to) __attribute__((always_inline)) {
        if constexpr (F32) {
            float* dst = static_cast<float*>(args.d) + to;
#pragma unroll
            for (int q = 0; q < FN; q += 4)
                put(reinterpret_cast<v4f*>(dst + q), (v4f){acc[fm][q][r], acc[fm][q + 1][r], acc[fm][q + 2][r], acc[fm][q + 3][r]});
        } else {
            uint32_t pk[FN / 2];
#pragma unroll
            for (int q = 0; q < FN; q += 2) {
                const v2f x = {acc[fm][q][r], acc[fm][q + 1][r]};
                pk[q / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2bf));
            }
            uint16_t* dst = static_cast<uint16_t*>(args.d) + to;
            if constexpr (FN == 8) put(reinterpret_cast<v4i*>(dst), (v4i){(int)pk[0], (int)pk[1], (int)pk[2], (int)pk[3]});
            else put(reinterpret_cast<v2u*>(dst), (v2u){pk[0], pk[1]});
        }
    };
    const int lane_row = wm * WM + 4 * g;
    if (list) {
        // all row numbers first: one wait for them (a load and a wait per row: 3.7 us of 12.5 at 300 x 7168 x 2048)
        int rows[FM][4];
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int r = 0; r < 4; ++r) rows[fm][r] = args.perm[row0 + lane_row + fm * 16 + r];
        asm volatile("" ::: "memory");
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (rows[fm][r] >= 0) store(fm, r, (size_t)rows[fm][r] * args.N + col0);
    } else {
        const size_t first = (size_t)(row0 + lane_row) * args.N + col0;
        if (count >= BM) {
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
#pragma unroll
                for (int r = 0; r < 4; ++r) store(fm, r, first + (size_t)(fm * 16 + r) * args.N);
        } else {
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (lane_row + fm * 16 + r < count) store(fm, r, first + (size_t)(fm * 16 + r) * args.N);
        }
    }
#endif
}

template <int BM, int WAVES_M, int WAVES_N, bool F32, bool NT, AScales S>
__global__ __launch_bounds__(256, BM == 64 ? 2 : 1) void gemm_fp4_tiled(GemmFp4Args args) {
    using C = Fp4Cfg<BM, WAVES_M, WAVES_N, S>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS_BYTES];
    const RowTiles rt = row_tiles(args, BM);
    const int v = xcd_tile(rt.total * ((args.N + kBN - 1) / kBN), blockIdx.x);
    if (v < 0) return;
    tiled_part<BM, WAVES_M, WAVES_N, F32, NT, S>(args, smem, rt, v, 0);
}

// 256 x 256 tiles in rounds of one per CU; a last round at most half full runs as parts of 64 rows where those are no more than
// the CUs, else of 128 rows, so that more of them work, and each starts when a CU is through with the rounds before.
template <bool F32>
__global__ __launch_bounds__(256, 1) void gemm_fp4_rounds(GemmFp4Args args) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[160 * 1024];
    const RowTiles rt = row_tiles(args, 256);
    const int total = rt.total * ((args.N + kBN - 1) / kBN);
    const int rem = total % kCus, full = rem <= kCus / 2 ? total - rem : total;
    if ((int)blockIdx.x < full) {
        tiled_part<256, 2, 2, F32, false>(args, smem, rt, xcd_tile(full, blockIdx.x), 0);
        return;
    }
    const int parts = rem <= kCus / 4 ? 4 : 2;
    const int u = xcd_tile((total - full) * parts, blockIdx.x - full);
    if (u < 0) return;
    if (parts == 4) tiled_part<64, 1, 4, F32, false>(args, smem, rt, full + u / 4, u % 4);
    else tiled_part<128, 2, 2, F32, false>(args, smem, rt, full + u / 2, u % 2);
}

template <int BM, int WAVES_M, int WAVES_N, AScales S>
hipError_t launch_tiled(unsigned grid, bool nt, const GemmFp4Args& a, hipStream_t stream) {
    if (a.out_f32) {
        if (nt) gemm_fp4_tiled<BM, WAVES_M, WAVES_N, true, true, S><<<grid, 256, 0, stream>>>(a);
        else gemm_fp4_tiled<BM, WAVES_M, WAVES_N, true, false, S><<<grid, 256, 0, stream>>>(a);
    } else {
        if (nt) gemm_fp4_tiled<BM, WAVES_M, WAVES_N, false, true, S><<<grid, 256, 0, stream>>>(a);
        else gemm_fp4_tiled<BM, WAVES_M, WAVES_N, false, false, S><<<grid, 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <int FM, int FN, int WAVES, int DEPTH>
hipError_t launch_skinny(bool nt, const GemmFp4Args& a, hipStream_t stream) {
    const size_t units = a.dense_rows > 0 ? cdiv(a.dense_rows, 16 * FM) : (size_t)a.max_tiles * (4 / FM);
    const size_t tiles = units * (size_t)(cdiv(a.N, 128) * (8 / FN));
    constexpr int T = WAVES * 64;
    if (tiles >= (size_t(1) << 32) / T) return hipErrorInvalidConfiguration;   // a launch wraps there
    const unsigned grid = (unsigned)tiles;
    if (a.out_f32) {
        if (nt) gemm_fp4_skinny<FM, FN, WAVES, DEPTH, true, true><<<grid, T, 0, stream>>>(a);
        else gemm_fp4_skinny<FM, FN, WAVES, DEPTH, true, false><<<grid, T, 0, stream>>>(a);
    } else {
        if (nt) gemm_fp4_skinny<FM, FN, WAVES, DEPTH, false, true><<<grid, T, 0, stream>>>(a);
        else gemm_fp4_skinny<FM, FN, WAVES, DEPTH, false, false><<<grid, T, 0, stream>>>(a);
    }
    return hipGetLastError();
}

// Microseconds of a product with each kernel. Tiled: rounds of the workgroups that the CUs hold, each fixed + step per 128 K
// (64 rows: two on a CU, a last round of one on a CU takes 0.57 of it, and where K is a multiple of 512 a step 0.9). Skinny:
// fixed + the larger of wave per pair of K steps that a wave takes and, per 256 workgroups, step per 128 K; + each per 256
// workgroups. Fitted to 260 products from 1 x 16 x 128 to 7698 x 2704 x 3200, 512 x 4096 x 7168 and 32 groups of about 150 rows,
// each timed with every kernel, weights from memory: what the model picks is 1.8 % slower than the best of the kernels on
// average, a third slower at worst (24 groups of about one row, 320 x 2816).
// A masked or listed product's 64-row tiles with few rows leave most workgroups of 16 or 32 rows without any and the others to
// a part of the CUs, so that there all count.
struct Cost {
    Fp4Kernel kernel;
    int block_m, bm, bn;       // rows of its row tiles, rows and columns per workgroup
    int waves;                 // sharing K; 0: tiled
    double fixed, step, wave, each;
};
constexpr Cost kCosts[] = {{Fp4Kernel::kTiled256, 256, 256, 256, 0, 7.9, 0.8, 0, 0},
                           {Fp4Kernel::kTiled128, 128, 128, 256, 0, 5.75, 0.504, 0, 0},
                           {Fp4Kernel::kTiled64, 64, 64, 256, 0, 6.0, 0.729, 0, 0},
                           {Fp4Kernel::kSkinny64x64, 64, 64, 64, 8, 1.50, 0.237, 3.00, 3.95},
                           {Fp4Kernel::kSkinny32x64, 64, 32, 64, 8, 1.66, 0.198, 2.24, 1.50},
                           {Fp4Kernel::kSkinny32x32, 64, 32, 32, 8, 1.66, 0.150, 1.62, 0.27},
                           {Fp4Kernel::kSkinny16x32, 64, 16, 32, 8, 1.14, 0.087, 1.27, 0.40},
                           {Fp4Kernel::kSkinny16, 64, 16, 16, 16, 2.08, 0.065, 0.98, 0.65}};
constexpr double kAlone64 = 0.574, kQuads64 = 0.895;

// Row tiles of bm rows. Groups of unknown length: spread from half to one and a half times the expected rows
double row_tiles_of(int groups, double rows, int most, bool ragged, int bm) {
    if (!ragged) return groups * std::ceil(rows / bm);
    double tiles = 0;
    for (int i = 0; i < 8; ++i) tiles += std::ceil(std::min<double>(most, rows * (9 + 2 * i) / 16) / bm);
    return groups * tiles / 8;
}

}  // namespace

Fp4Plan fp4_plan(int groups, double rows, int most, int max_rows, bool ragged, int N, int K) {
    Fp4Plan best{};
    double least = 0;
    const int steps = K / kBK;
    for (const Cost& c : kCosts) {
        const int cols = c.waves ? cdiv(N, 128) * (128 / c.bn) : cdiv(N, kBN);
        // a launch has fewer than 2^32 threads (the caller has checked this for kTiled128); the 256-row tiles' last round may take
        // kCus workgroups more
        const uint64_t grid = (uint64_t)most_row_tiles(max_rows, groups, c.block_m) * (c.block_m / c.bm) * cols +
                              (c.kernel == Fp4Kernel::kTiled256 ? kCus : 0);
        if (c.kernel != Fp4Kernel::kTiled128 && grid * (c.waves ? c.waves * 64 : 256) >= (1ull << 32)) continue;
        const int unit = ragged ? std::max(c.bm, 64) : c.bm;
        const double tiles = std::ceil(row_tiles_of(groups, rows, most, ragged, unit) * (unit / c.bm)) * cols;
        double t = 0;
        if (c.waves) {
            const double share = tiles / kCus;
            t = c.fixed + std::max(c.wave * cdiv(cdiv(steps, 2), c.waves), share * c.step * steps) + share * c.each;
        } else {
            const bool two = c.kernel == Fp4Kernel::kTiled64;
            const double round = c.fixed + c.step * (two && K % 512 == 0 ? kQuads64 : 1.0) * steps, slots = two ? 2 * kCus : kCus;
            const double rounds = std::floor(tiles / slots), rem = tiles - rounds * slots;
            t = rounds * round;
            // the parts of the 256-row tiles' last round: of 64 rows, kCosts[2], or 128, kCosts[1]
            if (c.kernel == Fp4Kernel::kTiled256 && rem > 0 && rem <= kCus / 4) t += kCosts[2].fixed + kCosts[2].step * steps;
            else if (c.kernel == Fp4Kernel::kTiled256 && rem > 0 && rem <= kCus / 2) t += kCosts[1].fixed + kCosts[1].step * steps;
            else if (two && rem > 0 && rem <= kCus) t += kAlone64 * round;
            else if (rem > 0) t += round;
        }
        if (best.block_m == 0 || t < least) {
            best = Fp4Plan{c.kernel, c.block_m, rows <= c.block_m};
            least = t;
        }
    }
    return best;
}

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
        case Fp4Kernel::kTiled128: return launch_tiled<128, 2, 2, AScales::kStaged>((unsigned)grid, plan.stream, a, stream);
        case Fp4Kernel::kTiled64:
            if (a.K % 512 == 0) return launch_tiled<64, 1, 4, AScales::kQuads>((unsigned)grid, plan.stream, a, stream);
            return launch_tiled<64, 1, 4, AScales::kWords>((unsigned)grid, plan.stream, a, stream);
        case Fp4Kernel::kSkinny64x64: return launch_skinny<4, 4, 8, 1>(plan.stream, a, stream);
        case Fp4Kernel::kSkinny32x64: return launch_skinny<2, 4, 8, 1>(plan.stream, a, stream);
        case Fp4Kernel::kSkinny32x32: return launch_skinny<2, 2, 8, 1>(plan.stream, a, stream);
        case Fp4Kernel::kSkinny16x32: return launch_skinny<1, 2, 8, 1>(plan.stream, a, stream);
        case Fp4Kernel::kSkinny16: return launch_skinny<1, 1, 16, 2>(plan.stream, a, stream);
    }
    return hipGetLastError();
}

}  // namespace moe
