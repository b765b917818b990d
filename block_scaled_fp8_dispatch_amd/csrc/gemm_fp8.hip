// FP8 x FP8 GEMMs with one UE8M0 scale per 1x128 block of A and per 128x128 block of B, on
// v_mfma_scale_f32_16x16x128_f8f6f4: one instruction spans exactly one block along K, so both
// scales go into it (every lane's scale byte is its row's, or its 128-column block's) and the
// sum over K stays in the FP32 accumulators. That instruction adds the products of 8
// consecutive K after aligning them to the largest of the 8 and drops what lies more than 13
// bits below it (measured on gfx950: 2^16 + 270 within 8 gives 2^16 + 264; across groups of 8 the
// sum is FP32's). That is about 1.5e-5 of the result's norm on normal data, 5e-5 on codes of every
// magnitude alike, at most 2^-10 of the sum over the groups of max|a| max|b|: far below a bf16
// output's rounding (1.7e-3) unless products cancel, but not FP32. FP32 outputs therefore go through v_mfma_f32_16x16x32_bf16,
// at half its rate, whose sums are FP32's: an e4m3 value times its block's power of two is exact
// in bf16 (3 mantissa bits of 7, the exponent range of FP32) for scale bytes 3 to 246. Rows with a
// byte outside, their own or their columns', are computed again from the codes alone, both
// scales going to each block's sum (add_block).
//
// Tiled kernel (bf16 outputs). A workgroup of 4 waves owns a BM x 256 tile of D. Both operands
// of a K step (BM x 128 and 256 x 128 bytes) go straight from memory into LDS rings
// (direct-to-LDS buffer loads, XOR-swizzled 16-byte chunks); rows of B are placed so that the
// 16 rows of a fragment are adjacent and a lane ends up with adjacent columns of D. There is
// one barrier per K step, before its last row of MFMAs: it waits for this wave's loads of the
// next step. Behind it the next step's B fragments are read into the registers of the current
// ones, each right after its last use, and the loads that refill the slots just freed go out,
// one per MFMA, on into the next step: B of DB and A of DA steps ahead, so that a load has
// DB - 1 (DA - 1) steps less that window to arrive. Scales come one 32-bit word per 4 K steps;
// the instruction's byte select picks the step.
//
// Workgroups go round-robin to the 8 XCDs; each XCD owns a contiguous range of tile ids, which
// walk groups of 4 row tiles across all column tiles, so the tiles resident on one XCD share
// rows of A and B in its L2.
//
// Bound by the matrix units at the clock that the power limit leaves: 2.4 to 2.7 PFLOP/s in full
// rounds of 256 x 256 tiles (4096 x 4096 x 7168: 90 to 102 us on different cards; a library product
// with one scale per tensor reaches 2.62 to 2.66 at 4096 x 7168 x 18432, these kernels 2.5). 64-row tiles that stream B once
// (32 groups of about 32 rows, 4096 x 7168 each) run at 5.9 TB/s.
#include <algorithm>
#include <cmath>

#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kGroupM = 4;
constexpr int kCus = 256;                 // compute units of an MI355X

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// 2^(byte - 127) as the operand of the scaled conversions, which read its exponent field
__device__ inline float scale_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

// The largest `byte - 3` (unsigned) of a row's scale bytes: above kBf16Holds where an e4m3 value times 2^(byte - 127)
// need not be a bf16 number (448 * 2^119 is below bf16's largest, 2^-9 * 2^-124 its smallest). The loops keep it, at
// two instructions a byte, and what it says is looked at once behind them (a branch in every step: 128 x 32 x 7168 6.0 us
// instead of 5.5, 33 x 7168 x 2048 9.2 instead of 6.9).
constexpr uint32_t kBf16Holds = 246 - 3;
// (pinned: done before the byte's register is loaded again, else the byte is copied, which waits for that load)
__device__ inline void keep_beyond(uint32_t& far, uint32_t byte) {
    far = max(far, byte - 3u);
    asm volatile("" : "+v"(far));
}

// two words of e4m3 codes (8 values) times 2^(byte - 127), exact in bf16 for bytes 3 to 246
__device__ inline v8bf to_bf16(int w0, int w1, float scale) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
    return (v8bf){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// sum += the products of one K step for a fragment's rows and columns, from the codes unscaled (exact in bf16) and
// both scales on the block's sum, so that nothing on the way leaves FP32's range unless the result does. row: the
// scale bytes of the lane's rows 4g .. 4g+3, col: the columns'
__device__ inline void add_block(v4f& sum, const v8i& a, const v8i& b, const uint32_t (&row)[4], uint32_t col) {
    v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16(a[2 * q], a[2 * q + 1], 1.0f), to_bf16(b[2 * q], b[2 * q + 1], 1.0f),
                                                    x, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        sum[r] += row[r] == 255u || col == 255u ? __uint_as_float(0x7fc00000u) : __builtin_ldexpf(x[r], (int)(row[r] + col) - 254);
}

// A lane's codes of K step ks from memory, as a fragment read from LDS has them
__device__ inline v8i load_block(__amdgpu_buffer_rsrc_t rs, uint32_t at, int ks) {
    const v4i lo = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, at, ks * kBK, 0));
    const v4i hi = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, at + 64, ks * kBK, 0));
    return (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

// Stores the first `left` of n adjacent columns of a row. A row may start at any element, so the
// wide store's address is aligned to the element only, which the hardware takes (one store per
// element instead: 8192 x 7001 x 2048 176 us against 142; aligned chunks taken apart: 142 against
// 147).
template <int n, class T>
__device__ inline void store_columns(T* dst, const T (&x)[n], int left) {
    if (left >= n) {
        if constexpr (sizeof(x) == 16) {
            if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
                __builtin_memcpy(__builtin_assume_aligned(dst, 16), x, sizeof(x));
                return;
            }
        }
        __builtin_memcpy(dst, x, sizeof(x));
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i < left) dst[i] = x[i];
    }
}

// Workgroups go round-robin to the XCDs: tile id of workgroup `block` with each XCD (workgroup id
// mod 8) owning a contiguous range of ids. -1: none left.
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

constexpr int kRsrcWord3 = 0x00020000;   // raw buffer descriptor: byte offsets, no swizzle
constexpr int kAllRecords = -1;
#define MOE_LPTR(p) ((__attribute__((address_space(3))) void*)(p))

// Skinny kernel: few rows, or too few tiles for the tiled kernel. A workgroup owns a BM x BN tile
// of D and its WAVES waves share K, wave w taking steps w, w + WAVES, ... and keeping sums of its
// own. Each wave fills LDS slots of its own (rows of A and B as the tiled kernel lays them
// out), so there is no barrier before the end: it waits for its oldest slot, reads and multiplies
// it, and refills it. The waves' sums meet in LDS, the upper half of the waves onto the lower, then
// those in wave order.
//
// Bound by latency where tiles are few (128 x 32 x 7168, FP32: 5.7 us in 16 tiles of 16 x 16 with two slots
// a wave; 32 x 32: 9.0), by weights in flight where they are many (4 x 7168 x 7168: 11.2 us, 4.6 TB/s,
// in tiles of 16 x 32). Two workgroups or more on a CU with one slot a wave beat one with two (33 x 7168 x
// 2048, 32 x 32: 7.5 us against 9.3). Operands straight from memory to registers instead were tried
// and were slower: a fragment read takes half a line of 16 rows at a time, and the chunks in flight
// do not fit the registers.
constexpr int kSkinnyWaves = 8;

template <int BM, int BN, int WAVES, int SLOTS>
struct SkinnyCfg {
    static constexpr int FM = BM / 16, FN = BN / 16;
    static constexpr int SLOT = (BM + BN) * kBK;
    static constexpr int A_DMA = BM / 8, B_DMA = BN / 8, NS = FM + 1;
    static constexpr int PITCH = BN + 4;           // floats per row of a wave's sums
    static constexpr int LDS_BYTES = SLOTS * WAVES * SLOT;
    static_assert(LDS_BYTES <= 160 * 1024 && BN <= 128, "");
    static_assert(WAVES / 2 * BM * PITCH * 4 <= LDS_BYTES, "the sums reuse the slots");
};

template <int BM, int BN, int WAVES, int SLOTS, bool F32>
__global__ __launch_bounds__(WAVES * 64) void gemm_fp8_skinny(GemmFp8Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
    using C = SkinnyCfg<BM, BN, WAVES, SLOTS>;
    constexpr int FM = C::FM, FN = C::FN, SUB = 64 / BM, PITCH = C::PITCH;
    __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS_BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l = lane & 15;
    const bool dense = p.dense_rows > 0;
    // units of BM rows: of a dense product's rows, or of the 64-row tiles in the list
    const int units = dense ? (p.dense_rows + BM - 1) / BM : min(__builtin_amdgcn_readfirstlane(p.meta[0]), p.max_tiles) * SUB;
    const int NT = (p.N + BN - 1) / BN;
    const int v = xcd_tile(units * NT, blockIdx.x);
    if (v < 0) return;
    // groups of 4 row tiles across all column tiles: their rows of A stay in the XCD's L2
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
    auto a_row = [&](int r) __attribute__((always_inline)) -> uint32_t {
        const int d = d_row(r);
        return d < 0 ? 0u : (uint32_t)d;           // padding rows read row 0 and are never stored
    };
    // padding comes last in a row tile: nothing but padding here
    if (__builtin_amdgcn_readfirstlane(d_row(0)) < 0) return;

    uint8_t* const mine = smem + wave * SLOTS * C::SLOT;
    const int chunk = (lane & 7) ^ (lane >> 3);
    uint32_t a_off[C::A_DMA], b_off[C::B_DMA], sa_off[FM];
#pragma unroll
    for (int j = 0; j < C::A_DMA; ++j) a_off[j] = a_row(8 * j + (lane >> 3)) * (uint32_t)p.K + chunk * 16;
#pragma unroll
    for (int j = 0; j < C::B_DMA; ++j)
        b_off[j] = (uint32_t)(min(nt * BN + 8 * j + (lane >> 3), p.N - 1) - nt * BN) * (uint32_t)p.K + chunk * 16;
#pragma unroll
    for (int f = 0; f < FM; ++f) sa_off[f] = a_row(f * 16 + l) * (uint32_t)p.sf_stride;
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)p.a, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_asf = __builtin_amdgcn_make_buffer_rsrc((void*)p.a_sf, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.b + ((size_t)group * p.N + (size_t)nt * BN) * p.K), 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_bsf = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.b_sf + ((size_t)group * ((p.N + 127) / 128) + nt * BN / 128) * p.sf_stride), 0, kAllRecords, kRsrcWord3);

    uint32_t sa[SLOTS][FM], sb[SLOTS];
    auto issue = [&](int ks, auto slot_c) __attribute__((always_inline)) {
        constexpr int S = decltype(slot_c)::value;
        uint8_t* dst = mine + S * C::SLOT;
#pragma unroll
        for (int f = 0; f < FM; ++f) sa[S][f] = __builtin_amdgcn_raw_buffer_load_b8(rs_asf, sa_off[f], ks, 0);
        sb[S] = __builtin_amdgcn_raw_buffer_load_b8(rs_bsf, 0, ks, 0);
#pragma unroll
        for (int j = 0; j < C::B_DMA; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, MOE_LPTR(dst + BM * kBK + j * 1024), 16, b_off[j], ks * kBK, 0, 0);
#pragma unroll
        for (int j = 0; j < C::A_DMA; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, MOE_LPTR(dst + j * 1024), 16, a_off[j], ks * kBK, 0, 0);
    };
    const uint32_t rd_lo = (uint32_t)(l * kBK + ((g ^ (l & 7)) << 4));
    const uint32_t rd_hi = (uint32_t)(l * kBK + (((g + 4) ^ (l & 7)) << 4));
    auto read = [&](const uint8_t* q) __attribute__((always_inline)) -> v8i {
        const v4i lo = *reinterpret_cast<const v4i*>(q + rd_lo);
        const v4i hi = *reinterpret_cast<const v4i*>(q + rd_hi);
        return (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };
    v4f acc[FM][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[f][n] = (v4f){0.f, 0.f, 0.f, 0.f};
    uint32_t far_a[FM] = {}, far_b = 0;            // F32: keep_beyond() of this wave's steps
    const int nks = p.K / kBK;
    // step ks of this wave, in slot S: wait until only the younger slots' loads (if any) are in
    // flight, multiply, refill
    constexpr int W = C::NS + C::A_DMA + C::B_DMA;
    auto wait = [&](auto younger_c) __attribute__((always_inline)) {
        constexpr int V = decltype(younger_c)::value * W;
        static_assert(V < 64, "vmcnt range");
        __builtin_amdgcn_s_waitcnt(0x0F70 | (V & 15) | (((V >> 4) & 3) << 14));
        asm volatile("s_waitcnt vmcnt(%0)" :: "n"(V) : "memory");
    };
    auto step = [&](int ks, auto slot_c) __attribute__((always_inline)) {
        constexpr int S = decltype(slot_c)::value;
        if (SLOTS > 1 && ks + WAVES < nks) wait(IntC<SLOTS - 1>{});
        else wait(IntC<0>{});
        const uint8_t* src = mine + S * C::SLOT;
        if constexpr (F32) {
            keep_beyond(far_b, sb[S]);
            v8bf bv[FN][4];
#pragma unroll
            for (int n = 0; n < FN; ++n) {
                const v8i w = read(src + (BM + n * 16) * kBK);
#pragma unroll
                for (int q = 0; q < 4; ++q) bv[n][q] = to_bf16(w[2 * q], w[2 * q + 1], scale_f32(sb[S]));
            }
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                keep_beyond(far_a[f], sa[S][f]);
                const v8i w = read(src + f * 16 * kBK);
                // the same 8 consecutive codes of a lane on both sides: any order of K will do
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v8bf av = to_bf16(w[2 * q], w[2 * q + 1], scale_f32(sa[S][f]));
#pragma unroll
                    for (int n = 0; n < FN; ++n)
                        acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv[n][q], acc[f][n], 0, 0, 0);
                }
            }
        } else {
            v8i bv[FN];
#pragma unroll
            for (int n = 0; n < FN; ++n) bv[n] = read(src + (BM + n * 16) * kBK);
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const v8i av = read(src + f * 16 * kBK);
#pragma unroll
                for (int n = 0; n < FN; ++n)
                    acc[f][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv[n], acc[f][n], 0, 0, 0, (int)sa[S][f], 0,
                                                                                 (int)sb[S]);
            }
        }
        if (ks + SLOTS * WAVES < nks) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // the slot's reads are done
            issue(ks + SLOTS * WAVES, slot_c);
        }
    };
    static_assert(SLOTS <= 2, "");
    auto each_slot = [&](int ks, auto&& f) __attribute__((always_inline)) {
        if (ks < nks) f(ks, IntC<0>{});
        if (SLOTS > 1 && ks + WAVES < nks) f(ks + WAVES, IntC<SLOTS - 1>{});
    };
    each_slot(wave, issue);
    for (int ks = wave; ks < nks; ks += SLOTS * WAVES) each_slot(ks, step);
    // F32: the rows that need add_block in some wave's steps, and whether there are any
    __shared__ uint8_t far_rows[F32 ? WAVES : 1][BM];
    __shared__ int far_any[WAVES];
    if constexpr (F32) {
        bool any = false;
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            const bool far = max(far_a[f], far_b) > kBf16Holds;
            far_rows[wave][f * 16 + l] = far;
            any |= far;
        }
        far_any[wave] = __ballot(any) != 0;
    }
    __syncthreads();                               // the sums reuse the slots of all waves
    float* const sums = reinterpret_cast<float*>(smem);
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
    // columns c .. c+3 of row r
    auto store = [&](int r, int c, const v4f& x) __attribute__((always_inline)) {
        const int row = d_row(r), n = nt * BN + c;
        if (row < 0) return;
        const size_t to = (size_t)row * p.N + n;
        if constexpr (F32) {
            const float out[4] = {x.x, x.y, x.z, x.w};
            store_columns<4>(static_cast<float*>(p.d) + to, out, p.N - n);
        } else {
            const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(((v2f){x.x, x.y}), v2bf));
            const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(((v2f){x.z, x.w}), v2bf));
            const uint16_t out[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
            store_columns<4>(static_cast<uint16_t*>(p.d) + to, out, p.N - n);
        }
    };
    // four adjacent columns per thread
    for (int i = tid; i < BM * BN / 4; i += WAVES * 64) {
        const int r = i / (BN / 4), c = i % (BN / 4) * 4;
        v4f x = *reinterpret_cast<const v4f*>(&at(0, r, c));
#pragma unroll
        for (int w = 1; w < WAVES / 2; ++w) x += *reinterpret_cast<const v4f*>(&at(w, r, c));
        store(r, c, x);
    }
    if constexpr (F32) {
        int any = 0;                               // (looked up before the stores: 0.2 us more)
#pragma unroll
        for (int w = 0; w < WAVES; ++w) any |= far_any[w];
        if (__builtin_amdgcn_readfirstlane(any) == 0) return;
        // fragment after fragment, operands straight from memory; the waves share K as before. Each element is
        // stored over by the thread that stored it.
        for (int i = 0; i < FM * FN; ++i) {
            const int f = i / FN, n = i % FN;
            bool far = false;                      // row 16f + l
            for (int w = 0; w < WAVES; ++w) far |= far_rows[w][f * 16 + l] != 0;
            const uint64_t rows = __ballot(far);
            if (rows == 0) continue;
            const uint32_t a_at = a_row(f * 16 + l) * (uint32_t)p.K + 16 * g;
            const uint32_t b_at = (uint32_t)(min(nt * BN + n * 16 + l, p.N - 1) - nt * BN) * (uint32_t)p.K + 16 * g;
            v4f sum = {0.f, 0.f, 0.f, 0.f};
            for (int ks = wave; ks < nks; ks += WAVES) {
                uint32_t row[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    row[r] = __builtin_amdgcn_raw_buffer_load_b8(rs_asf, a_row(f * 16 + 4 * g + r) * (uint32_t)p.sf_stride, ks, 0);
                add_block(sum, load_block(rs_a, a_at, ks), load_block(rs_b, b_at, ks), row,
                          __builtin_amdgcn_raw_buffer_load_b8(rs_bsf, 0, ks, 0));
            }
            __syncthreads();                       // what lies in the slots has been read
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[(wave * 16 + 4 * g + r) * 20 + l] = sum[r];
            __syncthreads();
            for (int j = tid; j < BM * BN / 4; j += WAVES * 64) {
                const int r = j / (BN / 4), c = j % (BN / 4) * 4;
                if (r / 16 != f || c / 16 != n || !((rows >> (r % 16)) & 1)) continue;
                v4f x = {0.f, 0.f, 0.f, 0.f};
                for (int w = 0; w < WAVES; ++w) x += *reinterpret_cast<const v4f*>(&sums[(w * 16 + r % 16) * 20 + c % 16]);
                store(r, c, x);
            }
        }
    }
#endif
}

// acc += A x B, both e4m3, scales from byte OPS of their words. As asm so that the accumulators
// stay in their registers; the operands are only ever written by LDS or buffer loads, and the
// kernel separates the accumulators' other accesses by s_nop, so no hazard needs padding.
template <int OPS>
__device__ inline void mfma_scaled(v4f& acc, const v8i& a, const v8i& b, uint32_t sa, uint32_t sb) {
    if constexpr (OPS == 0)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else if constexpr (OPS == 1)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0]"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else if constexpr (OPS == 2)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[1,1,0]"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0]"
                     : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
}

template <int BM, int BN, int WAVES_M, int WAVES_N>
struct Fp8Cfg {
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int FM = WM / 16, FN = WN / 16;
    static constexpr int A_BYTES = BM * kBK, B_BYTES = BN * kBK;
    // ring slots: all of the CU's 160 KB
    static constexpr int DB = BM == 256 ? 2 : BM == 128 ? 3 : 4;
    static constexpr int DA = BM == 256 ? 3 : 4;
    static constexpr int LDS_BYTES = DA * A_BYTES + DB * B_BYTES;
    static constexpr int A_DMA = A_BYTES / 1024 / 4, B_DMA = B_BYTES / 1024 / 4;   // 1 KB loads per wave and step
    static_assert(WAVES_M * WAVES_N == 4 && LDS_BYTES <= 160 * 1024, "");
    static_assert(DA == DB || DA == DB + 1, "issue order written for these");
    // a wave's columns lie in one scale block of B, or (224 columns) a lane's fragments each
    // have a scale word of their own
    static constexpr bool ONE_BLOCK = WN == 64 || WN == 128;
    static constexpr int NSB = ONE_BLOCK ? 1 : FN;
    static_assert(BN % (16 * WAVES_N) == 0 && B_BYTES % 4096 == 0, "");
};

// Part `part` (of BM rows) of tile v. Tile ids walk groups of 4 row tiles (of args.block_m rows)
// across all column tiles.
// STREAM: B is read by one row tile only, through non-temporal loads. WIDE: N % 8 == 0, every row
// and a lane's chunk aligned and a chunk wholly in or out, stored plainly.
template <int BM, int BN, int WAVES_M, int WAVES_N, bool STREAM, bool WIDE>
__device__ inline __attribute__((always_inline)) void tiled_part(const GemmFp8Args& args, uint8_t* smem, int num_mt, int v, int part) {
    // gfx950 buffer descriptors are a device-only type: the host pass sees an empty function
#if defined(__HIP_DEVICE_COMPILE__)
    using C = Fp8Cfg<BM, BN, WAVES_M, WAVES_N>;
    constexpr int WM = C::WM, WN = C::WN, FM = C::FM, FN = C::FN, DA = C::DA, DB = C::DB;
    constexpr int A_DMA = C::A_DMA, B_DMA = C::B_DMA, NSB = C::NSB;
    uint8_t* const bring = smem + DA * C::A_BYTES;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int g = lane >> 4, l = lane & 15;
    const bool dense = args.dense_rows > 0;
    const int NT = (args.N + BN - 1) / BN;
    const int grp = v / (kGroupM * NT), mt0 = grp * kGroupM;
    const int gm = min(kGroupM, num_mt - mt0), vin = v - grp * kGroupM * NT;
    const int mt = mt0 + vin % gm, nt = vin / gm;
    const int group = dense ? 0 : __builtin_amdgcn_readfirstlane(args.tile_expert[mt]);
    const int row0 = (dense ? mt * args.block_m : __builtin_amdgcn_readfirstlane(args.tile_row0[mt])) + part * BM;
    const int nks = args.K / kBK;
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
    // Load j of wave w fills LDS rows 8*(w*DMA + j) .. +7 of a tile; lane l lands at row + l/8,
    // physical 16-byte chunk l%8, which holds logical chunk (l%8) ^ (row%8).
    const int chunk = (lane & 7) ^ (lane >> 3);
    uint32_t a_off[A_DMA], b_off[B_DMA];
#pragma unroll
    for (int j = 0; j < A_DMA; ++j) a_off[j] = a_row(8 * (wave * A_DMA + j) + (lane >> 3)) * (uint32_t)args.K + chunk * 16;
    // LDS row 16*f + j of B (fragment f, lane column j) is column base + j*FN + f%FN of D, so that
    // a lane's FN fragments hold FN adjacent columns; rows past N read row N-1 and are not stored
#pragma unroll
    for (int j = 0; j < B_DMA; ++j) {
        const int r = 8 * (wave * B_DMA + j) + (lane >> 3);
        const int f = r >> 4;
        const int n = nt * BN + (f / FN) * WN + (r & 15) * FN + f % FN;
        b_off[j] = (uint32_t)(min(n, args.N - 1) - nt * BN) * (uint32_t)args.K + chunk * 16;
    }
    uint32_t sa_off[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) sa_off[f] = a_row(wm * WM + f * 16 + l) * (uint32_t)args.sf_stride;
    const int nblk = (args.N + 127) / 128;
    uint32_t sb_off[NSB];
#pragma unroll
    for (int f = 0; f < NSB; ++f) {
        const int n = nt * BN + wn * WN + (C::ONE_BLOCK ? 0 : l * FN + f);
        sb_off[f] = (uint32_t)min(n >> 7, nblk - 1) * (uint32_t)args.sf_stride;
    }
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)args.a, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_asf = __builtin_amdgcn_make_buffer_rsrc((void*)args.a_sf, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(args.b + ((size_t)group * args.N + (size_t)nt * BN) * args.K), 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_bsf = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(args.b_sf + (size_t)group * nblk * args.sf_stride), 0, kAllRecords, kRsrcWord3);

    auto load_a = [&](int ks, int j) __attribute__((always_inline)) {
        const int kc = min(ks, nks - 1);      // steps past the last reload it into a free slot
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, MOE_LPTR(smem + (ks % DA) * C::A_BYTES + (wave * A_DMA + j) * 1024), 16,
                                                 a_off[j], kc * kBK, 0, 0);
    };
    auto load_b = [&](int ks, int j) __attribute__((always_inline)) {
        const int kc = min(ks, nks - 1);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, MOE_LPTR(bring + (ks % DB) * C::B_BYTES + (wave * B_DMA + j) * 1024), 16,
                                                 b_off[j], kc * kBK, 0, STREAM ? 2 : 0);
    };
    uint32_t sa[2][FM], sb[2][NSB];
    auto load_scale = [&](int kb, int i, int set) __attribute__((always_inline)) {
        if (i < FM) sa[set][i] = __builtin_amdgcn_raw_buffer_load_b32(rs_asf, sa_off[i], kb * 4, 0);
        else sb[set][i - FM] = __builtin_amdgcn_raw_buffer_load_b32(rs_bsf, sb_off[i - FM], kb * 4, 0);
    };
    const uint32_t rd_lo = (uint32_t)(l * kBK + ((g ^ (l & 7)) << 4));
    const uint32_t rd_hi = (uint32_t)(l * kBK + (((g + 4) ^ (l & 7)) << 4));
    auto read = [&](const uint8_t* p) __attribute__((always_inline)) -> v8i {
        const v4i lo = *reinterpret_cast<const v4i*>(p + rd_lo);
        const v4i hi = *reinterpret_cast<const v4i*>(p + rd_hi);
        return (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };
    auto read_a = [&](int ks, int f) __attribute__((always_inline)) -> v8i {
        return read(smem + (ks % DA) * C::A_BYTES + (wm * FM + f) * 16 * kBK);
    };
    auto read_b = [&](int ks, int f) __attribute__((always_inline)) -> v8i {
        return read(bring + (ks % DB) * C::B_BYTES + (wn * FN + f) * 16 * kBK);
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

    // prologue: the scale words of block 0, then the loads that the steps before step 0 would
    // have issued (step s: B of s+DB, then A of s+DA)
    constexpr int NS = FM + NSB, SOPS = 4 - DB;
    const int last_kb = (nks - 1) >> 2;
#pragma unroll
    for (int i = 0; i < NS; ++i) load_scale(0, i, 0);
    if constexpr (DA == DB + 1) {
#pragma unroll
        for (int j = 0; j < A_DMA; ++j) load_a(0, j);
    }
#pragma unroll
    for (int s = 0; s < DB - 1; ++s) {
#pragma unroll
        for (int j = 0; j < B_DMA; ++j) load_b(s, j);
#pragma unroll
        for (int j = 0; j < A_DMA; ++j) load_a(s + DA - DB, j);
    }
    // of the step before step 0 only what goes out in its last row; step 0 issues the rest
#pragma unroll
    for (int op = 0; op < FN; ++op) {
        if (op < B_DMA) load_b(DB - 1, op);
        else if (op < B_DMA + A_DMA) load_a(DA - 1, op - B_DMA);
    }
    // everything after A and B of step 0
    constexpr int PART = FN < A_DMA + B_DMA ? FN : A_DMA + B_DMA;
    constexpr int WAIT0 = PART + (DB - 2) * (A_DMA + B_DMA) + (DA == DB ? 0 : A_DMA);
    __builtin_amdgcn_s_waitcnt(0x0F70 | (WAIT0 & 15) | (((WAIT0 >> 4) & 3) << 14));
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"(WAIT0) : "memory");
    v8i bq[FN], a_cur, a_nx;
#pragma unroll
    for (int f = 0; f < FN; ++f) bq[f] = read_b(0, f);
    a_nx = read_a(0, 0);

    // One K step. Its barrier stands before the last row of MFMAs: this wave's loads of step
    // ks+1 have landed (in flight may be what was issued after B of ks+1), its LDS reads of step
    // ks are done. Then go, one per MFMA, through the last row and the next step's first rows,
    // the loads into the slots that are free now: the next block's scale words (in one step
    // of four), B of step ks+DB, A of step ks+DA.
    auto step = [&](int ks, auto ops_c, auto set_c) __attribute__((always_inline)) {
        constexpr int OPS = decltype(ops_c)::value, SET = decltype(set_c)::value;
        auto issue = [&](int kp, int ns, int op) __attribute__((always_inline)) {
            if (op < ns) load_scale(min((kp >> 2) + 1, last_kb), op, SET ^ 1);
            else if (op < ns + B_DMA) load_b(kp + DB, op - ns);
            else if (op < ns + B_DMA + A_DMA) load_a(kp + DA, op - ns - B_DMA);
        };
        constexpr int NS_HERE = OPS == SOPS ? NS : 0, NS_PREV = (OPS + 3) % 4 == SOPS ? NS : 0;
        static_assert(NS + B_DMA + A_DMA <= FM * FN, "a step's loads fit between its MFMAs");
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            if (fm == FM - 1) {
                // issued after B of step ks+1: its A (where A runs further ahead), and the issues
                // of steps ks+2-DB .. ks-1
                constexpr int SCW = DB >= 3 && (OPS + 3) % 4 == SOPS ? NS : DB >= 4 && (OPS + 2) % 4 == SOPS ? NS : 0;
                constexpr int WN_ = (DA == DB ? 0 : A_DMA) + (DB - 2) * (A_DMA + B_DMA) + SCW;
                static_assert(WN_ < 64, "vmcnt range");
                __builtin_amdgcn_s_waitcnt(0x0070 | (WN_ & 15) | (((WN_ >> 4) & 3) << 14));
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(WN_) : "memory");
                if constexpr (OPS == 3) {
                    // the next block's scale words have landed: no wait of the compiler's own for them
#pragma unroll
                    for (int f = 0; f < FM; ++f) asm volatile("" : "+v"(sa[SET ^ 1][f]));
#pragma unroll
                    for (int f = 0; f < NSB; ++f) asm volatile("" : "+v"(sb[SET ^ 1][f]));
                }
            }
            a_cur = a_nx;
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) {
                mfma_scaled<OPS>(acc[fm][fn], a_cur, bq[fn], sa[SET][fm], sb[SET][C::ONE_BLOCK ? 0 : fn]);
                if (fn == 0) a_nx = fm + 1 < FM ? read_a(ks, fm + 1) : read_a(ks + 1, 0);
                if (fm == FM - 1) {
                    bq[fn] = read_b(ks + 1, fn);
                    issue(ks, NS_HERE, fn);
                } else {
                    issue(ks - 1, NS_PREV, FN + fm * FN + fn);
                }
                __builtin_amdgcn_sched_barrier(0x7);
            }
        }
    };

    // 8 steps per iteration: two 4-step scale blocks, one per scale set
    int ks0 = 0;
    for (; ks0 + 8 <= nks; ks0 += 8) {
        step(ks0, IntC<0>{}, IntC<0>{});
        step(ks0 + 1, IntC<1>{}, IntC<0>{});
        step(ks0 + 2, IntC<2>{}, IntC<0>{});
        step(ks0 + 3, IntC<3>{}, IntC<0>{});
        step(ks0 + 4, IntC<0>{}, IntC<1>{});
        step(ks0 + 5, IntC<1>{}, IntC<1>{});
        step(ks0 + 6, IntC<2>{}, IntC<1>{});
        step(ks0 + 7, IntC<3>{}, IntC<1>{});
    }
    if (ks0 < nks) step(ks0, IntC<0>{}, IntC<0>{});
    if (ks0 + 1 < nks) step(ks0 + 1, IntC<1>{}, IntC<0>{});
    if (ks0 + 2 < nks) step(ks0 + 2, IntC<2>{}, IntC<0>{});
    if (ks0 + 3 < nks) step(ks0 + 3, IntC<3>{}, IntC<0>{});
    if (ks0 + 4 < nks) step(ks0 + 4, IntC<0>{}, IntC<1>{});
    if (ks0 + 5 < nks) step(ks0 + 5, IntC<1>{}, IntC<1>{});
    if (ks0 + 6 < nks) step(ks0 + 6, IntC<2>{}, IntC<1>{});
    // the last steps' reloads must land before the workgroup's LDS is given back
    __builtin_amdgcn_s_waitcnt(0x0F70);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    // the accumulators' reads stay behind the wait states that the last MFMA's result needs
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) asm volatile("" : "+a"(acc[fm][fn]));

    // ---- epilogue: rows 16*fm + 4g + r, columns col0 .. col0 + FN-1 ----------------------------
    const int col0 = nt * BN + wn * WN + l * FN;
    uint16_t* const d = static_cast<uint16_t*>(args.d);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = d_row(wm * WM + fm * 16 + 4 * g + r);
            if (row < 0) continue;
            uint32_t pk[(FN + 1) / 2];
#pragma unroll
            for (int q = 0; q < FN; q += 2) {
                const v2f x = {acc[fm][q][r], acc[fm][q + 1 < FN ? q + 1 : q][r]};
                pk[q / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2bf));
            }
            uint16_t* dst = d + (size_t)row * args.N + col0;
            if constexpr (WIDE) {
                static_assert(FN == 8 || FN == 4, "");
                if (col0 >= args.N) continue;
                if constexpr (FN == 8) *reinterpret_cast<v4i*>(dst) = (v4i){(int)pk[0], (int)pk[1], (int)pk[2], (int)pk[3]};
                else *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
            } else {
                uint16_t out[FN];
#pragma unroll
                for (int q = 0; q < FN; ++q) out[q] = (uint16_t)(pk[q / 2] >> (16 * (q & 1)));
                store_columns<FN>(dst, out, args.N - col0);
            }
        }
    }
#endif
}

// The row tiles in use: their number lies on the device unless the product is dense
__device__ inline int row_tiles(const GemmFp8Args& args, int bm) {
    const int n = args.dense_rows > 0 ? (args.dense_rows + bm - 1) / bm : __builtin_amdgcn_readfirstlane(args.meta[0]);
    return min(n, args.max_tiles);
}

template <int BM, int BN, int WAVES_M, int WAVES_N, bool STREAM, bool WIDE>
__global__ __launch_bounds__(256, 1) void gemm_fp8_tiled(GemmFp8Args args) {
    using C = Fp8Cfg<BM, BN, WAVES_M, WAVES_N>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS_BYTES];
    const int num_mt = row_tiles(args, BM);
    const int v = xcd_tile(num_mt * ((args.N + BN - 1) / BN), blockIdx.x);
    if (v < 0) return;
    tiled_part<BM, BN, WAVES_M, WAVES_N, STREAM, WIDE>(args, smem, num_mt, v, 0);
}

// 256 x 256 tiles in rounds of one per CU; a last round at most half full runs as parts of 64 rows where
// those are no more than the CUs, else of 128 rows, so that more of them work, and each starts when a CU
// is through with the rounds before (as launches of their own the parts wait for the last of these
// workgroups: 3 to 5 us of 260 more at 8192 rows in 8 groups, 4096 x 7168).
template <bool WIDE>
__global__ __launch_bounds__(256, 1) void gemm_fp8_rounds(GemmFp8Args args) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[160 * 1024];
    const int num_mt = row_tiles(args, 256), total = num_mt * ((args.N + 255) / 256);
    const int rem = total % kCus, full = rem <= kCus / 2 ? total - rem : total;
    if ((int)blockIdx.x < full) {
        tiled_part<256, 256, 2, 2, false, WIDE>(args, smem, num_mt, xcd_tile(full, blockIdx.x), 0);
        return;
    }
    const int parts = rem <= kCus / 4 ? 4 : 2;
    const int u = xcd_tile((total - full) * parts, blockIdx.x - full);
    if (u < 0) return;
    if (parts == 4) tiled_part<64, 256, 1, 4, false, WIDE>(args, smem, num_mt, full + u / 4, u % 4);
    else tiled_part<128, 256, 2, 2, false, WIDE>(args, smem, num_mt, full + u / 2, u % 2);
}

// FP32 outputs with enough tiles: 128 x 256 of D per workgroup, 2 x 2 waves of 64 x 128, LDS rings of
// three steps. Each step converts its operands to bf16 (exact) and feeds
// v_mfma_f32_16x16x32_bf16. One barrier per step: behind it the loads of two steps ahead go into
// the slot that every wave has finished reading. Bound by the conversions (192 per wave and step
// beside 128 MFMAs): 224 us, 1.07 PFLOP/s at 4096 x 4096 x 7168, 124 us at 32768 x 256 x 7168; accumulators kept in place by asm and
// conversions placed between the MFMAs by hand measured 6 % slower.
constexpr int kF32Rows = 128;

__global__ __launch_bounds__(256, 1) void gemm_fp8_tiled_f32(GemmFp8Args args) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int BM = kF32Rows, FM = 4, FN = 8, SLOTS = 3, A_BYTES = BM * kBK, B_BYTES = kBN * kBK;
    constexpr int A_DMA = A_BYTES / 4096, B_DMA = B_BYTES / 4096;
    __shared__ __attribute__((aligned(16))) uint8_t smem[SLOTS * (A_BYTES + B_BYTES)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int g = lane >> 4, l = lane & 15;
    const bool dense = args.dense_rows > 0;
    int num_mt = dense ? (args.dense_rows + BM - 1) / BM : __builtin_amdgcn_readfirstlane(args.meta[0]);
    if (num_mt > args.max_tiles) num_mt = args.max_tiles;
    const int NT = (args.N + kBN - 1) / kBN;
    const int v = xcd_tile(num_mt * NT, blockIdx.x);
    if (v < 0) return;
    const int grp = v / (kGroupM * NT), mt0 = grp * kGroupM;
    const int gm = min(kGroupM, num_mt - mt0), vin = v - grp * kGroupM * NT;
    const int mt = mt0 + vin % gm, nt = vin / gm;
    const int group = dense ? 0 : __builtin_amdgcn_readfirstlane(args.tile_expert[mt]);
    const int row0 = dense ? mt * BM : __builtin_amdgcn_readfirstlane(args.tile_row0[mt]);
    const int nks = args.K / kBK;
    auto d_row = [&](int r) __attribute__((always_inline)) -> int {
        if (dense) return row0 + r < args.dense_rows ? row0 + r : -1;
        return args.perm[row0 + r];
    };
    auto a_row = [&](int r) __attribute__((always_inline)) -> uint32_t {
        const int d = d_row(r);
        return d < 0 ? 0u : (uint32_t)d;           // padding rows read row 0 and are never stored
    };
    const int chunk = (lane & 7) ^ (lane >> 3);
    uint32_t a_off[A_DMA], b_off[B_DMA], sa_off[FM];
#pragma unroll
    for (int j = 0; j < A_DMA; ++j) a_off[j] = a_row(8 * (wave * A_DMA + j) + (lane >> 3)) * (uint32_t)args.K + chunk * 16;
    // B rows in fragment order, as in the tiled kernel: a lane ends up with 8 adjacent columns
#pragma unroll
    for (int j = 0; j < B_DMA; ++j) {
        const int r = 8 * (wave * B_DMA + j) + (lane >> 3), f = r >> 4;
        const int n = nt * kBN + (f / FN) * 128 + (r & 15) * FN + f % FN;
        b_off[j] = (uint32_t)(min(n, args.N - 1) - nt * kBN) * (uint32_t)args.K + chunk * 16;
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) sa_off[f] = a_row(wm * 64 + f * 16 + l) * (uint32_t)args.sf_stride;
    const int nblk = (args.N + 127) / 128, blk = min(nt * 2 + wn, nblk - 1);
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)args.a, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_asf = __builtin_amdgcn_make_buffer_rsrc((void*)args.a_sf, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(args.b + ((size_t)group * args.N + (size_t)nt * kBN) * args.K), 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_bsf = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(args.b_sf + ((size_t)group * nblk + blk) * args.sf_stride), 0, kAllRecords, kRsrcWord3);
    uint32_t sa[2][FM], sb[2];
    // loads of step ks into ring slot ks % 3; the scale bytes into set S
    auto issue = [&](int ks, auto set_c) __attribute__((always_inline)) {
        constexpr int S = decltype(set_c)::value;
        const int kc = min(ks, nks - 1);           // steps past the last reload it into a free slot
        uint8_t* dst = smem + (ks % SLOTS) * (A_BYTES + B_BYTES);
#pragma unroll
        for (int f = 0; f < FM; ++f) sa[S][f] = __builtin_amdgcn_raw_buffer_load_b8(rs_asf, sa_off[f], kc, 0);
        sb[S] = __builtin_amdgcn_raw_buffer_load_b8(rs_bsf, 0, kc, 0);
#pragma unroll
        for (int j = 0; j < B_DMA; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, MOE_LPTR(dst + A_BYTES + (wave * B_DMA + j) * 1024), 16, b_off[j],
                                                     kc * kBK, 0, 0);
#pragma unroll
        for (int j = 0; j < A_DMA; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, MOE_LPTR(dst + (wave * A_DMA + j) * 1024), 16, a_off[j], kc * kBK, 0,
                                                     0);
    };
    const uint32_t rd_lo = (uint32_t)(l * kBK + ((g ^ (l & 7)) << 4));
    const uint32_t rd_hi = (uint32_t)(l * kBK + (((g + 4) ^ (l & 7)) << 4));
    auto read = [&](const uint8_t* p) __attribute__((always_inline)) -> v8i {
        const v4i lo = *reinterpret_cast<const v4i*>(p + rd_lo);
        const v4i hi = *reinterpret_cast<const v4i*>(p + rd_hi);
        return (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };
    v4f acc[FM][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[f][n] = (v4f){0.f, 0.f, 0.f, 0.f};
    uint32_t far_a[FM] = {}, far_b = 0;            // keep_beyond() of all steps
    // the scale bytes of a step are copied out of their set before the set is loaded again
    auto step = [&](int ks, auto set_c) __attribute__((always_inline)) {
        constexpr int S = decltype(set_c)::value;
        constexpr int W = FM + 1 + A_DMA + B_DMA;  // the loads of step ks+1
        __builtin_amdgcn_s_waitcnt(0x0070 | (W & 15) | (((W >> 4) & 3) << 14));
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(W) : "memory");
        float fa[FM];
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            fa[f] = scale_f32(sa[S][f]);
            keep_beyond(far_a[f], sa[S][f]);
        }
        const float fb = scale_f32(sb[S]);
        keep_beyond(far_b, sb[S]);
        issue(ks + 2, set_c);
        const uint8_t* src = smem + (ks % SLOTS) * (A_BYTES + B_BYTES);
        v8bf av[FM][4];
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            const v8i w = read(src + (wm * FM + f) * 16 * kBK);
#pragma unroll
            for (int q = 0; q < 4; ++q) av[f][q] = to_bf16(w[2 * q], w[2 * q + 1], fa[f]);
        }
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            const v8i w = read(src + A_BYTES + (wn * FN + n) * 16 * kBK);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v8bf bv = to_bf16(w[2 * q], w[2 * q + 1], fb);
#pragma unroll
                for (int f = 0; f < FM; ++f) acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[f][q], bv, acc[f][n], 0, 0, 0);
            }
        }
    };
    issue(0, IntC<0>{});
    issue(1, IntC<1>{});
    for (int ks = 0; ks < nks; ks += 2) {
        step(ks, IntC<0>{});
        if (ks + 1 < nks) step(ks + 1, IntC<1>{});
    }
    // the last steps' reloads must land before the workgroup's LDS is given back
    __builtin_amdgcn_s_waitcnt(0x0F70);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");

    const int col0 = nt * kBN + wn * 128 + l * FN;
    float* const d = static_cast<float*>(args.d);
#pragma unroll
    for (int f = 0; f < FM; ++f) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = d_row(wm * 64 + f * 16 + 4 * g + r);
            if (row < 0) continue;
            float out[FN];
#pragma unroll
            for (int n = 0; n < FN; ++n) out[n] = acc[f][n][r];
            store_columns<FN>(d + (size_t)row * args.N + col0, out, args.N - col0);
        }
    }
    // rows that need add_block: all of K again, operands from memory, stored over by the lanes that stored them
    uint64_t far[FM], any = 0;                     // bit l: row 16f + l
#pragma unroll
    for (int f = 0; f < FM; ++f) any |= far[f] = __ballot(max(far_a[f], far_b) > kBf16Holds);
    if (any == 0) return;
    static_assert(FM == 4, "");
    for (int f = 0; f < FM; ++f) {
        const uint64_t rows = f == 0 ? far[0] : f == 1 ? far[1] : f == 2 ? far[2] : far[3];
        if (rows == 0) continue;
        v4f sum[FN];
        uint32_t b_at[FN], row_at[4];
        const uint32_t a_at = a_row(wm * 64 + f * 16 + l) * (uint32_t)args.K + 16 * g;
#pragma unroll
        for (int r = 0; r < 4; ++r) row_at[r] = a_row(wm * 64 + f * 16 + 4 * g + r) * (uint32_t)args.sf_stride;
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            sum[n] = (v4f){0.f, 0.f, 0.f, 0.f};
            b_at[n] = (uint32_t)(min(col0 + n, args.N - 1) - nt * kBN) * (uint32_t)args.K + 16 * g;
        }
        for (int ks = 0; ks < nks; ++ks) {
            uint32_t row[4];
            const uint32_t col = __builtin_amdgcn_raw_buffer_load_b8(rs_bsf, 0, ks, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) row[r] = __builtin_amdgcn_raw_buffer_load_b8(rs_asf, row_at[r], ks, 0);
            const v8i a = load_block(rs_a, a_at, ks);
#pragma unroll
            for (int n = 0; n < FN; ++n) add_block(sum[n], a, load_block(rs_b, b_at[n], ks), row, col);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = d_row(wm * 64 + f * 16 + 4 * g + r);
            if (row < 0 || !((rows >> (4 * g + r)) & 1)) continue;
            float out[FN];
#pragma unroll
            for (int n = 0; n < FN; ++n) out[n] = sum[n][r];
            store_columns<FN>(d + (size_t)row * args.N + col0, out, args.N - col0);
        }
    }
#endif
}

template <int BM, int BN, int SLOTS>
void launch_skinny(const GemmFp8Args& a, hipStream_t stream) {
    const size_t units = a.dense_rows > 0 ? cdiv(a.dense_rows, BM) : (size_t)a.max_tiles * (64 / BM);
    const unsigned grid = (unsigned)(units * (size_t)cdiv(a.N, BN));
    if (a.out_f32) gemm_fp8_skinny<BM, BN, kSkinnyWaves, SLOTS, true><<<grid, kSkinnyWaves * 64, 0, stream>>>(a);
    else gemm_fp8_skinny<BM, BN, kSkinnyWaves, SLOTS, false><<<grid, kSkinnyWaves * 64, 0, stream>>>(a);
}

template <int BM, int WAVES_M, int WAVES_N, bool STREAM>
void launch_tiled(unsigned grid, const GemmFp8Args& a, hipStream_t stream) {
    if (a.N % 8 == 0) gemm_fp8_tiled<BM, kBN, WAVES_M, WAVES_N, STREAM, true><<<grid, 256, 0, stream>>>(a);
    else gemm_fp8_tiled<BM, kBN, WAVES_M, WAVES_N, STREAM, false><<<grid, 256, 0, stream>>>(a);
}

// Microseconds of a product with each kernel. Tiled: rounds of 256 workgroups, each fixed + step per
// 128 K. Skinny: fixed + wave per step that a wave takes + for every 256 workgroups tile + step per
// 128 K. Fitted to 35 products (FP32: 23) from 1 x 256 x 512 to 2 x 20000 x 7168, 2048 x 2048 x 18432
// and 4096 x 4096 x 2048, each timed with every kernel, weights from memory, and the tiled ones to
// 4096 x 4096 x 7168 (256 rows: 90 to 100 us) and 4096 x 7168 x 18432 (256 columns 453, 224 432) too:
// what the model picks is 1 to 2 % slower than the best of the kernels on average, 10 % at most.
// Of a list's 64-row tiles with few rows 3 in 4 workgroups of 16 rows have none and the others share a
// quarter of the CUs, so that there all count (16 x 4096 x 4096 so: 13.6 us, without the empty ones 6.9).
struct Cost {
    Fp8Kernel kernel;
    int block_m, bm, bn;       // rows of its row tiles, rows and columns per workgroup
    int threads;
    double fixed, step, wave, tile;
};
constexpr Cost kBf16[] = {{Fp8Kernel::kTiled256, 256, 256, 256, 256, 10.8, 1.50, 0, 0},
                          {Fp8Kernel::kTiled128, 128, 128, 256, 256, 7.0, 0.80, 0, 0},
                          {Fp8Kernel::kTiled64, 64, 64, 256, 256, 4.6, 0.72, 0, 0},
                          {Fp8Kernel::kTiled256x224, 256, 256, 224, 256, 13.5, 1.38, 0, 0},
                          {Fp8Kernel::kSkinny64, 64, 64, 64, 512, 2.26, 0.185, 2.05, 2.89},
                          {Fp8Kernel::kSkinny32, 64, 32, 32, 512, 1.89, 0.093, 0.95, 0.75},
                          {Fp8Kernel::kSkinny16x32, 64, 16, 32, 512, 2.12, 0.064, 0.68, 0.40},
                          {Fp8Kernel::kSkinny16, 64, 16, 16, 512, 2.05, 0.043, 0.42, 0.65}};
constexpr Cost kF32[] = {{Fp8Kernel::kTiled128, 128, 128, 256, 256, 8.0, 1.92, 0, 0},
                         {Fp8Kernel::kSkinny64, 64, 64, 64, 512, 2.78, 0.223, 1.81, 3.47},
                         {Fp8Kernel::kSkinny32, 64, 32, 32, 512, 2.07, 0.090, 0.89, 1.01},
                         {Fp8Kernel::kSkinny16x32, 64, 16, 32, 512, 2.02, 0.056, 0.76, 0.52},
                         {Fp8Kernel::kSkinny16, 64, 16, 16, 512, 2.01, 0.040, 0.51, 0.74}};

template <size_t NK>
Fp8Plan cheapest(const Cost (&costs)[NK], int groups, double rows, int max_rows, bool ragged, int N, int K) {
    Fp8Plan best{};
    double least = 0;
    const int steps = K / 128;
    for (const Cost& c : costs) {
        // a launch has fewer than 2^32 threads (the caller has checked this for kTiled128)
        const uint64_t grid = (uint64_t)(max_rows / c.block_m + groups) * (c.block_m / c.bm) * cdiv(N, c.bn);
        if (c.kernel != Fp8Kernel::kTiled128 && grid * c.threads >= (1ull << 32)) continue;
        // groups of unknown length end in a tile that is half full on average
        double mt = groups * (ragged ? rows / c.bm + 0.5 : std::ceil(rows / c.bm));
        if (ragged && c.bm < 32) mt = groups * std::max(1.0, rows / 64 + 0.5) * (64 / c.bm);
        const double tiles = std::ceil(mt) * std::ceil((double)N / c.bn);
        double t = 0;
        if (c.wave > 0) {
            t = c.fixed + c.wave * cdiv(steps, kSkinnyWaves) + tiles / kCus * (c.tile + c.step * steps);
        } else {
            double rounds = std::floor(tiles / kCus);
            const double rem = tiles - rounds * kCus;
            if (rem > 0) {
                // the parts of the 256-row tiles' last round: kBf16[2] and kBf16[1]
                if (c.kernel == Fp8Kernel::kTiled256 && rem <= kCus / 4) t = kBf16[2].fixed + kBf16[2].step * steps;
                else if (c.kernel == Fp8Kernel::kTiled256 && rem <= kCus / 2) t = kBf16[1].fixed + kBf16[1].step * steps;
                else rounds += 1;
            }
            t += rounds * (c.fixed + c.step * steps);
        }
        if (best.block_m == 0 || t < least) {
            best = Fp8Plan{c.kernel, c.block_m, rows <= c.block_m};
            least = t;
        }
    }
    return best;
}

}  // namespace

Fp8Plan fp8_plan(int groups, double rows_per_group, int max_rows, bool ragged, int N, int K, bool out_f32) {
    return out_f32 ? cheapest(kF32, groups, rows_per_group, max_rows, ragged, N, K)
                   : cheapest(kBf16, groups, rows_per_group, max_rows, ragged, N, K);
}

hipError_t launch_gemm_fp8(const Fp8Plan& plan, const GemmFp8Args& a, hipStream_t stream) {
    const size_t mt = a.dense_rows > 0 ? cdiv(a.dense_rows, plan.block_m) : a.max_tiles;
    // one workgroup per possible tile; those past the tiles in use return at once
    const size_t grid = mt * (size_t)cdiv(a.N, kBN);
    switch (plan.kernel) {
        case Fp8Kernel::kTiled256: {
            // the parts are at most 256
            const unsigned blocks = (unsigned)(a.dense_rows > 0 ? (grid % kCus == 0 || grid % kCus > kCus / 2 ? grid : grid - grid % kCus + kCus) : grid + kCus);
            if (a.N % 8 == 0) gemm_fp8_rounds<true><<<blocks, 256, 0, stream>>>(a);
            else gemm_fp8_rounds<false><<<blocks, 256, 0, stream>>>(a);
            break;
        }
        case Fp8Kernel::kTiled256x224:
            gemm_fp8_tiled<256, 224, 2, 2, false, false><<<(unsigned)(mt * cdiv(a.N, 224)), 256, 0, stream>>>(a);
            break;
        case Fp8Kernel::kTiled128:
            if (a.out_f32) gemm_fp8_tiled_f32<<<(unsigned)grid, 256, 0, stream>>>(a);
            else launch_tiled<128, 2, 2, false>((unsigned)grid, a, stream);
            break;
        case Fp8Kernel::kTiled64:
            if (plan.stream) launch_tiled<64, 1, 4, true>((unsigned)grid, a, stream);
            else launch_tiled<64, 1, 4, false>((unsigned)grid, a, stream);
            break;
        case Fp8Kernel::kSkinny64: launch_skinny<64, 64, 1>(a, stream); break;
        case Fp8Kernel::kSkinny32: launch_skinny<32, 32, 1>(a, stream); break;
        case Fp8Kernel::kSkinny16x32: launch_skinny<16, 32, 1>(a, stream); break;
        case Fp8Kernel::kSkinny16: launch_skinny<16, 16, 2>(a, stream); break;
    }
    return hipGetLastError();
}

}  // namespace moe
