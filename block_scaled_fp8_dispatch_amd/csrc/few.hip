// The MoE forward of a few tokens (at most 32) in two kernels, on the packed weights of
// moe_prepare_weights:
//   few_linear1  h8 = Q8( silu(x Wg^T) * (x Wu^T) ) per chosen expert and 128-column block
//   few_linear2  y[t] = bf16( sum over chosen experts e of w[t,e] * (h8[t,e] W2_e^T) )
// where w[t,e] is the sum of the top-k weights of t's slots that name e.
//
// With so few rows every product is a stream of packed weights, each fragment (16 columns x
// 128 K, 1 KB) read once from memory straight into the registers of the one wave that
// multiplies it (v_mfma_scale_f32_16x16x128_f8f6f4, the expert's tokens as rows). What counts is
// bytes in flight: a wave loads one chunk of K steps ahead of the one it multiplies, about
// 128 KB per CU in all. There is no routing pass: each workgroup of few_linear1 derives the
// chosen experts from the T*k ids, as one bit mask of tokens per expert in LDS (bits are set by
// integer atomics, whose order does not matter), and the first workgroup of each expert leaves
// its (slot, weight) rows in the workspace for few_linear2.
//
// few_linear1: a workgroup owns one 128-wide block of h of one chosen expert; wave w of 8 the
// gate fragment w and the up fragment w, so the block's largest |h| of a row meets in LDS and
// the row is requantised there. With few workgroups a second set of 8 waves takes the upper
// half of K (the sums meet in LDS). few_linear2: a workgroup owns 32 output columns; its 8 waves
// share the (expert, 512 K) pieces, each adds w * (its partial products) per token into its own
// FP32 tile in LDS, and the tiles are added in wave order.
#include <type_traits>

#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kMaxT = MOE_FEW_MAX_TOKENS;
// Largest x kept in LDS (beside 31.5 KB of few_linear1's own)
constexpr size_t kMaxXLds = 120 * 1024;
constexpr int kRsrcWord3 = 0x00020000;   // raw buffer descriptor: byte offsets, no swizzle
constexpr int kAllRecords = -1;
constexpr int kNt = 2;                   // buffer loads: non-temporal

// A row of a chosen expert: the token's first slot that names it, and its weights' sum
struct FewRow {
    int32_t slot;
    float weight;
};
// A chosen expert and its rows
struct FewSeg {
    int32_t expert, first, count;
};

__device__ inline int few_scale_byte(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int ex = (int)((bits >> 23) & 0xffu);
    const uint32_t mant = bits & 0x7fffffu;
    int b = ex - 8 + (mant > 0x600000u ? 1 : 0);   // 448 = 1.75 * 2^8
    b = b < 0 ? 0 : b;
    return amax == 0.f ? 127 : b;
}

// silu(g) * u with the hardware exp2 and reciprocal (about 1 ulp each)
__device__ inline float few_swiglu(float g, float u) {
    const float e = __builtin_amdgcn_exp2f(-g * 1.4426950408889634f);
    return g * u * __builtin_amdgcn_rcpf(1.0f + e);
}

__device__ inline v4i load_nt(const uint8_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const v4i*>(p));
}
__device__ inline uint32_t load_nt_word(const uint8_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
}

template <int OPS>
__device__ inline v4f mfma(const v8i& a, const v4i& b, const v4f& c, uint32_t sa, uint32_t sb) {
    const v8i b8 = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b8, c, 0, 4, OPS, (int)sa, OPS, (int)sb);
}

struct FewArgs {
    const uint8_t* x;
    const uint8_t* x_sf;
    const int32_t* idx;
    const float* weights;
    int T, k, E, H, I;
    const uint8_t *w1d, *w1s, *w2d, *w2s;
    size_t w1d_expert, w1d_ntile, w1s_expert, w1s_ntile;
    size_t w2d_expert, w2d_ntile, w2s_expert, w2s_ntile;
    uint8_t* h8;        // [T*k][I], the row of a (token, expert) pair being its first slot
    uint8_t* h_sf;      // [T*k][4*ceil(I/512)]
    FewRow* rows;       // [T*k] the rows of the chosen experts, expert after expert
    FewSeg* segs;       // [min(E, T*k)] the chosen experts, ascending, with their rows
    int32_t* n_used;
    uint16_t* y;
};

// C consecutive K steps of one wave: B fragments of two columns' sets and the A rows
template <int C, int FM>
struct Chunk {
    v4i b0[C], b1[C];
    v8i a[FM][C];
    uint32_t s0, s1, sa[FM];
};

template <int C, int FM, int OPS0>
__device__ inline void multiply(const Chunk<C, FM>& c, int ks, int nks, v4f (&c0)[FM], v4f (&c1)[FM]) {
    auto step = [&](auto i) __attribute__((always_inline)) {
        constexpr int S = decltype(i)::value;
        if constexpr (S < C) {
            if (ks + S < nks) {
#pragma unroll
                for (int f = 0; f < FM; ++f) {
                    c0[f] = mfma<OPS0 + S>(c.a[f][S], c.b0[S], c0[f], c.sa[f], c.s0);
                    c1[f] = mfma<OPS0 + S>(c.a[f][S], c.b1[S], c1[f], c.sa[f], c.s1);
                }
            }
        }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
}

// One wave's gate and up sums over K steps [k0, k1) for the expert's first 16 * FM tokens
// (XLDS: x rows in LDS at xl, read right before their use, so that the registers hold weights only)
template <int C, int FM, bool XLDS>
__device__ inline void linear1_sums(const FewArgs& p, const int* tok, int cnt, const uint8_t* bd, const uint8_t* bs, int k0,
                                    int k1, int lane, const uint8_t* xl, v4f (&ag)[FM], v4f (&au)[FM]) {
    const int g = lane >> 4, l = lane & 15;
    const int xsfs = 4 * ((p.H + 511) / 512);
    // (buffers with 32-bit offsets: at most 32 rows, and 64-bit addresses of each row would spill)
    uint32_t xa[FM], xs[FM];
    int sw[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int t = tok[min(f * 16 + l, cnt - 1)];     // rows past the last repeat it, unused
        xa[f] = (uint32_t)t * (uint32_t)p.H + (XLDS ? 0 : 16 * g);
        xs[f] = (uint32_t)t * (uint32_t)xsfs;
        sw[f] = t & 7;
    }
    const __amdgpu_buffer_rsrc_t rs_x = __builtin_amdgcn_make_buffer_rsrc((void*)p.x, 0, kAllRecords, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs_xsf = __builtin_amdgcn_make_buffer_rsrc((void*)p.x_sf, 0, kAllRecords, kRsrcWord3);
    auto load = [&](Chunk<C, FM>& c, int ks) __attribute__((always_inline)) {
        // steps past the last reload it (never multiplied)
        const int kb = min(ks, k1 - 1) >> 2;
        const __amdgpu_buffer_rsrc_t rs_s =
            __builtin_amdgcn_make_buffer_rsrc((void*)(bs + (size_t)kb * kBScaleBlockBytes), 0, kAllRecords, kRsrcWord3);
        c.s0 = __builtin_amdgcn_raw_buffer_load_b32(rs_s, lane * 4, 0, kNt);
        c.s1 = __builtin_amdgcn_raw_buffer_load_b32(rs_s, lane * 4, 8 * 256, kNt);
#pragma unroll
        for (int f = 0; f < FM; ++f) c.sa[f] = __builtin_amdgcn_raw_buffer_load_b32(rs_xsf, xs[f], 4 * kb, 0);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int kc = min(ks + i, k1 - 1);
            const __amdgpu_buffer_rsrc_t rs_b =
                __builtin_amdgcn_make_buffer_rsrc((void*)(bd + (size_t)kc * kBTileBytes), 0, kAllRecords, kRsrcWord3);
            c.b0[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_b, lane * 16, 0, kNt));
            c.b1[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_b, lane * 16, 8 * kFragBytes, kNt));
            if constexpr (XLDS) continue;
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const v4i lo = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_x, xa[f], kc * 128, 0));
                const v4i hi = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_x, xa[f] + 64, kc * 128, 0));
                c.a[f][i] = (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            }
        }
    };
    auto rows = [&](Chunk<C, FM>& c, int ks) __attribute__((always_inline)) {
        if constexpr (XLDS) {
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int f = 0; f < FM; ++f) {
                    const uint8_t* x = xl + xa[f] + min(ks + i, k1 - 1) * 128;
                    const v4i lo = *reinterpret_cast<const v4i*>(x + ((g ^ sw[f]) << 4));
                    const v4i hi = *reinterpret_cast<const v4i*>(x + (((g + 4) ^ sw[f]) << 4));
                    c.a[f][i] = (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                }
        }
    };
    if (k0 >= k1) return;
    Chunk<C, FM> even, odd;
    load(even, k0);
    for (int ks = k0; ks < k1; ks += 2 * C) {
        load(odd, ks + C);
        rows(even, ks);
        multiply<C, FM, 0>(even, ks, k1, ag, au);
        load(even, ks + 2 * C);
        rows(odd, ks + C);
        multiply<C, FM, C == 2 ? 2 : 0>(odd, ks + C, k1, ag, au);
    }
}

// FM: 16-row fragments an expert's tokens may need; KS: parts of K; C: K steps per chunk
template <int FM, int KS, int C>
__global__ __launch_bounds__(512 * KS, 4) void few_linear1(FewArgs p) {
    constexpr int kThreads = 512 * KS;
    __shared__ uint32_t mask[MOE_MAX_EXPERTS];
    __shared__ int ids[kMaxT * MOE_MAX_TOPK];
    __shared__ int tok[kMaxT], slot[kMaxT];        // the expert's tokens, ascending, and their first slots
    extern __shared__ __attribute__((aligned(16))) uint8_t xlds[];     // KS > 1: x, T * H bytes
    __shared__ uint32_t red[8][FM * 16];
    __shared__ __attribute__((aligned(16))) uint8_t codes[FM * 16][128];
    __shared__ v4f part[KS > 1 ? 8 : 1][2 * FM][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int cw = wave & 7, kp = wave >> 3;
    const int g = lane >> 4, l = lane & 15;
    const int NB = p.I / 128;
    const int nb = blockIdx.x % NB, u = blockIdx.x / NB;      // the u-th chosen expert

    // mask[e]: bit t set where token t names expert e
    for (int e = tid; e < p.E; e += kThreads) mask[e] = 0;
    __syncthreads();
    for (int s = tid; s < p.T * p.k; s += kThreads) {
        const int e = p.idx[s];
        ids[s] = e;
        if (e >= 0 && e < p.E) atomicOr(&mask[e], 1u << (s / p.k));
    }
    if constexpr (KS > 1) {
        // x into LDS, 16-byte chunk c of a 128-byte step at chunk c ^ (token % 8)
        for (int i = tid; i < p.T * (p.H / 16); i += kThreads) {
            const int t = i / (p.H / 16), c = i - t * (p.H / 16);
            *reinterpret_cast<v4i*>(xlds + (size_t)t * p.H + ((c ^ (t & 7)) << 4)) =
                *reinterpret_cast<const v4i*>(p.x + (size_t)i * 16);
        }
    }
    __syncthreads();
    int expert = -1, used = 0, row_base = 0;       // rows of the experts before this one
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        const uint32_t m = e0 + lane < p.E ? mask[e0 + lane] : 0u;
        uint64_t b = __ballot(m != 0);
        const int n = __popcll(b);
        const int nth = used + __popcll(b & ((1ull << lane) - 1));    // this lane's expert is the nth chosen
        if (expert < 0) {
            const uint64_t hit = __ballot(m != 0 && nth == u);
            if (nb == 0) {                             // uniform
                int before = nth < u ? __popc(m) : 0;
                for (int d = 1; d < 64; d <<= 1) before += __shfl_xor(before, d, 64);
                row_base += before;
            }
            if (hit) expert = e0 + __ffsll((unsigned long long)hit) - 1;
        }
        used += n;
    }
    expert = __builtin_amdgcn_readfirstlane(expert);
    if (blockIdx.x == 0 && tid == 0) *p.n_used = used;
    if (expert < 0) return;                        // fewer chosen experts than the grid allows for
    const uint32_t m = mask[expert];
    const int cnt = __popc(m);
    if (tid < 32 && ((m >> tid) & 1u)) {
        const int i = __popc(m & ((1u << tid) - 1));
        int first = tid * p.k;
        while (ids[first] != expert) ++first;            // the mask says that one is there
        tok[i] = tid;
        slot[i] = first;
        if (nb == 0) {
            float w = 0.f;
            for (int j = first; j < (tid + 1) * p.k; ++j)
                if (ids[j] == expert) w += p.weights[j];
            p.rows[row_base + i] = FewRow{first, w};
        }
    }
    if (nb == 0 && tid == 0) p.segs[u] = FewSeg{expert, row_base, cnt};
    __syncthreads();

    const uint8_t* bd = p.w1d + (size_t)expert * p.w1d_expert + (size_t)nb * p.w1d_ntile + cw * kFragBytes;
    const uint8_t* bs = p.w1s + (size_t)expert * p.w1s_expert + (size_t)nb * p.w1s_ntile + cw * 256;
    v4f ag[FM], au[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) ag[f] = au[f] = (v4f){0.f, 0.f, 0.f, 0.f};
    const int nkb = (p.H / 128 + 3) / 4;
    const int k0 = nkb * kp / KS * 4, k1 = min(nkb * (kp + 1) / KS * 4, p.H / 128);    // this wave's K steps
    if (FM == 1 || cnt <= 16) {
        v4f g1[1] = {ag[0]}, u1[1] = {au[0]};
        linear1_sums<C, 1, (KS > 1)>(p, tok, cnt, bd, bs, k0, k1, lane, xlds, g1, u1);
        ag[0] = g1[0];
        au[0] = u1[0];
    } else {
        linear1_sums<C, FM, (KS > 1)>(p, tok, cnt, bd, bs, k0, k1, lane, xlds, ag, au);
    }
    if constexpr (KS > 1) {
        if (kp > 0) {
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                part[cw][2 * f][lane] = ag[f];
                part[cw][2 * f + 1][lane] = au[f];
            }
        }
        __syncthreads();
        if (kp == 0) {
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                ag[f] += part[cw][2 * f][lane];
                au[f] += part[cw][2 * f + 1][lane];
            }
        }
    }
    // h of rows 16f + 4g + r, column 64*(cw/4) + 4*l + cw%4 of the block (the packed rows
    // are interleaved so); the largest |h| of a row over the block: DPP row, then the waves
    float h[FM][4];
    if (kp == 0) {
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                h[f][r] = few_swiglu(ag[f][r], au[f][r]);
                uint32_t a = __float_as_uint(fabsf(h[f][r]));
                a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xF, 0xF, false));
                a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xF, 0xF, false));
                a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x141, 0xF, 0xF, false));
                a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x140, 0xF, 0xF, false));
                if (l == 0) red[cw][f * 16 + 4 * g + r] = a;
            }
    }
    __syncthreads();
    if (kp == 0) {
        const int col = 64 * (cw >> 2) + 4 * l + (cw & 3);
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = f * 16 + 4 * g + r;
                uint32_t a = red[0][row];
#pragma unroll
                for (int w = 1; w < 8; ++w) a = max(a, red[w][row]);
                const float mul = __uint_as_float((uint32_t)(254 - few_scale_byte(__uint_as_float(a))) << 23);
                codes[row][col] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(h[f][r] * mul, 0.f, 0, false);
            }
    }
    __syncthreads();
    // 8 threads per row store its 128 codes, the first also its scale byte
    const int row = tid >> 3, piece = tid & 7;
    if (row < cnt) {
        const size_t s = slot[row];
        *reinterpret_cast<v4i*>(p.h8 + s * p.I + nb * 128 + piece * 16) =
            *reinterpret_cast<const v4i*>(&codes[row][piece * 16]);
        if (piece == 0) {
            uint32_t a = red[0][row];
            for (int w = 1; w < 8; ++w) a = max(a, red[w][row]);
            p.h_sf[s * (size_t)(4 * ((p.I + 511) / 512)) + nb] = (uint8_t)few_scale_byte(__uint_as_float(a));
        }
    }
}

// Output columns per workgroup: two fragments
constexpr int kFewCols = 32;

template <int FM>
__global__ __launch_bounds__(kFewThreads) void few_linear2(FewArgs p) {
    constexpr int C = 4;
    // a token's row of a wave's tile: 36 floats, so that the 4 rows of a lane group fall into
    // different banks
    constexpr int kPitch = kFewCols + 4;
    __shared__ float tile[kFewWaves][FM * 16][kPitch];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l = lane & 15;
    // The experts and their rows in LDS: a dependent read from memory between the pieces would
    // wait for every weight load in flight (entries past the last are copied, not used)
    __shared__ FewRow rows[kMaxT * MOE_MAX_TOPK];
    __shared__ FewSeg segs[MOE_MAX_EXPERTS];
    for (int i = tid; i < p.T * p.k; i += kFewThreads) rows[i] = p.rows[i];
    for (int i = tid; i < min(p.E, p.T * p.k); i += kFewThreads) segs[i] = p.segs[i];
    for (int i = lane; i < FM * 16 * kPitch; i += 64) (&tile[wave][0][0])[i] = 0.f;
    // each XCD (workgroup id mod 8) takes adjacent column tiles
    const int v = (int)(blockIdx.x & 7) * (int)(gridDim.x >> 3) + (int)(blockIdx.x >> 3);
    const int frag = (v & 7) * 2, nt = v >> 3;
    const int nks = p.I / 128, nkb = (nks + 3) / 4;
    const int items = __builtin_amdgcn_readfirstlane(*p.n_used) * nkb;
    const int first = (int)((long long)items * wave / kFewWaves), last = (int)((long long)items * (wave + 1) / kFewWaves);
    const size_t hsfs = 4 * (size_t)nkb;
    v4f c0[FM], c1[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) c0[f] = c1[f] = (v4f){0.f, 0.f, 0.f, 0.f};

    // where the loads stand: expert `lu` and its rows
    int lu = -1;
    int lcnt = 0;
    const uint8_t *ha[FM], *hs[FM], *bd = nullptr, *bs = nullptr;
    auto load = [&](Chunk<C, FM>& c, int it) __attribute__((always_inline)) {
        it = min(it, last - 1);                    // past the last piece: reload it, never multiplied
        const int u = it / nkb, kb = it - u * nkb;
        if (u != lu) {
            lu = u;
            const FewSeg s = segs[u];
            const int e = __builtin_amdgcn_readfirstlane(s.expert);
            lcnt = __builtin_amdgcn_readfirstlane(s.count);
            bd = p.w2d + (size_t)e * p.w2d_expert + (size_t)nt * p.w2d_ntile + frag * kFragBytes + lane * 16;
            bs = p.w2s + (size_t)e * p.w2s_expert + (size_t)nt * p.w2s_ntile + frag * 256 + lane * 4;
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const int slot = rows[s.first + min(f * 16 + l, s.count - 1)].slot;
                ha[f] = p.h8 + (size_t)slot * p.I + 16 * g;
                hs[f] = p.h_sf + slot * hsfs;
            }
        }
        c.s0 = load_nt_word(bs + (size_t)kb * kBScaleBlockBytes);
        c.s1 = load_nt_word(bs + (size_t)kb * kBScaleBlockBytes + 256);
#pragma unroll
        for (int f = 0; f < FM; ++f) c.sa[f] = *reinterpret_cast<const uint32_t*>(hs[f] + 4 * kb);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int kc = min(4 * kb + i, nks - 1);
            c.b0[i] = load_nt(bd + (size_t)kc * kBTileBytes);
            c.b1[i] = load_nt(bd + (size_t)kc * kBTileBytes + kFragBytes);
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                if (f > 0 && lcnt <= 16) break;    // its rows are not used: whatever is there will do
                const v4i lo = *reinterpret_cast<const v4i*>(ha[f] + kc * 128);
                const v4i hi = *reinterpret_cast<const v4i*>(ha[f] + kc * 128 + 64);
                c.a[f][i] = (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            }
        }
    };
    // adds the products of the piece's expert to its tokens' sums once its last piece here is done
    auto finish = [&](int it) __attribute__((always_inline)) {
        const int u = it / nkb;
        if (it + 1 < last && (it + 1) / nkb == u) return;
        const FewSeg s = segs[u];
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = f * 16 + 4 * g + r;
                if (row < s.count) {
                    const FewRow e = rows[s.first + row];
                    float* y = tile[wave][e.slot / p.k];
                    y[l] = __builtin_fmaf(e.weight, c0[f][r], y[l]);
                    y[16 + l] = __builtin_fmaf(e.weight, c1[f][r], y[16 + l]);
                }
                c0[f][r] = c1[f][r] = 0.f;
            }
    };
    __syncthreads();
    if (first < last) {
        Chunk<C, FM> even{}, odd{};
        load(even, first);
        for (int it = first; it < last; it += 2) {
            load(odd, it + 1);
            multiply<C, FM, 0>(even, (it % nkb) * 4, nks, c0, c1);
            finish(it);
            load(even, it + 2);
            if (it + 1 < last) {
                multiply<C, FM, 0>(odd, ((it + 1) % nkb) * 4, nks, c0, c1);
                finish(it + 1);
            }
        }
    }
    __syncthreads();
    // tile column 16*q + j: lane column j of fragment frag + q, row 128*(f/8) + 8*j + f%8 of the
    // 256-row tile; a thread stores the two adjacent columns of both fragments
    const int col0 = nt * 256 + 128 * (frag >> 3) + (frag & 7);
    for (int i = tid; i < p.T * 16; i += kFewThreads) {
        const int t = i >> 4, j = i & 15;
        float a = tile[0][t][j], b = tile[0][t][16 + j];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) {
            a += tile[w][t][j];
            b += tile[w][t][16 + j];
        }
        const int col = col0 + 8 * j;
        if (col < p.H) {
            const uint32_t lo = __builtin_bit_cast(uint16_t, (__bf16)a), hi = __builtin_bit_cast(uint16_t, (__bf16)b);
            *reinterpret_cast<uint32_t*>(p.y + (size_t)t * p.H + col) = lo | (hi << 16);
        }
    }
}

}  // namespace

FewLayout few_layout(const moe_shape_t& s) {
    FewLayout L{};
    const size_t T = s.max_tokens < kMaxT ? s.max_tokens : kMaxT;
    const size_t slots = T * s.num_topk, I = s.intermediate;
    L.h8 = 0;
    L.h_sf = align_up(slots * I, 256);
    L.rows = L.h_sf + align_up(slots * 4 * ((I + 511) / 512), 256);
    L.segs = L.rows + align_up(slots * sizeof(FewRow), 256);
    L.n_used = L.segs + align_up(slots * sizeof(FewSeg), 256);
    L.total = L.n_used + 256;
    return L;
}

hipError_t launch_few(const moe_shape_t& s, const PackedLayout& P, const uint8_t* x, const uint8_t* x_sf,
                      const int32_t* idx, const float* weights, int T, const uint8_t* packed, uint8_t* ws, uint16_t* y,
                      hipStream_t stream) {
    const FewLayout W = few_layout(s);
    FewArgs p{};
    p.x = x;
    p.x_sf = x_sf;
    p.idx = idx;
    p.weights = weights;
    p.T = T;
    p.k = s.num_topk;
    p.E = s.num_experts;
    p.H = s.hidden;
    p.I = s.intermediate;
    p.w1d = packed + P.w1d;
    p.w1s = packed + P.w1s;
    p.w2d = packed + P.w2d;
    p.w2s = packed + P.w2s;
    p.w1d_expert = P.w1d_expert;
    p.w1d_ntile = P.w1d_ntile;
    p.w1s_expert = P.w1s_expert;
    p.w1s_ntile = P.w1s_ntile;
    p.w2d_expert = P.w2d_expert;
    p.w2d_ntile = P.w2d_ntile;
    p.w2s_expert = P.w2s_expert;
    p.w2s_ntile = P.w2s_ntile;
    p.h8 = ws + W.h8;
    p.h_sf = ws + W.h_sf;
    p.rows = reinterpret_cast<FewRow*>(ws + W.rows);
    p.segs = reinterpret_cast<FewSeg*>(ws + W.segs);
    p.n_used = reinterpret_cast<int32_t*>(ws + W.n_used);
    p.y = y;
    // at most one expert per slot can be chosen
    const int max_used = s.num_experts < T * s.num_topk ? s.num_experts : T * s.num_topk;
    const unsigned g1 = (unsigned)max_used * (unsigned)(s.intermediate / 128), g2 = (unsigned)cdiv(s.hidden, 256) * 8u;
    // With fewer workgroups than CUs, twice the waves in each, with x in LDS where it fits (the
    // registers then hold weights only)
    const size_t x_bytes = (size_t)T * s.hidden;
    const bool split = g1 < 256 && T <= 16 && s.hidden >= 1024 && x_bytes <= kMaxXLds;
    if (T <= 16) {
        if (split) few_linear1<1, 2, 4><<<g1, 1024, x_bytes, stream>>>(p);
        else few_linear1<1, 1, 2><<<g1, 512, 0, stream>>>(p);
        few_linear2<1><<<g2, kFewThreads, 0, stream>>>(p);
    } else {
        few_linear1<2, 1, 2><<<g1, 512, 0, stream>>>(p);
        few_linear2<2><<<g2, kFewThreads, 0, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace moe
