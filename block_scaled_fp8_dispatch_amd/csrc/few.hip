// The MoE forward of a few tokens (at most 32) in two kernels, on the packed weights of
// moe_prepare_weights:
//   few_linear1  h8 = Q8( silu(x Wg^T) * (x Wu^T) ) per chosen expert and 128-column block
//   few_linear2  y[t] = bf16( sum over chosen experts e of w[t,e] * (h8[t,e] W2_e^T) )
// where w[t,e] is the sum of the top-k weights of t's slots that name e.
//
// With so few rows every product is a stream of packed weights, each fragment (16 columns x
// 128 K, 1 KB) read once from memory straight into the registers of the one wave that
// multiplies it; the tokens are the rows of v_mfma_scale_f32_16x16x128_f8f6f4, row i of a
// 16-row fragment being token i for every expert (rows of tokens that did not choose the
// expert are computed and dropped: the matrix units idle anyway). There is no routing pass:
// each workgroup derives the chosen experts from the T*k ids, as one bit mask of tokens per
// expert in LDS (bits are set by integer atomics, whose order does not matter).
//
// Linear1: a workgroup of 8 waves owns one 128-wide block of h of one chosen expert; wave w
// the gate fragment w and the up fragment w over the whole K, so the block's largest |h| of a
// row meets in LDS and the row is requantised there. Linear2: a workgroup owns 16 output
// columns; its 8 waves share the (expert, 512 K) pieces, each adds w * (its partial products)
// per token in FP32, and the waves' sums are added in wave order.
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

// mask[e] = bit t set where token t names expert e (all kFewThreads threads; ends in a barrier)
__device__ inline void token_masks(const int32_t* __restrict__ idx, int T, int k, int E, uint32_t* mask) {
    for (int e = threadIdx.x; e < E; e += kFewThreads) mask[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < T * k; s += kFewThreads) {
        const int e = idx[s];
        if (e >= 0 && e < E) atomicOr(&mask[e], 1u << (s / k));
    }
    __syncthreads();
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
    uint16_t* y;
};

// FM: 16-row fragments (tokens / 16)
template <int FM>
__global__ __launch_bounds__(kFewThreads) void few_linear1(FewArgs p) {
    __shared__ uint32_t mask[MOE_MAX_EXPERTS];
    __shared__ uint32_t red[kFewWaves][FM * 16];
    __shared__ __attribute__((aligned(16))) uint8_t codes[FM * 16][128];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l = lane & 15;
    const int NB = p.I / 128;
    const int nb = blockIdx.x % NB;
    int u = blockIdx.x / NB;                       // the u-th chosen expert
    token_masks(p.idx, p.T, p.k, p.E, mask);
    int expert = -1;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        uint64_t b = __ballot(e0 + lane < p.E && mask[e0 + lane] != 0);
        const int n = __popcll(b);
        if (u < n) {
            for (; u > 0; --u) b &= b - 1;
            expert = e0 + __ffsll((unsigned long long)b) - 1;
            break;
        }
        u -= n;
    }
    expert = __builtin_amdgcn_readfirstlane(expert);
    if (expert < 0) return;                        // fewer chosen experts than the grid allows for

    const int xsfs = 4 * ((p.H + 511) / 512);
    const uint8_t *xa[FM], *xs[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int t = min(f * 16 + l, p.T - 1);
        xa[f] = p.x + (size_t)t * p.H + 16 * g;
        xs[f] = p.x_sf + (size_t)t * xsfs;
    }
    const uint8_t* bd = p.w1d + (size_t)expert * p.w1d_expert + (size_t)nb * p.w1d_ntile + wave * kFragBytes + lane * 16;
    const uint8_t* bs = p.w1s + (size_t)expert * p.w1s_expert + (size_t)nb * p.w1s_ntile + wave * 256 + lane * 4;
    v4f ag[FM], au[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) ag[f] = au[f] = (v4f){0.f, 0.f, 0.f, 0.f};
    const int nks = p.H / 128;
    for (int kb = 0; kb * 4 < nks; ++kb) {
        const uint32_t sg = load_nt_word(bs + (size_t)kb * kBScaleBlockBytes);
        const uint32_t su = load_nt_word(bs + (size_t)kb * kBScaleBlockBytes + 8 * 256);
        uint32_t sa[FM];
#pragma unroll
        for (int f = 0; f < FM; ++f) sa[f] = *reinterpret_cast<const uint32_t*>(xs[f] + 4 * kb);
        auto step = [&](int s, auto ops) __attribute__((always_inline)) {
            constexpr int OPS = decltype(ops)::value;
            const int ks = kb * 4 + s;
            if (ks >= nks) return;
            const v4i bg = load_nt(bd + (size_t)ks * kBTileBytes);
            const v4i bu = load_nt(bd + (size_t)ks * kBTileBytes + 8 * kFragBytes);
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const v4i lo = *reinterpret_cast<const v4i*>(xa[f] + ks * 128);
                const v4i hi = *reinterpret_cast<const v4i*>(xa[f] + ks * 128 + 64);
                const v8i a = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                ag[f] = mfma<OPS>(a, bg, ag[f], sa[f], sg);
                au[f] = mfma<OPS>(a, bu, au[f], sa[f], su);
            }
        };
        step(0, std::integral_constant<int, 0>{});
        step(1, std::integral_constant<int, 1>{});
        step(2, std::integral_constant<int, 2>{});
        step(3, std::integral_constant<int, 3>{});
    }
    // h of rows 16f + 4g + r, column 64*(wave/4) + 4*l + wave%4 of the block (the packed rows
    // are interleaved so); the largest |h| of a row over the block: DPP row, then the waves
    float h[FM][4];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            h[f][r] = few_swiglu(ag[f][r], au[f][r]);
            uint32_t m = __float_as_uint(fabsf(h[f][r]));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
            if (l == 0) red[wave][f * 16 + 4 * g + r] = m;
        }
    __syncthreads();
    const int col = 64 * (wave >> 2) + 4 * l + (wave & 3);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = f * 16 + 4 * g + r;
            uint32_t m = red[0][row];
#pragma unroll
            for (int w = 1; w < kFewWaves; ++w) m = max(m, red[w][row]);
            const float mul = __uint_as_float((uint32_t)(254 - few_scale_byte(__uint_as_float(m))) << 23);
            codes[row][col] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(h[f][r] * mul, 0.f, 0, false);
        }
    __syncthreads();
    // 8 threads per row store its 128 codes, the first also its scale byte
    const int row = tid >> 3, part = tid & 7;
    if (row < p.T && ((mask[expert] >> row) & 1u)) {
        int j = 0;
        while (p.idx[row * p.k + j] != expert) ++j;      // the mask says that one is there
        const size_t slot = (size_t)row * p.k + j;
        *reinterpret_cast<v4i*>(p.h8 + slot * p.I + nb * 128 + part * 16) =
            *reinterpret_cast<const v4i*>(&codes[row][part * 16]);
        if (part == 0) {
            uint32_t m = red[0][row];
            for (int w = 1; w < kFewWaves; ++w) m = max(m, red[w][row]);
            p.h_sf[slot * (size_t)(4 * ((p.I + 511) / 512)) + nb] = (uint8_t)few_scale_byte(__uint_as_float(m));
        }
    }
}

template <int FM>
__global__ __launch_bounds__(kFewThreads) void few_linear2(FewArgs p) {
    __shared__ uint32_t mask[MOE_MAX_EXPERTS];
    __shared__ int16_t used[MOE_MAX_EXPERTS];      // the chosen experts, ascending
    __shared__ int n_used;
    __shared__ float red[kFewWaves][FM * 16][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l = lane & 15;
    token_masks(p.idx, p.T, p.k, p.E, mask);
    if (wave == 0) {
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const bool on = e0 + lane < p.E && mask[e0 + lane] != 0;
            const uint64_t b = __ballot(on);
            if (on) used[n + __popcll(b & ((1ull << lane) - 1))] = (int16_t)(e0 + lane);
            n += __popcll(b);
        }
        if (lane == 0) n_used = n;
    }
    __syncthreads();

    const int frag = blockIdx.x & 15, nt = blockIdx.x >> 4;
    const int nks = p.I / 128, nkb = (nks + 3) / 4;
    const int items = n_used * nkb;
    const int first = (int)((long long)items * wave / kFewWaves), last = (int)((long long)items * (wave + 1) / kFewWaves);
    const size_t hsfs = 4 * (size_t)nkb;
    v4f ysum[FM], acc[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) ysum[f] = acc[f] = (v4f){0.f, 0.f, 0.f, 0.f};
    int cur = -1;
    float wt[FM];
    const uint8_t *ha[FM], *hs[FM];
    bool on[FM];
    uint32_t bits = 0;
    const uint8_t *bd = nullptr, *bs = nullptr;
    auto flush = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 4 * g + r;
                const float w = __shfl(wt[f], t, 64);
                // dropped, not multiplied by 0: a row of another token may hold a NaN
                if ((bits >> (f * 16 + t)) & 1u) ysum[f][r] = __builtin_fmaf(w, acc[f][r], ysum[f][r]);
                acc[f][r] = 0.f;
            }
    };
    for (int it = first; it < last; ++it) {
        const int u = it / nkb, kb = it - u * nkb;
        if (u != cur) {
            if (cur >= 0) flush();
            cur = u;
            const int e = __builtin_amdgcn_readfirstlane((int)used[u]);
            bits = (uint32_t)__builtin_amdgcn_readfirstlane((int)mask[e]);
            bd = p.w2d + (size_t)e * p.w2d_expert + (size_t)nt * p.w2d_ntile + frag * kFragBytes + lane * 16;
            bs = p.w2s + (size_t)e * p.w2s_expert + (size_t)nt * p.w2s_ntile + frag * 256 + lane * 4;
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const int t = f * 16 + l;
                on[f] = (bits >> t) & 1u;
                int slot = 0;
                float w = 0.f;
                if (on[f]) {
                    slot = -1;
                    for (int j = 0; j < p.k; ++j)
                        if (p.idx[t * p.k + j] == e) {
                            w += p.weights[t * p.k + j];
                            if (slot < 0) slot = t * p.k + j;
                        }
                }
                wt[f] = w;
                ha[f] = p.h8 + (size_t)slot * p.I + 16 * g;
                hs[f] = p.h_sf + slot * hsfs;
            }
        }
        const uint32_t sb = load_nt_word(bs + (size_t)kb * kBScaleBlockBytes);
        uint32_t sa[FM];
#pragma unroll
        for (int f = 0; f < FM; ++f) sa[f] = on[f] ? *reinterpret_cast<const uint32_t*>(hs[f] + 4 * kb) : 0x7f7f7f7fu;
        auto step = [&](int s, auto ops) __attribute__((always_inline)) {
            constexpr int OPS = decltype(ops)::value;
            const int ks = kb * 4 + s;
            if (ks >= nks) return;
            const v4i b = load_nt(bd + (size_t)ks * kBTileBytes);
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                v4i lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
                if (on[f]) {
                    lo = *reinterpret_cast<const v4i*>(ha[f] + ks * 128);
                    hi = *reinterpret_cast<const v4i*>(ha[f] + ks * 128 + 64);
                }
                const v8i a = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                acc[f] = mfma<OPS>(a, b, acc[f], sa[f], sb);
            }
        };
        step(0, std::integral_constant<int, 0>{});
        step(1, std::integral_constant<int, 1>{});
        step(2, std::integral_constant<int, 2>{});
        step(3, std::integral_constant<int, 3>{});
    }
    if (cur >= 0) flush();
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][f * 16 + 4 * g + r][l] = ysum[f][r];
    __syncthreads();
    if (tid < FM * 16 * 16) {
        const int row = tid >> 4, j = tid & 15;
        float s = red[0][row][j];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) s += red[w][row][j];
        // lane column j of fragment f is row 128*(f/8) + 8*j + f%8 of the 256-row tile
        const int col = nt * 256 + 128 * (frag >> 3) + 8 * j + (frag & 7);
        if (row < p.T && col < p.H) {
            const __bf16 v = (__bf16)s;
            p.y[(size_t)row * p.H + col] = __builtin_bit_cast(uint16_t, v);
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
    L.total = L.h_sf + align_up(slots * 4 * ((I + 511) / 512), 256);
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
    p.y = y;
    // at most one expert per slot can be chosen
    const int max_used = s.num_experts < T * s.num_topk ? s.num_experts : T * s.num_topk;
    const unsigned g1 = (unsigned)max_used * (unsigned)(s.intermediate / 128), g2 = (unsigned)s.hidden / 16u;
    if (T <= 16) {
        few_linear1<1><<<g1, kFewThreads, 0, stream>>>(p);
        few_linear2<1><<<g2, kFewThreads, 0, stream>>>(p);
    } else {
        few_linear1<2><<<g1, kFewThreads, 0, stream>>>(p);
        few_linear2<2><<<g2, kFewThreads, 0, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace moe
