// Root-mean-square norm of bf16 rows, with the residual's addition in front and the FP8 cast behind (the cast:
// chenxutan.com/d/1930 section 9.2, the activation as FP8 codes and scale factors before the MoE call; section 11.1, a
// block's scale follows its largest magnitude):
//
//   h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  n = h * r * weight
//
// residual_out = bf16(h), normed = bf16(n); codes and scales are moe_cast_to_fp8's rule applied to n. Everything between is
// FP32: n is not rounded to bf16 before the cast.
//
// A workgroup owns a row and keeps it in registers: 8 columns per lane and chunk, so that the 16 lanes of a DPP row hold one
// 128-column block, whose largest magnitude is four steps within them. One pass over memory: 8192 x 7168 with a residual read and
// written moves 411 MB in 68 us, 6.0 TB/s, where a copy moves 5.1; 515 x 18432 with every output 85.6 MB in 19. Few rows are two
// barriers, the loads' and the sum's latency (16 x 7168 3.1 us in a graph, an empty launch 1.95). Narrow rows leave lanes idle
// (2^20 x 128 286 us, 1.4 TB/s), and rows past 32768 columns are read twice (1000 x 65536 with a residual 128 us, 3.6 TB/s).
#include "moe_internal.h"
#include "moe_serving.h"

namespace moe {
namespace {

template <int N>
struct IntC {
    static constexpr int value = N;
};

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));

// NT: past the caches
template <bool NT, class V>
__device__ inline V get(const void* p) {
    if constexpr (NT) return __builtin_nontemporal_load(static_cast<const V*>(p));
    else return *static_cast<const V*>(p);
}
template <bool NT, class V>
__device__ inline void put(void* p, const V& v) {
    if constexpr (NT) __builtin_nontemporal_store(v, static_cast<V*>(p));
    else *static_cast<V*>(p) = v;
}

constexpr int kMaxThreads = 1024;
constexpr int kCus = 256;                 // compute units of an MI355X

// The sum over 16 lanes, in each of them: neighbours, pairs, the mirrored half row, the mirrored row
__device__ inline float sum_of_16(float s) {
    auto add = [&](auto ctrl) __attribute__((always_inline)) {
        s += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(s), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    add(IntC<0xB1>{});
    add(IntC<0x4E>{});
    add(IntC<0x141>{});
    add(IntC<0x140>{});
    return s;
}

// The sum over the workgroup, in every thread, in a fixed order: 16 lanes, the wave's four rows of 16, the waves (at most 16)
__device__ inline float block_sum(float s, float* part) {
    const int b = (int)__float_as_uint(sum_of_16(s));
    s = (__uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 0)) + __uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 16))) +
        (__uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 32)) + __uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 48)));
    const int waves = blockDim.x >> 6;
    if (waves == 1) return s;
    static_assert(kMaxThreads == 16 * 64, "");
    __syncthreads();                                   // `part` may still be read from the sum before
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    const int w = threadIdx.x & 15;
    return sum_of_16(w < waves ? part[w] : 0.f);
}

__device__ inline void unpack8(const v4u& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

__device__ inline v4u pack8(const float (&f)[8]) {
    typedef float v8f __attribute__((ext_vector_type(8)));
    typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
    const v8f v = {f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
    return __builtin_bit_cast(v4u, __builtin_convertvector(v, v8bf));
}

struct NormArgs {
    const uint16_t* x;
    const uint16_t* residual;      // or null
    const void* weight;
    uint8_t* q;
    uint8_t* sf;
    uint16_t* normed;              // or null
    uint16_t* residual_out;        // or null
    uint32_t cols, sf_stride;      // (cols < 2^31: a column counter that steps past it stays within 32 bits, unsigned)
    float eps;
};

// h of the 8 columns at c of a row that starts at `at`
template <bool NT>
__device__ inline void load_h(const NormArgs& p, size_t at, uint32_t c, float (&h)[8]) {
    unpack8(get<NT, v4u>(p.x + at + c), h);
    if (p.residual) {
        float r[8];
        unpack8(get<NT, v4u>(p.residual + at + c), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += r[j];
    }
}

template <bool WF32>
__device__ inline void load_w(const NormArgs& p, uint32_t c, float (&w)[8]) {
    if constexpr (WF32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p.weight) + c);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p.weight) + c + 4);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
        unpack8(get<false, v4u>(static_cast<const uint16_t*>(p.weight) + c), w);
    }
}

// UE8M0 byte of a block whose largest magnitude has FP32 bit pattern `bits` (sign clear): 448 = 1.75 * 2^8
__device__ inline uint32_t fp8_scale_byte(uint32_t bits) {
    if (bits == 0) return 127u;
    if (bits >= 0x7f800000u) return 255u;              // an infinity or a NaN in the block
    const int b = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return b < 0 ? 0u : (uint32_t)b;
}

__device__ inline uint32_t max_of_16(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
}

// n of 8 columns -> normed, codes, and (every 16th lane) the block's scale byte. Past cols: zeros, past sf_stride * 128: nothing
template <bool NT>
__device__ inline void store_n(const NormArgs& p, size_t row, uint32_t c, const float (&n)[8]) {
    const bool active = c < p.cols;
    const size_t at = row * p.cols + c;
    if (active && p.normed) put<NT>(p.normed + at, pack8(n));
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(n[j]) & 0x7fffffffu);
    const uint32_t byte = fp8_scale_byte(max_of_16(m));
    // 2^-(byte - 127); NaN for a block of NaN, so that its codes are NaN too
    const float mul = byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - byte) << 23);
    if (active) {
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(n[0] * mul, n[1] * mul, 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(n[2] * mul, n[3] * mul, a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(n[4] * mul, n[5] * mul, 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(n[6] * mul, n[7] * mul, b, true);
        put<NT>(p.q + at, (v2u){(uint32_t)a, (uint32_t)b});
    }
    if ((threadIdx.x & 15) == 0 && (c >> 7) < p.sf_stride) p.sf[row * p.sf_stride + (c >> 7)] = active ? (uint8_t)byte : (uint8_t)0;
}

// Squares leave FP32's range where |h| passes 2^64 or, with a tiny eps, where all of the row is below about 2^-63; with an eps
// near its end their mean and eps do together. Such rows are scaled by a power of two before they are squared (a large eps hides
// the squares that this loses). `f`: that power, or 1
__device__ inline float square_scale(float sum, float eps) {
    if (!(sum <= 3.4028235e38f) || eps > 0x1p100f) return 0x1p-80f;
    return sum < 0x1p-100f && eps < 0x1p-80f ? 0x1p80f : 1.0f;
}

__device__ inline float inverse_root(float sum, float cols, float eps, float f) {
    return 1.0f / __builtin_sqrtf(sum / cols + eps * f * f);
}

// h * f * r of a row whose squares were scaled by f, as first * second: a row scaled down has columns that f would take below FP32's
// normal numbers, and |h| * r is at most 2^80 times the root of the columns; a row scaled up has columns that r would
struct Factors {
    float first, second;
};
__device__ inline Factors factors(float f, float r) { return f < 1.0f ? Factors{r, f} : Factors{f, r}; }

// The threads hold CH chunks of 8 columns each in registers (CH = 0: any number, read again for each pass, through the caches)
template <int CH, bool WF32, bool NT>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_kernel(NormArgs p, int row0) {
    __shared__ float part[kMaxThreads / 64];
    const size_t row = (size_t)row0 + blockIdx.x, at = row * p.cols;
    const uint32_t t8 = threadIdx.x * 8, span = blockDim.x * 8;
    const float cols = (float)p.cols;
    if constexpr (CH > 0) {
        float h[CH][8], s = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const uint32_t c = k * span + t8;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] = 0.f;
            if (c < p.cols) load_h<NT>(p, at, c, h[k]);
        }
        float f = 1.0f;
        auto squares = [&]() __attribute__((always_inline)) {
            float q = 0.f;
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) q += (h[k][j] * f) * (h[k][j] * f);
            return block_sum(q, part);
        };
        s = squares();
        f = square_scale(s, p.eps);
        if (f != 1.0f) s = squares();
        const Factors by = factors(f, inverse_root(s, cols, p.eps, f));
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const uint32_t c = k * span + t8;
            float n[8] = {};
            if (c < p.cols) {
                if (p.residual_out) put<NT>(p.residual_out + at + c, pack8(h[k]));
                float w[8];
                load_w<WF32>(p, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) n[j] = (h[k][j] * by.first) * by.second * w[j];
            }
            store_n<NT>(p, row, c, n);
        }
    } else {
        const uint32_t end = (p.cols + 511) / 512 * 512;     // whole waves
        float f = 1.0f;
        // The chunks' sums are added in 64 bits: a thread takes up to 2^18 of them, and FP32 would round each into a sum that grows
        // past it (2^30 equal columns: n 0.4 % off)
        auto squares = [&]() {
            double all = 0.0;
            for (uint32_t c = t8; c < p.cols; c += span) {
                float h[8], q = 0.f;
                load_h<false>(p, at, c, h);
#pragma unroll
                for (int j = 0; j < 8; ++j) q += (h[j] * f) * (h[j] * f);
                all += (double)q;
            }
            return block_sum((float)all, part);
        };
        float s = squares();
        f = square_scale(s, p.eps);
        if (f != 1.0f) s = squares();
        const Factors by = factors(f, inverse_root(s, cols, p.eps, f));
        for (uint32_t c = t8; c < end; c += span) {
            float h[8], n[8] = {};
            if (c < p.cols) {
                load_h<false>(p, at, c, h);
                // (the lane has read these columns of both inputs: either may be residual_out)
                if (p.residual_out) put<false>(p.residual_out + at + c, pack8(h));
                float w[8];
                load_w<WF32>(p, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) n[j] = (h[j] * by.first) * by.second * w[j];
            }
            store_n<false>(p, row, c, n);
        }
    }
}

// ceil(cols / n) of 1 to 2^31 - 1 columns
int chunks_of(uint32_t cols, uint32_t n) { return (int)((cols - 1) / n + 1); }

template <int CH>
void launch(const NormArgs& p, bool wf32, bool nt, int row0, unsigned rows, hipStream_t stream) {
    // as many waves as the row needs
    const int threads = CH > 0 ? 64 * chunks_of(p.cols, 512 * CH) : kMaxThreads;
    constexpr bool PAST = CH > 0;              // (CH = 0 has no form past the caches)
    if (wf32) {
        if (PAST && nt) rmsnorm_kernel<CH, true, PAST><<<rows, threads, 0, stream>>>(p, row0);
        else rmsnorm_kernel<CH, true, false><<<rows, threads, 0, stream>>>(p, row0);
    } else {
        if (PAST && nt) rmsnorm_kernel<CH, false, PAST><<<rows, threads, 0, stream>>>(p, row0);
        else rmsnorm_kernel<CH, false, false><<<rows, threads, 0, stream>>>(p, row0);
    }
}

}  // namespace

hipError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const void* weight, int weight_type, int rows, int cols,
                          float eps, uint8_t* q, uint8_t* sf, uint16_t* normed, uint16_t* residual_out, hipStream_t stream) {
    NormArgs p{x, residual, weight, q, sf, normed, residual_out, (uint32_t)cols, 4u * chunks_of(cols, 512), eps};
    const bool wf32 = weight_type == MOE_F32;
    // From a few MB on, loads and stores of rows that registers hold go past the caches: calls in turn over 1.2 GB, residual read
    // and written, 256 x 7168 4.8 -> 4.6 us, 400 x 7168 7.8 -> 5.8, 1000 x 7168 13.8 -> 9.8, 8192 x 7168 75 -> 68. Between a kernel
    // that writes x and one that reads normed, all three as often on the same few MB, 15.3 -> 14.6, 20.1 -> 18.0 and 27.0 -> 27.8;
    // 128 x 7168, below, 11.9 and 12.2.
    const bool nt = (size_t)rows * cols > (size_t(1) << 20);
    // Chunks per thread: one, or as few as 1024 threads allow, while at most two rows share a CU, so that a row has as many waves as
    // it can (16 x 7168: 3.1 us with one chunk, 3.6 with two, 4.9 with four; 400 x 7168 5.8, 6.5, 8.8). With more rows 8 waves a
    // row, so that four of them are under way on a CU (515 x 7168 8.7 with one chunk, 6.9 with two; 1000 x 10240 16.1 with two, 12.7
    // with three; 8192 x 7168 73 with one, 68 with two); four chunks up to three rows a CU (515 x 16384 14.7 with two, 11.9 with four;
    // 4000 x 16384 76 and 78). The last rule misses up to a fifth: 1000 x 16384 22.0 with two, 19.9 with four, and past 8 waves
    // 515 x 18432 19.8 with three, 16.0 with four, where 3000 x 18432 takes 67 and 70.
    const int least = chunks_of(cols, 8 * kMaxThreads), eight = chunks_of(cols, 8 * 512);
    const int ch = rows > 2 * kCus && eight <= (rows <= 3 * kCus ? 4 : 3) ? eight : least;
    constexpr int kMost = 1 << 21;                      // rows of a launch: at most 2^31 threads
    for (int row0 = 0; row0 < rows; row0 += kMost) {
        const unsigned n = (unsigned)(rows - row0 < kMost ? rows - row0 : kMost);
        switch (ch) {
            case 1: launch<1>(p, wf32, nt, row0, n, stream); break;
            case 2: launch<2>(p, wf32, nt, row0, n, stream); break;
            case 3: launch<3>(p, wf32, nt, row0, n, stream); break;
            case 4: launch<4>(p, wf32, nt, row0, n, stream); break;
            default: launch<0>(p, wf32, nt, row0, n, stream);
        }
        if (rows - row0 <= kMost) break;                // (row0 + kMost may pass 2^31)
    }
    return hipGetLastError();
}

}  // namespace moe
