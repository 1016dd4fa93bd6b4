// summaries.cu -- key summaries of a paged cache, and the selection of blocks by them.
//
// A summary is a box around the keys of one (block, KV head): per channel the least and the greatest K of the block's
// tokens, as integers of 8 bits in units of one power of two,
//     lo_d = floor(min_t K_td 2^-e),  hi_d = ceil(max_t K_td 2^-e),  e the least with max |K| <= 127 2^e:
//   summaries [NB][H_kv][2][D] int8 (lo, hi), sum_scales [NB][H_kv] bytes, b standing for 2^(b - 127).
// No key of the block has a larger product with a query q than sum_d max(q_d lo_d, q_d hi_d) 2^e: that sum is the
// block's score.  With q in integers of 9 bits and a sign (q_d 2^-f rounded, f the least with max |q| <= 511 2^f) every
// sum is an integer below 128 * 127 * 511 < 2^23, hence exact in fp32 in any order: the selection does not depend on
// how the sum is split.
#include <algorithm>
#include <type_traits>

#include "quant.cuh"

namespace pa {

constexpr int kBoxTop = 127, kQueryTop = 511;

// Least e in [kScaleMin, kScaleMax] with a <= top 2^e (a >= 0, kScaleMax where there is none), top = 2^BITS - 1.
template <int BITS>
__device__ __forceinline__ int int_exponent(float a) {
    constexpr uint32_t kTopMantissa = ((1u << BITS) - 1u) << (24 - BITS) & 0x7fffffu;  // of 2^BITS - 1
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - (BITS - 1) + ((u & 0x7fffffu) > kTopMantissa ? 1 : 0);
    return min(max(e, kScaleMin), kScaleMax);
}

// ----------------------------------------------------------------------------- summaries

// L lanes per (block, KV head), each with its own channels, walk the block's tokens.  Minima and maxima that start as
// NaN ignore NaN elements: the instructions return the other operand.
constexpr int kSumThreads = 256;

// K rows of 16 bits: 8 channels per lane, minima and maxima in the rows' own type.
template <typename T>
struct Pair;
template <>
struct Pair<__half> {
    static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
};
template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
};

struct SummaryParams {
    int8_t* boxes;
    uint8_t* box_scales;
    const void* pool;
    const uint8_t* scales;
    const int32_t* tables;
    const int32_t* ctx_lens;
    const int32_t* q_start;  // null: every block of the context
    int64_t units;           // N * touched * H_kv
    int H_kv, MB, NB, touched, max_q_len;
    int* err;
};

// One lane's channels of one box: C channels from lo/hi (NaN where the channel has no value), the row's exponent over
// its L lanes, 8-bit integers out.
template <int L, int C>
__device__ __forceinline__ void store_box(const float (&lo)[C], const float (&hi)[C], int8_t* row, int D, int sub,
                                          uint8_t* scale, unsigned mask) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) m = fmaxf(m, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
    const int e = int_exponent<7>(m);
    const float inv = pow2i(-e);
    uint32_t wl[C / 4], wh[C / 4];
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
        wl[i] = wh[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // (what 127 2^40 does not hold saturates; a channel without a value is the box [0, 0])
            const int a = max(__float2int_rd(fmaxf(lo[4 * i + j] * inv, -1000.f)), -kBoxTop);
            const int b = min(__float2int_ru(fminf(hi[4 * i + j] * inv, 1000.f)), kBoxTop);
            const bool some = lo[4 * i + j] == lo[4 * i + j];
            wl[i] |= (uint32_t)((some ? min(a, kBoxTop) : 0) & 0xff) << (8 * j);
            wh[i] |= (uint32_t)((some ? max(b, -kBoxTop) : 0) & 0xff) << (8 * j);
        }
    }
    if constexpr (C == 8) {
        reinterpret_cast<uint2*>(row)[sub] = make_uint2(wl[0], wl[1]);
        reinterpret_cast<uint2*>(row + D)[sub] = make_uint2(wh[0], wh[1]);
    } else {
        reinterpret_cast<uint4*>(row)[sub] = make_uint4(wl[0], wl[1], wl[2], wl[3]);
        reinterpret_cast<uint4*>(row + D)[sub] = make_uint4(wh[0], wh[1], wh[2], wh[3]);
    }
    if (sub == 0) *scale = (uint8_t)(e + kScaleBias);
}

// T: __half, __nv_bfloat16, or uint8_t for a quantised cache.
template <typename T, int D, int LGB>
__global__ void __launch_bounds__(kSumThreads) summarize_kernel(const SummaryParams p) {
    constexpr bool kQuant = std::is_same<T, uint8_t>::value;
    constexpr int B = 1 << LGB, C = kQuant ? 16 : 8, L = D / C;
    griddep_wait();
    griddep_launch_dependents();
    const int sub = threadIdx.x % L;
    const unsigned mask = ((1ull << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
    for (int64_t u = (int64_t)blockIdx.x * (kSumThreads / L) + threadIdx.x / L; u < p.units;
         u += (int64_t)gridDim.x * (kSumThreads / L)) {
        const int64_t sb = u / p.H_kv;
        const int h = (int)(u - sb * p.H_kv), s = (int)(sb / p.touched), i = (int)(sb - (int64_t)s * p.touched);
        const int ctx = p.ctx_lens[s];
        int n = ctx;
        if (p.q_start) {
            const int q0 = p.q_start[s];
            n = p.q_start[s + 1] - q0;
        }
        if (n < 0 || n > p.max_q_len || ctx < n || ctx > p.MB * B) {
            if (i == 0 && h == 0 && sub == 0) flag_error(p.err, PA_DEV_ERR_CTX);
            continue;
        }
        const int b = ((ctx - n) >> LGB) + i;
        if (n == 0 || b * (int64_t)B >= ctx) continue;
        const int blk = p.tables[(int64_t)s * p.MB + b];
        if ((unsigned)blk >= (unsigned)p.NB) {
            if (h == 0 && sub == 0) flag_error(p.err, PA_DEV_ERR_BLOCK);
            continue;
        }
        const int nv = min(B, ctx - b * B);
        float lo[C], hi[C];
        if constexpr (kQuant) {
            const uint8_t* k = static_cast<const uint8_t*>(p.pool) + ((int64_t)blk * p.H_kv + h) * (2 * B * D);
            const uint8_t* sc = p.scales + ((int64_t)blk * p.H_kv + h) * (2 * B);
#pragma unroll
            for (int j = 0; j < C; ++j) lo[j] = hi[j] = __uint_as_float(0x7fffffffu);
#pragma unroll 4
            for (int t = 0; t < nv; ++t) {
                const uint4 x = reinterpret_cast<const uint4*>(k + t * D)[sub];
                const float f = pow2i(scale_of(sc[t]));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float2 v = Mma<__half>::unpack(e4m3x2_to_f16x2(w[j / 2] >> (16 * (j & 1))));
                    v.x *= f;
                    v.y *= f;
                    lo[2 * j] = fminf(lo[2 * j], v.x);
                    hi[2 * j] = fmaxf(hi[2 * j], v.x);
                    lo[2 * j + 1] = fminf(lo[2 * j + 1], v.y);
                    hi[2 * j + 1] = fmaxf(hi[2 * j + 1], v.y);
                }
            }
        } else {
            const T* k = static_cast<const T*>(p.pool) + ((int64_t)blk * B * 2 * p.H_kv + h) * D;
            const int64_t step = (int64_t)2 * p.H_kv * D;
            uint32_t a[4], z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = z[j] = 0x7fff7fffu;
#pragma unroll 8
            for (int t = 0; t < nv; ++t) {
                const uint4 x = reinterpret_cast<const uint4*>(k + t * step)[sub];
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[j] = Pair<T>::lo(a[j], w[j]);
                    z[j] = Pair<T>::hi(z[j], w[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Mma<T>::unpack(a[j]), g = Mma<T>::unpack(z[j]);
                lo[2 * j] = f.x;
                lo[2 * j + 1] = f.y;
                hi[2 * j] = g.x;
                hi[2 * j + 1] = g.y;
            }
        }
        const int64_t row = (int64_t)blk * p.H_kv + h;
        store_box<L, C>(lo, hi, p.boxes + row * 2 * D, D, sub, p.box_scales + row, mask);
    }
}

static int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        sms = 1;
    return sms;
}

template <typename T, int D>
static cudaError_t summarize_d(const SummaryParams& p, int B, cudaStream_t st) {
    const int64_t per = kSumThreads / (D / (sizeof(T) == 1 ? 16 : 8));
    const unsigned grid = (unsigned)std::min<int64_t>((p.units + per - 1) / per, 0x7fffffff);
    auto kern = B == 8 ? summarize_kernel<T, D, 3> : B == 16 ? summarize_kernel<T, D, 4> : summarize_kernel<T, D, 5>;
    return launch_kernel(kern, dim3(grid), dim3(kSumThreads), 0, st, p);
}

pa_status launch_summarize(const SummarizeArgs& a) {
    SummaryParams p;
    p.boxes = static_cast<int8_t*>(a.summaries);
    p.box_scales = static_cast<uint8_t*>(a.sum_scales);
    p.pool = a.pool;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.q_start = a.q_start;
    p.H_kv = a.H_kv;
    p.MB = a.MB;
    p.NB = a.NB;
    p.max_q_len = a.max_q_len;
    // blocks that max_q_len newest tokens can lie in
    const int64_t t = a.q_start ? ((int64_t)a.max_q_len + a.B - 2) / a.B + 1 : ((int64_t)a.max_q_len + a.B - 1) / a.B;
    p.touched = (int)std::min<int64_t>(t, a.MB);
    p.units = (int64_t)a.N * p.touched * a.H_kv;
    p.err = a.dev_err;
    cudaError_t e;
    if (a.kv_dtype == PA_E4M3)
        e = a.D == 128 ? summarize_d<uint8_t, 128>(p, a.B, a.stream) : summarize_d<uint8_t, 64>(p, a.B, a.stream);
    else if (a.kv_dtype == PA_BF16)
        e = a.D == 128 ? summarize_d<__nv_bfloat16, 128>(p, a.B, a.stream)
                       : summarize_d<__nv_bfloat16, 64>(p, a.B, a.stream);
    else
        e = a.D == 128 ? summarize_d<__half, 128>(p, a.B, a.stream) : summarize_d<__half, 64>(p, a.B, a.stream);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "summarize launch");
}

// ----------------------------------------------------------------------------- selection

struct SelectParams {
    int32_t* selected;
    const void* q;
    const int8_t* boxes;
    const uint8_t* box_scales;
    const int32_t* tables;
    const int32_t* ctx_lens;
    float* keys;  // [N][H_kv][stride]
    int64_t stride;
    int H_kv, G, lgB, MB, NB, max_ctx, top_k, sink, recent;
    int* err;
};

// Blocks of sequence s, 0 where its length is out of range.
__device__ __forceinline__ int context_blocks(const SelectParams& p, int s) {
    const int ctx = p.ctx_lens[s];
    return ctx < 1 || ctx > p.max_ctx || ctx > (int64_t)p.MB << p.lgB ? 0 : (ctx + (1 << p.lgB) - 1) >> p.lgB;
}

// Scores: one warp per (sequence, KV head, 16 blocks), mma.sync m16n8k16 with the blocks on M and the query heads of
// the KV head on N.  max(q lo, q hi) is q hi for q >= 0 and q lo below, so a box's score is one product of length 2 D,
// [max(q, 0), min(q, 0)] . [hi, lo]; box and query integers are exact in fp16.
constexpr int kScoreWarps = 8;

// Four 8-bit integers as two fp16 pairs: v + 128 in the low byte of 0x6400 is 1024 + 128 + v.
__device__ __forceinline__ void int8x4_to_f16(uint32_t x, uint32_t& a, uint32_t& b) {
    const uint32_t u = x ^ 0x80808080u;
    const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
    uint32_t r0 = __byte_perm(u, 0x64646464u, 0x4140), r1 = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 h0 = __hsub2(*reinterpret_cast<__half2*>(&r0), bias), h1 = __hsub2(*reinterpret_cast<__half2*>(&r1), bias);
    a = *reinterpret_cast<const uint32_t*>(&h0);
    b = *reinterpret_cast<const uint32_t*>(&h1);
}

template <typename T, int D>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const SelectParams p) {
    constexpr int NC = D / 64;  // 16-byte chunks of a lane: t4, t4 + 4 of each half of the box
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
    const int h = blockIdx.y, s = blockIdx.z;
    const int nb = context_blocks(p, s);
    if (nb <= p.top_k) return;  // nothing to choose
    const int tile = blockIdx.x * kScoreWarps + (threadIdx.x >> 5);
    if (16 * tile >= nb) return;
    // the query integers of head g4, in the order of the box's bytes: word w of chunk c holds channels 64 c + 16 t4 +
    // 4 w on, the k-columns 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 of k-step (c, w)
    float x[NC][16];
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (g4 < p.G)
                v = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                   (((int64_t)s * p.H_kv + h) * p.G + g4) * D + 64 * c + 16 * t4)[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Mma<T>::unpack(w[j]);
                x[c][8 * i + 2 * j] = f.x;
                x[c][8 * i + 2 * j + 1] = f.y;
                m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));  // (a NaN counts as nothing)
            }
        }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int f = int_exponent<9>(m);
    const float inv = pow2i(-f);
    const float f0 = pow2i(__shfl_sync(0xffffffffu, f, 8 * t4)), f1 = pow2i(__shfl_sync(0xffffffffu, f, 8 * t4 + 4));
    uint32_t up[NC][4][2], dn[NC][4][2];  // max(q, 0) and min(q, 0)
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float y = x[c][2 * i + k];
                v[k] = y == y ? fminf(fmaxf(rintf(y * inv), -(float)kQueryTop), (float)kQueryTop) : 0.f;
            }
            up[c][i / 2][i & 1] = Mma<__half>::pack(fmaxf(v[0], 0.f), fmaxf(v[1], 0.f));
            dn[c][i / 2][i & 1] = Mma<__half>::pack(fminf(v[0], 0.f), fminf(v[1], 0.f));
        }
    // the boxes of blocks g4 and g4 + 8 of the tile
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int64_t row[2];
    bool good[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int b = 16 * tile + g4 + 8 * r;
        const int blk = b < nb ? p.tables[(int64_t)s * p.MB + b] : 0;
        good[r] = (unsigned)blk < (unsigned)p.NB;
        if (!good[r] && t4 == 0 && h == 0) flag_error(p.err, PA_DEV_ERR_BLOCK);
        row[r] = (int64_t)(good[r] ? blk : 0) * p.H_kv + h;
    }
    uint4 v[2][2][NC];  // [block][lo, hi][chunk]
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                v[r][k][c] = reinterpret_cast<const uint4*>(p.boxes + (row[r] * 2 + k) * D + 64 * c)[t4];
    float unit[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) unit[r] = pow2i(scale_of(p.box_scales[row[r]]));
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint32_t w0[4] = {v[0][k][c].x, v[0][k][c].y, v[0][k][c].z, v[0][k][c].w};
            const uint32_t w1[4] = {v[1][k][c].x, v[1][k][c].y, v[1][k][c].z, v[1][k][c].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t a0, a1, a2, a3;
                int8x4_to_f16(w0[w], a0, a2);
                int8x4_to_f16(w1[w], a1, a3);
                const uint32_t(&qf)[2] = k ? up[c][w] : dn[c][w];
                Mma<__half>::run(acc, a0, a1, a2, a3, qf[0], qf[1]);
            }
        }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float y = -INFINITY;
        if (2 * t4 < p.G) y = acc[2 * r] * f0;
        if (2 * t4 + 1 < p.G) y = fmaxf(y, acc[2 * r + 1] * f1);
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
        const int b = 16 * tile + g4 + 8 * r;
        if (t4 == 0 && b < nb) p.keys[((int64_t)s * p.H_kv + h) * p.stride + b] = good[r] ? y * unit[r] : -INFINITY;
    }
}

// The top_k of a (sequence, KV head): a radix search from the top digit down for the key of the last one taken, then
// one pass in index order that lists every key above it and the first ones equal to it.
constexpr int kTopThreads = 256;

// Unsigned integers order as the floats do.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kTopThreads) top_blocks_kernel(const SelectParams p) {
    __shared__ int hist[256];
    __shared__ int warp_sum[2][kTopThreads / 32];
    __shared__ int s_digit, s_left;
    griddep_wait();
    griddep_launch_dependents();
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nb = context_blocks(p, s);
    const int64_t r = (int64_t)s * p.H_kv + h;
    int32_t* out = p.selected + r * p.top_k;
    if (nb == 0 && h == 0 && tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
    if (nb <= p.top_k) {
        for (int i = tid; i < p.top_k; i += kTopThreads) out[i] = i < nb ? i : -1;
        return;
    }
    const float* keys = p.keys + r * p.stride;
    auto key = [&](int b) -> uint32_t {
        return b < p.sink || b >= nb - p.recent ? 0xffffffffu : ordered(keys[b]);
    };
    uint32_t prefix = 0;
    int left = p.top_k;  // keys still to take among those that share the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int b = tid; b < nb; b += kTopThreads) {
            const uint32_t k = key(b);
            if (shift == 24 || k >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&hist[k >> shift & 255], 1);
        }
        __syncthreads();
        // keys with a larger digit than tid's
        int v = hist[255 - tid];
        const int own_count = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) warp_sum[0][warp] = v;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += warp_sum[0][w];
        const int above = before + v - own_count;
        if (above < left && above + own_count >= left) {
            s_digit = 255 - tid;
            s_left = left - above;
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        left = s_left;
        __syncthreads();
    }
    int taken = 0, ties = 0;  // listed, and equal keys met, before the chunk
    for (int b0 = 0; b0 < nb; b0 += kTopThreads) {
        const int b = b0 + tid;
        const uint32_t k = b < nb ? key(b) : 0;
        const bool eq = b < nb && k == prefix;
        const unsigned me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) warp_sum[0][warp] = __popc(me);
        __syncthreads();
        int e = ties + __popc(me & ((1u << lane) - 1u));
        for (int w = 0; w < kTopThreads / 32; ++w) {
            if (w < warp) e += warp_sum[0][w];
            ties += warp_sum[0][w];
        }
        const bool take = b < nb && (k > prefix || (eq && e < left));
        const unsigned mt = __ballot_sync(0xffffffffu, take);
        if (lane == 0) warp_sum[1][warp] = __popc(mt);
        __syncthreads();
        int at = taken + __popc(mt & ((1u << lane) - 1u));
        for (int w = 0; w < kTopThreads / 32; ++w) {
            if (w < warp) at += warp_sum[1][w];
            taken += warp_sum[1][w];
        }
        if (take) out[at] = b;
    }
}

size_t select_workspace_bytes(int N, int H_kv, int max_ctx, int B) {
    if (N <= 0 || N > 65535 || H_kv <= 0 || H_kv > 65535 || max_ctx <= 0 || (B != 8 && B != 16 && B != 32)) return 0;
    const size_t stride = ((size_t)max_ctx + B - 1) / B;
    return (size_t)N * H_kv * stride * sizeof(float);
}

pa_status launch_select(const SelectArgs& a) {
    SelectParams p;
    p.selected = a.selected;
    p.q = a.q;
    p.boxes = static_cast<const int8_t*>(a.summaries);
    p.box_scales = static_cast<const uint8_t*>(a.sum_scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.keys = static_cast<float*>(a.workspace);
    p.stride = ((int64_t)a.max_ctx + a.B - 1) / a.B;
    p.H_kv = a.H_kv;
    p.G = a.H_q / a.H_kv;
    p.lgB = a.B == 8 ? 3 : a.B == 16 ? 4 : 5;
    p.MB = a.MB;
    p.NB = a.NB;
    p.max_ctx = a.max_ctx;
    p.top_k = a.top_k;
    p.sink = a.sink;
    p.recent = a.recent;
    p.err = a.dev_err;
    const int64_t nb = std::min<int64_t>(p.stride, a.MB);
    if (nb > a.top_k) {
        const unsigned gx = (unsigned)((nb + 16 * kScoreWarps - 1) / (16 * kScoreWarps));
        auto kern = a.q_dtype == PA_BF16 ? (a.D == 128 ? score_kernel<__nv_bfloat16, 128> : score_kernel<__nv_bfloat16, 64>)
                                         : (a.D == 128 ? score_kernel<__half, 128> : score_kernel<__half, 64>);
        const cudaError_t e = launch_kernel(kern, dim3(gx, (unsigned)a.H_kv, (unsigned)a.N), dim3(kScoreWarps * 32), 0,
                                            a.stream, p);
        count_launch();
        if (e != cudaSuccess) return cuda_fail(e, "score launch");
    }
    const cudaError_t e = launch_kernel(top_blocks_kernel, dim3((unsigned)a.H_kv, (unsigned)a.N), dim3(kTopThreads), 0,
                                        a.stream, p);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "top_blocks launch");
}

}  // namespace pa
