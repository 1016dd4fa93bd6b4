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
#include "runs.cuh"

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
constexpr int kSumThreads = 128;
constexpr int kSumBatch = 8;  // tokens of a block on their way at a time

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

// v 2^-e as an integer, rounded down or up, in the low bits of an fp32 number above 2^23 (|v 2^-e| < 2^22).
__device__ __forceinline__ uint32_t int_down(float v, float inv) {
    return __float_as_uint(__fmaf_rd(v, inv, 12582912.f));  // 1.5 * 2^23
}
__device__ __forceinline__ uint32_t int_up(float v, float inv) {
    return __float_as_uint(__fmaf_ru(v, inv, 12582912.f));
}

// One lane's channels of one box: C channels from lo/hi (NaN where the channel has no value), the row's exponent over
// its L lanes, 8-bit integers out.
template <int L, int C>
__device__ __forceinline__ void store_box(float (&lo)[C], float (&hi)[C], int8_t* row, int D, int sub, uint8_t* scale,
                                          unsigned mask) {
    float m = 0.f;
    bool none = false;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        m = fmaxf(m, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
        none = none || lo[i] != lo[i];
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
    const int e = int_exponent<7>(m);
    const float inv = pow2i(-e), top = kBoxTop * pow2i(kScaleMax);
    if (none || m > top) {  // rare: channels without a value, magnitudes past the largest box
#pragma unroll
        for (int i = 0; i < C; ++i) {
            lo[i] = lo[i] == lo[i] ? fminf(fmaxf(lo[i], -top), top) : 0.f;
            hi[i] = hi[i] == hi[i] ? fminf(fmaxf(hi[i], -top), top) : 0.f;
        }
    }
    uint32_t wl[C / 4], wh[C / 4];
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
        wl[i] = __byte_perm(__byte_perm(int_down(lo[4 * i], inv), int_down(lo[4 * i + 1], inv), 0x0040),
                            __byte_perm(int_down(lo[4 * i + 2], inv), int_down(lo[4 * i + 3], inv), 0x0040), 0x5410);
        wh[i] = __byte_perm(__byte_perm(int_up(hi[4 * i], inv), int_up(hi[4 * i + 1], inv), 0x0040),
                            __byte_perm(int_up(hi[4 * i + 2], inv), int_up(hi[4 * i + 3], inv), 0x0040), 0x5410);
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
            uint32_t sw[B / 4];  // the tokens' scale bytes
#pragma unroll
            for (int j = 0; j < B / 8; ++j) {
                const uint2 x = reinterpret_cast<const uint2*>(sc)[j];
                sw[2 * j] = x.x;
                sw[2 * j + 1] = x.y;
            }
            // the largest and the least byte of the block's tokens (those past the last one repeat it)
            uint32_t top2 = 0, low2 = 0x00ff00ffu;
            if (nv < B) {
                const uint32_t last = (uint32_t)sc[nv - 1] * 0x01010101u;
#pragma unroll
                for (int j = 0; j < B / 4; ++j) {
                    const int in = min(max(nv - 4 * j, 0), 4);  // bytes of the word that count
                    const uint32_t keep = in == 4 ? 0xffffffffu : (1u << (8 * in)) - 1u;
                    sw[j] = (sw[j] & keep) | (last & ~keep);
                }
            }
#pragma unroll
            for (int j = 0; j < B / 4; ++j) {
                const uint32_t even = sw[j] & 0x00ff00ffu, odd = sw[j] >> 8 & 0x00ff00ffu;
                top2 = vmax_u16x2(top2, vmax_u16x2(even, odd));
                low2 = vmin_u16x2(low2, vmin_u16x2(even, odd));
            }
            const int top = (int)max(top2 & 0xffffu, top2 >> 16), low = (int)min(low2 & 0xffffu, low2 >> 16);
            if (top - low <= 14 && low >= kScaleMin + kScaleBias && top <= kScaleMax + kScaleBias) {
                // rows in units of the largest scale: e4m3 is a multiple of 2^-9, so down to 2^-14 of it fp16 is exact
                uint32_t a[8], z[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = z[j] = 0x7fff7fffu;
#pragma unroll
                for (int t0 = 0; t0 < B; t0 += kSumBatch) {
                    if (t0 < nv) {
                        uint4 x[kSumBatch];
#pragma unroll
                        for (int t = 0; t < kSumBatch; ++t)  // (past the last token: the last one again)
                            x[t] = reinterpret_cast<const uint4*>(k + min(t0 + t, nv - 1) * D)[sub];
#pragma unroll
                        for (int t = 0; t < kSumBatch; ++t) {
                            const int byte = (int)(sw[(t0 + t) / 4] >> (8 * (t & 3)) & 0xffu);
                            const uint32_t f = (uint32_t)(byte - top + 15) * 0x04000400u;  // 2^(byte - top), twice
                            const uint32_t w[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t q = e4m3x2_to_f16x2(w[j / 2] >> (16 * (j & 1)));
                                const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&q),
                                                          *reinterpret_cast<const __half2*>(&f));
                                const uint32_t v = *reinterpret_cast<const uint32_t*>(&y);
                                a[j] = Pair<__half>::lo(a[j], v);
                                z[j] = Pair<__half>::hi(z[j], v);
                            }
                        }
                    }
                }
                const float unit = pow2i(top - kScaleBias);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = Mma<__half>::unpack(a[j]), g = Mma<__half>::unpack(z[j]);
                    lo[2 * j] = f.x * unit;
                    lo[2 * j + 1] = f.y * unit;
                    hi[2 * j] = g.x * unit;
                    hi[2 * j + 1] = g.y * unit;
                }
            } else {
#pragma unroll
                for (int j = 0; j < C; ++j) lo[j] = hi[j] = __uint_as_float(0x7fffffffu);
                for (int t = 0; t < nv; ++t) {
                    const uint4 x = reinterpret_cast<const uint4*>(k + t * D)[sub];
                    const float f = pow2i(scale_of(sc[t]));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 v = Mma<__half>::unpack(e4m3x2_to_f16x2(w[j / 2] >> (16 * (j & 1))));
                        lo[2 * j] = fminf(lo[2 * j], v.x * f);
                        hi[2 * j] = fmaxf(hi[2 * j], v.x * f);
                        lo[2 * j + 1] = fminf(lo[2 * j + 1], v.y * f);
                        hi[2 * j + 1] = fmaxf(hi[2 * j + 1], v.y * f);
                    }
                }
            }
        } else {
            const T* k = static_cast<const T*>(p.pool) + ((int64_t)blk * B * 2 * p.H_kv + h) * D;
            const int64_t step = (int64_t)2 * p.H_kv * D;
            uint32_t a[4], z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = z[j] = 0x7fff7fffu;
#pragma unroll
            for (int t0 = 0; t0 < B; t0 += kSumBatch) {
                if (t0 < nv) {
                    uint4 x[kSumBatch];
#pragma unroll
                    for (int t = 0; t < kSumBatch; ++t)  // (past the last token: the last one again)
                        x[t] = reinterpret_cast<const uint4*>(k + min(t0 + t, nv - 1) * step)[sub];
#pragma unroll
                    for (int t = 0; t < kSumBatch; ++t) {
                        const uint32_t w[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a[j] = Pair<T>::lo(a[j], w[j]);
                            z[j] = Pair<T>::hi(z[j], w[j]);
                        }
                    }
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
    uint32_t* keys;  // [N][H_kv][stride], ordered as the scores
    int64_t stride;
    int N, H_kv, G, lgB, MB, NB, max_ctx, top_k, sink, recent;
    int* err;
};

// Blocks of sequence s, 0 where its length is out of range.
__device__ __forceinline__ int context_blocks(const SelectParams& p, int s) {
    const int ctx = p.ctx_lens[s];
    return ctx < 1 || ctx > p.max_ctx || ctx > (int64_t)p.MB << p.lgB ? 0 : (ctx + (1 << p.lgB) - 1) >> p.lgB;
}

// Unsigned integers order as the floats do.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Scores: mma.sync m16n8k16 with 16 blocks on M and the query heads of the KV head on N.  max(q lo, q hi) is q hi for q >= 0 and q lo below, so a box's score is one product of length 2 D,
// [max(q, 0), min(q, 0)] . [hi, lo]; box and query integers are exact in fp16.
constexpr int kScoreWarps = 4;
constexpr int kScoreCtas = 4;  // per SM

// Four 8-bit integers as two fp16 pairs: v + 128 in the low byte of 0x6400 is 1024 + 128 + v.
__device__ __forceinline__ void int8x4_to_f16(uint32_t x, uint32_t& a, uint32_t& b) {
    const uint32_t u = x ^ 0x80808080u;
    const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
    uint32_t r0 = __byte_perm(u, 0x64646464u, 0x4140), r1 = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 h0 = __hsub2(*reinterpret_cast<__half2*>(&r0), bias), h1 = __hsub2(*reinterpret_cast<__half2*>(&r1), bias);
    a = *reinterpret_cast<const uint32_t*>(&h0);
    b = *reinterpret_cast<const uint32_t*>(&h1);
}

// Tiles of each row of a sequence with something to choose.
__device__ __forceinline__ int row_tiles(const SelectParams& p, int s) {
    const int nb = context_blocks(p, s);
    return nb > p.top_k ? (nb + 15) / 16 : 0;
}

// The tiles of all rows -- (sequence, KV head) -- in order are cut into runs of equal length, one per warp.  While a tile
// is scored, the next one's boxes are on their way, and the block ids of the one after that.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreWarps * 32, kScoreCtas) score_kernel(const SelectParams p) {
    constexpr int NC = D / 64;  // 16-byte chunks of a lane: t4, t4 + 4 of each half of the box
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
    const auto tiles_of = [&](int s) { return row_tiles(p, s); };
    const RowScan<decltype(tiles_of)> scan(tiles_of, p.N, p.H_kv);
    const int total = scan.total(), warps = min((int)gridDim.x * kScoreWarps, total);
    const int w = (int)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;  // neighbouring runs on different SMs
    if (w >= warps) return;
    const Cut cut(total, warps);
    const int u0 = cut.start(w);
    int left = cut.start(w + 1) - u0;

    // A tile of the run, and this lane's block ids in it: blocks g4 and g4 + 8.
    struct Pos {
        int s, h, t, tiles, nb, blk[2];
    };
    auto look_up = [&](Pos& x) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int b = 16 * x.t + g4 + 8 * r;
            x.blk[r] = b < x.nb ? p.tables[(int64_t)x.s * p.MB + b] : 0;
        }
    };
    auto step = [&](Pos x) -> Pos {  // the run's next tile after x
        if (++x.t == x.tiles) {
            x.t = 0;
            if (++x.h == p.H_kv) {
                x.h = 0;
                do x.tiles = row_tiles(p, ++x.s);
                while (x.tiles == 0);  // (ends: the run has tiles left)
                x.nb = context_blocks(p, x.s);
            }
        }
        look_up(x);
        return x;
    };
    Pos cur;
    int first;
    cur.s = scan.find(u0, cur.tiles, first);
    cur.h = (u0 - first) / cur.tiles;
    cur.t = u0 - first - cur.h * cur.tiles;
    cur.nb = context_blocks(p, cur.s);
    look_up(cur);

    // The query integers of head g4, in the order of the box's bytes: word w of chunk c holds channels 64 c + 16 t4 + 4 w
    // on, the k-columns 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 of k-step (c, w).
    uint32_t up[NC][8], dn[NC][8];  // max(q, 0) and min(q, 0)
    float f0 = 0.f, f1 = 0.f;       // units of heads 2 t4 and 2 t4 + 1
    auto read_query = [&](int s, int h) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (g4 < p.G)
                    v = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                       (((int64_t)s * p.H_kv + h) * p.G + g4) * D + 64 * c + 16 * t4)[i];
                up[c][4 * i] = v.x;
                up[c][4 * i + 1] = v.y;
                up[c][4 * i + 2] = v.z;
                up[c][4 * i + 3] = v.w;
            }
    };
    auto make_query = [&]() {
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = Mma<T>::unpack(up[c][i]);
                m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));  // (a NaN counts as nothing)
            }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int f = int_exponent<9>(m);
        const float inv = pow2i(-f);
        f0 = pow2i(__shfl_sync(0xffffffffu, f, 8 * t4));
        f1 = pow2i(__shfl_sync(0xffffffffu, f, 8 * t4 + 4));
        auto integer = [&](float x) {
            return x == x ? fminf(fmaxf(rintf(x * inv), -(float)kQueryTop), (float)kQueryTop) : 0.f;
        };
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 x = Mma<T>::unpack(up[c][i]);
                const uint32_t q = Mma<__half>::pack(integer(x.x), integer(x.y));
                up[c][i] = Pair<__half>::hi(q, 0);
                dn[c][i] = Pair<__half>::lo(q, 0);
            }
    };
    // A tile's boxes: [block g4, g4 + 8][lo, hi][chunk], and the units of the two blocks (0: no such block).  As soon as a
    // piece has been multiplied, its registers receive the next tile's.
    uint4 v[2][2][NC];
    float unit[2], next_unit[2] = {0.f, 0.f};
    const int8_t* box[2];
    auto find = [&](const Pos& x, float (&unit)[2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool good = (unsigned)x.blk[r] < (unsigned)p.NB;
            if (!good && t4 == 0 && x.h == 0) flag_error(p.err, PA_DEV_ERR_BLOCK);
            const int64_t row = (int64_t)(good ? x.blk[r] : 0) * p.H_kv + x.h;
            box[r] = p.boxes + row * 2 * D + 16 * t4;
            unit[r] = good ? pow2i(scale_of(p.box_scales[row])) : 0.f;
        }
    };
    auto load = [&](int k, int c) {
#pragma unroll
        for (int r = 0; r < 2; ++r) v[r][k][c] = *reinterpret_cast<const uint4*>(box[r] + k * D + 64 * c);
    };
    read_query(cur.s, cur.h);
    find(cur, unit);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < NC; ++c) load(k, c);
    make_query();
    Pos nxt = cur;
    if (left > 1) nxt = step(cur);
    for (; left > 0; --left) {
        Pos after = nxt;
        if (left > 1) find(nxt, next_unit);
        if (left > 2) after = step(nxt);
        float acc[2][4] = {};
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
                    // the query's negative half meets lo, its positive half hi
                    const uint32_t* q = k ? up[c] : dn[c];
                    Mma<__half>::run(acc[k], a0, a1, a2, a3, q[2 * w], q[2 * w + 1]);
                }
                if (left > 1) load(k, c);
            }
        uint32_t* keys = p.keys + ((int64_t)cur.s * p.H_kv + cur.h) * p.stride;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float y = -INFINITY;
            if (2 * t4 < p.G) y = (acc[0][2 * r] + acc[1][2 * r]) * f0;
            if (2 * t4 + 1 < p.G) y = fmaxf(y, (acc[0][2 * r + 1] + acc[1][2 * r + 1]) * f1);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
            const int b = 16 * cur.t + g4 + 8 * r;
            if (t4 == 0 && b < cur.nb) keys[b] = ordered(unit[r] > 0.f ? y * unit[r] : -INFINITY);
            unit[r] = next_unit[r];
        }
        if (left > 1 && (nxt.s != cur.s || nxt.h != cur.h)) {
            read_query(nxt.s, nxt.h);
            make_query();
        }
        cur = nxt;
        nxt = after;
    }
}

// The top_k of a (sequence, KV head): one CTA, each thread with neighbouring keys, in registers (K of them) or read anew
// (K = 0).  The key of the last block taken is found by a histogram over the eight bits below those that all competing
// keys share, then among the keys of one bin: ranked against one another where there are no more than threads' worth of
// them, else by the next eight bits.  One scan then gives every taken block its place.
constexpr int kBins = 256;

// Key k competes and agrees with the prefix above its low `open` bits.
__device__ __forceinline__ bool agree(uint32_t k, uint32_t prefix, int open) {
    return k != 0 && (open == 32 || (k ^ prefix) >> open == 0);
}

template <int THREADS, int K>
__global__ void __launch_bounds__(THREADS) top_blocks_kernel(const SelectParams p) {
    constexpr int W = THREADS / 32;
    static_assert(THREADS >= kBins, "a thread per bin");
    __shared__ uint2 s_sum[W];
    __shared__ uint32_t s_bin[kBins], s_list[kBins], s_warp[kBins / 32];
    __shared__ uint32_t s_digit, s_above, s_count, s_cut, s_left;
    griddep_wait();
    griddep_launch_dependents();
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nb = context_blocks(p, s);
    const int64_t r = (int64_t)s * p.H_kv + h;
    int32_t* out = p.selected + r * p.top_k;
    if (nb == 0 && h == 0 && tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
    if (nb <= p.top_k) {
        for (int i = tid; i < p.top_k; i += THREADS) out[i] = i < nb ? i : -1;
        return;
    }
    const uint32_t* keys = p.keys + r * p.stride;
    const int n = ((nb + THREADS - 1) / THREADS + 3) & ~3;  // keys per thread, in fours (the row is padded to a four)
    const int b0 = tid * n;
    // Keys that do not compete count as 0, below every score: blocks kept anyway, places past the context.
    auto masked = [&](uint32_t k, int b) -> uint32_t { return b < p.sink || b >= nb - p.recent ? 0u : k; };
    uint32_t reg[K ? K : 1];
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; i += 4) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i < n && b0 + i < nb) v = *reinterpret_cast<const uint4*>(keys + b0 + i);
            reg[i] = masked(v.x, b0 + i);
            reg[i + 1] = masked(v.y, b0 + i + 1);
            reg[i + 2] = masked(v.z, b0 + i + 2);
            reg[i + 3] = masked(v.w, b0 + i + 3);
        }
    }
    // f(key, block) for each of this thread's keys
    auto each = [&](auto f) {
        if constexpr (K > 0) {
#pragma unroll
            for (int i = 0; i < K; i += 4)
                if (i < n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) f(reg[i + j], b0 + i + j);
                }
        } else {
            for (int i = 0; i < n && b0 + i < nb; ++i) f(masked(keys[b0 + i], b0 + i), b0 + i);
        }
    };
    uint32_t want = (uint32_t)(p.top_k - p.sink - p.recent);  // of the keys that compete, fewer than there are
    uint32_t cut = 0xffffffffu, ties_taken = 0;               // taken: keys above cut, the first ties_taken equal ones
    if (want > 0) {
        if (tid < kBins) s_bin[tid] = 0;
        if (tid == 0) s_count = 0;
        uint32_t lo = 0xffffffffu, hi = 0;
        each([&](uint32_t k, int) {
            if (k) lo = min(lo, k);
            hi = max(hi, k);
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) s_sum[warp] = make_uint2(lo, hi);
        __syncthreads();
        const uint2 v = lane < W ? s_sum[lane] : make_uint2(0xffffffffu, 0);
        lo = __reduce_min_sync(0xffffffffu, v.x);
        hi = __reduce_max_sync(0xffffffffu, v.y);
        // the keys that compete agree above their low `open` bits with `prefix`
        int open = 32 - __clz(lo ^ hi);
        uint32_t prefix = hi;
        while (true) {
            const int shift = max(0, open - 8);
            each([&](uint32_t k, int) {
                if (agree(k, prefix, open)) atomicAdd(&s_bin[k >> shift & 255], 1u);
            });
            __syncthreads();
            // thread t: bin 255 - t, and the keys in higher bins
            uint32_t mine = 0, x = 0;
            if (tid < kBins) {
                mine = x = s_bin[kBins - 1 - tid];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (lane == 31) s_warp[warp] = x;
            }
            __syncthreads();
            if (tid < kBins) {
                const uint32_t below = lane < warp ? s_warp[lane] : 0u;
                const uint32_t above = x - mine + __reduce_add_sync(0xffffffffu, below);
                if (above < want && above + mine >= want) {
                    s_digit = kBins - 1 - tid;
                    s_above = above;
                    s_left = mine;
                }
            }
            __syncthreads();
            const uint32_t digit = s_digit, count = s_left;
            want -= s_above;
            prefix = (open == 32 ? 0u : prefix >> open << open) | digit << shift;
            if (count == want) {  // the whole bin
                cut = prefix ? prefix - 1 : 0;  // (a key that competes is above 0)
                break;
            }
            open = shift;
            if (shift == 0) {  // equal keys
                cut = prefix;
                ties_taken = want;
                break;
            }
            if (count <= kBins) {
                each([&](uint32_t k, int) {
                    if (agree(k, prefix, shift)) s_list[atomicAdd(&s_count, 1u)] = k;
                });
                __syncthreads();
                if (tid < (int)count) {
                    const uint32_t k = s_list[tid];
                    uint32_t above = 0, equal = 0;
                    for (uint32_t i = 0; i < count; ++i) {
                        above += s_list[i] > k;
                        equal += s_list[i] == k;
                    }
                    if (above < want && above + equal >= want) {  // (equal keys write the same)
                        s_cut = k;
                        s_above = want - above;
                    }
                }
                __syncthreads();
                cut = s_cut;
                ties_taken = s_above;
                break;
            }
            if (tid < kBins) s_bin[tid] = 0;
            __syncthreads();
        }
    }
    // places: blocks kept and keys above cut before this thread's, and equal ones, of which ties_taken count
    uint32_t sure = 0, ties = 0;
    each([&](uint32_t k, int b) {
        sure += b < p.sink || (b >= nb - p.recent && b < nb) || k > cut;
        ties += k == cut;
    });
    uint32_t a = sure, t = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) {
            a += x;
            t += y;
        }
    }
    if (lane == 31) s_sum[warp] = make_uint2(a, t);
    __syncthreads();
    const uint2 v = lane < warp ? s_sum[lane] : make_uint2(0, 0);
    a += __reduce_add_sync(0xffffffffu, v.x) - sure;
    t += __reduce_add_sync(0xffffffffu, v.y) - ties;
    each([&](uint32_t k, int b) {
        const bool is_sure = b < p.sink || (b >= nb - p.recent && b < nb) || k > cut, tie = k == cut;
        if (is_sure || (tie && t < ties_taken)) out[a + min(t, ties_taken)] = b;
        a += is_sure;
        t += tie;
    });
}

// Keys of a row, in whole vectors of four.
static int64_t key_stride(int max_ctx, int B) { return (((int64_t)max_ctx + B - 1) / B + 3) & ~int64_t(3); }

size_t select_workspace_bytes(int N, int H_kv, int max_ctx, int B) {
    if (N <= 0 || N > 65535 || H_kv <= 0 || H_kv > 65535 || max_ctx <= 0 || (B != 8 && B != 16 && B != 32)) return 0;
    return (size_t)N * H_kv * (size_t)key_stride(max_ctx, B) * sizeof(uint32_t);
}

pa_status launch_select(const SelectArgs& a) {
    SelectParams p;
    p.selected = a.selected;
    p.q = a.q;
    p.boxes = static_cast<const int8_t*>(a.summaries);
    p.box_scales = static_cast<const uint8_t*>(a.sum_scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.keys = static_cast<uint32_t*>(a.workspace);
    p.stride = key_stride(a.max_ctx, a.B);
    p.N = a.N;
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
    const int64_t nb = std::min<int64_t>(((int64_t)a.max_ctx + a.B - 1) / a.B, a.MB);  // the longest context's
    if (nb > a.top_k) {
        const int64_t tiles = (nb + 15) / 16 * a.N * a.H_kv;
        if (tiles >= 1LL << 31) return fail(PA_ERR_UNSUPPORTED, "too many blocks to score");
        const unsigned grid = (unsigned)std::min<int64_t>((tiles + kScoreWarps - 1) / kScoreWarps,
                                                          (int64_t)sm_count() * kScoreCtas);
        auto kern = a.q_dtype == PA_BF16 ? (a.D == 128 ? score_kernel<__nv_bfloat16, 128> : score_kernel<__nv_bfloat16, 64>)
                                         : (a.D == 128 ? score_kernel<__half, 128> : score_kernel<__half, 64>);
        const cudaError_t e = launch_kernel(kern, dim3(grid), dim3(kScoreWarps * 32), 0, a.stream, p);
        count_launch();
        if (e != cudaSuccess) return cuda_fail(e, "score launch");
    }
    // keys in registers up to 16 per thread (32 spill)
    void (*top)(SelectParams) = top_blocks_kernel<1024, 0>;
    int threads = 1024;
    if (nb <= 256 * 8) {
        top = top_blocks_kernel<256, 8>;
        threads = 256;
    } else if (nb <= 1024 * 8) {
        top = top_blocks_kernel<1024, 8>;
    } else if (nb <= 1024 * 16) {
        top = top_blocks_kernel<1024, 16>;
    }
    const cudaError_t e = launch_kernel(top, dim3((unsigned)a.H_kv, (unsigned)a.N), dim3((unsigned)threads), 0, a.stream, p);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "top_blocks launch");
}

}  // namespace pa
