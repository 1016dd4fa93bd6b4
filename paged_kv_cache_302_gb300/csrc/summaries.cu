// summaries.cu -- key summaries of a paged cache, rebuilt from the pool (the format is in summary.cuh).
#include <algorithm>
#include <type_traits>

#include "summary.cuh"

namespace pa {

// L lanes per (block, KV head), each with its own channels, walk the block's tokens: a lane has all rows it needs, and
// the heads of a 16-bit token, which lie side by side, go to neighbouring lanes.  Minima and maxima that start as NaN
// ignore NaN elements: the instructions return the other operand.  16-bit rows are compared as they are, two channels
// at a time; e4m3 rows as fp16 pairs in units of the block's largest scale, exact while the scales lie within 2^14 of
// one another (fp32 otherwise).  A box is rounded to integers by a multiply-add with directed rounding that leaves the
// integer in the low bits.  Bound by memory: 8 contexts of 16384 tokens with 8 heads (285 MB) take 46 us, 6.2 TB/s; 32
// ragged chunks over e4m3 (101 MB) 22.5 us, 4.5 TB/s, are bound by latency: rows wait for the scale bytes, one read more
// in the chain, with 40 % of the SM's warps resident; the ALU pipe and the issue slots are half busy.  CTAs of 128
// threads took 46 us where 256 took 48 (the last wave is shorter); 16 tokens on their way at a time instead of 8 46 and
// 51, 4 of them 51.  Over e4m3 minima and maxima in fp32 took 50 us, fp16 pairs with a rounding function per channel 26.
constexpr int kSumThreads = 128;
constexpr int kSumBatch = 8;  // tokens of a block on their way at a time

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
        const int64_t chunk = p.q_start ? (int64_t)p.q_start[s + 1] - p.q_start[s] : ctx;
        if (chunk < 0 || chunk > p.max_q_len || ctx < chunk || ctx > p.MB * B) {
            if (i == 0 && h == 0 && sub == 0) flag_error(p.err, PA_DEV_ERR_CTX);
            continue;
        }
        const int n = (int)chunk;
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

}  // namespace pa
