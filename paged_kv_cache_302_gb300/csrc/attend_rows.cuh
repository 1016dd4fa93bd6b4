// attend_rows.cuh -- attention of one (query row, query head) per CTA over a paged cache, 16-bit or quantised: the
// plain two-product form with an online softmax over tiles of 128 keys.
#pragma once

#include "quant.cuh"

namespace pa {

struct RowsParams {
    void* out;
    int out_dtype;
    const void* q;
    const void* pool;         // 16-bit [NB][B][2][H_kv][D], or e4m3 [NB][H_kv][2][B][D]
    const uint8_t* scales;    // null for a 16-bit pool
    const int32_t* tables;
    const int32_t* ctx_lens;
    const int32_t* q_start;   // null: one row per sequence that sees its whole context
    const uint32_t* mask;
    int mask_words, N, T, H_q, G, H_kv, lgB, MB, NB, max_ctx, max_q_len;
    float scale_log2;
    int* err;
};

template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(128) attend_rows_kernel(const RowsParams p) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float sq[D], sp[128], sred[4];
    const int tid = threadIdx.x, row = blockIdx.x, h = blockIdx.y, g = h / p.G;
    int s = row, n = 1, i = 0;
    if (p.q_start) {
        if (row == 0 && h == 0)
            for (int j = tid; j < p.N; j += 128) {
                const int a = p.q_start[j], b = p.q_start[j + 1];
                if (a < 0 || b < a || b > p.T || b - a > p.max_q_len || (b > a && p.ctx_lens[j] < b - a))
                    flag_error(p.err, PA_DEV_ERR_CTX);
            }
        int lo = 0, hi = p.N;  // the last sequence that starts at or before the row
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.q_start[mid] <= row) lo = mid; else hi = mid;
        }
        s = lo;
        i = row - p.q_start[s];
        n = p.q_start[s + 1] - p.q_start[s];
        if (i < 0 || i >= n) return;
    }
    const int ctx = p.ctx_lens[s], B = 1 << p.lgB;
    if (ctx < 1 || ctx > p.max_ctx || ctx > p.MB * B || (p.q_start && (n > ctx || n > p.max_q_len || p.q_start[s] < 0 || row - i + n > p.T))) {
        if (tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
        return;
    }
    const T* q = static_cast<const T*>(p.q) + ((size_t)row * p.H_q + h) * D;
    for (int d = tid; d < D; d += 128) sq[d] = (float)q[d];
    __syncthreads();
    float M = -INFINITY, l = 0.f, acc = 0.f;
    for (int k0 = 0; k0 < ctx; k0 += 128) {
        const int t = k0 + tid;
        float y = -INFINITY, es = 1.f;
        if (t < ctx) {
            const int j = t - (ctx - n);
            const bool seen = !p.q_start || j < 0 || (p.mask[(size_t)row * p.mask_words + (j >> 5)] >> (j & 31) & 1u);
            int blk = p.tables[(size_t)s * p.MB + (t >> p.lgB)];
            const int off = t & (B - 1);
            const bool good = (unsigned)blk < (unsigned)p.NB;
            if (!good) flag_error(p.err, PA_DEV_ERR_BLOCK);
            float dot = 0.f;
            int ek = 0, ev = 0;
            if (good) {
                if constexpr (QUANT) {
                    const size_t r = ((((size_t)blk * p.H_kv + g) * 2) << p.lgB) + off;
                    const uint8_t* kr = static_cast<const uint8_t*>(p.pool) + r * D;
                    for (int d = 0; d < D; d += 2) {
                        const float2 f = Mma<__half>::unpack(
                            e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kr + d)));
                        dot += f.x * sq[d] + f.y * sq[d + 1];
                    }
                    ek = scale_of(p.scales[r]);
                    ev = scale_of(p.scales[r + B]);
                } else {
                    const T* kr = static_cast<const T*>(p.pool) + ((((size_t)blk << p.lgB) + off) * 2 * p.H_kv + g) * D;
                    for (int d = 0; d < D; ++d) dot += (float)kr[d] * sq[d];
                }
            }
            if (seen) y = dot * pow2i(ek) * p.scale_log2 + (float)ev;
            es = pow2i(-ev);
        }
        float mx = y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((tid & 31) == 0) sred[tid >> 5] = mx;
        __syncthreads();
        const float Mn = fmaxf(M, fmaxf(fmaxf(sred[0], sred[1]), fmaxf(sred[2], sred[3])));
        const float Mu = Mn == -INFINITY ? 0.f : Mn;
        const float a = fast_exp2(M - Mu), pr = fast_exp2(y - Mu);
        M = Mn;
        l = l * a + pr * es;
        sp[tid] = pr;
        __syncthreads();
        acc *= a;
        if (tid < D) {
            const int nk = min(128, ctx - k0);
            for (int j = 0; j < nk; ++j) {
                const float w = sp[j];
                if (w == 0.f) continue;  // a key that is not seen, whatever its V holds
                const int blk = p.tables[(size_t)s * p.MB + ((k0 + j) >> p.lgB)], off = (k0 + j) & (B - 1);
                if ((unsigned)blk >= (unsigned)p.NB) continue;
                if constexpr (QUANT) {
                    const size_t r = ((((size_t)blk * p.H_kv + g) * 2 + 1) << p.lgB) + off;
                    acc += w * Mma<__half>::unpack(e4m3x2_to_f16x2(static_cast<const uint8_t*>(p.pool)[r * D + tid])).x;
                } else {
                    acc += w * (float)static_cast<const T*>(
                                   p.pool)[(((((size_t)blk << p.lgB) + off) * 2 + 1) * p.H_kv + g) * D + tid];
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if ((tid & 31) == 0) sred[tid >> 5] = l;
    __syncthreads();
    l = sred[0] + sred[1] + sred[2] + sred[3];
    const float o = l > 0.f || l != l ? acc / l : 0.f;  // a row that sees nothing is zero
    if (tid < D) {
        const size_t at = ((size_t)row * p.H_q + h) * D + tid;
        if (p.out_dtype == PA_F32)
            static_cast<float*>(p.out)[at] = o;
        else
            static_cast<T*>(p.out)[at] = from_float<T>(o);
    }
}

static inline pa_status launch_attend_rows(const RowsParams& p, int rows, int q_dtype, int D, cudaStream_t stream) {
    auto go = [&](auto kern) { return launch_kernel(kern, dim3(rows, p.H_q), dim3(128), 0, stream, p); };
    cudaError_t e;
    if (q_dtype == PA_BF16)
        e = D == 128 ? (p.scales ? go(attend_rows_kernel<__nv_bfloat16, 128, true>)
                                 : go(attend_rows_kernel<__nv_bfloat16, 128, false>))
                     : (p.scales ? go(attend_rows_kernel<__nv_bfloat16, 64, true>)
                                 : go(attend_rows_kernel<__nv_bfloat16, 64, false>));
    else
        e = D == 128 ? (p.scales ? go(attend_rows_kernel<__half, 128, true>) : go(attend_rows_kernel<__half, 128, false>))
                     : (p.scales ? go(attend_rows_kernel<__half, 64, true>) : go(attend_rows_kernel<__half, 64, false>));
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "attention launch");
}

}  // namespace pa
