// decode_sparse.cu -- single-token decode attention over listed blocks of each (sequence, KV head).
#include <algorithm>
#include <type_traits>

#include "quant.cuh"

namespace pa {

// One CTA per (sequence, KV head), its warps on the listed tokens in turn, each with a running maximum, sum and output
// of its own for every query head; joined through shared memory at the end.
constexpr int kSparseWarps = 8;

struct SparseParams {
    void* out;
    int out_dtype;
    const void* q;
    const void* pool;
    const uint8_t* scales;
    const int32_t* tables;
    const int32_t* ctx_lens;
    const int32_t* selected;
    int top_k, H_kv, G, B, MB, NB;
    float scale_log2;
    int* err;
};

template <typename T, bool kQuant, int D>
__global__ void __launch_bounds__(kSparseWarps * 32) decode_sparse_kernel(const SparseParams p) {
    constexpr int V = D / 32;
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float s_m[kSparseWarps][kMaxGroup], s_l[kSparseWarps][kMaxGroup];
    __shared__ float s_o[kSparseWarps][kMaxGroup][D];
    const int h = blockIdx.x, s = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctx = p.ctx_lens[s];
    if (ctx < 1 || ctx > (int64_t)p.MB * p.B) {
        if (h == 0 && threadIdx.x == 0) flag_error(p.err, PA_DEV_ERR_CTX);
        return;
    }
    const int64_t row0 = ((int64_t)s * p.H_kv + h) * p.G;
    float q[kMaxGroup][V], o[kMaxGroup][V], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            q[g][v] = g < p.G ? (float)static_cast<const T*>(p.q)[(row0 + g) * D + lane * V + v] : 0.f;
            o[g][v] = 0.f;
        }
    }
    const int32_t* list = p.selected + ((int64_t)s * p.H_kv + h) * p.top_k;
    const int nblk = (ctx + p.B - 1) / p.B;
    for (int i = warp; i < p.top_k; i += kSparseWarps) {
        const int e = list[i];
        if (e < 0) continue;
        const int blk = e < nblk ? p.tables[(int64_t)s * p.MB + e] : -1;
        if ((unsigned)blk >= (unsigned)p.NB) {
            if (lane == 0) flag_error(p.err, PA_DEV_ERR_BLOCK);
            continue;
        }
        const int nv = min(p.B, ctx - e * p.B);
        for (int t = 0; t < nv; ++t) {
            float k[V], w[V];
            if constexpr (kQuant) {
                const int64_t row = ((int64_t)blk * p.H_kv + h) * 2 * p.B + t;
                const uint8_t* kp = static_cast<const uint8_t*>(p.pool) + row * D + lane * V;
                const float fk = pow2i(scale_of(p.scales[row])), fv = pow2i(scale_of(p.scales[row + p.B]));
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    const float2 a = Mma<__half>::unpack(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kp + v)));
                    const float2 b = Mma<__half>::unpack(
                        e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kp + (int64_t)p.B * D + v)));
                    k[v] = a.x * fk;
                    k[v + 1] = a.y * fk;
                    w[v] = b.x * fv;
                    w[v + 1] = b.y * fv;
                }
            } else {
                const T* kp = static_cast<const T*>(p.pool) + ((((int64_t)blk * p.B + t) * 2) * p.H_kv + h) * D + lane * V;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    k[v] = (float)kp[v];
                    w[v] = (float)kp[(int64_t)p.H_kv * D + v];
                }
            }
#pragma unroll
            for (int g = 0; g < kMaxGroup; ++g) {
                if (g < p.G) {
                    float x = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v) x += q[g][v] * k[v];
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    x *= p.scale_log2;
                    const float n = fmaxf(m[g], x), a = exp2f(m[g] - n), y = exp2f(x - n);
                    m[g] = n;
                    l[g] = l[g] * a + y;
#pragma unroll
                    for (int v = 0; v < V; ++v) o[g][v] = o[g][v] * a + y * w[v];
                }
            }
        }
    }
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
        if (lane == 0) {
            s_m[warp][g] = m[g];
            s_l[warp][g] = l[g];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) s_o[warp][g][lane * V + v] = o[g][v];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.G * D; i += kSparseWarps * 32) {
        const int g = i / D, d = i % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int w = 0; w < kSparseWarps; ++w) M = fmaxf(M, s_m[w][g]);
        if (M > -INFINITY) {
            for (int w = 0; w < kSparseWarps; ++w) {
                const float f = exp2f(s_m[w][g] - M);
                L += f * s_l[w][g];
                O += f * s_o[w][g][d];
            }
            O /= L;
        }
        if (p.out_dtype == PA_F32)
            static_cast<float*>(p.out)[row0 * D + i] = O;
        else
            static_cast<T*>(p.out)[row0 * D + i] = from_float<T>(O);
    }
}

size_t decode_sparse_workspace_bytes(int N, int H_q, int H_kv, int D, int B, int top_k) {
    if (N <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || H_q / H_kv > kMaxGroup || (D != 64 && D != 128) ||
        (B != 8 && B != 16 && B != 32) || top_k <= 0)
        return 0;
    return 256;
}

pa_status launch_decode_sparse(const DecodeSparseArgs& a) {
    SparseParams p;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.q = a.q;
    p.pool = a.pool;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.selected = a.selected;
    p.top_k = a.top_k;
    p.H_kv = a.H_kv;
    p.G = a.H_q / a.H_kv;
    p.B = a.B;
    p.MB = a.MB;
    p.NB = a.NB;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);  // log2(e)
    p.err = a.dev_err;
    auto pick = [&](auto q, auto d) {
        constexpr int D = decltype(d)::value;
        return a.kv_dtype == PA_E4M3 ? decode_sparse_kernel<decltype(q), true, D>
                                     : decode_sparse_kernel<decltype(q), false, D>;
    };
    auto by_dim = [&](auto q) {
        return a.D == 128 ? pick(q, std::integral_constant<int, 128>()) : pick(q, std::integral_constant<int, 64>());
    };
    auto kern = a.q_dtype == PA_BF16 ? by_dim(__nv_bfloat16()) : by_dim(__half());
    const cudaError_t e = launch_kernel(kern, dim3((unsigned)a.H_kv, (unsigned)a.N), dim3(kSparseWarps * 32), 0, a.stream, p);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "decode_sparse launch");
}

}  // namespace pa
