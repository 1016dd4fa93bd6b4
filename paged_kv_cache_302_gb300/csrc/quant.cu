// quant.cu -- the quantised cache: the write that quantises through slot_mapping, and the read that restores blocks
// of a 16-bit pool.  The format is in quant.cuh.
#include <algorithm>
#include <type_traits>

#include "quant.cuh"

namespace pa {

// ----------------------------------------------------------------------------- write

// A row's D / 16 lanes take 16 elements (32 bytes) each, find the row's largest magnitude with xor shuffles -- as
// 16-bit integers, two at a time: magnitudes order as their bits do -- and write 16 bytes each; lane 0 of the row
// writes the scale byte.  Rows are numbered (token, K/V, head).  Bound by memory: 4 D bytes read and 2 D + 2 written
// per (token, head): 16387 tokens of 8 heads (101 MB) take 17.6 us, 5.7 TB/s.  16 elements per lane and one row at a
// time with 32 registers, 8 CTAs on an SM, measured best: 8 elements per lane took 26 us (half as many bytes in flight,
// the shuffles and the scale shared by half as many elements), two rows at a time with 4 CTAs 19, four with 2 CTAs 25,
// a CTA for every 32 rows 20.
constexpr int kQuantThreads = 256;
constexpr int kQuantCtasPerSm = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kQuantThreads, kQuantCtasPerSm)
    quant_cache_kernel(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ qpool,
                       uint8_t* __restrict__ scales, const int64_t* __restrict__ slots, int64_t rows, int64_t nslots,
                       int H_kv, int lgB, int* err) {
    constexpr int L = D / 16;                  // lanes per row
    constexpr int kPer = kQuantThreads / L;    // rows of a CTA at a time
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    griddep_wait();
    griddep_launch_dependents();
    const int sub = threadIdx.x % L, R = 2 * H_kv;
    const unsigned mask = ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
    // token and row in the token of this thread's next row, and the step to the one after
    const int64_t step = (int64_t)gridDim.x * kPer;
    int64_t r = (int64_t)blockIdx.x * kPer + threadIdx.x / L, i = r / R;
    int rem = (int)(r - i * R);
    const int64_t di = step / R;
    const int dr = (int)(step - di * R);
    for (; r < rows; r += step) {
        const int which = rem >= H_kv, h = rem - which * H_kv;
        const int64_t slot = slots[i];
        // (read whether or not the slot is good: the loads need not wait for it)
        const uint4* src = reinterpret_cast<const uint4*>((which ? v : k) + (i * H_kv + h) * D) + 2 * sub;
        const uint4 x0 = src[0], x1 = src[1];
        if (slot >= nslots && rem == 0 && sub == 0) flag_error(err, PA_DEV_ERR_SLOT);
        i += di;
        rem += dr;
        if (rem >= R) {
            rem -= R;
            ++i;
        }
        if (slot < 0 || slot >= nslots) continue;  // uniform over the row's lanes
        const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = vmax_u16x2(m, w[j] & 0x7fff7fffu);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = vmax_u16x2(m, __shfl_xor_sync(mask, m, o));
        m = max(m & 0xffffu, m >> 16);
        if (m > kInf) {  // a NaN, which counts as nothing
            m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t lo = w[j] & 0x7fffu, hi = w[j] >> 16 & 0x7fffu;
                m = max(m, max(lo <= kInf ? lo : 0u, hi <= kInf ? hi : 0u));
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
        }
        const int e = scale_exponent(Mma<T>::unpack(m).x);
        const float inv = pow2i(-e);
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f0 = Mma<T>::unpack(w[2 * j]), f1 = Mma<T>::unpack(w[2 * j + 1]);
            q[j] = to_e4m3x2(f0.x * inv, f0.y * inv) | to_e4m3x2(f1.x * inv, f1.y * inv) << 16;
        }
        const int64_t blk = slot >> lgB, off = slot - (blk << lgB);
        const int64_t row = (((blk * H_kv + h) * 2 + which) << lgB) + off;
        reinterpret_cast<uint4*>(qpool + row * D)[sub] = make_uint4(q[0], q[1], q[2], q[3]);
        if (sub == 0) scales[row] = (uint8_t)(e + kScaleBias);
    }
}

static int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        sms = 1;
    return sms;
}

template <typename T>
static cudaError_t quant_cache_d(const void* k, const void* v, void* qpool, void* scales, const int64_t* slots, int T_,
                                 int64_t nslots, int H_kv, int D, int lgB, int* err, cudaStream_t st) {
    const int64_t rows = (int64_t)T_ * 2 * H_kv, per = kQuantThreads / (D / 16);
    const unsigned grid = (unsigned)std::min<int64_t>((rows + per - 1) / per, (int64_t)sm_count() * kQuantCtasPerSm);
    auto kern = D == 128 ? quant_cache_kernel<T, 128> : quant_cache_kernel<T, 64>;
    return launch_kernel(kern, dim3(grid), dim3(kQuantThreads), 0, st, static_cast<const T*>(k),
                         static_cast<const T*>(v), static_cast<uint8_t*>(qpool), static_cast<uint8_t*>(scales), slots,
                         rows, nslots, H_kv, lgB, err);
}

pa_status launch_quant_cache(const void* k, const void* v, void* qpool, void* scales, const int64_t* slot_mapping,
                             int T, int NB, int B, int H_kv, int D, int dtype, int* dev_err, cudaStream_t stream) {
    if (T == 0) return PA_OK;
    const int lgB = B == 8 ? 3 : B == 16 ? 4 : 5;
    const int64_t nslots = (int64_t)NB * B;
    const cudaError_t e = dtype == PA_BF16 ? quant_cache_d<__nv_bfloat16>(k, v, qpool, scales, slot_mapping, T, nslots,
                                                                          H_kv, D, lgB, dev_err, stream)
                                           : quant_cache_d<__half>(k, v, qpool, scales, slot_mapping, T, nslots, H_kv,
                                                                   D, lgB, dev_err, stream);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "quant_cache launch");
}

// ----------------------------------------------------------------------------- read

// A row's D / 16 lanes read 16 values each and write 32 bytes each, one whole sector where the pool allows.  grid.x =
// pair, grid.y = chunk of the block's rows (numbered (head, K/V, token), the order they lie in).  Bound by memory: 4001
// blocks of 16 tokens and 8 heads, D = 128 (394 MB read and written): 63.7 us, 6.2 TB/s; with two 16-byte stores per
// lane 64.4.
constexpr int kDequantThreads = 256;

template <typename T>
__device__ __forceinline__ uint32_t restore2(uint32_t e4m3x2, float s) {
    const uint32_t h = e4m3x2_to_f16x2(e4m3x2);
    float2 f = Mma<__half>::unpack(h);
    f.x *= s;
    f.y *= s;
    if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
        // a magnitude that fp16 cannot hold becomes its largest (NaN stays)
        if (fabsf(f.x) > 65504.f) f.x = copysignf(65504.f, f.x);
        if (fabsf(f.y) > 65504.f) f.y = copysignf(65504.f, f.y);
    }
    return Mma<T>::pack(f.x, f.y);
}

template <typename T, int D>
__global__ void __launch_bounds__(kDequantThreads) dequant_blocks_kernel(T* __restrict__ pool,
                                                                         const uint8_t* __restrict__ qpool,
                                                                         const uint8_t* __restrict__ scales,
                                                                         const int64_t* __restrict__ pairs, int NB_dst,
                                                                         int NB_src, int H_kv, int lgB, int* err) {
    constexpr int L = D / 16;  // lanes per row
    griddep_wait();
    griddep_launch_dependents();
    const int64_t src = pairs[2 * (int64_t)blockIdx.x], dst = pairs[2 * (int64_t)blockIdx.x + 1];
    if (src < 0 || src >= NB_src || dst < 0 || dst >= NB_dst) {
        if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(err, PA_DEV_ERR_BLOCK);
        return;
    }
    const int rows = (2 * H_kv) << lgB, B = 1 << lgB;
    const bool sector = (reinterpret_cast<uintptr_t>(pool) & 31u) == 0;
    const int sub = threadIdx.x % L;
    for (int r = blockIdx.y * (kDequantThreads / L) + threadIdx.x / L; r < rows;
         r += gridDim.y * (kDequantThreads / L)) {
        const int64_t row = src * rows + r;
        const uint4 x = reinterpret_cast<const uint4*>(qpool + row * D)[sub];
        const float s = pow2i(scale_of(scales[row]));
        const int t = r & (B - 1), which = (r >> lgB) & 1, h = r >> (lgB + 1);
        uint4 o[2];
        o[0] = make_uint4(restore2<T>(x.x, s), restore2<T>(x.x >> 16, s), restore2<T>(x.y, s),
                          restore2<T>(x.y >> 16, s));
        o[1] = make_uint4(restore2<T>(x.z, s), restore2<T>(x.z >> 16, s), restore2<T>(x.w, s),
                          restore2<T>(x.w >> 16, s));
        T* d = pool + ((((dst << lgB) + t) * 2 + which) * H_kv + h) * D + 16 * sub;
        if (sector) {  // a lane's 32 bytes are one sector
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "r"(o[0].x), "r"(o[0].y),
                         "r"(o[0].z), "r"(o[0].w), "r"(o[1].x), "r"(o[1].y), "r"(o[1].z), "r"(o[1].w)
                         : "memory");
        } else {
            reinterpret_cast<uint4*>(d)[0] = o[0];
            reinterpret_cast<uint4*>(d)[1] = o[1];
        }
    }
}

pa_status launch_dequant_blocks(void* pool, int NB_dst, const void* qpool, const void* scales, int NB_src,
                                const int64_t* pairs, int n, int B, int H_kv, int D, int dtype, int* dev_err,
                                cudaStream_t stream) {
    if (n == 0) return PA_OK;
    const int lgB = B == 8 ? 3 : B == 16 ? 4 : 5;
    const int64_t rows = (int64_t)2 * H_kv * B, per = kDequantThreads / (D / 16);
    const unsigned gy = (unsigned)std::min<int64_t>((rows + per - 1) / per, 65535);
    auto go = [&](auto kern, auto* p) {
        return launch_kernel(kern, dim3((unsigned)n, gy), dim3(kDequantThreads), 0, stream, p,
                             static_cast<const uint8_t*>(qpool), static_cast<const uint8_t*>(scales), pairs, NB_dst,
                             NB_src, H_kv, lgB, dev_err);
    };
    cudaError_t e;
    if (dtype == PA_BF16)
        e = go(D == 128 ? dequant_blocks_kernel<__nv_bfloat16, 128> : dequant_blocks_kernel<__nv_bfloat16, 64>,
               static_cast<__nv_bfloat16*>(pool));
    else
        e = go(D == 128 ? dequant_blocks_kernel<__half, 128> : dequant_blocks_kernel<__half, 64>,
               static_cast<__half*>(pool));
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "dequant_blocks launch");
}

}  // namespace pa
