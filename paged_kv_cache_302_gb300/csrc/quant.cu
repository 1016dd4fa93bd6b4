// quant.cu -- the quantised cache: the write that quantises through slot_mapping, and the read that restores blocks
// of a 16-bit pool.  The format is in quant.cuh.
#include <algorithm>
#include <type_traits>

#include "quant.cuh"

namespace pa {

// ----------------------------------------------------------------------------- write

// A row's D / 8 lanes take 8 elements (16 bytes) each, find the row's largest magnitude with xor shuffles, and
// write 8 bytes each; lane 0 of the row writes the scale byte.  Rows are numbered (token, K/V, head).
constexpr int kQuantThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kQuantThreads) quant_cache_kernel(const T* __restrict__ k, const T* __restrict__ v,
                                                                    uint8_t* __restrict__ qpool,
                                                                    uint8_t* __restrict__ scales,
                                                                    const int64_t* __restrict__ slots, int T_,
                                                                    int64_t nslots, int H_kv, int lgB, int* err) {
    constexpr int L = D / 8;  // lanes per row
    griddep_wait();
    griddep_launch_dependents();
    const int sub = threadIdx.x % L;
    const int64_t rows = (int64_t)T_ * 2 * H_kv;
    const int64_t stride = (int64_t)gridDim.x * (kQuantThreads / L);
    for (int64_t r = (int64_t)blockIdx.x * (kQuantThreads / L) + threadIdx.x / L; r < rows; r += stride) {
        const int64_t i = r / (2 * H_kv);
        const int rem = (int)(r - i * 2 * H_kv), which = rem >= H_kv, h = rem - which * H_kv;
        const int64_t slot = slots[i];
        const bool ok = slot >= 0 && slot < nslots;
        if (slot >= nslots && rem == 0 && sub == 0) flag_error(err, PA_DEV_ERR_SLOT);
        if (!ok) continue;  // uniform over the row's lanes
        const uint4 x = reinterpret_cast<const uint4*>((which ? v : k) + (i * H_kv + h) * D)[sub];
        const float2 f[4] = {Mma<T>::unpack(x.x), Mma<T>::unpack(x.y), Mma<T>::unpack(x.z), Mma<T>::unpack(x.w)};
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = fmaxf(a, fmaxf(fabsf(f[j].x), fabsf(f[j].y)));  // NaN counts as nothing
        const unsigned mask = (L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1)));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(mask, a, o));
        const int e = scale_exponent(a);
        const float inv = pow2i(-e);
        uint2 q;
        q.x = to_e4m3x2(f[0].x * inv, f[0].y * inv) | to_e4m3x2(f[1].x * inv, f[1].y * inv) << 16;
        q.y = to_e4m3x2(f[2].x * inv, f[2].y * inv) | to_e4m3x2(f[3].x * inv, f[3].y * inv) << 16;
        const int64_t blk = slot >> lgB, off = slot - (blk << lgB);
        const int64_t row = (((blk * H_kv + h) * 2 + which) << lgB) + off;
        reinterpret_cast<uint2*>(qpool + row * D)[sub] = q;
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
    const int64_t rows = (int64_t)T_ * 2 * H_kv, per = kQuantThreads / (D / 8);
    const unsigned grid = (unsigned)std::min<int64_t>((rows + per - 1) / per, (int64_t)sm_count() * 8);
    auto kern = D == 128 ? quant_cache_kernel<T, 128> : quant_cache_kernel<T, 64>;
    return launch_kernel(kern, dim3(grid), dim3(kQuantThreads), 0, st, static_cast<const T*>(k),
                         static_cast<const T*>(v), static_cast<uint8_t*>(qpool), static_cast<uint8_t*>(scales), slots,
                         T_, nslots, H_kv, lgB, err);
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

// A row's D / 16 lanes read 16 values each and write 32 bytes each.  grid.x = pair, grid.y = chunk of the block's
// rows (numbered (head, K/V, token), the order they lie in).
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
        uint4* d = reinterpret_cast<uint4*>(pool + ((((dst << lgB) + t) * 2 + which) * H_kv + h) * D) + 2 * sub;
        d[0] = o[0];
        d[1] = o[1];
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
