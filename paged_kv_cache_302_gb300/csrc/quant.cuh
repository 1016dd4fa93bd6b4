// quant.cuh -- the quantised cache's format, shared by its writer, its reader and the attention kernels.
//
// A row is the D elements of one token's K or V for one KV head.  It is held as D e4m3 values (1 sign, 4 exponent,
// 3 mantissa bits, largest finite 448) and one scale byte b that stands for 2^(b - 127): element d is
// q_d 2^(b - 127).  The scale is the smallest power of two that brings the row's largest magnitude to 448 or
// below.  e4m3 is a floating format, so a scale finer than a power of two would gain no relative precision, and
// with a power of two scaling and restoring are exact: an element's only rounding is the one to e4m3 (half a step:
// 2^-4 of its magnitude, or 2^-10 of the scale below 2^-6 of it).
//   qpool  [NB][H_kv][2][B][D] e4m3: a (block, head)'s K rows then V rows, one contiguous chunk of 2 B D bytes
//   scales [NB][H_kv][2][B] bytes
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kScaleBias = 127;
// Exponents a scale takes.  In attention exp2(y), y = score + V exponent, serves both the output and (times 2^-e)
// the exponential sum: with |e| <= 40 neither product leaves the normal fp32 range for a term that matters.
constexpr int kScaleMin = -40, kScaleMax = 40;

// Exponent e of the scale for a row whose largest magnitude is a (>= 0): the smallest e with a <= 448 2^e.
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - kScaleBias - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
    return min(max(e, kScaleMin), kScaleMax);
}

// Exponent a scale byte stands for (a byte the writer cannot have written counts as the nearest it can).
__device__ __forceinline__ int scale_of(int byte) { return min(max(byte - kScaleBias, kScaleMin), kScaleMax); }

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two fp32 values as e4m3 (x in the low byte), round to nearest even, magnitudes above 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float x, float y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
}

// Two e4m3 values (the low 16 bits) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

// 3-D tiled tensor load into shared memory, completion counted on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}

}  // namespace pa
