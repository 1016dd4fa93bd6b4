// summary.cuh -- the format of key summaries, shared by the kernel that makes them and the one that selects blocks by
// them.
//
// A summary is a box around the keys of one (block, KV head): per channel the least and the greatest K of the block's
// tokens, as integers of 8 bits in units of one power of two,
//     lo_d = floor(min_t K_td 2^-e),  hi_d = ceil(max_t K_td 2^-e),  e the least with max |K| <= 127 2^e:
//   summaries [NB][H_kv][2][D] int8 (lo, hi), sum_scales [NB][H_kv] bytes, b standing for 2^(b - 127).
// No key of the block has a larger product with a query q than sum_d max(q_d lo_d, q_d hi_d) 2^e (as long as none
// saturates).  A block's score is that sum for q in integers of 9 bits and a sign (q_d 2^-f rounded, f the least with
// max |q| <= 511 2^f): it bounds the products with q itself up to the rounding, 2^(f - 1) sum_d |K_d|.  Every such sum
// is an integer below 128 * 127 * 511 < 2^23, hence exact in fp32 in any order: the selection does not depend on how
// the sum is split.
#pragma once

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

// Minima and maxima of 16-bit pairs; of a NaN and a number the number.
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

}  // namespace pa
