// runs.cuh -- the work of a batch cut into runs of equal length.
//
// A row is one (sequence, KV head); all H_kv rows of a sequence have the same number of units, which follows from its
// context.  The units of all rows, in order, are cut into `parts` runs whose lengths differ by at most one.  A warp
// finds its run by itself: it reads the lengths once, the first kScanSeqs of them in one go.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kScanSeqs = 128;

struct Cut {
    int len, longer;  // the first `longer` runs have one unit more than len
    __device__ __forceinline__ Cut(int total, int parts) : len(total / parts), longer(total - total / parts * parts) {}
    __device__ __forceinline__ int start(int i) const { return i * len + min(i, longer); }
    __device__ __forceinline__ int run_of(int unit) const {  // the run that holds a unit
        const int head = longer * (len + 1);
        return unit < head ? unit / (len + 1) : longer + (unit - head) / len;
    }
};

// Units of a row of each sequence, as units(s) gives them (0 for a sequence that has none).
template <typename F>
struct RowScan {
    F units;
    int N, H_kv;
    int w[kScanSeqs / 32];

    __device__ __forceinline__ RowScan(F f, int n, int h) : units(f), N(n), H_kv(h) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kScanSeqs / 32; ++i) w[i] = 32 * i + lane < N ? units(32 * i + lane) : 0;
    }
    // Units of the whole batch.
    __device__ __forceinline__ int total() const {
        int t = 0;
#pragma unroll
        for (int i = 0; i < kScanSeqs / 32; ++i)
            if (32 * i < N) t += w[i];
        for (int s = kScanSeqs + (threadIdx.x & 31); s < N; s += 32) t += units(s);
        return __reduce_add_sync(0xffffffffu, t) * H_kv;
    }
    // The sequence that holds unit u (below the total): its units per row in `n`, its first unit in `first`.  (The last
    // one, should the lengths have changed since: nothing is ever looked up behind the batch.)
    __device__ __forceinline__ int find(int u, int& n, int& first) const {
        const int lane = threadIdx.x & 31;
        int before = 0, s = -1;
        n = 1;
        first = u;
        auto look = [&](int s0, int x) {
            int v = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            const int hi = before + v * H_kv;
            const unsigned hit = __ballot_sync(0xffffffffu, u < hi);
            if (hit) {
                const int src = __ffs(hit) - 1;
                s = s0 + src;
                n = __shfl_sync(0xffffffffu, x, src);
                first = __shfl_sync(0xffffffffu, hi, src) - n * H_kv;
            }
            before = __shfl_sync(0xffffffffu, hi, 31);
        };
#pragma unroll
        for (int i = 0; i < kScanSeqs / 32; ++i)
            if (s < 0 && 32 * i < N) look(32 * i, w[i]);
        for (int s0 = kScanSeqs; s < 0 && s0 < N; s0 += 32) look(s0, s0 + lane < N ? units(s0 + lane) : 0);
        return s < 0 ? N - 1 : s;
    }
};

}  // namespace pa
