// compact.cu -- compaction: a sequence's kept tokens moved together, in place.
//
// Kept token j moves from position src_j to dst_j = base + j.  The kept positions ascend from base on, so src_j >= dst_j:
// no token is written to a place that a later one is still read from.  A CTA therefore walks its sequence in order, a
// chunk of tokens at a time, reads a chunk before it writes it, and needs no second buffer.  CTAs of one sequence work
// on different columns of the tokens' rows and never meet.
#include <algorithm>
#include <climits>

#include "pa_device.cuh"

namespace pa {

struct CompactParams {
    uint8_t* data;
    const int32_t* tables;
    const int32_t* ctx_lens;
    const int32_t* base;
    const int32_t* keep;
    const int32_t* keep_start;
    int T, MB, NB, lgB;
    // A token's row in `data`: `cols` vectors, vector c at block * block_bytes + (c / run) * run_step + offset *
    // token_step + (c % run) * sizeof(vector).
    int64_t block_bytes, token_step, run_step;
    int cols, run;
    int* err;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// V: uint4 for rows of values, uint8_t for scale bytes.  grid.x: groups of `width` columns, grid.y: sequences.
template <typename V>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p, int width) {
    __shared__ int s_bad;  // first entry of the list that is out of order or out of range
    griddep_wait();
    griddep_launch_dependents();
    const int s = blockIdx.y;
    const int k0 = p.keep_start[s], k1 = p.keep_start[s + 1], base = p.base[s], ctx = p.ctx_lens[s];
    if (k0 < 0 || k1 < k0 || k1 > p.T || base < 0 || ctx < 0 || ctx > (int64_t)p.MB << p.lgB) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.err, PA_DEV_ERR_CTX);
        return;
    }
    const int n = k1 - k0, lane = threadIdx.x % width, tok = threadIdx.x / width, per = kMoveThreads / width;
    const int c = blockIdx.x * width + lane;
    const int64_t col = (int64_t)(c / p.run) * p.run_step + (int64_t)(c % p.run) * sizeof(V);
    const bool mine = c < p.cols && tok < per;
    const int32_t* table = p.tables + (int64_t)s * p.MB;
    const int B1 = (1 << p.lgB) - 1;
    if (threadIdx.x == 0) s_bad = INT_MAX;
    __syncthreads();
    for (int j0 = 0; j0 < n; j0 += per * kMoveUnroll) {
        V v[kMoveUnroll];
        int src_blk[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int j = j0 + u * per + tok;
            src_blk[u] = -1;
            if (!mine || j >= n) continue;
            const int src = p.keep[k0 + j], before = j ? p.keep[k0 + j - 1] : base - 1;
            if (src <= before || src < 0 || src >= ctx) {
                atomicMin(&s_bad, j);
                continue;
            }
            if (src == base + j) continue;  // stays
            const int blk = table[src >> p.lgB];
            if ((unsigned)blk >= (unsigned)p.NB) {
                flag_error(p.err, PA_DEV_ERR_BLOCK);
                continue;
            }
            src_blk[u] = blk;
            v[u] = *reinterpret_cast<const V*>(p.data + blk * p.block_bytes + (src & B1) * p.token_step + col);
        }
        __syncthreads();  // the chunk is read
        const int bad = s_bad;
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int j = j0 + u * per + tok;
            if (src_blk[u] < 0 || j >= bad) continue;
            const int dst = base + j;  // below the position it comes from
            const int blk = table[dst >> p.lgB];
            if ((unsigned)blk >= (unsigned)p.NB) {
                flag_error(p.err, PA_DEV_ERR_BLOCK);
                continue;
            }
            *reinterpret_cast<V*>(p.data + blk * p.block_bytes + (dst & B1) * p.token_step + col) = v[u];
        }
        if (bad < INT_MAX) {
            if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.err, PA_DEV_ERR_CTX);
            return;
        }
        __syncthreads();  // s_bad is read
    }
}

pa_status launch_compact(const CompactArgs& a) {
    CompactParams p;
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.base = a.base;
    p.keep = a.keep;
    p.keep_start = a.keep_start;
    p.T = a.T;
    p.MB = a.MB;
    p.NB = a.NB;
    p.lgB = a.B == 8 ? 3 : a.B == 16 ? 4 : 5;
    p.err = a.dev_err;
    const bool quant = a.kv_dtype == PA_E4M3;
    p.data = static_cast<uint8_t*>(a.pool);
    const int64_t row = (int64_t)2 * a.H_kv * a.D * (quant ? 1 : 2);
    p.block_bytes = row * a.B;
    p.cols = (int)(row / 16);
    p.run = quant ? a.D / 16 : p.cols;
    p.run_step = quant ? (int64_t)a.B * a.D : 0;
    p.token_step = quant ? a.D : row;
    const int width = 4;
    cudaError_t e = launch_kernel(compact_kernel<uint4>, dim3((unsigned)((p.cols + width - 1) / width), (unsigned)a.N),
                                  dim3(kMoveThreads), 0, a.stream, p, width);
    count_launch();
    if (e == cudaSuccess && quant) {
        p.data = static_cast<uint8_t*>(a.scales);
        p.block_bytes = (int64_t)2 * a.H_kv * a.B;
        p.cols = 2 * a.H_kv;
        p.run = 1;
        p.run_step = a.B;
        p.token_step = 1;
        e = launch_kernel(compact_kernel<uint8_t>, dim3((unsigned)((p.cols + width - 1) / width), (unsigned)a.N),
                          dim3(kMoveThreads), 0, a.stream, p, width);
        count_launch();
    }
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "compact launch");
}

}  // namespace pa
