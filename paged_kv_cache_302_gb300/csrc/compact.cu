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
    uint8_t* scales;  // null for a 16-bit pool
    const int32_t* tables;
    const int32_t* ctx_lens;
    const int32_t* base;
    const int32_t* keep;
    const int32_t* keep_start;
    int T, MB, NB, lgB;
    // A token's row: `cols` vectors of 16 bytes, vector c at block * block_bytes + (c / run) * run_step + offset *
    // token_step + (c % run) * 16.  A quantised row's run is one head's K or V, whose scale byte lies at (block * cols /
    // run + c / run) * B + offset.
    int64_t block_bytes, token_step, run_step;
    int cols, run;
    int* err;
};

// The threads of a CTA are 2^lgw columns times the tokens of a quarter chunk, and each takes kMoveUnroll tokens of a
// chunk.  While chunk c is stored, chunk c + 1 is on its way into registers and the positions of chunk c + 2 are looked
// up.  One barrier per chunk separates its reads, all issued before, from its writes; four buffers of looked-up
// positions, because a thread may be one barrier behind another.
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;
constexpr int kMinWidth = 2;  // columns of a CTA: at least one 32-byte sector
constexpr int kMoveCtas = 152 * 8;
constexpr int kMaxChunk = kMoveThreads / kMinWidth * kMoveUnroll;

template <bool kQuant>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p, int lgw) {
    __shared__ int2 s_row[4][kMaxChunk];  // pool rows (block * B + offset) a token comes from (-1: stays) and goes to
    __shared__ int s_bad;                 // first entry of the list that is out of order or out of range
    griddep_wait();
    griddep_launch_dependents();
    const int s = blockIdx.y, tid = threadIdx.x;
    const int k0 = p.keep_start[s], k1 = p.keep_start[s + 1], base = p.base[s], ctx = p.ctx_lens[s];
    if (k0 < 0 || k1 < k0 || k1 > p.T || base < 0 || ctx < 0 || ctx > (int64_t)p.MB << p.lgB) {
        if (blockIdx.x == 0 && tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
        return;
    }
    const int n = k1 - k0, per = kMoveThreads >> lgw, chunk = per * kMoveUnroll;
    const int tok = tid >> lgw, c = (blockIdx.x << lgw) + (tid & ((1 << lgw) - 1));
    const bool mine = c < p.cols;
    const int r = c / p.run;
    const int64_t col = r * p.run_step + (int64_t)(c - r * p.run) * 16;
    const bool scale_too = kQuant && mine && c == r * p.run;
    const int runs = p.cols / p.run;
    const int32_t* table = p.tables + (int64_t)s * p.MB;
    const int32_t* keep = p.keep + k0;
    const int B1 = (1 << p.lgB) - 1;

    // looks up the rows of chunk i
    auto look_up = [&](int i) {
#pragma unroll
        for (int x = 0; x < kMaxChunk / kMoveThreads; ++x) {
            const int at = tid + x * kMoveThreads;
            const int64_t j = (int64_t)i * chunk + at;
            if (at >= chunk) break;
            int2 row = make_int2(-1, -1);
            if (j < n) {
                const int src = keep[j], before = j ? keep[j - 1] : base - 1;
                if (src <= before || src < 0 || src >= ctx) {
                    atomicMin(&s_bad, (int)j);
                } else if (src != base + j && base + j < ctx) {  // (not below src only behind an entry out of order)
                    const int dst = base + (int)j;
                    const int sb = table[src >> p.lgB], db = table[dst >> p.lgB];
                    if ((unsigned)sb < (unsigned)p.NB && (unsigned)db < (unsigned)p.NB)
                        row = make_int2((sb << p.lgB) + (src & B1), (db << p.lgB) + (dst & B1));
                    else
                        flag_error(p.err, PA_DEV_ERR_BLOCK);
                }
            }
            s_row[i & 3][at] = row;
        }
    };
    auto place = [&](int row) -> int64_t {
        return (int64_t)(row >> p.lgB) * p.block_bytes + (row & B1) * p.token_step + col;
    };
    auto scale_place = [&](int row) -> int64_t { return (((int64_t)(row >> p.lgB) * runs + r) << p.lgB) + (row & B1); };
    auto load = [&](int i, uint4 (&v)[kMoveUnroll], uint32_t& sc) {
        sc = 0;
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int src = s_row[i & 3][u * per + tok].x;
            if (src < 0 || !mine) continue;
            v[u] = *reinterpret_cast<const uint4*>(p.data + place(src));
            if (scale_too) sc |= (uint32_t)p.scales[scale_place(src)] << (8 * u);
        }
    };

    if (tid == 0) s_bad = INT_MAX;
    __syncthreads();
    look_up(0);
    look_up(1);
    __syncthreads();
    uint4 v[kMoveUnroll];
    uint32_t sc;
    load(0, v, sc);
    for (int i = 0; (int64_t)i * chunk < n; ++i) {
        uint4 next[kMoveUnroll];
        uint32_t next_sc;
        load(i + 1, next, next_sc);
        look_up(i + 2);
        __syncthreads();  // chunk i is read
        const int64_t bad = s_bad, j0 = (int64_t)i * chunk;
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int2 row = s_row[i & 3][u * per + tok];
            if (row.x < 0 || !mine || j0 + u * per + tok >= bad) continue;
            *reinterpret_cast<uint4*>(p.data + place(row.y)) = v[u];
            if (scale_too) p.scales[scale_place(row.y)] = (uint8_t)(sc >> (8 * u));
        }
        if (bad < j0 + chunk) {
            if (blockIdx.x == 0 && tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
            return;
        }
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) v[u] = next[u];
        sc = next_sc;
    }
}

pa_status launch_compact(const CompactArgs& a) {
    CompactParams p;
    const bool quant = a.kv_dtype == PA_E4M3;
    p.data = static_cast<uint8_t*>(a.pool);
    p.scales = static_cast<uint8_t*>(a.scales);
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
    const int64_t row = (int64_t)2 * a.H_kv * a.D * (quant ? 1 : 2);
    p.block_bytes = row * a.B;
    p.cols = (int)(row / 16);
    p.run = quant ? a.D / 16 : p.cols;
    p.run_step = quant ? (int64_t)a.B * a.D : 0;
    p.token_step = quant ? a.D : row;
    // Columns per CTA: a chunk no longer than the lists are on average, and, as far as a sector per token allows, enough
    // CTAs to fill the device several times.
    const int64_t mean = a.T / a.N;
    int lgw = 1;
    while (lgw < 8 && (1 << lgw) < p.cols &&
           ((int64_t)(kMoveThreads >> lgw) * kMoveUnroll > mean || ((int64_t)p.cols * a.N) >> lgw > kMoveCtas))
        ++lgw;
    const int64_t gx = (p.cols + (1 << lgw) - 1) >> lgw;
    const cudaError_t e = launch_kernel(quant ? compact_kernel<true> : compact_kernel<false>,
                                        dim3((unsigned)gx, (unsigned)a.N), dim3(kMoveThreads), 0, a.stream, p, lgw);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "compact launch");
}

}  // namespace pa
