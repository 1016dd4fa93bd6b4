// compact.cu -- compaction: a sequence's kept tokens moved together, in place.
//
// Kept token j moves from position src_j to dst_j = base + j.  The kept positions ascend from base on, so src_j >=
// dst_j: no token is written to a place that a later one is still read from.  A CTA therefore walks its sequence in
// order, a chunk of tokens at a time, reads a chunk before it writes it, and needs no second buffer.  CTAs of one
// sequence work on different columns of the tokens' rows and never meet.
//
// Bound by memory, each moved row read once and written once: 8 sequences of 16384 tokens, half of them kept (537 MB),
// take 97 us, 5.5 TB/s.  A few sequences are bound by the chain of their chunks instead: 5 of up to 8192 tokens over
// e4m3 rows (77 MB) take 24.6 us.  64 drafts of 24 tokens, 6 of them accepted: 3.3 us on the device.  A chunk read into
// registers and stored without more took 155 us; the next chunk read ahead 133; a ring of asynchronous copies with rows
// looked up chunk by chunk 115 to 172 (each chunk waited for its own look-up), a span of chunks ahead 97.
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
    // token_step + (c % run) * 16.  A quantised row's run is one head's K or V, whose scale byte lies at (block * cols
    // / run + c / run) * B + offset.
    int64_t block_bytes, token_step, run_step;
    int cols, run;
    int* err;
};

// A CTA's threads are 2^lgw columns times kMoveThreads / 2^lgw tokens, and each takes kMoveUnroll tokens of a chunk.
// Chunks go through a ring of shared-memory stages: kMoveStages - 1 of them are on their way while one is stored.  The
// rows that tokens come from and go to (a list entry and two block-table entries each) are looked up kSpan tokens at a
// time, in three steps during the first three chunks of the span before, so that no step waits for its own loads.
// Every thread stores what it copied itself; the one barrier per chunk puts all reads of a chunk before its first
// write. Columns: 8 sequences took 97 us with 8 per CTA, 115 to 140 with 4 or 16 (fewer tokens in flight per CTA, or
// fewer CTAs); 5 e4m3 sequences 24.6 us with 2, 30 with 4.  Two stages instead of three took 137.
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;
constexpr int kMoveStages = 3;
constexpr int kSpan = 2048;
constexpr int kMinLgw = 1, kMaxLgw = 8;  // columns of a CTA: at least one 32-byte sector
constexpr int kLook = kSpan / kMoveThreads;
constexpr int kMoveCtas = 152 * 5 / 2;  // as many as the columns are spread over (time only; by the device built for)
constexpr size_t kMoveSmem = (size_t)kMoveStages * kMoveThreads * kMoveUnroll * 16 + 2 * kSpan * sizeof(int2);
// the copies of chunk i + kMoveStages - 1 follow chunk i's barrier, the third step comes before that of a span's third
static_assert(kSpan / ((kMoveThreads >> kMinLgw) * kMoveUnroll) >= kMoveStages + 1, "a span's rows are there in time");

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A sequence's list.
struct KeepList {
    const int32_t* keep;
    const int32_t* table;
    int n, base, ctx, lgB, NB;

    // Whether the list's token j moves.  `bad` receives the least j that is out of order or out of range.
    __device__ __forceinline__ bool moves(int64_t j, int src, int before, int* bad) const {
        if (j >= n) return false;
        if (src <= before || src < 0 || src >= ctx) {
            atomicMin(bad, (int)j);
            return false;
        }
        return src != base + j && base + j < ctx;  // (the latter fails only behind an entry out of order)
    }
    // Rows (block * B + offset) that it comes from and goes to, of its block-table entries; (-1, -1) without a block.
    __device__ __forceinline__ int2 rows(int64_t j, int src, int sb, int db, int* err) const {
        const int B1 = (1 << lgB) - 1;
        if ((unsigned)sb >= (unsigned)NB || (unsigned)db >= (unsigned)NB) {
            flag_error(err, PA_DEV_ERR_BLOCK);
            return make_int2(-1, -1);
        }
        return make_int2((sb << lgB) + (src & B1), (db << lgB) + ((base + (int)j) & B1));
    }
    __device__ __forceinline__ int block_from(int src) const { return table[src >> lgB]; }
    __device__ __forceinline__ int block_to(int64_t j) const { return table[(base + (int)j) >> lgB]; }
    __device__ __forceinline__ int source(int64_t j) const { return j < n ? keep[j] : 0; }
    __device__ __forceinline__ int source_before(int64_t j) const {
        return j <= 0 ? base - 1 : j <= n ? keep[j - 1] : 0;
    }
};

template <bool kQuant>
__global__ void __launch_bounds__(kMoveThreads, 2) compact_kernel(const CompactParams p, int lgw) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_bad;  // first entry of the list that is out of order or out of range
    griddep_wait();
    griddep_launch_dependents();
    const int s = blockIdx.y, tid = threadIdx.x;
    const int k0 = p.keep_start[s], k1 = p.keep_start[s + 1], base = p.base[s], ctx = p.ctx_lens[s];
    if (k0 < 0 || k1 < k0 || k1 > p.T || base < 0 || ctx < 0 || ctx > (int64_t)p.MB << p.lgB) {
        if (blockIdx.x == 0 && tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
        return;
    }
    const KeepList list = {p.keep + k0, p.tables + (int64_t)s * p.MB, k1 - k0, base, ctx, p.lgB, p.NB};
    const int n = list.n, B1 = (1 << p.lgB) - 1, runs = kQuant ? p.cols / p.run : 0;
    if (tid == 0) s_bad = INT_MAX;
    __syncthreads();

    if (kQuant && (int)blockIdx.x < runs) {
        // Scale bytes, one CTA per (head, K or V): a thread per token, its bytes in registers over the barrier.
        constexpr int kU = 4;
        auto place = [&](int row) -> int64_t {
            return (((int64_t)(row >> p.lgB) * runs + blockIdx.x) << p.lgB) + (row & B1);
        };
        for (int64_t j0 = 0; j0 < n; j0 += kMoveThreads * kU) {
            int2 row[kU];
            uint8_t v[kU];
            int src[kU], sb[kU], db[kU];
            bool go[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int64_t j = j0 + u * kMoveThreads + tid;
                src[u] = list.source(j);
                go[u] = list.moves(j, src[u], list.source_before(j), &s_bad);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                sb[u] = go[u] ? list.block_from(src[u]) : 0;
                db[u] = go[u] ? list.block_to(j0 + u * kMoveThreads + tid) : 0;
            }
#pragma unroll
            for (int u = 0; u < kU; ++u)
                row[u] = go[u] ? list.rows(j0 + u * kMoveThreads + tid, src[u], sb[u], db[u], p.err)
                               : make_int2(-1, -1);
#pragma unroll
            for (int u = 0; u < kU; ++u) v[u] = row[u].x >= 0 ? p.scales[place(row[u].x)] : (uint8_t)0;
            __syncthreads();
            const int bad = s_bad;
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (row[u].x >= 0 && j0 + u * kMoveThreads + tid < bad) p.scales[place(row[u].y)] = v[u];
            if (bad < j0 + kMoveThreads * kU) {
                if (blockIdx.x == 0 && tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
                return;
            }
            __syncthreads();  // (a thread ahead may lower s_bad for its next tokens)
        }
        return;
    }

    const int per = kMoveThreads >> lgw, chunk = per * kMoveUnroll, tok = tid >> lgw;
    const int c = (((int)blockIdx.x - runs) << lgw) + (tid & ((1 << lgw) - 1));
    const bool mine = c < p.cols;
    const int64_t col = (int64_t)(c / p.run) * p.run_step + (int64_t)(c % p.run) * 16;
    const uint32_t ring = smem_addr(smem) + tid * 16;  // this thread's vectors: kMoveThreads vectors apart
    int2* s_row = reinterpret_cast<int2*>(smem + (size_t)kMoveStages * kMoveThreads * kMoveUnroll * 16);
    auto place = [&](int row) -> int64_t {
        return (int64_t)(row >> p.lgB) * p.block_bytes + (row & B1) * p.token_step + col;
    };
    auto vector = [&](int stage, int u) -> uint32_t {
        return ring + (uint32_t)(stage * kMoveUnroll + u) * (kMoveThreads * 16);
    };
    auto row_of = [&](int64_t j) -> int2 { return s_row[j & (2 * kSpan - 1)]; };
    auto copy = [&](int64_t j0, int stage) {  // the chunk from token j0 on
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int src = row_of(j0 + u * per + tok).x;
            if (src >= 0 && mine) copy_async16(vector(stage, u), p.data + place(src));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int src[kLook], sb[kLook], db[kLook];
    bool go[kLook];
    int before[kLook];
    auto read_entries = [&](int64_t j0) {  // of the span from token j0 on
#pragma unroll
        for (int x = 0; x < kLook; ++x) {
            src[x] = list.source(j0 + x * kMoveThreads + tid);
            before[x] = list.source_before(j0 + x * kMoveThreads + tid);
        }
    };
    auto read_blocks = [&](int64_t j0) {
#pragma unroll
        for (int x = 0; x < kLook; ++x) {
            const int64_t j = j0 + x * kMoveThreads + tid;
            go[x] = list.moves(j, src[x], before[x], &s_bad);
            sb[x] = go[x] ? list.block_from(src[x]) : 0;
            db[x] = go[x] ? list.block_to(j) : 0;
        }
    };
    auto write_rows = [&](int64_t j0) {
#pragma unroll
        for (int x = 0; x < kLook; ++x) {
            const int64_t j = j0 + x * kMoveThreads + tid;
            s_row[j & (2 * kSpan - 1)] = go[x] ? list.rows(j, src[x], sb[x], db[x], p.err) : make_int2(-1, -1);
        }
    };
    read_entries(0);
    read_blocks(0);
    write_rows(0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMoveStages - 1; ++i) copy(i * chunk, i);
    int stage = 0;
    for (int64_t j0 = 0; j0 < n; j0 += chunk) {
        const int at = (int)j0 & (kSpan - 1);  // in its span
        const int64_t next = j0 - at + kSpan;
        if (next < n) {
            if (at == 0) read_entries(next);
            if (at == chunk) read_blocks(next);
        }
        if (at == 2 * chunk) {
            if (next >= n) {
#pragma unroll
                for (int x = 0; x < kLook; ++x) go[x] = false;  // the copies run past the list's end
            }
            write_rows(next);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kMoveStages - 2) : "memory");
        __syncthreads();  // the chunk is read
        const int64_t bad = s_bad;
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int64_t j = j0 + u * per + tok;
            const int2 row = row_of(j);
            if (row.x < 0 || !mine || j >= bad) continue;
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(vector(stage, u))
                         : "memory");
            *reinterpret_cast<uint4*>(p.data + place(row.y)) = v;
        }
        if (bad < j0 + chunk) {
            if (blockIdx.x == 0 && tid == 0) flag_error(p.err, PA_DEV_ERR_CTX);
            break;
        }
        copy(j0 + (kMoveStages - 1) * chunk, stage == 0 ? kMoveStages - 1 : stage - 1);
        if (++stage == kMoveStages) stage = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
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
    // Columns per CTA: a chunk no longer than the lists are on average, and, as far as two sectors per token allow, two
    // CTAs per SM.
    const int64_t mean = a.T / a.N;
    int lgw = kMinLgw;
    while (lgw < kMaxLgw && (1 << lgw) < p.cols &&
           ((int64_t)(kMoveThreads >> lgw) * kMoveUnroll > mean || ((int64_t)p.cols * a.N) >> lgw > kMoveCtas))
        ++lgw;
    const int64_t gx = ((p.cols + (1 << lgw) - 1) >> lgw) + (quant ? p.cols / p.run : 0);
    auto kern = quant ? compact_kernel<true> : compact_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMoveSmem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(compact)");
    e = launch_kernel(kern, dim3((unsigned)gx, (unsigned)a.N), dim3(kMoveThreads), kMoveSmem, a.stream, p, lgw);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "compact launch");
}

}  // namespace pa
