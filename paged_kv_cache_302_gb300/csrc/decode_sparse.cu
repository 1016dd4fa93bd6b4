// decode_sparse.cu -- single-token decode attention over listed blocks of each (sequence, KV head).
//
// Two kernels per call.  attend_sparse_kernel: every row -- one (sequence, KV head) with its list -- counts as many
// units of 32 listed tokens as its list can hold of its context; the units of all rows in order are cut into runs of
// equal length, one run per CTA, so that every CTA reads as much as the others whatever the batch.  A row that lies
// inside a run is finished there; of a row that a cut divides, each CTA writes its part's maximum, sum and output, and
// join_sparse_kernel joins them.  A CTA is two warps.  Warp 0 (producer) finds the run, walks the lists, drops padding
// and bad entries, and streams the blocks' K and V of the row's head through a ring of shared-memory stages of 32
// tokens by TMA, the row's query heads with its first stage.  Warp 1 (consumer) computes with mma.sync m16n8k16 (tokens
// on M, the <= 8 query heads of the KV head on N) and an online softmax in base 2, over 16-bit rows as
//     S^T = K Q^T,  O^T += V^T P^T  with P in a high and a low 16-bit part,
// and over e4m3 rows (quant.cuh) with rows converted to fp16 in registers, exactly, as
//     raw = K8 q'^T,  y = raw 2^ek c + ev,  p = 2^(y - M),  O += p V8,  l += p 2^-ev:
// the exponent of V's scale inside the maximum keeps p <= 1 next to the e4m3 values it weighs, |ev| <= 40 keeps l in
// fp32.  q' is the query in fp16, a bf16 one scaled row by row with a power of two.
// Short lists and few rows take one kernel instead, a cluster of CTAs per row (below).
//
// Bound by memory, 4 D (2 D + 2) bytes per listed token and head: 64 sequences of 128 blocks of 16 tokens, 8 heads (528
// MB) take 83-86 us, 6.3 TB/s, a plain kernel with a CTA per row 556; 16 of 256 blocks over e4m3 rows (136 MB) 31.6 us,
// 4.3 TB/s: five of them pass before the first block arrives (lengths, list, block table, block), three in the join.
// One sequence of 64 blocks, by clusters: 6.5 us on the device.
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "quant.cuh"
#include "runs.cuh"
#include "tensor_map.h"

namespace pa {

constexpr int kUnitTok = 32;       // tokens of a unit: one pipeline stage
constexpr int kSpThreads = 64;
// No more runs than one for this many units: few long rows are not cut into more parts than the join is worth.  8 rows
// of 4096 tokens, D = 128, e4m3: 12.9 us, 14.2 with six, 21.0 with one; of 8192 tokens 17.2, 16.6, 22.8.
constexpr int kMinRun = 4;

// CTAs per SM.  Fewer leave a CTA more stages in flight, more run more consumer chains beside one another: e4m3, D =
// 128, 1024 rows of 2048 tokens 79 us with seven, 81 with six, 86 with eight; 16 bits, D = 128, the same 137 with four,
// 139 with three, 140 with five; e4m3, D = 64, 512 such rows 32 with eight or ten, 34 with nine or seven; 16 bits, D =
// 64, the same 54 with six or seven, 63 with five or eight, but 224 rows of 4096 tokens 44 with six, 232 rows 60 with
// seven.
constexpr int sparse_ctas(bool quant, int D) { return D == 128 ? (quant ? 7 : 4) : quant ? 8 : 6; }
// Of the workspace, whose size is asked without a device: one with more SMs than 152 takes no more CTAs.
constexpr int kSpMaxCtas = 152 * sparse_ctas(true, 64);
// Calls that take a cluster per row: the largest size, up to 8, at which the device holds the clusters of all rows at
// once, provided that a CTA's share of the list is short.  One kernel instead of two, and nothing to find.  By clusters
// against by runs, 256 tokens to a CTA, D = 128: 48 rows over e4m3 12.7 us against 13.9, 232 rows 17.5 against 18.8; 24
// rows over 16 bits 11.5 against 12.7, 128 rows 16.1 against 17.7.  Longer shares pay where the clusters fill seven
// eighths of the device and equal runs have little to gain: 504 rows of 1024 tokens over e4m3 28.8 against 29.7 (312
// such rows 26.9 against 22.1; 504 rows of 2048 even), 72 rows of 8192 tokens over 16 bits 49.3 against 51.7 (24 rows
// of 4096 18.4 against 17.2).
constexpr int kSpMaxCluster = 8;
constexpr int kSpShare = 256;                              // tokens of a CTA's share
constexpr int kSpShareFull16 = 1024, kSpShareFull8 = 512;  // the same on a device that is seven eighths full
constexpr int kJoinWarps = 8;

enum : int { kSpFirst = 1, kSpLast = 2, kSpDone = 4 };

// What the consumer needs to know of a stage.
struct __align__(16) SpMeta {
    int row;        // sequence * H_kv + KV head
    int flags;
    uint32_t seen;  // bit t: token t of the stage takes part
    int part;       // where the row's part goes (-1: the row is whole, the output itself)
};

struct SpParams {
    void* out;
    int out_dtype;
    const void* q;
    const uint8_t* scales;
    const int32_t* tables;
    const int32_t* ctx_lens;
    const int32_t* selected;
    int top_k, N, H_kv, G, MB, NB;
    int ctas;          // CTAs that the workspace has parts for
    int64_t cap;       // tokens a block-table row holds
    float scale_log2;
    int2* cuts;        // [N * H_kv]: first and last CTA of a divided row, (-1, -1) for a whole one
    float* part_m;     // [2 * CTAs][G]: part 2 c of the row that CTA c continues, 2 c + 1 of the one it leaves open
    float* part_l;
    float* part_acc;   // [2 * CTAs][G][D]
    int cluster;       // CTAs per row where the parts are joined over a cluster
    uint64_t wait_ns;
    int* err;
};

// Ring geometry: per stage the rows (1024-byte aligned for the swizzle), scale bytes (e4m3), the query heads, the
// description, two barriers.
template <bool kQuant, int D>
struct SpGeo {
    static constexpr uint32_t kSlot = kUnitTok * D * (kQuant ? 2 : 4);
    static constexpr uint32_t kScales = kQuant ? kUnitTok * 2 : 0;
    static constexpr uint32_t kQ = kMaxGroup * D * 2;
    static constexpr uint32_t kPerStage = kSlot + kScales + kQ + sizeof(SpMeta) + 16;
    static constexpr int kCtas = sparse_ctas(kQuant, D);
    static constexpr int kStages = (233472 / kCtas - 1024 - 1024 - 16) / (int)kPerStage;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kPerStage + 16;
    static_assert((2 * kMaxGroup + kMaxGroup * D) * sizeof(float) <= kSlot, "a part fits a stage");
    static_assert(kStages >= 2 && kCtas * (kSmem + 1024) <= 233472, "the CTAs of an SM fit its shared memory");
};

__device__ __forceinline__ uint4 sp_lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 sp_lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t sp_lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Units of every row of a sequence of ctx tokens (0: the context is out of range).
template <int LGB>
__device__ __forceinline__ int row_units(const SpParams& p, int ctx) {
    constexpr int kPerUnit = kUnitTok >> LGB;  // (in blocks: a list's tokens may be 2^31)
    if (ctx < 1 || ctx > p.cap) return 0;
    const int nb = (ctx + (1 << LGB) - 1) >> LGB;
    return (min(nb, p.top_k) + kPerUnit - 1) / kPerUnit;
}

// The run of a CTA, walked chunk by chunk of at most 32 list entries.  Everything is uniform over the warp.
template <int LGB>
struct Run {
    int s, h;      // row
    int units;     // of a row of this sequence
    int ctx;
    int unit;      // the row's first
    int left;      // units of the run behind this segment
    int e, e_end;  // list entries of the segment still to come
    int part;
    bool first;    // the next chunk is the segment's first

    // Enters the segment that starts at unit j of the row and sets the row's cuts.
    __device__ __forceinline__ void enter(const SpParams& p, int j, const Cut& cut) {
        constexpr int kPerUnit = kUnitTok >> LGB;
        const int cta = blockIdx.x;
        const bool to_end = units - j <= left;
        const int j1 = to_end ? units : j + left;
        part = j > 0 ? 2 * cta : to_end ? -1 : 2 * cta + 1;
        e = j * kPerUnit;
        e_end = to_end ? p.top_k : j1 * kPerUnit;  // (what stands behind the last unit is padding, or counts here)
        first = true;
        if (j == 0 && (threadIdx.x & 31) == 0)
            p.cuts[(int64_t)s * p.H_kv + h] = to_end ? make_int2(-1, -1) : make_int2(cta, cut.run_of(unit + units - 1));
        left -= j1 - j;
    }
};

// kCluster: a cluster of CTAs per row instead, each with an equal part of the list; the parts are joined over the
// cluster's shared memory.
template <typename T, bool kQuant, int D, int LGB, bool kCluster>
__global__ void __launch_bounds__(kSpThreads) attend_sparse_kernel(const __grid_constant__ CUtensorMap tm,
                                                                   const SpParams p) {
    using Geo = SpGeo<kQuant, D>;
    constexpr int nstage = Geo::kStages, B = 1 << LGB, BPS = kUnitTok / B;
    constexpr uint32_t kBox = 2u * B * D * (kQuant ? 1 : 2);  // bytes of a block's K and V of one head
    constexpr int NSUB = kUnitTok / 16, NT = D / 16, DH = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sc_g = base + (size_t)nstage * Geo::kSlot;
    uint8_t* q_g = sc_g + (size_t)nstage * Geo::kScales;
    SpMeta* meta = reinterpret_cast<SpMeta*>(q_g + (size_t)nstage * Geo::kQ);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(meta + nstage);
    uint64_t* empty_bar = full_bar + nstage;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(empty_bar + nstage);
    const uint32_t slots_s = smem_addr(base), sc_s = smem_addr(sc_g), q_s = smem_addr(q_g);
    const uint32_t full_s = smem_addr(full_bar), empty_s = smem_addr(empty_bar);

    if (threadIdx.x == 0) {
        for (int i = 0; i < nstage; ++i) {
            mbar_init(full_s + 8 * i, 1);
            mbar_init(empty_s + 8 * i, 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
        // The SM hands a CTA's two warps neighbouring slots: the CTAs in every other group of four slots swap the
        // roles, so that the consumers spread over its four schedulers.
        uint32_t wid;
        asm volatile("mov.u32 %0, %%warpid;" : "=r"(wid));
        abort_flag[1] = (int)(wid >> 2 & 1);
        prefetch_tmap(&tm);
    }
    __syncthreads();
    const bool producer = (int)(threadIdx.x >> 5) == abort_flag[1];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const float NEG_INF = -INFINITY;
    // This CTA's part of its row for the cluster's join: maxima and sums of the query heads, then their outputs.  It
    // lies in the ring, which is empty by then: a cluster's CTA has one segment.
    float* share = reinterpret_cast<float*>(base);
    // A cluster's CTA takes an equal share of whole units, of the list as it lies (an empty share is a list of
    // padding). Its first entries are on their way beside the length.
    [[maybe_unused]] int share0 = 0, share1 = 0, entry0 = -1;
    if constexpr (kCluster) {
        const int row = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
        const int len = ((p.top_k + p.cluster - 1) / p.cluster + BPS - 1) / BPS * BPS;
        share0 = min(rank * len, p.top_k);
        share1 = min(share0 + len, p.top_k);
        if (producer && share0 + lane < share1) entry0 = p.selected[(int64_t)row * p.top_k + share0 + lane];
        const int ctx = p.ctx_lens[row / p.H_kv];
        if (ctx < 1 || ctx > p.cap) {  // (the whole cluster returns)
            if (threadIdx.x == 0 && blockIdx.x % (p.cluster * p.H_kv) == 0) flag_error(p.err, PA_DEV_ERR_CTX);
            return;
        }
    }

    auto produce = [&]() {
        // ------------------------------------------------------------------ producer warp
        Run<LGB> run;
        const auto units_of = [&](int s) { return row_units<LGB>(p, p.ctx_lens[s]); };
        const RowScan<decltype(units_of)> scan(units_of, kCluster ? 0 : p.N, p.H_kv);
        const int total = kCluster ? 1 : scan.total();
        const int ctas = min((int)gridDim.x, (total - 1) / kMinRun + 1);
        const Cut cut(total, ctas);
        run.e = run.e_end = run.left = 0;
        run.first = false;
        if constexpr (kCluster) {
            const int row = blockIdx.x / p.cluster;
            run.s = row / p.H_kv;
            run.h = row % p.H_kv;
            run.ctx = p.ctx_lens[run.s];
            run.e = share0;
            run.e_end = share1;
            run.part = 0;
            run.first = true;
        } else {
            if (blockIdx.x == 0) {
                for (int s = lane; s < p.N; s += 32)
                    if (units_of(s) == 0) flag_error(p.err, PA_DEV_ERR_CTX);
            }
            if ((int)blockIdx.x < ctas && total > 0) {
                const int u0 = cut.start(blockIdx.x);
                run.left = cut.start(blockIdx.x + 1) - u0;
                int first;
                run.s = scan.find(u0, run.units, first);
                run.ctx = p.ctx_lens[run.s];
                run.h = (u0 - first) / run.units;
                run.unit = first + run.h * run.units;
                run.enter(p, u0 - run.unit, cut);
            }
        }
        const uint64_t pol = policy_evict_first();
        int slot = 0;
        uint32_t ephase = 0;
        int narm = 0;  // stages armed so far (stage i's k-th arm completes phase k of full_bar[i])
        bool ok = true;

        // One stage: the blocks of lanes src[0 .. nb-1] (their physical blocks in `blk`, tokens that count in `nv`).
        auto arm = [&](int row, int h, int part, bool first, bool last, int nb, int blk, int nv, unsigned from) {
            if (lane == 0) ok = mbar_wait_bounded(empty_s + 8 * slot, ephase ^ 1, abort_flag, p.wait_ns);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) return;
            ++narm;  // armed below: expect_tx and every copy of the stage, with no wait in between
            const uint32_t bar = full_s + 8 * slot;
            // block b of the stage: the b-th set bit of `from`; lane b copies its rows, lane 16 + b its scale bytes
            const int b = lane & 15;
            unsigned rest = from;
            uint32_t seen = 0;
            int mine = 0;
#pragma unroll
            for (int i = 0; i < BPS; ++i) {
                const int src = rest ? __ffs(rest) - 1 : 0;
                rest &= rest - 1;
                const int n = __shfl_sync(0xffffffffu, nv, src), e = __shfl_sync(0xffffffffu, blk, src);
                if (i < nb) seen |= (n < 32 ? (1u << n) - 1u : 0xffffffffu) << (i * B % 32);
                if (i == b) mine = e;
            }
            if (lane == 0) {
                SpMeta m;
                m.row = row;
                m.flags = (first ? kSpFirst : 0) | (last ? kSpLast : 0);
                m.seen = seen;
                m.part = part;
                meta[slot] = m;
                const uint32_t q_bytes = first ? (uint32_t)p.G * D * 2 : 0u;
                mbar_arrive_expect_tx(bar, (uint32_t)nb * (kBox + (kQuant ? 2 * B : 0)) + q_bytes);
                if (first)
                    bulk_load(q_s + slot * Geo::kQ, static_cast<const T*>(p.q) + (int64_t)row * p.G * D, q_bytes, bar);
            }
            __syncwarp();
            if (b < nb) {
                if constexpr (kQuant) {
                    if (lane < 16)
                        tma_load_3d(slots_s + slot * Geo::kSlot + b * kBox, &tm, bar, 0, 0, mine * p.H_kv + h, pol);
                    else
                        bulk_load(sc_s + slot * Geo::kScales + b * 2 * B,
                                  p.scales + ((int64_t)mine * p.H_kv + h) * (2 * B), 2 * B, bar);
                } else if (lane < 16) {
                    tma_load_5d(slots_s + slot * Geo::kSlot + b * kBox, &tm, bar, 0, mine * B, 0, h, 0, pol);
                }
            }
            if (++slot == nstage) {
                slot = 0;
                ephase ^= 1;
            }
        };

        // A chunk: up to 32 entries of a segment's list, one per lane.
        struct Chunk {
            int row, s, h, part, ctx, entry;  // entry: this lane's
            bool first, last, some;
        };
        auto next_chunk = [&]() -> Chunk {
            Chunk c;
            c.some = false;
            c.row = c.s = c.h = c.part = c.ctx = 0;
            c.entry = -1;
            c.first = c.last = false;
            if (run.e >= run.e_end && !(kCluster && run.first)) {
                if (run.left <= 0) return c;
                run.unit += run.units;
                if (++run.h == p.H_kv) {
                    run.h = 0;
                    do {  // (the run has units left, so a sequence follows)
                        if (++run.s >= p.N) {
                            run.left = 0;
                            return c;
                        }
                        run.ctx = p.ctx_lens[run.s];
                        run.units = row_units<LGB>(p, run.ctx);
                    } while (run.units == 0);
                }
                run.enter(p, 0, cut);
            }
            c.some = true;
            c.s = run.s;
            c.h = run.h;
            c.row = run.s * p.H_kv + run.h;
            c.part = run.part;
            c.ctx = run.ctx;
            c.first = run.first;
            const int n = min(32, run.e_end - run.e);
            if (kCluster && run.first)
                c.entry = entry0;
            else if (lane < n)
                c.entry = p.selected[(int64_t)c.row * p.top_k + run.e + lane];
            run.first = false;
            run.e += n;
            c.last = run.e >= run.e_end;
            return c;
        };
        // physical block of this lane's entry, -1 where there is none; nv its tokens
        auto look_up = [&](const Chunk& c, int& nv) -> int {
            nv = 0;
            if (!c.some || c.entry < 0) return -1;
            if (c.entry >= min((c.ctx + B - 1) >> LGB, p.MB)) return -1;
            nv = min(B, c.ctx - (c.entry << LGB));
            return p.tables[(int64_t)c.s * p.MB + c.entry];
        };
        Chunk cur = next_chunk();
        int nv, blk = look_up(cur, nv);
        Chunk nxt = next_chunk();
        bool open = false;  // the segment's first stage is out
        while (cur.some && ok) {
            // the next chunk's blocks and the entries of the one after that are on their way while this one streams
            int nv1;
            const int blk1 = look_up(nxt, nv1);
            const Chunk after = next_chunk();
            const bool good = (unsigned)blk < (unsigned)p.NB;
            if (cur.entry >= 0 && !good) flag_error(p.err, PA_DEV_ERR_BLOCK);
            if (cur.first) open = false;
            unsigned from = __ballot_sync(0xffffffffu, good);
            if (from == 0 && cur.last) {
                arm(cur.row, cur.h, cur.part, !open, true, 0, blk, nv, 0);  // a segment always ends with a stage
            }
            while (from && ok) {
                const int n = min(BPS, __popc(from));
                unsigned rest = from;
#pragma unroll
                for (int i = 0; i < BPS; ++i) rest &= rest - 1;
                arm(cur.row, cur.h, cur.part, !open, cur.last && rest == 0, n, blk, nv, from);
                open = true;
                from = rest;
            }
            cur = nxt;
            blk = blk1;
            nv = nv1;
            nxt = after;
        }
        if constexpr (!kCluster) {
            // a wait that ran out: the run's other rows still get their cuts, which the join reads
            while (!ok && nxt.some) nxt = next_chunk();
        }
        if (ok && lane == 0) {
            ok = mbar_wait_bounded(empty_s + 8 * slot, ephase ^ 1, abort_flag, p.wait_ns);
            if (ok) {
                meta[slot].flags = kSpDone;
                mbar_arrive(full_s + 8 * slot);
                ++narm;
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (lane == 0) {
            if (!ok) {
                flag_error(p.err, PA_DEV_ERR_TIMEOUT);
                *abort_flag = 1;
            }
            // Copies land in this CTA's shared memory, so it may not exit while one is in flight: wait for the phase
            // that the last arm of each stage completes (each earlier arm was consumed before the next).
            for (int i = 0; i < nstage && i < narm; ++i) {
                const int m = (narm - 1 - i) / nstage;
                mbar_wait_bounded(full_s + 8 * i, (uint32_t)(m & 1), nullptr, kWaitLimitNs);
            }
        }
    };

    // ---------------------------------------------------------------------- consumer warp
    auto consume = [&]() {
        const int g4 = lane >> 2, t4 = lane & 3;
        float O[NT][4];
        uint32_t qf[NT][2];
        float m0 = NEG_INF, m1 = NEG_INF, l0 = 0.f, l1 = 0.f;
        float c0 = p.scale_log2, c1 = p.scale_log2;  // raw scores of heads 2 t4, 2 t4 + 1 to base-2 units
        int slot = 0;
        uint32_t fphase = 0;

        // Addresses.  e4m3: the thread holds token rt (and rt + 8) of each tile of K, in an order of the 8 rows that
        // spreads the 16- and 8-byte reads of both products over all banks under the stage's swizzle, and of V^T the
        // elements from d0 on of tokens va, vb (and + 8), the ones whose probabilities the score product left in rows 2
        // t4 and 2 t4 + 1.  16 bit: ldmatrix rows.
        auto row_token = [](int i) -> int {
            return D == 128 ? ((i >> 1) | ((i & 1) << 2)) : (int)((0x65742130u >> (4 * i)) & 7u);
        };
        const int rt = kQuant ? row_token(g4) : g4;
        auto qtok_ofs = [](int n) -> uint32_t { return (uint32_t)((n >> LGB) * 2 * B + (n & (B - 1))) * D; };
        auto qsc_ofs = [](int n) -> uint32_t { return (uint32_t)((n >> LGB) * 2 * B + (n & (B - 1))); };
        const uint32_t qk_ofs = D == 128 ? rt * 128 + ((t4 ^ rt) << 4) : rt * 64 + ((t4 ^ (rt >> 1 & 3)) << 4);
        const int va = row_token(2 * t4), vb = row_token(2 * t4 + 1);
        const int vch = D == 128 ? row_token(g4) : g4;
        const int d0 = vch * 2 * NT;
        auto qv_ofs = [&](int tok) -> uint32_t {
            return (uint32_t)(B * D) + (D == 128 ? tok * 128 + ((vch ^ tok) << 4)
                                                 : tok * 64 + (((vch >> 1) ^ (tok >> 1 & 3)) << 4) + ((vch & 1) << 3));
        };
        uint32_t kofs[NSUB][DH], kx[NSUB][DH], vofs[NSUB][DH], vx[NSUB][DH];
        if constexpr (!kQuant) {
            const int k_tok = (lane & 7) + ((lane >> 3) & 1) * 8, k_hi = lane >> 4;
            const int v_tok = (lane & 7) + ((lane >> 4) & 1) * 8, v_hi = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < NSUB; ++j)
#pragma unroll
                for (int dh = 0; dh < DH; ++dh) {
                    int tok = 16 * j + k_tok;
                    int row = (tok >> LGB) * (2 * DH * B) + dh * B + (tok & (B - 1));
                    kofs[j][dh] = (uint32_t)row * 128;
                    kx[j][dh] = (uint32_t)((k_hi ^ (row & 7)) << 4);
                    tok = 16 * j + v_tok;
                    row = (tok >> LGB) * (2 * DH * B) + (DH + dh) * B + (tok & (B - 1));
                    vofs[j][dh] = (uint32_t)row * 128;
                    vx[j][dh] = (uint32_t)((v_hi ^ (row & 7)) << 4);
                }
        }

        while (true) {
            if (!mbar_wait_bounded(full_s + 8 * slot, fphase, abort_flag, p.wait_ns)) {
                if (lane == 0) {
                    flag_error(p.err, PA_DEV_ERR_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            const SpMeta mt = meta[slot];
            if (mt.flags & kSpDone) break;
            const uint32_t kv = slots_s + slot * Geo::kSlot, scb = sc_s + slot * Geo::kScales;
            if (mt.flags & kSpFirst) {
                if constexpr (kQuant) {
                    float a = 0.f;
                    const uint32_t qrow = q_s + slot * Geo::kQ + g4 * D * 2 + t4 * 32;
#pragma unroll
                    for (int w = 0; w < NT; ++w) {
                        const uint2 x = g4 < p.G ? sp_lds64(qrow + (w >> 2) * 128 + (w & 3) * 8) : make_uint2(0, 0);
                        qf[w][0] = x.x;
                        qf[w][1] = x.y;
                        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                            const float2 f0 = Mma<T>::unpack(x.x), f1 = Mma<T>::unpack(x.y);
                            a = fmaxf(a, fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))));
                        }
                    }
                    c0 = c1 = p.scale_log2;
                    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                        // The row's largest magnitude goes to [2^14, 2^15): elements down to 2^-28 of it are normal
                        // fp16 numbers and exact, smaller ones are off by at most 2^-40 of it.
                        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                        const int ex = (int)(__float_as_uint(a) >> 23) - 127;
                        const int e = ex > 127 || a == 0.f ? 0 : max(ex - 14, -126);
                        const float inv = pow2i(-e);
#pragma unroll
                        for (int w = 0; w < NT; ++w)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float2 f = Mma<T>::unpack(qf[w][i]);
                                qf[w][i] = Mma<__half>::pack(f.x * inv, f.y * inv);
                            }
                        const float up = pow2i(e);
                        c0 *= __shfl_sync(0xffffffffu, up, 8 * t4);  // lane 4 n holds head n's
                        c1 *= __shfl_sync(0xffffffffu, up, 8 * t4 + 4);
                    }
                } else {
                    const uint8_t* qs = q_g + (size_t)slot * Geo::kQ;
#pragma unroll
                    for (int ks = 0; ks < NT; ++ks) {
                        const int d = 16 * ks + 2 * t4;
                        const uint32_t* row = reinterpret_cast<const uint32_t*>(qs + ((size_t)g4 * D + d) * 2);
                        qf[ks][0] = g4 < p.G ? row[0] : 0u;
                        qf[ks][1] = g4 < p.G ? row[4] : 0u;
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.f;
                m0 = m1 = NEG_INF;
                l0 = l1 = 0.f;
            }
            // the running maximum moves to n0, n1
            auto rescale = [&](float n0, float n1) {
                const float a0 = fast_exp2(m0 - n0), a1 = fast_exp2(m1 - n1);
                m0 = n0;
                m1 = n1;
                if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        O[i][0] *= a0;
                        O[i][1] *= a1;
                        O[i][2] *= a0;
                        O[i][3] *= a1;
                    }
                    l0 *= a0;
                    l1 *= a1;
                }
            };
            // one copy for whole stages, without a branch between the tiles, and one for the others
            auto stage = [&](auto full_c) {
                constexpr bool kFull = decltype(full_c)::value;
                float y[NSUB][4];                   // scores in base-2 units
                [[maybe_unused]] float iv[NSUB][2]; // 2^-ev of tokens rt and rt + 8 (e4m3)
                float top0 = NEG_INF, top1 = NEG_INF;
#pragma unroll
                for (int j = 0; j < NSUB; ++j) {
                    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (kQuant) {
#pragma unroll
                        for (int c = 0; c < NT / 4; ++c) {
                            const uint4 lo = sp_lds128(kv + qtok_ofs(16 * j) + (qk_ofs ^ (c * 64)));
                            const uint4 hi = sp_lds128(kv + qtok_ofs(16 * j + 8) + (qk_ofs ^ (c * 64)));
                            const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                Mma<__half>::run(w & 1 ? b : a, e4m3x2_to_f16x2(wl[w]), e4m3x2_to_f16x2(wh[w]),
                                                 e4m3x2_to_f16x2(wl[w] >> 16), e4m3x2_to_f16x2(wh[w] >> 16),
                                                 qf[4 * c + w][0], qf[4 * c + w][1]);
                        }
                    } else {
#pragma unroll
                        for (int ks = 0; ks < NT; ++ks) {
                            const int dh = ks >> 2;
                            const uint32_t addr = kv + kofs[j][dh] + ((uint32_t)(((ks & 3) * 2) << 4) ^ kx[j][dh]);
                            uint32_t r0, r1, r2, r3;
                            ldmatrix_x4(addr, r0, r1, r2, r3);
                            Mma<T>::run(ks & 1 ? b : a, r0, r1, r2, r3, qf[ks][0], qf[ks][1]);
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int tok = 16 * j + 8 * half + rt;
                        float x0 = a[2 * half] + b[2 * half], x1 = a[2 * half + 1] + b[2 * half + 1], add = 0.f;
                        if constexpr (kQuant) {
                            const uint32_t at = scb + qsc_ofs(16 * j + 8 * half) + rt;
                            const float fk = pow2i(scale_of((int)sp_lds8(at)));
                            const int ev = scale_of((int)sp_lds8(at + B));
                            x0 *= fk;  // (before the query's factor, which may be as large as fp32 allows)
                            x1 *= fk;
                            add = (float)ev;
                            iv[j][half] = pow2i(-ev);
                        }
                        const bool in = kFull || (mt.seen >> tok & 1u);
                        y[j][2 * half] = in ? fmaf(x0, c0, add) : NEG_INF;
                        y[j][2 * half + 1] = in ? fmaf(x1, c1, add) : NEG_INF;
                    }
                    top0 = fmaxf(top0, fmaxf(y[j][0], y[j][2]));
                    top1 = fmaxf(top1, fmaxf(y[j][1], y[j][3]));
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
                    top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
                }
                rescale(fmaxf(m0, top0), fmaxf(m1, top1));
                if constexpr (!kQuant) {
                    // V rows of tokens that take no part may hold anything (even NaN): they become zeros
                    if (!kFull) {
                        for (int c = lane; c < kUnitTok * DH * 8; c += 32) {
                            const int tok = c / (DH * 8), dh = c / 8 % DH, ch = c & 7;
                            if (mt.seen >> tok & 1u) continue;
                            const int row = (tok >> LGB) * (2 * DH * B) + (DH + dh) * B + (tok & (B - 1));
                            const uint32_t at = kv + (uint32_t)row * 128 + ch * 16;
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int j = 0; j < NSUB; ++j) {
                    // probabilities as a high and a low 16-bit part, transposed into B fragments
                    using P = typename std::conditional<kQuant, __half, T>::type;
                    const float p0 = fast_exp2(y[j][0] - m0), p1 = fast_exp2(y[j][1] - m1);
                    const float p2 = fast_exp2(y[j][2] - m0), p3 = fast_exp2(y[j][3] - m1);
                    if constexpr (kQuant) {
                        l0 = fmaf(p0, iv[j][0], fmaf(p2, iv[j][1], l0));
                        l1 = fmaf(p1, iv[j][0], fmaf(p3, iv[j][1], l1));
                    } else {
                        l0 += p0 + p2;
                        l1 += p1 + p3;
                    }
                    const uint32_t h01 = Mma<P>::pack(p0, p1), h23 = Mma<P>::pack(p2, p3);
                    const float2 f01 = Mma<P>::unpack(h01), f23 = Mma<P>::unpack(h23);
                    const uint32_t lo01 = Mma<P>::pack(p0 - f01.x, p1 - f01.y);
                    const uint32_t lo23 = Mma<P>::pack(p2 - f23.x, p3 - f23.y);
                    const uint32_t bh0 = movmatrix_trans(h01), bh1 = movmatrix_trans(h23);
                    const uint32_t bl0 = movmatrix_trans(lo01), bl1 = movmatrix_trans(lo23);
                    if constexpr (kQuant) {
                        uint32_t w[4][NT / 2];  // tokens va, vb, va + 8, vb + 8
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t at = kv + qtok_ofs(16 * j + 8 * (t >> 1)) + qv_ofs(t & 1 ? vb : va);
                            if constexpr (D == 128) {
                                const uint4 x = sp_lds128(at);
                                w[t][0] = x.x;
                                w[t][1] = x.y;
                                w[t][2] = x.z;
                                w[t][3] = x.w;
                            } else {
                                const uint2 x = sp_lds64(at);
                                w[t][0] = x.x;
                                w[t][1] = x.y;
                            }
                            if (!kFull) {  // (as above)
                                const bool in = mt.seen >> (16 * j + 8 * (t >> 1) + (t & 1 ? vb : va)) & 1u;
#pragma unroll
                                for (int i = 0; i < NT / 2; ++i) w[t][i] = in ? w[t][i] : 0u;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < NT / 2; ++i) {
                            // (va, vb) pairs of elements 4 i .. 4 i + 3, then the same of the tokens 8 later
                            const uint32_t u[2] = {__byte_perm(w[0][i], w[1][i], 0x5140),
                                                   __byte_perm(w[0][i], w[1][i], 0x7362)};
                            const uint32_t z[2] = {__byte_perm(w[2][i], w[3][i], 0x5140),
                                                   __byte_perm(w[2][i], w[3][i], 0x7362)};
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t r0 = e4m3x2_to_f16x2(u[k]), r1 = e4m3x2_to_f16x2(u[k] >> 16),
                                               r2 = e4m3x2_to_f16x2(z[k]), r3 = e4m3x2_to_f16x2(z[k] >> 16);
                                Mma<__half>::run(O[2 * i + k], r0, r1, r2, r3, bh0, bh1);
                                Mma<__half>::run(O[2 * i + k], r0, r1, r2, r3, bl0, bl1);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const int dh = i >> 2;
                            const uint32_t addr = kv + vofs[j][dh] + ((uint32_t)(((i & 3) * 2) << 4) ^ vx[j][dh]);
                            uint32_t r0, r1, r2, r3;
                            ldmatrix_x4_trans(addr, r0, r1, r2, r3);
                            Mma<T>::run(O[i], r0, r1, r2, r3, bh0, bh1);
                            Mma<T>::run(O[i], r0, r1, r2, r3, bl0, bl1);
                        }
                    }
                }
            };
            if (mt.seen == 0xffffffffu)
                stage(std::true_type{});
            else if (mt.seen)
                stage(std::false_type{});
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_s + 8 * slot);

            if (mt.flags & kSpLast) {
                float L0 = l0, L1 = l1;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    L0 += __shfl_xor_sync(0xffffffffu, L0, o);
                    L1 += __shfl_xor_sync(0xffffffffu, L1, o);
                }
                const uint64_t keep = policy_evict_last();  // the join reads the parts right after this kernel
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int hd = 2 * t4 + hh;
                    if (hd >= p.G) continue;
                    const float L = hh ? L1 : L0;
                    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;  // an empty list: zeros
                    // element d(i, k): row k of the pair that this thread holds of tile i
                    auto d_of = [&](int i, int k) { return kQuant ? d0 + 2 * i + k : 16 * i + g4 + 8 * k; };
                    if constexpr (kCluster) {
                        if (g4 == 0) {
                            share[hd] = hh ? m1 : m0;
                            share[kMaxGroup + hd] = L;
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            share[2 * kMaxGroup + hd * D + d_of(i, 0)] = O[i][hh];
                            share[2 * kMaxGroup + hd * D + d_of(i, 1)] = O[i][2 + hh];
                        }
                    } else if (mt.part < 0) {
                        const int64_t o = ((int64_t)mt.row * p.G + hd) * D;
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const float v0 = O[i][hh] * inv, v1 = O[i][2 + hh] * inv;
                            if (kQuant && p.out_dtype == PA_F32) {
                                float* to = static_cast<float*>(p.out) + o + d_of(i, 0);
                                *reinterpret_cast<float2*>(to) = make_float2(v0, v1);
                            } else if (kQuant) {
                                T* to = static_cast<T*>(p.out) + o + d_of(i, 0);
                                *reinterpret_cast<uint32_t*>(to) = Mma<T>::pack(v0, v1);
                            } else if (p.out_dtype == PA_F32) {
                                static_cast<float*>(p.out)[o + d_of(i, 0)] = v0;
                                static_cast<float*>(p.out)[o + d_of(i, 1)] = v1;
                            } else {
                                static_cast<T*>(p.out)[o + d_of(i, 0)] = from_float<T>(v0);
                                static_cast<T*>(p.out)[o + d_of(i, 1)] = from_float<T>(v1);
                            }
                        }
                    } else {
                        const int64_t r = (int64_t)mt.part * p.G + hd;
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            st_hint(p.part_acc + r * D + d_of(i, 0), O[i][hh], keep);
                            st_hint(p.part_acc + r * D + d_of(i, 1), O[i][2 + hh], keep);
                        }
                        if (g4 == 0) {
                            st_hint(p.part_m + r, hh ? m1 : m0, keep);
                            st_hint(p.part_l + r, L, keep);
                        }
                    }
                }
            }
            if (++slot == nstage) {
                slot = 0;
                fphase ^= 1;
            }
        }
    };
    if (producer)
        produce();
    else
        consume();

    if constexpr (kCluster) {
        // every CTA of the cluster joins its slice of the row's outputs (every wait before has a limit: all get here)
        __syncwarp();
        cluster_sync();
        const int row = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
        const uint32_t at = smem_addr(share);
        const int n = p.G * D;
        for (int i = rank * kSpThreads + threadIdx.x; i < n; i += p.cluster * kSpThreads) {
            const int g = i / D;
            float m[kSpMaxCluster], M = NEG_INF, L = 0.f, o = 0.f;
#pragma unroll
            for (int c = 0; c < kSpMaxCluster; ++c) {
                m[c] = c < p.cluster ? ld_cluster(at + 4 * g, c) : NEG_INF;
                M = fmaxf(M, m[c]);
            }
            if (M > NEG_INF) {
#pragma unroll
                for (int c = 0; c < kSpMaxCluster; ++c) {
                    if (c >= p.cluster) continue;
                    const float f = fast_exp2(m[c] - M);
                    L += f * ld_cluster(at + 4 * (kMaxGroup + g), c);
                    o += f * ld_cluster(at + 4 * (2 * kMaxGroup + i), c);
                }
                o /= L;
            } else {  // no score, or none that is a number: zeros, or NaN like the sums
                for (int c = 0; c < p.cluster; ++c) o += ld_cluster(at + 4 * (kMaxGroup + g), c);
            }
            const int64_t to = (int64_t)row * n + i;
            if (p.out_dtype == PA_F32)
                static_cast<float*>(p.out)[to] = o;
            else
                static_cast<T*>(p.out)[to] = from_float<T>(o);
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its share
    }
}

// One warp per (row, query head): the parts of a divided row, in order.
template <typename OutT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_sparse_kernel(const SpParams p) {
    constexpr int V = D / 32, kBatch = 8;
    // (Without an early start for the next kernel: what comes in beside CTAs of this one lies so in the SM's shared
    // memory that its last CTA may find no room until its first one ends.  Calls after calls over 1024 rows of 2048
    // tokens, 16 bits, D = 128: 137 us, 162 with it; 8 rows 0.2 us more.)
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (r >= (int64_t)p.N * p.H_kv * p.G) return;
    const int64_t row = r / p.G;
    const int g = (int)(r - row * p.G);
    const int ctx = p.ctx_lens[row / p.H_kv];
    if (ctx < 1 || ctx > p.cap) return;
    const int2 cut = p.cuts[row];
    // A whole row.  (Or no cuts at all, should the lengths have changed since: no part is looked up behind the
    // workspace's.)
    if (cut.x < 0 || cut.y < cut.x || cut.y >= p.ctas) return;
    const int n = cut.y - cut.x + 1;
    auto part = [&](int i) -> int64_t { return (int64_t)(2 * (cut.x + i) + (i == 0 ? 1 : 0)) * p.G + g; };
    float M = -INFINITY, L = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
    for (int i0 = 0; i0 < n; i0 += kBatch) {
        float a[kBatch][V];
        const float m = lane < kBatch && i0 + lane < n ? p.part_m[part(i0 + lane)] : -INFINITY;
        const float l = lane < kBatch && i0 + lane < n ? p.part_l[part(i0 + lane)] : 0.f;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
#pragma unroll
            for (int v = 0; v < V; ++v) a[j][v] = 0.f;
            if (i0 + j < n) {
                const float* src = p.part_acc + part(i0 + j) * D + lane * V;
                if constexpr (V == 4)
                    *reinterpret_cast<float4*>(a[j]) = *reinterpret_cast<const float4*>(src);
                else
                    *reinterpret_cast<float2*>(a[j]) = *reinterpret_cast<const float2*>(src);
            }
        }
        float top = m;
#pragma unroll
        for (int k = kBatch / 2; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        top = fmaxf(M, __shfl_sync(0xffffffffu, top, 0));
        if (top == -INFINITY) {  // only parts without a score so far, or with none that is a number: sums of 0 or NaN
#pragma unroll
            for (int j = 0; j < kBatch; ++j) L += __shfl_sync(0xffffffffu, l, j);
            continue;
        }
        const float f = fast_exp2(M - top), w = fast_exp2(m - top);
        M = top;
        L *= f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= f;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            L += wj * __shfl_sync(0xffffffffu, l, j);
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] += wj * a[j][v];
        }
    }
    const float inv = M > -INFINITY ? 1.f / L : L;
    OutT* out = static_cast<OutT*>(p.out) + r * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = from_float<OutT>(o[v] * inv);
}

// ----------------------------------------------------------------------------- host side

struct SparseLayout {
    size_t m, l, acc, total;  // cuts lie at 0
    int ctas;
};

static bool sparse_layout(int N, int H_q, int H_kv, int D, int B, int top_k, SparseLayout* L) {
    if (N <= 0 || N > 65535 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || H_q / H_kv > kMaxGroup || (D != 64 && D != 128) ||
        (B != 8 && B != 16 && B != 32) || top_k <= 0)
        return false;
    const int64_t rows = (int64_t)N * H_kv, units = ((int64_t)top_k * B + kUnitTok - 1) / kUnitTok;
    if (units >= (1LL << 31) / rows || rows * (H_q / H_kv) > 0x7fffffffLL) return false;
    auto align = [](size_t x) { return (x + 255) & ~size_t(255); };
    L->ctas = (int)std::min<int64_t>(kSpMaxCtas, (rows * units + kMinRun - 1) / kMinRun);
    const size_t parts = (size_t)2 * L->ctas * (H_q / H_kv);
    L->m = align((size_t)rows * sizeof(int2));
    L->l = align(L->m + parts * sizeof(float));
    L->acc = align(L->l + parts * sizeof(float));
    L->total = align(L->acc + parts * D * sizeof(float));
    return true;
}

size_t decode_sparse_workspace_bytes(int N, int H_q, int H_kv, int D, int B, int top_k) {
    SparseLayout L;
    return sparse_layout(N, H_q, H_kv, D, B, top_k, &L) ? L.total : 0;
}

template <typename T, bool kQuant, int D, int LGB>
static pa_status run_sparse(const DecodeSparseArgs& a, SpParams& p, const SparseLayout& L) {
    using Geo = SpGeo<kQuant, D>;
    constexpr int B = 1 << LGB;
    CUtensorMap tm;
    pa_status st;
    if (kQuant) {
        st = quant_tensor_map(&tm, a.pool, a.NB, a.H_kv, a.B, D);
    } else {
        // dims (innermost first): 64 columns, token (NB*B), column half, kv head, K/V; one box is a block's rows of a
        // head
        const cuuint64_t dims[5] = {64, (cuuint64_t)a.NB * a.B, D / 64, (cuuint64_t)a.H_kv, 2};
        const cuuint64_t str[4] = {(cuuint64_t)4 * a.H_kv * D, 128, (cuuint64_t)2 * D, (cuuint64_t)2 * a.H_kv * D};
        const cuuint32_t box[5] = {64, (cuuint32_t)a.B, D / 64, 1, 2};
        st = encode_tensor_map(&tm, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                               5, a.pool, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (st != PA_OK) return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    auto in_cluster = attend_sparse_kernel<T, kQuant, D, LGB, true>;
    e = cudaFuncSetAttribute(in_cluster, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(attend_sparse)");
    static ClusterRoom room;
    const int64_t rows = (int64_t)a.N * a.H_kv, tokens = (int64_t)a.top_k * B;
    constexpr int kShareFull = kQuant ? kSpShareFull8 : kSpShareFull16;
    p.cluster = 0;
    for (int size = kSpMaxCluster; size > 0; size /= 2) {
        if (tokens > (int64_t)size * kShareFull) break;
        int held = 0;
        e = room.get(in_cluster, size, kSpThreads, Geo::kSmem, &held);
        if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters(attend_sparse)");
        if (rows > held) continue;
        if (tokens <= (int64_t)size * (8 * rows >= 7 * (int64_t)held ? kShareFull : kSpShare)) p.cluster = size;
        break;
    }
    if (p.cluster) {
        e = launch_clusters(in_cluster, p.cluster, dim3((unsigned)(rows * p.cluster)), dim3(kSpThreads), Geo::kSmem,
                            a.stream, tm, p);
    } else {
        auto kern = attend_sparse_kernel<T, kQuant, D, LGB, false>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo::kSmem);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(attend_sparse)");
        const int grid = std::max(1, std::min(Geo::kCtas * sms, L.ctas));
        e = launch_kernel(kern, dim3((unsigned)grid), dim3(kSpThreads), Geo::kSmem, a.stream, tm, p);
    }
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "attend_sparse launch");
}

template <typename T, bool kQuant>
static pa_status run_sparse_shape(const DecodeSparseArgs& a, SpParams& p, const SparseLayout& L) {
    if (a.D == 128)
        return a.B == 8    ? run_sparse<T, kQuant, 128, 3>(a, p, L)
               : a.B == 16 ? run_sparse<T, kQuant, 128, 4>(a, p, L)
                           : run_sparse<T, kQuant, 128, 5>(a, p, L);
    return a.B == 8    ? run_sparse<T, kQuant, 64, 3>(a, p, L)
           : a.B == 16 ? run_sparse<T, kQuant, 64, 4>(a, p, L)
                       : run_sparse<T, kQuant, 64, 5>(a, p, L);
}

pa_status launch_decode_sparse(const DecodeSparseArgs& a) {
    SparseLayout L;
    if (!sparse_layout(a.N, a.H_q, a.H_kv, a.D, a.B, a.top_k, &L))
        return fail(PA_ERR_UNSUPPORTED, "too many work records");
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    SpParams p;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.q = a.q;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.selected = a.selected;
    p.top_k = a.top_k;
    p.N = a.N;
    p.H_kv = a.H_kv;
    p.G = a.H_q / a.H_kv;
    p.MB = a.MB;
    p.NB = a.NB;
    p.ctas = L.ctas;
    p.cap = (int64_t)a.MB * a.B;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);  // log2(e)
    p.cuts = reinterpret_cast<int2*>(ws);
    p.part_m = reinterpret_cast<float*>(ws + L.m);
    p.part_l = reinterpret_cast<float*>(ws + L.l);
    p.part_acc = reinterpret_cast<float*>(ws + L.acc);
    p.wait_ns = wait_limit_ns();
    p.err = a.dev_err;
    const bool quant = a.kv_dtype == PA_E4M3;
    pa_status st;
    if (a.q_dtype == PA_BF16)
        st = quant ? run_sparse_shape<__nv_bfloat16, true>(a, p, L) : run_sparse_shape<__nv_bfloat16, false>(a, p, L);
    else
        st = quant ? run_sparse_shape<__half, true>(a, p, L) : run_sparse_shape<__half, false>(a, p, L);
    if (st != PA_OK || p.cluster) return st;
    const unsigned grid = (unsigned)(((int64_t)a.N * a.H_q + kJoinWarps - 1) / kJoinWarps);
    auto join = a.out_dtype == PA_F32 ? (a.D == 128 ? join_sparse_kernel<float, 128> : join_sparse_kernel<float, 64>)
                : a.out_dtype == PA_BF16
                    ? (a.D == 128 ? join_sparse_kernel<__nv_bfloat16, 128> : join_sparse_kernel<__nv_bfloat16, 64>)
                    : (a.D == 128 ? join_sparse_kernel<__half, 128> : join_sparse_kernel<__half, 64>);
    const cudaError_t e = launch_kernel(join, dim3(grid), dim3(kJoinWarps * 32), 0, a.stream, p);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "join_sparse launch");
}

}  // namespace pa
