// decode_quant.cu -- single-token decode attention over the quantised cache (quant.cuh).
//
// The same three kernels as the 16-bit decode (schedule, attention, merge), of which the schedule and the merge are
// those of decode.cu.  The attention kernel: CTAs of two warps.  Warp 1 (producer) streams each work record's (block,
// head) chunks into a ring of 32-token stages, one TMA box (K rows, then V rows, swizzled) and one bulk copy of the 2 B
// scale bytes per block.  Warp 0 (consumer) computes with mma.sync m16n8k16, tokens on M, the <= 8 query heads of the
// KV head on N:
//     raw = K8 q'^T,  q' the query in fp16 (bf16 queries scaled row by row with a power of two, exactly); y_t = raw_t
//     2^ek_t c + ev_t,  c = scale log2 e 2^(query's exponent), ek_t, ev_t the exponents of the row scales; p_t = 2^(y_t
//     - M), M the running maximum of y;  O += p V8,  l += p 2^-ev;  out = O / l.
// With the exponent of V's scale inside the maximum, p <= 1 weighs the e4m3 values themselves, so p rounds to fp16
// (here a high and a low part, 2^-22) relative to the largest contribution to the output, whatever the scales' spread.
// |ev| <= 40 keeps p 2^-ev and l within fp32.  K8 and V8 become fp16 in registers (exact: cvt e4m3x2 -> f16x2).
//
// Bound by memory: 2 D + 2 bytes per token and KV head.  256 sequences of ~1500 tokens with 8 KV heads, D = 128 (811
// MB): 132 us, 6.1 TB/s; 64 of ~1000 with 40 KV heads (758 MB): 115 us, 6.6 TB/s; 8 of 32768 with 7 query heads to a KV
// head (541 MB): 95 us, 5.7 TB/s.  One sequence of 1000 tokens: 11 us, the latency of three kernels.
#include <algorithm>
#include <type_traits>

#include "quant.cuh"
#include "tensor_map.h"

namespace pa {

// A consumer warp is bound by the latency of its own chain (scores, maximum, exponentials, products), so the SM needs
// several: with 32-token stages seven CTAs of three stages (D = 128) fit.  Measured on 256 sequences of ~1500 tokens
// with 8 KV heads / 8 of 32768 / 64 of ~1000 with 40 KV heads: 4 CTAs 141 / 103 / 125 us, 6 CTAs 131 / 96 / 123, 7 CTAs
// 131 / 94 / 115, 8 CTAs (two stages each) 138 / 101 / 120; 64-token stages with 4 CTAs 141 / 97 / 120.
constexpr int kQStageTok = 32;   // tokens of one KV head per pipeline stage
constexpr int kQCtasPerSm = 7;
constexpr int kQThreads = 64;

enum : int { kQFirst = 1, kQLast = 2, kQDone = 4 };

struct __align__(16) QStageMeta {
    int s, h, part, ctx;
    int n_valid, flags, pad0, pad1;
};

struct QuantParams {
    const int4* rec;
    int* header;
    const int32_t* tables;
    int MB, NB;
    const uint8_t* scales;
    const void* q;
    int H_q, G;
    void* out;
    int out_dtype;
    float* part_m2;
    float* part_l;
    float* part_acc;
    int P, PT;
    const int32_t* ctx_lens;
    int N, H_kv, max_ctx, cap;
    float scale_log2;
    uint64_t wait_ns;
    int* err;
};

// Shared memory: ring slots (kSlot bytes each, 1024-byte aligned for the swizzle), then per stage the scale bytes and
// the query rows, the stage's description and its two barriers.
template <int D>
struct QGeo {
    static constexpr uint32_t kSlot = kQStageTok * D * 2;
    static constexpr uint32_t kScales = kQStageTok * 2;
    static constexpr uint32_t kQ = kMaxGroup * D * 2;
    static constexpr uint32_t kPerStage = kSlot + kScales + kQ + sizeof(QStageMeta) + 16;
    static constexpr int kStages = (233472 / kQCtasPerSm - 1024 - 1024 - 16) / (int)kPerStage;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kPerStage + 16;
    static_assert(kQCtasPerSm * (kSmem + 1024) <= 233472, "the CTAs of an SM fit its shared memory");
};

// Token of row i (0..7) of an 8-row half of the mma's M, chosen so that the 16- and 8-byte shared-memory reads of
// both products spread over all banks under the stage's swizzle (16-byte chunk c of row r lies at c ^ (r & 7) for
// 128-byte rows, c ^ (r / 2 & 3) for 64-byte rows).
template <int D>
__device__ __forceinline__ int row_token(int i) {
    return D == 128 ? ((i >> 1) | ((i & 1) << 2)) : (int)((0x65742130u >> (4 * i)) & 7u);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ int incl_scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

template <typename T, int D, int LGB>
__global__ void __launch_bounds__(kQThreads) attend_quant_kernel(const __grid_constant__ CUtensorMap tm,
                                                                 const QuantParams p) {
    using Geo = QGeo<D>;
    constexpr int ST = kQStageTok, nstage = Geo::kStages;
    constexpr int B = 1 << LGB;
    constexpr int BPS = ST / B;                  // blocks per stage
    constexpr uint32_t kBox = 2u * B * D;        // bytes of one (block, head) chunk
    constexpr int NSUB = ST / 16;        // 16-token mma tiles per stage
    constexpr int NT = D / 16;                   // k-steps of the score product, m-tiles of the value product
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sc_g = base + (size_t)nstage * Geo::kSlot;
    uint8_t* q_g = sc_g + (size_t)nstage * Geo::kScales;
    QStageMeta* meta = reinterpret_cast<QStageMeta*>(q_g + (size_t)nstage * Geo::kQ);
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
    }
    // The SM hands a CTA's two warps neighbouring slots, so with fixed roles every consumer would sit on the same two
    // of its four schedulers: the CTAs in every other group of four slots swap the roles.
    if (threadIdx.x == 0) {
        uint32_t wid;
        asm volatile("mov.u32 %0, %%warpid;" : "=r"(wid));
        abort_flag[1] = (int)(wid >> 2 & 1);
        prefetch_tmap(&tm);
    }
    __syncthreads();
    const bool producer = (int)(threadIdx.x >> 5) != abort_flag[1];
    // As in the 16-bit kernel, everything up to join_schedule() overlaps the schedule kernel, right after which this
    // kernel is always launched: the call's inputs are final here, only the schedule's records need the wait.
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;

    if (producer) {
        // ------------------------------------------------------------------ producer warp
        int total = 0, nwhole = 0;
        bool joined = false;
        auto join_schedule = [&]() {
            griddep_wait();
            total = p.header[0];
            nwhole = p.header[2];
            joined = true;
        };
        const uint64_t pol = policy_evict_first();
        int slot = 0;
        uint32_t ephase = 0;
        int narm = 0;  // stages armed so far (stage i's k-th arm completes phase k of full_bar[i])
        bool ok = true;
        const int4 none = make_int4(-1, 0, 0, 0);
        // record order: whole partitions round robin, then the ragged tails from a shared counter, longest first
        auto after = [&](int i) -> int {
            const int j = i + (int)gridDim.x;
            return j < nwhole ? j : nwhole + atomicAdd(p.header + 1, 1);
        };
        // the CTA's first whole partition follows from the lengths alone when it lies in the first 256 sequences:
        // it is streamed before the schedule is written
        constexpr int kEarly = 8;
        auto early_record = [&]() -> int4 {
            if (p.PT >= kUnpartitioned) return none;
            const int j = (int)blockIdx.x / p.H_kv, h = (int)blockIdx.x % p.H_kv;
            int c[kEarly];
#pragma unroll
            for (int k = 0; k < kEarly; ++k) {
                const int sq = 32 * k + lane;
                int v = sq < p.N ? p.ctx_lens[sq] : 0;
                if (v < 1 || v > p.max_ctx || v > p.cap) v = 0;  // as the schedule: no records
                c[k] = v;
            }
            int run = 0;
#pragma unroll
            for (int k = 0; k < kEarly; ++k) {
                const int nf = c[k] / p.PT;
                const int incl = incl_scan(nf);
                const unsigned hit = __ballot_sync(0xffffffffu, run + incl - nf <= j && j < run + incl);
                if (hit) {
                    const int src = __ffs(hit) - 1;
                    const int first = __shfl_sync(0xffffffffu, run + incl - nf, src);
                    return make_int4(32 * k + src, h, j - first, __shfl_sync(0xffffffffu, c[k], src));
                }
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            return none;
        };
        int4 cur = early_record(), nxt = none;
        int nidx = 0, pend = 0;
        auto join_after_first = [&]() {
            join_schedule();
            if (lane == 0) nidx = after((int)blockIdx.x);
            nidx = __shfl_sync(0xffffffffu, nidx, 0);
            nxt = nidx < total ? p.rec[nidx] : none;
            if (lane == 0 && nxt.x >= 0) pend = after(nidx);
        };
        if (cur.x < 0) {
            join_schedule();
            if (lane == 0) nidx = after((int)blockIdx.x - (int)gridDim.x);
            nidx = __shfl_sync(0xffffffffu, nidx, 0);
            cur = nidx < total ? p.rec[nidx] : none;
            if (lane == 0) nidx = after(nidx);
            nidx = __shfl_sync(0xffffffffu, nidx, 0);
            nxt = nidx < total ? p.rec[nidx] : none;
            if (lane == 0 && nxt.x >= 0) pend = after(nidx);
        }
        // table entries of the 32 blocks of `it` from its block `cb` on
        auto load_entries = [&](const int4& it, int cb) -> int {
            const int t0 = it.z * p.PT;
            const int nblk = (min(p.PT, it.w - t0) + B - 1) / B;
            const int b = cb + lane;
            return b < nblk ? p.tables[(size_t)it.x * p.MB + t0 / B + b] : 0;
        };
        int ent = cur.x >= 0 ? load_entries(cur, 0) : 0;
        while (cur.x >= 0 && ok) {
            const int s = cur.x, h = cur.y, part = cur.z, ctx = cur.w;
            const int t0 = part * p.PT;
            const int ntok = min(p.PT, ctx - t0);
            const int nblk = (ntok + B - 1) / B;
            const int nst = (ntok + ST - 1) / ST;
            int st = 0;
            for (int cb = 0; cb < nblk && ok; cb += 32) {
                int ent_nx = 0;
                if (cb + 32 < nblk)
                    ent_nx = load_entries(cur, cb + 32);
                else if (joined && nxt.x >= 0)
                    ent_nx = load_entries(nxt, 0);
                const int cend = min(cb + 32, nblk);
                for (int b0 = cb; b0 < cend; b0 += BPS, ++st) {
                    if (!joined && st == nstage) {
                        // the ring is full of the early record: learn the next one while it drains
                        join_after_first();
                        if (cb + 32 >= nblk && nxt.x >= 0) ent_nx = load_entries(nxt, 0);
                    }
                    if (lane == 0) ok = mbar_wait_bounded(empty_s + 8 * slot, ephase ^ 1, abort_flag, p.wait_ns);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    ++narm;  // armed below: expect_tx and every copy of the stage, with no wait in between
                    const int nb = min(BPS, nblk - b0);
                    const bool first = st == 0, last = st == nst - 1;
                    const uint32_t bar = full_s + 8 * slot;
                    if (lane == 0) {
                        QStageMeta m;
                        m.s = s;
                        m.h = h;
                        m.part = part;
                        m.ctx = ctx;
                        m.n_valid = min(ST, ntok - st * ST);
                        m.flags = (first ? kQFirst : 0) | (last ? kQLast : 0);
                        m.pad0 = m.pad1 = 0;
                        meta[slot] = m;
                        mbar_arrive_expect_tx(bar, (uint32_t)nb * (kBox + 2 * B) +
                                                       (first ? (uint32_t)p.G * D * 2 : 0u));
                        if (first) {
                            const T* qsrc = static_cast<const T*>(p.q) + ((size_t)s * p.H_q + (size_t)h * p.G) * D;
                            bulk_load(q_s + slot * Geo::kQ, qsrc, (uint32_t)p.G * D * 2, bar);
                        }
                    }
                    __syncwarp();
                    // lane b copies block b's rows, lane 16 + b its scale bytes
                    const int b = lane & 15;
                    int e = __shfl_sync(0xffffffffu, ent, (b0 - cb + b) & 31);
                    if (b < nb) {
                        const bool good = (unsigned)e < (unsigned)p.NB;
                        if (lane < 16) {
                            if (!good) flag_error(p.err, PA_DEV_ERR_BLOCK);
                            // a bad entry reads past the tensor: TMA fills zeros
                            tma_load_3d(slots_s + slot * Geo::kSlot + b * kBox, &tm, bar, 0, 0,
                                        (good ? e : p.NB) * p.H_kv + h, pol);
                        } else {
                            bulk_load(sc_s + slot * Geo::kScales + b * 2 * B,
                                      p.scales + ((size_t)(good ? e : 0) * p.H_kv + h) * (2 * B), 2 * B, bar);
                        }
                    }
                    if (++slot == nstage) {
                        slot = 0;
                        ephase ^= 1;
                    }
                }
                ent = ent_nx;
            }
            if (!joined) {
                join_after_first();
                ent = nxt.x >= 0 ? load_entries(nxt, 0) : 0;
            }
            cur = nxt;
            nidx = __shfl_sync(0xffffffffu, pend, 0);
            nxt = nidx < total ? p.rec[nidx] : none;
            if (lane == 0 && nxt.x >= 0) pend = after(nidx);
        }
        if (ok && lane == 0) {
            ok = mbar_wait_bounded(empty_s + 8 * slot, ephase ^ 1, abort_flag, p.wait_ns);
            if (ok) {
                meta[slot].flags = kQDone;
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
        return;
    }

    // ---------------------------------------------------------------------- consumer warp
    const int g4 = lane >> 2, t4 = lane & 3;
    // Offset in a slot of the K rows of the 8 tokens from n on (n a multiple of 8); their V rows follow B rows later,
    // their scale bytes lie at n's place in the stage's scales.
    auto tok_ofs = [](int n) -> uint32_t { return (uint32_t)((n >> LGB) * 2 * B + (n & (B - 1))) * D; };
    auto sc_ofs = [](int n) -> uint32_t { return (uint32_t)((n >> LGB) * 2 * B + (n & (B - 1))); };
    // Score product, A = K: this thread holds token rt (and rt + 8) of each tile and, of the contraction, the 16-byte
    // chunks t4 and (D = 128) t4 + 4 of the row: word w covers elements 16 t4 + 4 w .. + 3, as the k-columns 2 t4,
    // 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 of k-step w (any order serves, the query's fragments follow the same one).
    const int rt = row_token<D>(g4);
    const uint32_t kofs = D == 128 ? rt * 128 + ((t4 ^ rt) << 4) : rt * 64 + ((t4 ^ (rt >> 1 & 3)) << 4);
    // Value product, A = V^T: rows are elements, columns tokens va, vb (and + 8) of the tile, the ones whose
    // probabilities the score product left in rows 2 t4 and 2 t4 + 1.  This thread's elements are the 2 NT from d0 on,
    // rows g4 and g4 + 8 of m-tile i being d0 + 2 i and d0 + 2 i + 1.
    const int va = row_token<D>(2 * t4), vb = row_token<D>(2 * t4 + 1);
    const int vch = D == 128 ? row_token<128>(g4) : g4;  // 16-byte (8-byte) piece of the row
    const int d0 = vch * 2 * NT;
    auto vofs_of = [&](int tok) -> uint32_t {
        return D == 128 ? tok * 128 + ((vch ^ tok) << 4)
                        : tok * 64 + (((vch >> 1) ^ (tok >> 1 & 3)) << 4) + ((vch & 1) << 3);
    };
    const uint32_t vofs_a = B * D + vofs_of(va), vofs_b = B * D + vofs_of(vb);
    float O[NT][4];
    uint32_t qf[NT][2];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float c0 = 0.f, c1 = 0.f;  // raw scores of heads 2 t4, 2 t4 + 1 to base-2 units
    int slot = 0;
    uint32_t fphase = 0;
    const float NEG_INF = -INFINITY;
    while (true) {
        if (!mbar_wait_bounded(full_s + 8 * slot, fphase, abort_flag, p.wait_ns)) {
            if (lane == 0) {
                flag_error(p.err, PA_DEV_ERR_TIMEOUT);
                *abort_flag = 1;
            }
            break;
        }
        const QStageMeta mt = meta[slot];
        if (mt.flags & kQDone) break;
        const uint32_t kv = slots_s + slot * Geo::kSlot, scb = sc_s + slot * Geo::kScales;
        if (mt.flags & kQFirst) {
            float a = 0.f;
            const uint32_t qrow = q_s + slot * Geo::kQ + g4 * D * 2 + t4 * 32;
#pragma unroll
            for (int w = 0; w < NT; ++w) {
                const uint2 x = g4 < p.G ? lds64(qrow + (w >> 2) * 128 + (w & 3) * 8) : make_uint2(0, 0);
                qf[w][0] = x.x;
                qf[w][1] = x.y;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    const float2 f0 = Mma<T>::unpack(x.x), f1 = Mma<T>::unpack(x.y);
                    a = fmaxf(a, fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))));
                }
            }
            c0 = c1 = p.scale_log2;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                // The row's largest magnitude goes to [2^14, 2^15): elements down to 2^-28 of it are normal fp16
                // numbers and exact, smaller ones are off by at most 2^-40 of it.
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
                c0 *= __shfl_sync(0xffffffffu, up, 8 * t4);      // lane 4 n holds head n's
                c1 *= __shfl_sync(0xffffffffu, up, 8 * t4 + 4);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.f;
            m0 = m1 = NEG_INF;
            l0 = l1 = 0.f;
        }
        const int nvalid = mt.n_valid;
        // one copy for whole stages, without a branch between the tiles, and one for a context's last
        auto stage = [&](auto full_c) {
            constexpr bool kFull = decltype(full_c)::value;
            // scores of every tile, to y = raw 2^ek c + ev
            float y[NSUB][4], iv[NSUB][2];  // iv: 2^-ev of tokens rt and rt + 8
            float x0 = NEG_INF, x1 = NEG_INF;
    #pragma unroll
            for (int j = 0; j < NSUB; ++j) {
                y[j][0] = y[j][1] = y[j][2] = y[j][3] = NEG_INF;
                iv[j][0] = iv[j][1] = 0.f;
                if (kFull || 16 * j < nvalid) {
                    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
                    for (int c = 0; c < NT / 4; ++c) {
                        const uint4 lo = lds128(kv + tok_ofs(16 * j) + (kofs ^ (c * 64)));
                        const uint4 hi = lds128(kv + tok_ofs(16 * j + 8) + (kofs ^ (c * 64)));
                        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
    #pragma unroll
                        for (int w = 0; w < 4; ++w)
                            Mma<__half>::run(w & 1 ? b : a, e4m3x2_to_f16x2(wl[w]), e4m3x2_to_f16x2(wh[w]),
                                             e4m3x2_to_f16x2(wl[w] >> 16), e4m3x2_to_f16x2(wh[w] >> 16), qf[4 * c + w][0],
                                             qf[4 * c + w][1]);
                    }
    #pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int tok = 16 * j + 8 * half + rt;
                        const uint32_t at = scb + sc_ofs(16 * j + 8 * half) + rt;
                        const int bk = (int)lds8(at), bv = (int)lds8(at + B);
                        const float fk = pow2i(scale_of(bk));
                        const int ev = scale_of(bv);
                        iv[j][half] = pow2i(-ev);
                        if (kFull || tok < nvalid) {
                            y[j][2 * half] = fmaf((a[2 * half] + b[2 * half]) * fk, c0, (float)ev);
                            y[j][2 * half + 1] = fmaf((a[2 * half + 1] + b[2 * half + 1]) * fk, c1, (float)ev);
                        }
                    }
                    x0 = fmaxf(x0, fmaxf(y[j][0], y[j][2]));
                    x1 = fmaxf(x1, fmaxf(y[j][1], y[j][3]));
                }
            }
    #pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
            }
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
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
            // O^T += V8^T p^T, p as a high and a low fp16 part transposed into B fragments
    #pragma unroll
            for (int j = 0; j < NSUB; ++j) {
                if (kFull || 16 * j < nvalid) {
                    const float p0 = fast_exp2(y[j][0] - n0), p1 = fast_exp2(y[j][1] - n1);
                    const float p2 = fast_exp2(y[j][2] - n0), p3 = fast_exp2(y[j][3] - n1);
                    l0 = fmaf(p0, iv[j][0], fmaf(p2, iv[j][1], l0));
                    l1 = fmaf(p1, iv[j][0], fmaf(p3, iv[j][1], l1));
                    const uint32_t h01 = Mma<__half>::pack(p0, p1), h23 = Mma<__half>::pack(p2, p3);
                    const float2 f01 = Mma<__half>::unpack(h01), f23 = Mma<__half>::unpack(h23);
                    const uint32_t lo01 = Mma<__half>::pack(p0 - f01.x, p1 - f01.y),
                                   lo23 = Mma<__half>::pack(p2 - f23.x, p3 - f23.y);
                    const uint32_t bh0 = movmatrix_trans(h01), bh1 = movmatrix_trans(h23);
                    const uint32_t bl0 = movmatrix_trans(lo01), bl1 = movmatrix_trans(lo23);
                    uint32_t w[4][NT / 2];  // tokens va, vb, va + 8, vb + 8
    #pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t at = kv + tok_ofs(16 * j + 8 * (t >> 1)) + (t & 1 ? vofs_b : vofs_a);
                        if constexpr (D == 128) {
                            const uint4 x = lds128(at);
                            w[t][0] = x.x;
                            w[t][1] = x.y;
                            w[t][2] = x.z;
                            w[t][3] = x.w;
                        } else {
                            const uint2 x = lds64(at);
                            w[t][0] = x.x;
                            w[t][1] = x.y;
                        }
                    }
                    // V rows past the context may hold anything (even NaN): they count as zeros
                    if (!kFull && 16 * j + 16 > nvalid) {
    #pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const bool in = 16 * j + 8 * (t >> 1) + (t & 1 ? vb : va) < nvalid;
    #pragma unroll
                            for (int i = 0; i < NT / 2; ++i) w[t][i] = in ? w[t][i] : 0u;
                        }
                    }
    #pragma unroll
                    for (int i = 0; i < NT / 2; ++i) {
                        // (va, vb) pairs of elements 4 i .. 4 i + 3, then the same of the tokens 8 later
                        const uint32_t u0 = __byte_perm(w[0][i], w[1][i], 0x5140);
                        const uint32_t u1 = __byte_perm(w[0][i], w[1][i], 0x7362);
                        const uint32_t u2 = __byte_perm(w[2][i], w[3][i], 0x5140);
                        const uint32_t u3 = __byte_perm(w[2][i], w[3][i], 0x7362);
                        {
                            const uint32_t r0 = e4m3x2_to_f16x2(u0), r1 = e4m3x2_to_f16x2(u0 >> 16),
                                           r2 = e4m3x2_to_f16x2(u2), r3 = e4m3x2_to_f16x2(u2 >> 16);
                            Mma<__half>::run(O[2 * i], r0, r1, r2, r3, bh0, bh1);
                            Mma<__half>::run(O[2 * i], r0, r1, r2, r3, bl0, bl1);
                        }
                        {
                            const uint32_t r0 = e4m3x2_to_f16x2(u1), r1 = e4m3x2_to_f16x2(u1 >> 16),
                                           r2 = e4m3x2_to_f16x2(u3), r3 = e4m3x2_to_f16x2(u3 >> 16);
                            Mma<__half>::run(O[2 * i + 1], r0, r1, r2, r3, bh0, bh1);
                            Mma<__half>::run(O[2 * i + 1], r0, r1, r2, r3, bl0, bl1);
                        }
                    }
                }
            }
        };
        if (nvalid == ST)
            stage(std::true_type{});
        else
            stage(std::false_type{});
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_s + 8 * slot);

        if (mt.flags & kQLast) {
            float L0 = l0, L1 = l1;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                L0 += __shfl_xor_sync(0xffffffffu, L0, o);
                L1 += __shfl_xor_sync(0xffffffffu, L1, o);
            }
            const int np = p.PT >= kUnpartitioned ? 1 : (mt.ctx + p.PT - 1) / p.PT;
            const size_t qrow0 = (size_t)mt.s * p.H_q + (size_t)mt.h * p.G;
            // the merge reads the partials right after this kernel: keep them in L2
            const uint64_t keep = policy_evict_last();
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int hd = 2 * t4 + hh;
                if (hd >= p.G) continue;
                if (np == 1) {
                    const float inv = 1.f / (hh ? L1 : L0);
                    const size_t o = (qrow0 + hd) * D + d0;
                    if (p.out_dtype == PA_F32) {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
#pragma unroll
                        for (int i = 0; i < NT / 2; ++i)
                            dst[i] = make_float4(O[2 * i][hh] * inv, O[2 * i][2 + hh] * inv, O[2 * i + 1][hh] * inv,
                                                 O[2 * i + 1][2 + hh] * inv);
                    } else {
                        uint2* dst = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + o);
#pragma unroll
                        for (int i = 0; i < NT / 2; ++i)
                            dst[i] = make_uint2(Mma<T>::pack(O[2 * i][hh] * inv, O[2 * i][2 + hh] * inv),
                                                Mma<T>::pack(O[2 * i + 1][hh] * inv, O[2 * i + 1][2 + hh] * inv));
                    }
                } else {
                    const size_t r = (qrow0 + hd) * p.P + mt.part;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        st_hint(p.part_acc + r * D + d0 + 2 * i, O[i][hh], keep);
                        st_hint(p.part_acc + r * D + d0 + 2 * i + 1, O[i][2 + hh], keep);
                    }
                    if (g4 == 0) {
                        st_hint(p.part_m2 + r, hh ? m1 : m0, keep);
                        st_hint(p.part_l + r, hh ? L1 : L0, keep);
                    }
                }
            }
        }
        if (++slot == nstage) {
            slot = 0;
            fphase ^= 1;
        }
    }
}

// ----------------------------------------------------------------------------- host side

template <typename T, int D, int LGB>
static pa_status run_attend_quant(const DecodeQuantArgs& a, const WorkspaceLayout& L, const CUtensorMap& tm) {
    auto kern = attend_quant_kernel<T, D, LGB>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    int sms = 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    constexpr size_t smem = QGeo<D>::kSmem;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(attend_quant)");
    const long maxrec = std::min<long>((long)a.N * L.P * a.H_kv, 1L << 30);
    const int grid = (int)std::max<long>(1, std::min<long>((long)kQCtasPerSm * sms, maxrec));

    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    QuantParams p;
    p.rec = reinterpret_cast<const int4*>(ws + L.records);
    p.header = reinterpret_cast<int*>(ws + L.header);
    p.tables = a.tables;
    p.MB = a.MB;
    p.NB = a.NB;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.q = a.q;
    p.H_q = a.H_q;
    p.G = a.H_q / a.H_kv;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.part_m2 = L.P > 1 ? reinterpret_cast<float*>(ws + L.part_m2) : nullptr;
    p.part_l = L.P > 1 ? reinterpret_cast<float*>(ws + L.part_l) : nullptr;
    p.part_acc = L.P > 1 ? reinterpret_cast<float*>(ws + L.part_acc) : nullptr;
    p.P = L.P;
    p.PT = L.PT;
    p.ctx_lens = a.ctx_lens;
    p.N = a.N;
    p.H_kv = a.H_kv;
    p.max_ctx = a.max_ctx;
    p.cap = (int)std::min<long long>((long long)a.MB * a.B, 0x7fffffff);
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);  // log2(e)
    p.wait_ns = wait_limit_ns();
    p.err = a.dev_err;
    if (a.attend_events && a.attend_events[0]) {
        e = cudaEventRecord(static_cast<cudaEvent_t>(a.attend_events[0]), a.stream);
        if (e != cudaSuccess) return cuda_fail(e, "cudaEventRecord");
    }
    e = launch_kernel(kern, dim3(grid), dim3(kQThreads), smem, a.stream, tm, p);
    count_launch();
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
    if (a.attend_events && a.attend_events[1]) {
        e = cudaEventRecord(static_cast<cudaEvent_t>(a.attend_events[1]), a.stream);
        if (e != cudaSuccess) return cuda_fail(e, "cudaEventRecord");
    }
    return PA_OK;
}

template <typename T, int D>
static pa_status dispatch_block(const DecodeQuantArgs& a, const WorkspaceLayout& L, const CUtensorMap& tm) {
    return a.B == 8    ? run_attend_quant<T, D, 3>(a, L, tm)
           : a.B == 16 ? run_attend_quant<T, D, 4>(a, L, tm)
                       : run_attend_quant<T, D, 5>(a, L, tm);
}

pa_status quant_tensor_map(CUtensorMap* m, const void* qpool, int NB, int H_kv, int B, int D) {
    // dims (innermost first): D bytes, the chunk's 2 B rows, chunk (block, head); one box is one chunk
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)2 * B, (cuuint64_t)NB * H_kv};
    const cuuint64_t str[2] = {(cuuint64_t)D, (cuuint64_t)2 * B * D};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)2 * B, 1};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, qpool, dims, str, box,
                             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// The consumer warps resident on a GB300 (kQCtasPerSm on each of its 152 SMs; the length may not depend on the device at
// hand, for a workspace is sized by it) each take a record at a time, in about 1 us per 32 tokens.  Where no length is
// named, a batch with fewer whole default partitions than warps is cut finer, down to 64 tokens (two
// stages; shorter ones leave the merge more than they save): one sequence of 1000 tokens and 8 KV heads took 28 us in
// partitions of 512 and takes 11 in partitions of 64.  (Lengths that would fill the last round over the warps made no
// difference to larger batches: 8 sequences of 32768 tokens took 96 us with 512, 97 with 576, 95 with 768.)
int quant_partition(int N, int H_kv, int max_ctx) {
    if (const int pt = named_partition()) return pt;
    constexpr long kWarps = 152 * kQCtasPerSm;
    const long tokens = (long)N * H_kv * max_ctx;
    const long pt = ((tokens + kWarps - 1) / kWarps + kStageTok - 1) / kStageTok * kStageTok;
    return (int)std::min<long>(kDefaultPartition, std::max<long>(64, pt));
}

pa_status launch_decode_quant(const DecodeQuantArgs& a) {
    WorkspaceLayout L;
    const int pt = quant_partition(a.N, a.H_kv, a.max_ctx);
    if (!(a.partition_tokens == 0 && workspace_layout(a.N, a.H_q, a.H_kv, a.D, a.max_ctx, pt, &L) &&
          L.total <= a.ws_bytes) &&
        !workspace_layout(a.N, a.H_q, a.H_kv, a.D, a.max_ctx, a.partition_tokens, &L))
        return fail(PA_ERR_INVALID, "invalid workspace arguments");
    if (a.ws_bytes < L.total) return fail(PA_ERR_INVALID, "workspace too small: %zu < %zu", a.ws_bytes, L.total);
    CUtensorMap tm;
    pa_status st = quant_tensor_map(&tm, a.qpool, a.NB, a.H_kv, a.B, a.D);
    if (st != PA_OK) return st;
    const int cap = (int)std::min<long long>((long long)a.MB * a.B, 0x7fffffff);
    st = launch_plan(a.ctx_lens, nullptr, a.N, a.H_kv, a.max_ctx, cap, 0, a.workspace, L, a.dev_err, a.stream);
    if (st != PA_OK) return st;
    if (a.q_dtype == PA_BF16)
        st = a.D == 128 ? dispatch_block<__nv_bfloat16, 128>(a, L, tm) : dispatch_block<__nv_bfloat16, 64>(a, L, tm);
    else
        st = a.D == 128 ? dispatch_block<__half, 128>(a, L, tm) : dispatch_block<__half, 64>(a, L, tm);
    if (st != PA_OK || L.P == 1) return st;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    return launch_partition_reduce(a.out, a.out_dtype, reinterpret_cast<float*>(ws + L.part_m2),
                                   reinterpret_cast<float*>(ws + L.part_l), reinterpret_cast<float*>(ws + L.part_acc),
                                   reinterpret_cast<int*>(ws + L.nparts), a.H_q, a.N * a.H_q, L.P, a.D, true,
                                   a.dev_err, a.stream);
}

}  // namespace pa
