// tree.cu -- attention of drafted tokens over a paged cache (16-bit or quantised) under a tree mask.
//
// Row (drafted token i, query head) of sequence s sees the context before the draft and the drafted tokens its mask
// names.  The query rows of one KV head -- 128 / G tokens times the G heads -- form row tiles of up to 128 (tcgen05's
// M), so each K/V byte serves every row of a tile, and a (sequence, KV head, row tile) is a unit of ceil(ctx / 128) key
// tiles.
//
// tree_kernel: one persistent CTA per SM.  All key tiles of the call, in unit order, are cut into runs of equal cost,
// one per CTA, so the GPU is evenly loaded whatever the lengths; a CTA walks its run as segments (consecutive tiles of
// one unit), and a unit that several CTAs share leaves partial results (m, l, unnormalised O) that tree_merge_kernel
// joins.  A CTA leaves at most two (its first and its last segment), so the workspace has a fixed size.  Roles:
//   * warps 0-3 and 4-7, two softmax warpgroups: warpgroup w takes keys 64 w .. 64 w + 63 of every tile; each thread
//     owns one TMEM lane = one query row.  It reads its 64 scores (tcgen05.ld), masks, keeps a running maximum of its
//     own (its O is rescaled only when that grows by more than 2^8) and writes the probabilities to TMEM, over the
//     scores it has just read.  The warpgroups have accumulators of their own, O_0 and O_1, joined at the segment's
//     end, so they never wait for one another in between;
//   * warp 8 (TMA): query rows (16-bit pool), K and V tiles into rings, block by block through the block table;
//   * warp 9 (one thread): S = Q K^T into one of two buffers (TMEM columns 0 .. 127 and 128 .. 255), so that a tile's
//     score product runs under the softmax of the tile before it; warp 10 (one thread): O_w += P_w V (columns 256 + D
//     w), P read from TMEM;
//   * quantised pool, warps 12-19: e4m3 tiles from the raw ring to fp16 tiles in the K and V rings, and the query rows.
// The value product takes P in V's 16-bit type: for bf16, or an fp32 output, as a high and a low part (two products).
//
// Quantised pool: query rows are scaled to fp16's range by a power of two (exact); K8 is converted to fp16 times 2^(ek
// - emax + 7), emax the tile's largest exponent (keys 2^22 below it count as zero: a score is off by at most 2^-22 of
// the largest that a key of the tile could give), V8 likewise where that is exact (see kTreeSpan); with E the exponent
// taken out of V (per tile, else per key): y = raw c 2^(emax - 7) + E, p = 2^(y - M), O += p (V 2^-E), l += p 2^-E, as
// in decode_quant.cu.
//
// What bounds it, measured at D = 128.  64 sequences with trees of up to 24 tokens, 32 / 8 heads, bf16: 90 us, 4.8 TB/s
// of K and V.  The bytes alone are 64 us; inside a run a tile takes about 2700 cycles, 64 KB at 7 TB/s over the GPU,
// and the rest is the launch, the first tiles and the ends of 512 units.  16 trees of up to 63 tokens over 4500
// quantised tokens each: 111 us, about 2800 cycles per tile of 128 x 128, bound by the roles' own instructions and
// waits (the SM issues 2.1 of 4 instructions a cycle, the tensor pipe is 28 % busy, memory 20 %).  Of 117 us with all
// in place, a copy without the conversion to fp16 took 88, without exponentials 113, without both products 109, without
// all three 83.  What the time was spent on before: one group of converters (114 us), one score buffer (128), masked
// and keyed tiles in line (138) and spin waits unrolled by the compiler (180), both of which pushed the usual tile's
// code out of the instruction cache.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "quant.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace pa {

constexpr int kTRows = 128;    // query rows per tile (tcgen05 M), one TMEM lane each
constexpr int kTKeys = 128;    // keys per tile (N of S, K of P V)
constexpr uint32_t kTRegion = kTRows * 128;  // [128 rows][64 columns] 16-bit, 128-byte swizzled
constexpr uint32_t kTTmem = 512;
constexpr int kTreeMaxCtas = 160;  // CTAs of a call at most (the workspace holds two partial results for each)
// Cost of a unit's start and end (query rows, first scores, joining the warpgroups, storing) in key tiles.  Two to four
// make no difference (512 units of 13 tiles: 89, 91, 91 us; 6: 97).
constexpr int kTreeUnitCost = 2;
constexpr int kConvWarps = 8;  // two groups of four: one for the even tiles, one for the odd
// Probabilities are relative to a reference kPHeadroom below the row's maximum, which may grow by 2^8 before O is
// rescaled: they reach 2^15, the top of fp16's range, so that the smallest keep as many bits as fp16 allows (an
// absolute 2^-25 is 2^-32 of the largest).
constexpr float kPHeadroom = 7.f;
// Quantised V: while the exponents of a tile's scales lie within kTreeSpan of one another, one exponent serves the tile
// (V8 2^(ev - vmax + 7) is exact in fp16); otherwise (kTreeKeyed) each key's enters the scores.  With the headroom a
// probability's absolute rounding then weighs no more than it does keyed, where the largest product is the reference.
constexpr int kTreeSpan = 7;
constexpr float kTreeKeyed = 1e30f;

struct TreeParams {
    const void* q;
    int q_bf16;
    const int32_t* tables;
    const int32_t* ctx_lens;
    const int32_t* q_start;
    const uint32_t* mask;
    const uint8_t* scales;
    int W, N, T, H_q, H_kv, G, TQ, lgB, MB, NB, max_q_len;
    void* out;
    int out_dtype;
    float scale_log2;
    int4* desc;       // per CTA: the unit it starts and leaves unfinished (sequence, unit, pieces), pieces 0: none
    float* part_ml;   // [2 * CTAs][128][2]
    float* part_acc;  // [2 * CTAs][128][D]
    uint64_t wait_ns;
    int* err;
};

// mbar_wait_bounded for hand-offs that usually take well under a microsecond: the clock, whose read takes longer than
// that, is consulted only every 64 tries (every try when the limit is below a microsecond).  Kept short in code: a
// kernel whose roles wait at many places fits the instruction cache only so.
__device__ __forceinline__ bool mbar_wait_spin(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    const uint32_t tries = limit_ns < 1000 ? 1 : 64;
    uint64_t t0 = 0;
#pragma unroll 1
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n\t"
            "AGAIN:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "@p bra DONE;\n\tsub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra AGAIN;\n\t"
            "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(tries)
            : "memory");
        if (ok) return true;
        if (*abort) return false;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > limit_ns) return false;
    }
}

// A scale byte held to the range the writer produces.
__device__ __forceinline__ int clamp_scale(uint32_t b) { return scale_of((int)b) + kScaleBias; }

// Eight words to one 32-byte sector (32-byte aligned), or to two halves of one.
__device__ __forceinline__ void st_words8(void* d, const uint32_t* v, bool sector) {
    if (sector) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        static_cast<uint4*>(d)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4*>(d)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// ----------------------------------------------------------------------------- work distribution

struct TreeSeq {
    int ctx, n, qs, nt, nmt;  // nt: key tiles (0: nothing to do), nmt: row tiles
};

// A sequence's work; an invalid one has none (and is flagged when `flag`).
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int s, bool flag) {
    TreeSeq q;
    const int a = p.q_start[s], b = p.q_start[s + 1];
    q.ctx = p.ctx_lens[s];
    q.qs = a;
    q.n = b - a;
    q.nt = 0;
    q.nmt = 0;
    if (a < 0 || b < a || b > p.T || q.n > p.max_q_len ||
        (q.n > 0 && (q.ctx < q.n || (int64_t)q.ctx > ((int64_t)p.MB << p.lgB)))) {
        if (flag) flag_error(p.err, PA_DEV_ERR_CTX);
        return q;
    }
    if (q.n > 0) {
        q.nt = (q.ctx - 1) / kTKeys + 1;
        q.nmt = (q.n + p.TQ - 1) / p.TQ;
    }
    return q;
}

__device__ __forceinline__ int64_t tree_cost(const TreeParams& p, const TreeSeq& q) {
    return q.nt > 0 ? (int64_t)(q.nt + kTreeUnitCost) * q.nmt * p.H_kv : 0;
}

// Consecutive key tiles j0 .. j1 - 1 of one unit.
struct TreeSeg {
    int s, h, mt, j0, j1, nt, ctx, n, qs;
};

// a / b of positive numbers: a 64-bit division is a long subroutine, and calls whose tiles need one are rare.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return (a | b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Walks a CTA's run segment by segment.  Positions count cost: a unit is kTreeUnitCost, then one per tile.
struct TreeWalk {
    int s, u, o;  // sequence, unit in it, position in the unit
    int64_t left;
    TreeSeq q;
    __device__ __forceinline__ void start(const TreeSeq& q0, int s0, int64_t rem, int64_t count) {
        s = s0;
        left = count;
        q = q0;
        u = (int)divide(rem, q.nt + kTreeUnitCost);
        o = (int)(rem - (int64_t)u * (q.nt + kTreeUnitCost));
    }
    __device__ __forceinline__ bool next(const TreeParams& p, TreeSeg& g) {
        while (left > 0) {
            const int size = q.nt + kTreeUnitCost;
            const int o1 = (int)min((int64_t)size, o + left);
            g.s = s;
            g.h = u / q.nmt;
            g.mt = u - g.h * q.nmt;
            g.j0 = max(0, o - kTreeUnitCost);
            g.j1 = max(0, o1 - kTreeUnitCost);
            g.nt = q.nt;
            g.ctx = q.ctx;
            g.n = q.n;
            g.qs = q.qs;
            left -= o1 - o;
            o = 0;
            if (++u == q.nmt * p.H_kv && left > 0) {
                u = 0;
                do {
                    q = tree_seq(p, ++s, false);
                } while (q.nt == 0);
            }
            if (g.j1 > g.j0) return true;
        }
        return false;
    }
};

// The CTA's run [lo, hi) of the call's cost, and the sequence it starts in with the part of it that lies before. Every
// thread of the block calls it; `buf`: 40 words of 8 bytes.  Up to 32 sequences every warp finds it by itself, one lane
// to a sequence: without barriers and second reads of the lengths the first tiles of 4 sequences start 1 us sooner.
struct TreeRun {
    int64_t per, lo, hi, rem;
    int s;
    TreeSeq q;
};

__device__ __forceinline__ int64_t shfl64(int64_t x, int lane) {
    return (int64_t)__shfl_sync(0xffffffffu, (unsigned long long)x, lane);
}

template <int THREADS>
__device__ __forceinline__ TreeRun tree_run(const TreeParams& p, int cta, int ctas, bool flag, int64_t* buf) {
    constexpr int NW = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    TreeRun r;
    if (p.N <= 32) {
        TreeSeq q = {};
        if (lane < p.N) q = tree_seq(p, lane, flag && warp == 0);
        const int64_t c = tree_cost(p, q);
        int64_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = (int64_t)__shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
            if (lane >= o) incl += u;
        }
        const int64_t total = shfl64(incl, 31);
        r.per = divide(total + ctas - 1, ctas);
        r.lo = r.per * cta;
        r.hi = min(r.lo + r.per, total);
        // the sequence that holds position lo: the first whose end lies past it
        r.s = max(__ffs(__ballot_sync(0xffffffffu, incl > r.lo)) - 1, 0);
        r.rem = r.lo - shfl64(incl - c, r.s);
        r.q.ctx = __shfl_sync(0xffffffffu, q.ctx, r.s);
        r.q.n = __shfl_sync(0xffffffffu, q.n, r.s);
        r.q.qs = __shfl_sync(0xffffffffu, q.qs, r.s);
        r.q.nt = __shfl_sync(0xffffffffu, q.nt, r.s);
        r.q.nmt = __shfl_sync(0xffffffffu, q.nmt, r.s);
        return r;
    }
    int64_t sum = 0, c0 = 0;
    for (int s = tid; s < p.N; s += THREADS) {
        const int64_t c = tree_cost(p, tree_seq(p, s, flag));
        if (s < THREADS) c0 = c;
        sum += c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += (int64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)sum, o);
    if (lane == 0) buf[warp] = sum;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < NW; ++w) total += buf[w];
    r.per = divide(total + ctas - 1, ctas);  // (a run may hold no tile: a small call's tiles each have a CTA)
    r.lo = r.per * cta;
    r.hi = min(r.lo + r.per, total);
    r.s = 0;
    r.rem = 0;
    if (r.lo >= total) return r;  // uniform: nothing to do
    int64_t before = 0;
    for (int base = 0; base < p.N; base += THREADS) {
        const int s = base + tid;
        const int64_t c = base == 0 ? c0 : (s < p.N ? tree_cost(p, tree_seq(p, s, false)) : 0);
        int64_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = (int64_t)__shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
            if (lane >= o) incl += u;
        }
        __syncthreads();
        if (lane == 31) buf[warp] = incl;
        __syncthreads();
        int64_t pre = before, chunk = 0;
        for (int w = 0; w < NW; ++w) {
            if (w < warp) pre += buf[w];
            chunk += buf[w];
        }
        const int64_t first = pre + incl - c;
        if (c > 0 && first <= r.lo && r.lo < first + c) {
            buf[32] = s;
            buf[33] = r.lo - first;
        }
        before += chunk;
        if (before > r.lo) break;  // uniform
    }
    __syncthreads();
    r.s = (int)buf[32];
    r.rem = buf[33];
    r.q = tree_seq(p, r.s, false);
    return r;
}

// ----------------------------------------------------------------------------- masks

// Bits b = 0..31: whether drafted token `tok` of the sequence sees key k0 + b, j0 = k0 - (context before the draft).
__device__ __forceinline__ uint32_t tree_word(const uint32_t* row, int n, int x) {
    if (x < 0) return 0xffffffffu;
    if (32 * x >= n) return 0u;
    return row[x] & (n - 32 * x < 32 ? (1u << (n - 32 * x)) - 1u : 0xffffffffu);
}
__device__ __forceinline__ uint32_t tree_visible(const TreeParams& p, const TreeSeg& g, int tok, int j0) {
    if (j0 >= g.n) return 0u;
    if (j0 <= -32) return 0xffffffffu;
    const uint32_t* row = p.mask + (size_t)(g.qs + tok) * p.W;
    const int x = j0 >> 5;
    return __funnelshift_r(tree_word(row, g.n, x), tree_word(row, g.n, x + 1), j0 & 31);
}

// Keys k0 .. k0 + 32 NW - 1 that some row of the row tile sees: the same words in every lane.
template <int NW>
__device__ __forceinline__ void tree_union(const TreeParams& p, const TreeSeg& g, int k0, uint32_t (&u)[NW]) {
    const int lane = threadIdx.x & 31, tok0 = g.mt * p.TQ, ntok = min(p.TQ, g.n - tok0);
    uint32_t v[NW] = {};
    for (int t = lane; t < ntok; t += 32)
#pragma unroll
        for (int c = 0; c < NW; ++c) v[c] |= tree_visible(p, g, tok0 + t, k0 + 32 * c - (g.ctx - g.n));
#pragma unroll
    for (int c = 0; c < NW; ++c) u[c] = __reduce_or_sync(0xffffffffu, v[c]);
}

// Scores (64 TMEM columns from t_s on) of keys that are not seen become -inf.
__device__ __forceinline__ void tree_mask_scores(uint32_t t_s, uint32_t see0, uint32_t see1) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        const uint32_t see = (c & 2 ? see1 : see0) >> (16 * (c & 1));
        uint32_t x[16];
        tmem_ld16_async(t_s + 16 * c, x);
        tmem_loaded16(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = see >> i & 1u ? x[i] : 0xff800000u;
        tmem_st16(t_s + 16 * c, x);
    }
    tmem_wait_st();
}

// A row's reference for the probabilities of a tile with the given maximum, and the factor of what was summed before.
__device__ __forceinline__ float tree_reference(float m_tile, bool first, float& m_ref, float& alpha) {
    const float m_new = m_tile > m_ref + 8.f || m_ref == -INFINITY ? fmaxf(m_ref, m_tile) : m_ref;
    alpha = first || m_new == m_ref ? 1.f : fast_exp2(m_ref - m_new);
    m_ref = m_new;
    return m_new == -INFINITY ? 0.f : m_new;
}

// Probabilities of 64 keys with exponents of their own (scale bytes at shared address ex), over the scores at t_s.
// Such tiles are rare and are read twice, 32 columns at a time, out of line: with it in line the code of the usual
// tiles left the instruction cache (a sixth of the time).  Returns the exponential sum, the reference, and the factor
// of what was summed before.
template <typename PT, bool SPLIT>
__device__ __noinline__ float3 tree_probabilities_keyed(uint32_t t_s, uint32_t ex, float mul, bool first, float m_ref) {
    uint32_t x[32] = {}, e = 0;
    // of four neighbouring keys: their bytes; y = score + ev, and 2^-ev
    auto exponents = [&](int at) { asm volatile("ld.shared.u32 %0, [%1];" : "=r"(e) : "r"(ex + at)); };
    auto score = [&](int i, int k) {
        return fmaf(__uint_as_float(x[i + k]), mul, (float)((int)(e >> 8 * k & 0xffu) - kScaleBias));
    };
    auto weight = [&](int k) { return pow2i(kScaleBias - (int)(e >> 8 * k & 0xffu)); };
    float m_tile = -INFINITY, alpha, sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        tmem_ld32_async(t_s + c, x);
        tmem_loaded(x);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            exponents(c + i);
            m_tile = fmax3(fmax3(m_tile, score(i, 0), score(i, 1)), score(i, 2), score(i, 3));
        }
    }
    const float off = -tree_reference(m_tile - kPHeadroom, first, m_ref, alpha);
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        tmem_ld32_async(t_s + c, x);
        tmem_loaded(x);
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            exponents(c + i);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const float2 y = make_float2(fast_exp2(score(i, k) + off), fast_exp2(score(i, k + 1) + off));
                sum = fmaf(y.x, weight(k), fmaf(y.y, weight(k + 1), sum));
                const uint32_t h = Mma<PT>::pack(y.x, y.y);
                hi[(i + k) / 2] = h;
                if (SPLIT) {
                    const float2 f = fsub2(y, Mma<PT>::unpack(h));
                    lo[(i + k) / 2] = Mma<PT>::pack(f.x, f.y);
                }
            }
        }
        const uint32_t at = t_s + (SPLIT ? c : c / 2);  // columns whose scores have been read
        tmem_st16(at, hi);
        if (SPLIT) tmem_st16(at + 16, lo);
    }
    return make_float3(sum, m_ref, alpha);
}

// ----------------------------------------------------------------------------- the kernel

template <int D, bool QUANT>
struct TreeGeo {
    static constexpr int DH = D / 64;
    static constexpr uint32_t kTile = DH * kTRegion;      // one 16-bit tile, [8-row group][column half][8 rows][128 B]
    static constexpr uint32_t kGroup = DH * 1024;
    // V ring slots and K ring slots.  A converted K tile is free again as soon as its score product is done, long
    // before its V: one slot serves, and the space holds another raw tile on its way.
    static constexpr int NS = QUANT ? 2 : 3, KS = QUANT ? 1 : 3;
    static constexpr int KF = QUANT ? 2 : 3;  // "K read" barriers, by tile in turn
    static constexpr int NR = QUANT ? (D == 128 ? 3 : 6) : 0;      // raw ring slots: K and V rows of a tile, scales
    static constexpr uint32_t kRaw = 2u * kTKeys * D, kRawScales = 2 * kTKeys;
    static constexpr uint32_t kExp = QUANT ? kTKeys : 0;           // per V slot: each key's scale byte of V
    // Registers move from the copying and converting warpgroups to the two softmax warpgroups: the launch's share is
    // 96 (640 threads) or 168 (384) each, and 256 * kMore + (kThreads - 256) * kLess is exactly that total.
    static constexpr int kThreads = QUANT ? 640 : 384;
    static constexpr int kMore = QUANT ? 120 : 200, kLess = QUANT ? 80 : 104;
    static_assert(256 * kMore + (kThreads - 256) * kLess == kThreads * (QUANT ? 96 : 168), "register split");
    // Q | K ring | V ring | raw ring | raw scales | exponents | row exchange | query exponents | barriers, small things
    static constexpr uint32_t oK = kTile, oV = oK + KS * kTile, oRaw = oV + NS * kTile, oRawSc = oRaw + NR * kRaw,
                              oExp = oRawSc + NR * kRawScales, oXch = oExp + NS * kExp, oQe = oXch + 2 * kTRows * 4,
                              oBar = oQe + (QUANT ? kTRows : 0);
    static constexpr int kBars = 5 + KS + KF + 2 * NS + 6 + 2 * NR;
    static constexpr uint32_t oSmall = oBar + 8 * kBars;
    static constexpr size_t kSmem = oSmall + 64;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(8 * 40 <= kTile, "the Q tile's space also serves the start");
};

template <typename T, int D, bool QUANT, bool SPLIT>
__global__ void __launch_bounds__(TreeGeo<D, QUANT>::kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ TreeParams p) {
    using Geo = TreeGeo<D, QUANT>;
    constexpr int NS = Geo::NS, KS = Geo::KS, KF = Geo::KF, NR = Geo::NR;
    constexpr int NK = D / 16, NT = kTKeys / 32;  // k-steps of S, and of each warpgroup's value product
    constexpr bool kBf16 = !QUANT && std::is_same<T, __nv_bfloat16>::value;  // type of the products
    using PT = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
    static_assert(!kBf16 || SPLIT, "a bf16 value product takes P in two parts");
    constexpr uint32_t idesc_s = umma_idesc(kBf16, kTRows, kTKeys, false);
    constexpr uint32_t idesc_o = umma_idesc(kBf16, kTRows, D, true);
    constexpr uint32_t kTile = Geo::kTile, kGroup = Geo::kGroup;
    constexpr float NEG_INF = -INFINITY;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sb = smem_addr(smem_raw);
    const uint32_t sQ = sb, sK = sb + Geo::oK, sV = sb + Geo::oV, sBar = sb + Geo::oBar;
    // sfull, prdy, pvd: one for each of the two buffers of scores
    const uint32_t qfull = sBar, qfree = qfull + 8, qread = qfree + 8, sdone = qread + 8, pdone = sdone + 8,
                   kfull = pdone + 8, kfree = kfull + 8 * KS,
                   vfull = kfree + 8 * KF, vfree = vfull + 8 * NS, sfull = vfree + 8 * NS, pvd = sfull + 16,
                   prdy = pvd + 16, rfull = prdy + 16, rfree = rfull + 8 * NR;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + Geo::oSmall);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* armed = abort_flag + 1;  // K, V (quantised: raw) tiles and query tiles whose copies have been issued
    // Of the last four tiles (a tile is converted once the value products of the fourth before it are done): 2^(emax -
    // 7) of its K; the exponent that its V is scaled down by, or kTreeKeyed.
    float* kmul = reinterpret_cast<float*>(tmem_slot + 5);
    float* vexp = kmul + 4;
    int8_t* qexp = reinterpret_cast<int8_t*>(smem_raw + Geo::oQe);  // per query row: exponent it was scaled down by
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // (nothing up to the wait touches global memory: it runs under the kernel before)
    if (tid < Geo::kBars) {
        const uint32_t bar = sBar + 8 * tid;
        int count = 1;
        if (bar == prdy || bar == prdy + 8) count = 256;
        if (QUANT) {
            if (bar == qfull) count = kConvWarps;
            if (bar == qread) count = 8;
            if ((bar >= kfull && bar < kfree) || (bar >= vfull && bar < vfree) || bar >= rfree) count = kConvWarps / 2;
        }
        mbar_init(bar, count);
        fence_mbar_init();
    }
    if (tid == 0) {
        *abort_flag = 0;
        armed[0] = armed[1] = armed[2] = 0;
    }
    griddep_wait();
    griddep_launch_dependents();
    if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);  // before every exit: the merge reads it
    // swizzled tiles need the 1024-byte alignment that dynamic shared memory has when there is no static
    if (sb & 1023u) {
        if (tid == 0) flag_error(p.err, PA_DEV_ERR_TIMEOUT);
        return;
    }
    const TreeRun run =
        tree_run<Geo::kThreads>(p, blockIdx.x, gridDim.x, blockIdx.x == 0, reinterpret_cast<int64_t*>(smem_raw));
    if (run.lo >= run.hi) return;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // A wait that runs out sets the abort flag, after which every other wait returns at once: the softmax warps never
    // leave their loops early, so the barriers between them are always met.
    auto waited = [&](uint32_t bar, uint32_t parity) {
        const bool w = mbar_wait_spin(bar, parity, abort_flag, p.wait_ns);
        if (!w) *abort_flag = 1;
        return w;
    };
    // two waits at once (each barrier's first look costs about a hundred cycles)
    auto waited2 = [&](uint32_t a, uint32_t pa, uint32_t b, uint32_t pb) {
        const bool wa = mbar_try_wait(a, pa), wb = mbar_try_wait(b, pb);
        return (wa || waited(a, pa)) && (wb || waited(b, pb));
    };
    // TMEM columns: the scores of tile t, and on top of a warpgroup's own 64 the P of its 32 keys k (high parts in 16,
    // then low parts in 16)
    auto s_col = [](int t) { return (uint32_t)((t & 1) * kTKeys); };
    auto p_col = [&](int t, int w, int k) { return s_col(t) + (uint32_t)(w * 64 + k * (SPLIT ? 32 : 16)); };
    auto slot = [](int i) { return (uint32_t)(i % NS); };
    auto ph = [](int i) { return (uint32_t)((i / NS) & 1); };
    auto kslot = [](int i) { return (uint32_t)(i % KS); };
    auto kph = [](int i) { return (uint32_t)((i / KS) & 1); };
    bool ok = true;
    TreeWalk walk;
    walk.start(run.q, run.s, run.rem, run.hi - run.lo);
    TreeSeg g;
    const int B = 1 << p.lgB;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Geo::kLess));
        if (warp == 8) {
            // -------------------------------------------------------- TMA producer: lane b copies the tile's block b
            const uint64_t pol = policy_evict_first();
            int t = 0;  // tiles so far
            for (int seg = 0; ok && walk.next(p, g); ++seg) {
                auto entry = [&](int j) {
                    const int nblk = (min(kTKeys, g.ctx - j * kTKeys) + B - 1) >> p.lgB;
                    return lane < nblk ? p.tables[(size_t)g.s * p.MB + ((size_t)j * kTKeys >> p.lgB) + lane] : 0;
                };
                int mine = entry(g.j0);
                if constexpr (!QUANT) {
                    // the query rows, once the last segment's score products have read theirs
                    if (seg > 0) ok = waited(qfree, (uint32_t)((seg - 1) & 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        armed[2] = seg + 1;
                        mbar_arrive_expect_tx(qfull, (uint32_t)(D / 64) * p.G * p.TQ * 128);
                        for (int dh = 0; dh < D / 64; ++dh)
                            tma_load_4d(sQ + dh * kTRegion, &tm_q, qfull, 0, dh, g.h * p.G, g.qs + g.mt * p.TQ, pol);
                    }
                    __syncwarp();
                }
                for (int j = g.j0; j < g.j1 && ok; ++j, ++t) {
                    const int nblk = (min(kTKeys, g.ctx - j * kTKeys) + B - 1) >> p.lgB;
                    int e = mine;
                    if (j + 1 < g.j1) mine = entry(j + 1);
                    const bool good = (unsigned)e < (unsigned)p.NB;
                    if (lane < nblk && !good) flag_error(p.err, PA_DEV_ERR_BLOCK);
                    if (!good) e = p.NB;  // past the tensor: TMA fills zeros
                    if constexpr (QUANT) {
                        const uint32_t b = (uint32_t)(t % NR), bar = rfull + 8 * b;
                        if (t >= NR) ok = waited(rfree + 8 * b, (uint32_t)((t / NR - 1) & 1));
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lane == 0) {
                            armed[0] = t + 1;  // expect_tx and every copy below, with no wait in between
                            mbar_arrive_expect_tx(bar, (uint32_t)nblk * 2 * B * (D + 1));
                        }
                        __syncwarp();
                        if (lane < nblk) {
                            tma_load_3d(sb + Geo::oRaw + b * Geo::kRaw + (uint32_t)lane * 2 * B * D, &tm, bar, 0, 0,
                                        e * p.H_kv + g.h, pol);
                            bulk_load(sb + Geo::oRawSc + b * Geo::kRawScales + (uint32_t)lane * 2 * B,
                                      p.scales + ((size_t)(good ? e : 0) * p.H_kv + g.h) * (2 * B), 2 * B, bar);
                        }
                    } else {
                        const uint32_t b = slot(t);
                        for (int which = 0; which < 2 && ok; ++which) {
                            if (t >= NS) ok = waited((which ? vfree : kfree) + 8 * b, ph(t - NS));
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            const uint32_t bar = (which ? vfull : kfull) + 8 * b;
                            if (lane == 0) {
                                armed[which] = t + 1;  // as above
                                mbar_arrive_expect_tx(bar, (uint32_t)nblk * B * D * 2);
                            }
                            __syncwarp();
                            if (lane < nblk)
                                tma_load_5d((which ? sV : sK) + b * kTile + (uint32_t)lane * B * D * 2, &tm, bar, 0, 0,
                                            0, e * (B / 8), which * p.H_kv + g.h, pol);
                        }
                    }
                }
            }
        } else if (warp == 9) {
            // -------------------------------------------------------- score products
            if (lane == 0) {
                const uint64_t dq = umma_desc(sQ, 16, 1024);
                int t = 0;
                for (int seg = 0; ok && walk.next(p, g); ++seg) {
                    ok = waited(qfull, (uint32_t)(seg & 1));
                    for (int j = g.j0; j < g.j1 && ok; ++j, ++t) {
                        // the buffer is free once the value products of the tile before last have read its P
                        ok = t < 2 ? waited(kfull + 8 * kslot(t), kph(t))
                                   : waited2(pvd + 8 * (t & 1), (uint32_t)((t - 2) >> 1 & 1),
                                             kfull + 8 * kslot(t), kph(t));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t dk = umma_desc(sK + kslot(t) * kTile, 16, kGroup);
#pragma unroll
                        for (int ks = 0; ks < NK; ++ks)
                            umma_f16(tmem + s_col(t), dq + (ks >> 2) * (kTRegion >> 4) + (ks & 3) * 2,
                                     dk + (ks >> 2) * (1024 >> 4) + (ks & 3) * 2, idesc_s, ks > 0);
                        umma_commit(sfull + 8 * (t & 1));
                        umma_commit(kfree + 8 * (t % KF));
                    }
                    if (ok) umma_commit(qfree);  // (never before the rows have landed)
                }
                umma_commit(sdone);  // arrives once every product issued above has completed
            }
            __syncwarp();
        } else if (warp == 10) {
            // -------------------------------------------------------- value products
            if (lane == 0) {
                int t = 0;
                while (ok && walk.next(p, g)) {
                    for (int j = g.j0; j < g.j1 && ok; ++j, ++t) {
                        // (every softmax thread ready also means that all have read the last segment's O)
                        ok = waited2(vfull + 8 * slot(t), ph(t), prdy + 8 * (t & 1), (uint32_t)((t >> 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t dv = umma_desc(sV + slot(t) * kTile, 1024, kGroup);
                        // products of the two accumulators in turn: a product need not wait for the one before it
#pragma unroll
                        for (int ks = 0; ks < NT; ++ks) {
#pragma unroll
                            for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
                                for (int w = 0; w < 2; ++w)
                                    umma_f16_ta(tmem + 2 * kTKeys + (uint32_t)w * D,
                                                tmem + p_col(t, w, ks >> 1) + (ks & 1) * 8 + part * 16,
                                                dv + (uint64_t)((w * NT + ks) * ((2 * kGroup) >> 4)), idesc_o,
                                                j > g.j0 || ks > 0 || part > 0);
                        }
                        umma_commit(pvd + 8 * (t & 1));
                        umma_commit(vfree + 8 * slot(t));
                    }
                }
                umma_commit(pdone);
            }
            __syncwarp();
        } else if (warp >= 12) {
            // -------------------------------------------------------- converters (quantised pool)
            if constexpr (QUANT) {
                const int cw = warp - 12;
                // Four warps to a tile, so that one group's waits and scales run under the other's conversion.  A lane
                // converts a row, 16 values at a time, so that the row's factor stays in a register; eight neighbouring
                // rows' pieces lie in eight different bank groups on both sides, swizzled as they are.
                const int row = 32 * (cw & 3) + lane, mb = ~(B - 1);
                const uint32_t so = (uint32_t)(row + (row & mb)) * D, ro = (uint32_t)(row + (row & mb));
                const uint32_t to = (uint32_t)(row >> 3) * kGroup + (row & 7) * 128;
                int t = 0;
                for (int seg = 0; walk.next(p, g); ++seg) {
                    // the query rows as fp16, four lanes to a row: read, then written once the last segment's have been
                    // used
                    {
                        constexpr int C = D / 32;                   // 16-byte pieces of a row per lane
                        constexpr int R = kTRows / 8 / kConvWarps;  // rows per lane
                        const int tok0 = g.mt * p.TQ, rows = min(p.TQ, g.n - tok0) * p.G;
                        uint4 xs[R][C];
#pragma unroll
                        for (int k = 0; k < R; ++k) {
                            const int r = (cw + k * kConvWarps) * 8 + (lane >> 2);
                            const size_t row =
                                ((size_t)(g.qs + tok0 + r / p.G) * p.H_q + (size_t)g.h * p.G + r % p.G) * D;
                            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + row);
#pragma unroll
                            for (int i = 0; i < C; ++i)
                                xs[k][i] = r < rows ? src[4 * i + (lane & 3)] : make_uint4(0, 0, 0, 0);
                        }
                        if (seg > 0) {
                            ok = waited(qfree, (uint32_t)((seg - 1) & 1)) && ok;
                            ok = waited(qread, (uint32_t)((seg - 1) & 1)) && ok;
                        }
#pragma unroll
                        for (int k = 0; k < R; ++k) {
                            const int r = (cw + k * kConvWarps) * 8 + (lane >> 2);
                            uint4 (&x)[C] = xs[k];
                            int e = 0;
                            if (p.q_bf16) {
                                float a = 0.f;
#pragma unroll
                                for (int i = 0; i < C; ++i) {
                                    const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const float2 f = Mma<__nv_bfloat16>::unpack(v[k]);
                                        a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
                                    }
                                }
                                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                                // largest magnitude to [2^14, 2^15), as in decode_quant.cu
                                const int ex = (int)(__float_as_uint(a) >> 23) - 127;
                                e = ex > 127 || a == 0.f ? 0 : max(ex - 14, -126);
                                const float inv = pow2i(-e);
#pragma unroll
                                for (int i = 0; i < C; ++i) {
                                    uint32_t* v = reinterpret_cast<uint32_t*>(&x[i]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const float2 f = Mma<__nv_bfloat16>::unpack(v[k]);
                                        v[k] = Mma<__half>::pack(f.x * inv, f.y * inv);
                                    }
                                }
                            }
                            if ((lane & 3) == 0) qexp[r] = (int8_t)e;
#pragma unroll
                            for (int i = 0; i < C; ++i) {
                                const int ch = 4 * i + (lane & 3);  // piece of the row
                                const uint32_t dst =
                                    sQ + (uint32_t)(ch >> 3) * kTRegion + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst),
                                             "r"(x[i].x), "r"(x[i].y), "r"(x[i].z), "r"(x[i].w)
                                             : "memory");
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(qfull);
                    }
                    for (int j = g.j0; j < g.j1; ++j, ++t) {
                        if ((t & 1) != cw >> 2) continue;
                        const int k0 = j * kTKeys;
                        const uint32_t rb = (uint32_t)(t % NR);
                        const uint32_t raw = sb + Geo::oRaw + rb * Geo::kRaw;
                        const uint32_t rsc = sb + Geo::oRawSc + rb * Geo::kRawScales;
                        uint32_t u[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                        const bool masked = k0 + kTKeys > g.ctx - g.n;
                        if (masked) tree_union<4>(p, g, k0, u);  // keys past the context are in none
                        const uint32_t sl = slot(t);
                        ok = waited(rfull + 8 * rb, (uint32_t)((t / NR) & 1)) && ok;
                        // lane: keys 4 lane .. + 3, all of one block; the largest exponents of the keys that are seen
                        const uint32_t at = rsc + 4 * lane + ((4 * lane) & mb);
                        uint32_t kb, vb;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kb) : "r"(at));
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vb) : "r"(at + B));
                        uint32_t vlow = vb;  // (for the least of V's)
                        if (masked) {  // bytes of keys nobody sees: the least scale (for the least of V's: the largest)
                            const uint32_t four = u[lane >> 3] >> (4 * lane & 31) & 0xfu;
                            const uint32_t m = (four * 0x00204081u & 0x01010101u) * 255u;
                            kb = (kb & m) | (~m & 0x57575757u);
                            vlow = (vb & m) | (~m & 0xa7a7a7a7u);
                            vb = (vb & m) | (~m & 0x57575757u);
                        }
                        // largest of K's, largest and least of V's, held to the range the writer produces
                        const uint32_t kx = vmax_u16x2(kb & 0x00ff00ffu, kb >> 8 & 0x00ff00ffu);
                        const uint32_t vx = vmax_u16x2(vb & 0x00ff00ffu, vb >> 8 & 0x00ff00ffu);
                        const uint32_t vn = vmin_u16x2(vlow & 0x00ff00ffu, vlow >> 8 & 0x00ff00ffu);
                        const int em = clamp_scale(__reduce_max_sync(0xffffffffu, max(kx & 0xffffu, kx >> 16)));
                        const int vm = clamp_scale(__reduce_max_sync(0xffffffffu, max(vx & 0xffffu, vx >> 16)));
                        const int vl = clamp_scale(__reduce_min_sync(0xffffffffu, min(vn & 0xffffu, vn >> 16)));
                        const bool keyed = vm - vl > kTreeSpan;
                        // fp16 factors 2^(e - max + 7) of this lane's row: exponent field e - max + 7 + 15, or a factor
                        // of zero where that is not positive.  V8 as it is when keyed.  A row that nobody sees, past
                        // the context or padding, may hold anything: it counts as zeros.
                        const bool seen = u[cw & 3] >> lane & 1u;
                        uint32_t bk, bv;
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(bk) : "r"(rsc + ro));
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(bv) : "r"(rsc + ro + B));
                        const int ek = clamp_scale(bk), ev = clamp_scale(bv);
                        const uint32_t fk = seen ? (uint32_t)max(ek - em + 22, 0) * 0x04000400u : 0u;
                        const uint32_t scaled = keyed ? 0x3c003c00u : (uint32_t)max(ev - vm + 22, 0) * 0x04000400u;
                        const uint32_t fv = seen ? scaled : 0u;
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {  // K's and V's row, in halves
                            const int which = i >> 1, c0 = (i & 1) * (D / 32);
                            const uint32_t f2 = which ? fv : fk;
                            // the last K tile's score product has read it; the last V in this slot is used up
                            if (i == 0 && t >= 1)
                                ok = waited(kfree + 8 * ((t - 1) % KF), (uint32_t)((t - 1) / KF & 1)) && ok;
                            if (i == 2 && t >= NS) ok = waited(vfree + 8 * sl, ph(t - NS)) && ok;
                            // addresses of the half's pieces differ from its first's in the swizzled bits only
                            const uint32_t src =
                                raw + so + (which ? B * D : 0) + ((c0 ^ (D == 128 ? row & 7 : row >> 1 & 3)) << 4);
                            const uint32_t dst =
                                (which ? sV + sl * kTile : sK) + to +
                                (D == 128 ? (i & 1) * 1024 + ((row & 7) << 4) : ((2 * c0) ^ (row & 7)) << 4);
                            uint4 vs[D / 32];  // all read before the first is converted
#pragma unroll
                            for (int cc = 0; cc < D / 32; ++cc)
                                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(vs[cc].x), "=r"(vs[cc].y), "=r"(vs[cc].z), "=r"(vs[cc].w)
                                             : "r"(src ^ (cc << 4)));
                            if (masked && !seen) {  // (zero times NaN is NaN)
#pragma unroll
                                for (int cc = 0; cc < D / 32; ++cc) vs[cc] = make_uint4(0u, 0u, 0u, 0u);
                            }
#pragma unroll
                            for (int cc = 0; cc < D / 32; ++cc) {
                                const uint4 v = vs[cc];
                                uint32_t h[8] = {e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y),
                                                 e4m3x2_to_f16x2(v.y >> 16), e4m3x2_to_f16x2(v.z),
                                                 e4m3x2_to_f16x2(v.z >> 16), e4m3x2_to_f16x2(v.w),
                                                 e4m3x2_to_f16x2(v.w >> 16)};
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[k]),
                                                              *reinterpret_cast<const __half2*>(&f2));
                                    h[k] = *reinterpret_cast<const uint32_t*>(&y);
                                }
#pragma unroll
                                for (int o = 0; o < 2; ++o)
                                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                                     dst ^ ((2 * cc + o) << 4)),
                                                 "r"(h[4 * o]), "r"(h[4 * o + 1]), "r"(h[4 * o + 2]), "r"(h[4 * o + 3])
                                                 : "memory");
                            }
                            if (i == 2 && keyed) smem_raw[Geo::oExp + sl * Geo::kExp + row] = (uint8_t)ev;
                            if (i == 1 && row == 0) {
                                kmul[t & 3] = pow2i(em - kScaleBias - 7);
                                vexp[t & 3] = keyed ? kTreeKeyed : (float)(vm - kScaleBias - 7);
                            }
                            if (c0 == 0) continue;
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(which ? vfull + 8 * sl : kfull);
                        }
                        if (lane == 0 && ok) mbar_arrive(rfree + 8 * rb);  // (never before its copies have landed)
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Geo::kMore));
        // ------------------------------------------------------------ softmax warpgroup w: keys 64 w .. of each tile
        const int w = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_o = lanes + 2 * kTKeys;
        const int r = tid & (kTRows - 1);
        const uint32_t pair = 1 + (warp & 3);  // named barrier of the two warps that hold the same rows
        float* xch = reinterpret_cast<float*>(smem_raw + Geo::oXch);
        int t = 0;  // tiles so far
        while (walk.next(p, g)) {
            const int tok0 = g.mt * p.TQ, rows = min(p.TQ, g.n - tok0) * p.G;
            const int tok = tok0 + r / p.G;
            const bool row_ok = r < rows, warp_ok = (warp & 3) * 32 < rows;
            const int base = g.ctx - g.n;  // keys before the draft
            float cr = p.scale_log2;
            float m_ref = NEG_INF, l = 0.f;
            for (int j = g.j0; j < g.j1; ++j, ++t) {
                const int k0 = j * kTKeys + 64 * w;  // the warpgroup's first key
                const uint32_t par = (uint32_t)(t >> 1 & 1);
                const uint32_t t_s = lanes + s_col(t) + (uint32_t)w * 64;
                const bool masked = k0 + 64 > base;
                uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
                if (masked) {
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t v = row_ok ? tree_visible(p, g, tok, k0 + 32 * k - base) : 0u;
                        if (k == 0)
                            vis[0] = v;
                        else
                            vis[1] = v;
                    }
                }
                ok = waited(sfull + 8 * (t & 1), par) && ok;
                tc_fence_after();
                if (QUANT) {
                    if (j == g.j0) {
                        cr = p.scale_log2 * pow2i((int)qexp[r]);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(qread);
                    }
                }
                float alpha = 1.f;
                // E is the exponent of every key: the scores stay in registers.
                auto probabilities = [&](float mul, float E) {
                    uint32_t s[2][32];
                    tmem_ld32_async(t_s, s[0]);
                    tmem_ld32_async(t_s + 32, s[1]);
                    tmem_loaded(s[0]);
                    tmem_loaded(s[1]);
                    float mx[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
                    for (int k = 0; k < 64; k += 8) {
                        const uint32_t* x = &s[k >> 5][k & 31];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mx[i] = fmax3(mx[i], __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                    }
                    const float top = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                    const float m_tile = fmaf(top, mul, E) - kPHeadroom;  // (mul > 0: -inf stays so)
                    const float off = E - tree_reference(m_tile, j == g.j0, m_ref, alpha);
                    const float2 mul2 = make_float2(mul, mul), off2 = make_float2(off, off);
                    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t hi[2][16], lo[2][16];
#pragma unroll
                    for (int k = 0; k < 64; k += 2) {
                        const uint32_t* y = &s[k >> 5][k & 31];
                        float2 x = ffma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), mul2, off2);
                        x.x = fast_exp2(x.x);
                        x.y = fast_exp2(x.y);
                        ls[(k >> 1) & 1] = fadd2(ls[(k >> 1) & 1], x);
                        const uint32_t h = Mma<PT>::pack(x.x, x.y);
                        hi[k >> 5][(k & 31) / 2] = h;
                        if (SPLIT) {
                            const float2 f = fsub2(x, Mma<PT>::unpack(h));
                            lo[k >> 5][(k & 31) / 2] = Mma<PT>::pack(f.x, f.y);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        tmem_st16(lanes + p_col(t, w, k), hi[k]);
                        if (SPLIT) tmem_st16(lanes + p_col(t, w, k) + 16, lo[k]);
                    }
                    const float2 lsum = fadd2(ls[0], ls[1]);
                    float sum = lsum.x + lsum.y;
                    if (QUANT) sum *= pow2i(-(int)E);
                    l = fmaf(l, alpha, sum);
                };
                if (warp_ok) {
                    // The product may leave fp32's range downwards (small queries; 2^-47 of a tile that nobody sees), and
                    // -inf times zero is NaN: it is held to 2^-126.  A raw score is at most 2^39, so that moves a score
                    // by 2^-87 at most.
                    const float mul = QUANT ? fmaxf(cr * kmul[t & 3], 0x1p-126f) : cr;
                    const float E = QUANT ? vexp[t & 3] : 0.f;
                    if (masked) tree_mask_scores(t_s, vis[0], vis[1]);
                    if (QUANT && E == kTreeKeyed) {
                        ok = waited(vfull + 8 * slot(t), ph(t)) && ok;  // the exponents, with V
                        const uint32_t ex = sb + Geo::oExp + slot(t) * Geo::kExp + 64 * w;
                        const float3 r = tree_probabilities_keyed<PT, SPLIT>(t_s, ex, mul, j == g.j0, m_ref);
                        m_ref = r.y;
                        alpha = r.z;
                        l = fmaf(l, alpha, r.x);
                    } else {
                        probabilities(mul, E);
                    }
                    // O_w is rescaled (rarely) once the last tile's products have landed
                    if (__any_sync(0xffffffffu, alpha != 1.f)) {
                        ok = waited(pvd + 8 * ((t - 1) & 1), (uint32_t)(((t - 1) >> 1) & 1)) && ok;
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[16];
                            tmem_ld16_async(t_o + (uint32_t)w * D + k, o);
                            tmem_loaded16(o);
#pragma unroll
                            for (int b = 0; b < 16; ++b) o[b] = __float_as_uint(__uint_as_float(o[b]) * alpha);
                            tmem_st16(t_o + (uint32_t)w * D + k, o);
                        }
                    }
                    tmem_wait_st();
                }
                if (!QUANT && masked) {
                    // V rows nobody sees (past the context, padding) may hold anything, even NaN: zeros before the
                    // products meet them with P = 0.  Two threads to a row, one per half of it.
                    uint32_t u[2];
                    tree_union<2>(p, g, k0, u);
                    ok = waited(vfull + 8 * slot(t), ph(t)) && ok;
                    const int rr = (r & 63), key = 64 * w + rr;
                    if (!(u[rr >> 5] >> (rr & 31) & 1u)) {
                        const uint32_t vr = sV + slot(t) * kTile + (uint32_t)(key >> 3) * kGroup + (key & 7) * 128;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const int k = (r >> 6) * (D / 16) + i;
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vr + (k >> 3) * 1024 +
                                                                                          (k & 7) * 16),
                                         "r"(0)
                                         : "memory");
                        }
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                mbar_arrive(prdy + 8 * (t & 1));
            }
            // The two warps of the same rows exchange their maxima, then their sums, and each joins and stores one half
            // of the columns once the last products have landed.
            xch[w * kTRows + r] = m_ref;
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            const float m_other = xch[(w ^ 1) * kTRows + r];
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            xch[w * kTRows + r] = l;
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            const float l_other = xch[(w ^ 1) * kTRows + r];
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            const float M = fmaxf(m_ref, m_other);
            const float fo = m_ref == NEG_INF ? 0.f : fast_exp2(m_ref - M);
            const float fx = m_other == NEG_INF ? 0.f : fast_exp2(m_other - M);
            const float f0 = w ? fx : fo, f1 = w ? fo : fx;
            // both warps sum in the same order (a NaN exponential sum stays one)
            const float den = w ? l_other * f0 + l * f1 : l * f0 + l_other * f1;
            const bool whole = g.j0 == 0 && g.j1 == g.nt;
            const int part = 2 * blockIdx.x + (g.j0 == 0 ? 1 : 0);
            const size_t orow = ((size_t)(g.qs + tok) * p.H_q + (size_t)g.h * p.G + r % p.G) * D;
            const float inv = den == 0.f ? 0.f : 1.f / den;  // a row that sees nothing is zero
            ok = waited(pvd + 8 * ((t - 1) & 1), (uint32_t)(((t - 1) >> 1) & 1)) && ok;
            tc_fence_after();
            if (warp_ok) {
                // whole 32-byte sectors per lane where `out` or the workspace is aligned to them (a caller need align
                // either to 16 bytes only): half the store instructions.  (16 columns at a time: the code of a unit's
                // end is seldom in the instruction cache, so it is kept short.)
                const void* to = whole ? p.out : p.part_acc;
                const bool sector = (reinterpret_cast<uintptr_t>(to) & 31u) == 0;
                const bool f32 = !whole || p.out_dtype == PA_F32;
                const float f = whole ? inv : 1.f;
                const float g0 = den == 0.f && whole ? 0.f : f0 * f, g1 = den == 0.f && whole ? 0.f : f1 * f;
                char* dst = whole ? static_cast<char*>(p.out) + orow * (f32 ? 4 : 2)
                                  : reinterpret_cast<char*>(p.part_acc + ((size_t)part * kTRows + r) * D);
#pragma unroll 1
                for (int col = w * (D / 2); col < (w + 1) * (D / 2); col += 16) {
                    uint32_t a[16], b[16];
                    tmem_ld16_async(t_o + col, a);
                    tmem_ld16_async(t_o + D + col, b);
                    tmem_loaded16(a);
                    tmem_loaded16(b);
                    // an accumulator whose keys the row does not see holds nothing of it
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        a[x] = __float_as_uint((g0 == 0.f ? 0.f : __uint_as_float(a[x]) * g0) +
                                               (g1 == 0.f ? 0.f : __uint_as_float(b[x]) * g1));
                    if (row_ok && ok) {
                        if (f32) {
                            st_words8(dst + 4 * col, a, sector);
                            st_words8(dst + 4 * col + 32, a + 8, sector);
                        } else {
                            uint32_t h[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float lo = __uint_as_float(a[2 * x]), up = __uint_as_float(a[2 * x + 1]);
                                h[x] = p.out_dtype == PA_BF16 ? Mma<__nv_bfloat16>::pack(lo, up)
                                                              : Mma<__half>::pack(lo, up);
                            }
                            st_words8(dst + 2 * col, h, sector);
                        }
                    }
                }
            }
            if (!whole && row_ok && ok && w == 0)
                reinterpret_cast<float2*>(p.part_ml)[(size_t)part * kTRows + r] = make_float2(M, den);
            if (tid == 0 && g.j0 == 0 && !whole)
                p.desc[blockIdx.x] = make_int4(g.s, g.h, g.mt, 1 + (int)divide(g.nt - g.j1 + run.per - 1, run.per));
            tc_fence_before();  // O may be started afresh once this thread's next P is ready
        }
    }
    // Nothing issued may still be running when TMEM and shared memory are released: the tensor-core products (their
    // threads' last commits) and the copies (the last arm of every stage; earlier ones were consumed before it).
    if ((warp == 9 || warp == 10) && lane == 0) mbar_wait_bounded(warp == 9 ? sdone : pdone, 0, nullptr);
    if (warp == 8 && lane == 0) {
        if constexpr (QUANT) {
            const int n = armed[0];
            for (int b = 0; b < NR && b < n; ++b)
                mbar_wait_bounded(rfull + 8 * b, (uint32_t)(((n - 1 - b) / NR) & 1), nullptr);
        } else {
            for (int which = 0; which < 2; ++which) {
                const int n = armed[which];
                for (int b = 0; b < NS && b < n; ++b)
                    mbar_wait_bounded((which ? vfull : kfull) + 8 * b, (uint32_t)(((n - 1 - b) / NS) & 1), nullptr);
            }
            if (armed[2] > 0) mbar_wait_bounded(qfull, (uint32_t)((armed[2] - 1) & 1), nullptr);
        }
    }
    tc_fence_before();
    ok = __syncthreads_and(ok && !*abort_flag);
    if (!ok && tid == 0) flag_error(p.err, PA_DEV_ERR_TIMEOUT);
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTTmem) : "memory");
    }
}

// ----------------------------------------------------------------------------- joining the partial results

// Block (c, y): the unit CTA c started and left unfinished, rows 8 y .. + 7, one warp each.  Piece 0 is CTA c's last
// segment, piece i CTA c + i's first.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p) {
    constexpr int V = D / 32, kChunk = 8;
    griddep_wait();
    griddep_launch_dependents();
    const int4 d = p.desc[blockIdx.x];
    if (d.w < 2) return;
    const TreeSeq q = tree_seq(p, d.x, false);
    const int tok0 = d.z * p.TQ, rows = min(p.TQ, q.n - tok0) * p.G;
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= rows) return;
    auto at = [&](int i) { return ((size_t)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * kTRows + r); };
    float M = -INFINITY, den = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
    for (int b = 0; b < d.w; b += kChunk) {
        const int n = min(kChunk, d.w - b);
        const float2 ml =
            lane < n ? reinterpret_cast<const float2*>(p.part_ml)[at(b + lane)] : make_float2(-INFINITY, 0.f);
        float a[kChunk][V];
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) a[j][v] = j < n ? p.part_acc[at(b + j) * D + lane * V + v] : 0.f;
        float mc = ml.x;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, k));
        const float Mn = fmaxf(M, mc);
        const float f = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
        const float wl = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - Mn);
        M = Mn;
        den = den * f + wl * ml.y;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= f;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const float wj = __shfl_sync(0xffffffffu, wl, j);
            if (wj != 0.f) {  // a piece in which the row sees nothing counts for nothing
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = fmaf(wj, a[j][v], o[v]);
            }
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) den += __shfl_xor_sync(0xffffffffu, den, k);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const size_t row = ((size_t)(q.qs + tok0 + r / p.G) * p.H_q + (size_t)d.y * p.G + r % p.G) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float x = den == 0.f ? 0.f : o[v] * inv;
        if (p.out_dtype == PA_F32)
            static_cast<float*>(p.out)[row + v] = x;
        else if (p.out_dtype == PA_BF16)
            static_cast<__nv_bfloat16*>(p.out)[row + v] = from_float<__nv_bfloat16>(x);
        else
            static_cast<__half*>(p.out)[row + v] = from_float<__half>(x);
    }
}

// ----------------------------------------------------------------------------- host side

struct TreeWorkspace {
    size_t ml, acc, total;
};

static TreeWorkspace tree_workspace(int D) {
    TreeWorkspace w;
    w.ml = (sizeof(int4) * kTreeMaxCtas + 255) & ~size_t(255);
    w.acc = w.ml + sizeof(float) * 2 * 2 * kTreeMaxCtas * kTRows;
    w.total = w.acc + sizeof(float) * 2 * kTreeMaxCtas * kTRows * D;
    return w;
}

size_t tree_workspace_bytes(int N, int H_q, int H_kv, int D, int max_q_len) {
    if (N <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || (D != 64 && D != 128) || max_q_len <= 0) return 0;
    return tree_workspace(D).total;
}

template <typename T, int D, bool QUANT, bool SPLIT>
static pa_status run_tree(const TreeParams& p, const CUtensorMap& tm, const CUtensorMap& tm_q, int ctas,
                          cudaStream_t stream) {
    using Geo = TreeGeo<D, QUANT>;
    auto kern = tree_kernel<T, D, QUANT, SPLIT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(tree)");
    e = launch_kernel(kern, dim3(ctas), dim3(Geo::kThreads), Geo::kSmem, stream, tm, tm_q, p);
    count_launch();
    if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
    const int rows = std::min(p.TQ, p.max_q_len) * p.G;  // of a row tile at most
    e = launch_kernel(tree_merge_kernel<D>, dim3(ctas, (rows + 7) / 8), dim3(256), 0, stream, p);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "tree merge launch");
}

template <int D>
static pa_status dispatch_tree(const TreeArgs& a, const TreeParams& p, const CUtensorMap& tm, const CUtensorMap& tm_q,
                               int ctas) {
    const bool f32 = a.out_dtype == PA_F32;
    if (a.scales)
        return f32 ? run_tree<__half, D, true, true>(p, tm, tm_q, ctas, a.stream)
                   : run_tree<__half, D, true, false>(p, tm, tm_q, ctas, a.stream);
    if (a.q_dtype == PA_BF16) return run_tree<__nv_bfloat16, D, false, true>(p, tm, tm_q, ctas, a.stream);
    return f32 ? run_tree<__half, D, false, true>(p, tm, tm_q, ctas, a.stream)
               : run_tree<__half, D, false, false>(p, tm, tm_q, ctas, a.stream);
}

pa_status launch_tree(const TreeArgs& a) {
    const TreeWorkspace w = tree_workspace(a.D);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    TreeParams p;
    p.q = a.q;
    p.q_bf16 = a.q_dtype == PA_BF16;
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.q_start = a.q_start;
    p.mask = a.mask;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.W = a.mask_words;
    p.N = a.N;
    p.T = a.T;
    p.H_q = a.H_q;
    p.H_kv = a.H_kv;
    p.G = a.H_q / a.H_kv;
    p.TQ = kTRows / p.G;
    p.lgB = a.B == 8 ? 3 : a.B == 16 ? 4 : 5;
    p.MB = a.MB;
    p.NB = a.NB;
    p.max_q_len = a.max_q_len;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);  // log2(e)
    p.desc = reinterpret_cast<int4*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + w.ml);
    p.part_acc = reinterpret_cast<float*>(ws + w.acc);
    p.wait_ns = wait_limit_ns();
    p.err = a.dev_err;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    const int ctas = std::max(1, std::min(sms, kTreeMaxCtas));
    CUtensorMap tm, tm_q;
    std::memset(&tm_q, 0, sizeof tm_q);
    pa_status st;
    if (a.scales) {
        st = quant_tensor_map(&tm, a.pool, a.NB, a.H_kv, a.B, a.D);
    } else {
        const CUtensorMapDataType dt =
            a.q_dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        // queries [T][H_q][D]: dims 64 columns, column half, head, token; box = a row tile's half
        const cuuint64_t qd[4] = {64, (cuuint64_t)a.D / 64, (cuuint64_t)a.H_q, (cuuint64_t)a.T};
        const cuuint64_t qs[3] = {128, (cuuint64_t)a.D * 2, (cuuint64_t)a.H_q * a.D * 2};
        const cuuint32_t qb[4] = {64, 1, (cuuint32_t)p.G, (cuuint32_t)p.TQ};
        st = encode_tensor_map(&tm_q, dt, 4, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != PA_OK) return st;
        // the pool [NB][B][2][H_kv][D]: dims 64 columns, token within a group of 8, column half, group of 8 tokens
        // (over all blocks), K/V x KV head; box = the K or V rows of one block and head
        const cuuint64_t dims[5] = {64, 8, (cuuint64_t)a.D / 64, (cuuint64_t)a.NB * a.B / 8, (cuuint64_t)2 * a.H_kv};
        const cuuint64_t str[4] = {(cuuint64_t)2 * a.H_kv * a.D * 2, 128, (cuuint64_t)8 * 2 * a.H_kv * a.D * 2,
                                   (cuuint64_t)a.D * 2};
        const cuuint32_t box[5] = {64, 8, (cuuint32_t)a.D / 64, (cuuint32_t)(a.B / 8), 1};
        st = encode_tensor_map(&tm, dt, 5, a.pool, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (st != PA_OK) return st;
    return a.D == 128 ? dispatch_tree<128>(a, p, tm, tm_q, ctas) : dispatch_tree<64>(a, p, tm, tm_q, ctas);
}

}  // namespace pa
