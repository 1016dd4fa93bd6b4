// select.cu -- the blocks of each (sequence, KV head) that block-sparse decode reads, by their key summaries.
//
// Two kernels per call: the scores (the format and the score are in summary.cuh), then the top_k of each row -- one
// (sequence, KV head).  Up to a few hundred rows take one kernel instead, a cluster of CTAs per row, whose scores meet
// in the shared memory of one of them.
//
// Bound by the boxes' bytes, 2 D + 1 per (block, head), and by the latency around them.  64 sequences of up to 16384
// tokens (8 heads, 74 MB of boxes) take 24.5 us, of which 15 stream the boxes at 4.9 TB/s and 5 find the top_k; 16 of
// 32768 (68 MB, one kernel) 20 us; 1 of 16384 4.7 us on the device, a chain of five dependent reads and the search.
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "runs.cuh"
#include "summary.cuh"

namespace pa {

struct SelectParams {
    int32_t* selected;
    const void* q;
    const int8_t* boxes;
    const uint8_t* box_scales;
    const int32_t* tables;
    const int32_t* ctx_lens;
    uint32_t* keys;  // [N][H_kv][stride], ordered as the scores
    int64_t stride;
    int N, H_kv, G, lgB, MB, NB, max_ctx, top_k, sink, recent;
    int cluster;  // CTAs per row where a row is selected by one cluster
    int* err;
};

// Blocks of sequence s, 0 where its length is out of range.
__device__ __forceinline__ int context_blocks(const SelectParams& p, int s) {
    const int ctx = p.ctx_lens[s];
    return ctx < 1 || ctx > p.max_ctx || ctx > (int64_t)p.MB << p.lgB ? 0 : (ctx + (1 << p.lgB) - 1) >> p.lgB;
}

// Unsigned integers order as the floats do.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Scores: mma.sync m16n8k16 with 16 blocks on M and the query heads of the KV head on N.  max(q lo, q hi) is q hi for q
// >= 0 and q lo below, so a box's score is one product of length 2 D, [max(q, 0), min(q, 0)] . [hi, lo]; box and query
// integers are exact in fp16.
constexpr int kScoreWarps = 4;
constexpr int kScoreCtas = 5;  // per SM: 96 registers

// Four 8-bit integers as two fp16 pairs: v + 128 in the low byte of 0x6400 is 1024 + 128 + v.
__device__ __forceinline__ void int8x4_to_f16(uint32_t x, uint32_t& a, uint32_t& b) {
    const uint32_t u = x ^ 0x80808080u;
    const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
    uint32_t r0 = __byte_perm(u, 0x64646464u, 0x4140), r1 = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 h0 = __hsub2(*reinterpret_cast<__half2*>(&r0), bias);
    const __half2 h1 = __hsub2(*reinterpret_cast<__half2*>(&r1), bias);
    a = *reinterpret_cast<const uint32_t*>(&h0);
    b = *reinterpret_cast<const uint32_t*>(&h1);
}

// A tile: 16 blocks of a row, and this lane's block ids among them, of blocks g4 and g4 + 8.
struct Tile {
    int s, h, t, tiles, nb, blk[2];  // tiles, nb: of the row
};

// One warp's state.  The tile's boxes lie in registers; as soon as a piece has been multiplied, its registers receive
// the next tile's.
template <typename T, int D>
struct Scorer {
    static constexpr int NC = D / 64;  // 16-byte chunks of a lane: t4, t4 + 4 of each half of a box
    const SelectParams& p;
    const int g4, t4;
    // The query integers of head g4, in the order of the box's bytes: word w of chunk c holds channels 64 c + 16 t4 +
    // 4 w on, the k-columns 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 of k-step (c, w).  Their halves max(q, 0) and min(q, 0)
    // are taken anew for each product: kept, they cost the registers of one CTA in five (25.7 us against 24.5).
    uint32_t qi[NC][8];
    float f0, f1;                 // units of heads 2 t4 and 2 t4 + 1
    uint4 v[2][2][NC];            // [block g4, g4 + 8][lo, hi][chunk]
    float unit[2], next_unit[2];  // of the two blocks (0: no such block)
    const int8_t* box[2];

    __device__ __forceinline__ explicit Scorer(const SelectParams& q)
        : p(q), g4((threadIdx.x & 31) >> 2), t4(threadIdx.x & 3), f0(0.f), f1(0.f), next_unit{0.f, 0.f} {}

    __device__ __forceinline__ void look_up(Tile& x) const {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int b = 16 * x.t + g4 + 8 * r;
            x.blk[r] = b < x.nb ? p.tables[(int64_t)x.s * p.MB + b] : 0;
        }
    }
    __device__ __forceinline__ void read_query(int s, int h) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (g4 < p.G)
                    x = reinterpret_cast<const uint4*>(
                        static_cast<const T*>(p.q) + (((int64_t)s * p.H_kv + h) * p.G + g4) * D + 64 * c + 16 * t4)[i];
                qi[c][4 * i] = x.x;
                qi[c][4 * i + 1] = x.y;
                qi[c][4 * i + 2] = x.z;
                qi[c][4 * i + 3] = x.w;
            }
    }
    __device__ __forceinline__ void make_query() {  // of what read_query brought
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = Mma<T>::unpack(qi[c][i]);
                m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));  // (a NaN counts as nothing)
            }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int f = int_exponent<9>(m);
        const float inv = pow2i(-f);
        f0 = pow2i(__shfl_sync(0xffffffffu, f, 8 * t4));
        f1 = pow2i(__shfl_sync(0xffffffffu, f, 8 * t4 + 4));
        auto integer = [&](float x) {
            return x == x ? fminf(fmaxf(rintf(x * inv), -(float)kQueryTop), (float)kQueryTop) : 0.f;
        };
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 x = Mma<T>::unpack(qi[c][i]);
                const uint32_t q = Mma<__half>::pack(integer(x.x), integer(x.y));
                qi[c][i] = q;
            }
    }
    __device__ __forceinline__ void find(const Tile& x, float (&u)[2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool good = (unsigned)x.blk[r] < (unsigned)p.NB;
            if (!good && t4 == 0 && x.h == 0) flag_error(p.err, PA_DEV_ERR_BLOCK);
            const int64_t row = (int64_t)(good ? x.blk[r] : 0) * p.H_kv + x.h;
            box[r] = p.boxes + row * 2 * D + 16 * t4;
            u[r] = good ? pow2i(scale_of(p.box_scales[row])) : 0.f;
        }
    }
    __device__ __forceinline__ void load(int k, int c) {
#pragma unroll
        for (int r = 0; r < 2; ++r) v[r][k][c] = *reinterpret_cast<const uint4*>(box[r] + k * D + 64 * c);
    }
    // The scores of `left` tiles from cur on, each step(tile) after the one before, as emit(tile, block, key).
    template <typename Step, typename Emit>
    __device__ __forceinline__ void run(Tile cur, int left, Step step, Emit emit) {
        look_up(cur);
        read_query(cur.s, cur.h);
        find(cur, unit);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < NC; ++c) load(k, c);
        make_query();
        auto next = [&](Tile x) {
            step(x);
            look_up(x);
            return x;
        };
        Tile nxt = cur;
        if (left > 1) nxt = next(cur);
        for (; left > 0; --left) {
            Tile after = nxt;
            if (left > 1) find(nxt, next_unit);
            if (left > 2) after = next(nxt);
            float acc[2][4] = {};
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint32_t w0[4] = {v[0][k][c].x, v[0][k][c].y, v[0][k][c].z, v[0][k][c].w};
                    const uint32_t w1[4] = {v[1][k][c].x, v[1][k][c].y, v[1][k][c].z, v[1][k][c].w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a0, a1, a2, a3;
                        int8x4_to_f16(w0[w], a0, a2);
                        int8x4_to_f16(w1[w], a1, a3);
                        // the query's negative half meets lo, its positive half hi
                        const uint32_t x0 = qi[c][2 * w], x1 = qi[c][2 * w + 1];
                        Mma<__half>::run(acc[k], a0, a1, a2, a3, k ? Pair<__half>::hi(x0, 0) : Pair<__half>::lo(x0, 0),
                                         k ? Pair<__half>::hi(x1, 0) : Pair<__half>::lo(x1, 0));
                    }
                    if (left > 1) load(k, c);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float y = -INFINITY;
                if (2 * t4 < p.G) y = (acc[0][2 * r] + acc[1][2 * r]) * f0;
                if (2 * t4 + 1 < p.G) y = fmaxf(y, (acc[0][2 * r + 1] + acc[1][2 * r + 1]) * f1);
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
                const int b = 16 * cur.t + g4 + 8 * r;
                if (t4 == 0 && b < cur.nb) emit(cur, b, ordered(unit[r] > 0.f ? y * unit[r] : -INFINITY));
                unit[r] = next_unit[r];
            }
            if (left > 1 && (nxt.s != cur.s || nxt.h != cur.h)) {
                read_query(nxt.s, nxt.h);
                make_query();
            }
            cur = nxt;
            nxt = after;
        }
    }
};

// Tiles of each row of a sequence with something to choose.
__device__ __forceinline__ int row_tiles(const SelectParams& p, int s) {
    const int nb = context_blocks(p, s);
    return nb > p.top_k ? (nb + 15) / 16 : 0;
}

// The tiles of all rows in order are cut into runs of equal length, one per warp.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreWarps * 32, kScoreCtas) score_kernel(const SelectParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const auto tiles_of = [&](int s) { return row_tiles(p, s); };
    const RowScan<decltype(tiles_of)> scan(tiles_of, p.N, p.H_kv);
    const int total = scan.total(), warps = min((int)gridDim.x * kScoreWarps, total);
    const int w = (int)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;  // neighbouring runs on different SMs
    if (w >= warps) return;
    const Cut cut(total, warps);
    const int u0 = cut.start(w);
    Tile x;
    int first;
    x.s = scan.find(u0, x.tiles, first);
    x.h = (u0 - first) / x.tiles;
    x.t = u0 - first - x.h * x.tiles;
    x.nb = context_blocks(p, x.s);
    auto step = [&](Tile& y) {
        if (++y.t == y.tiles) {
            y.t = 0;
            if (++y.h == p.H_kv) {
                y.h = 0;
                while (y.s + 1 < p.N) {  // (the run has tiles left, so a sequence follows)
                    y.tiles = row_tiles(p, ++y.s);
                    if (y.tiles > 0) break;
                }
                y.nb = context_blocks(p, y.s);
            }
        }
    };
    Scorer<T, D> scorer(p);
    scorer.run(x, cut.start(w + 1) - u0, step, [&](const Tile& y, int b, uint32_t key) {
        p.keys[((int64_t)y.s * p.H_kv + y.h) * p.stride + b] = key;
    });
}

// The top_k of a row with more blocks than that: one CTA, each thread with neighbouring keys, in registers (K of them)
// or read anew (K = 0).  The key of the last block taken is found by a histogram over the bits below those that all
// competing keys share, eight at a time (seven for 128 threads), then among the keys of one bin: ranked against one
// another where there are no more than bins, else by their next bits.  One scan then gives every taken block its place.

// Key k competes and agrees with the prefix above its low `open` bits.
__device__ __forceinline__ bool agree(uint32_t k, uint32_t prefix, int open) {
    return k != 0 && (open == 32 || (k ^ prefix) >> open == 0);
}

template <int THREADS, int K>
__device__ __forceinline__ void top_blocks(const SelectParams& p, int nb, const uint32_t* keys, int32_t* out) {
    constexpr int W = THREADS / 32;
    constexpr int kBits = THREADS >= 256 ? 8 : 7, kBins = 1 << kBits;  // a bin per thread
    static_assert(THREADS >= kBins, "a thread per bin");
    __shared__ uint2 s_sum[W];
    __shared__ uint32_t s_bin[kBins], s_list[kBins], s_warp[kBins / 32];
    __shared__ uint32_t s_digit, s_above, s_count, s_cut, s_left;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = ((nb + THREADS - 1) / THREADS + 3) & ~3;  // keys per thread, in fours (the row is padded to a four)
    const int b0 = tid * n;
    // Keys that do not compete count as 0, below every score: blocks kept anyway, places past the context.
    auto masked = [&](uint32_t k, int b) -> uint32_t { return b < p.sink || b >= nb - p.recent ? 0u : k; };
    uint32_t reg[K ? K : 1];
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; i += 4) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i < n && b0 + i < nb) v = *reinterpret_cast<const uint4*>(keys + b0 + i);
            reg[i] = masked(v.x, b0 + i);
            reg[i + 1] = masked(v.y, b0 + i + 1);
            reg[i + 2] = masked(v.z, b0 + i + 2);
            reg[i + 3] = masked(v.w, b0 + i + 3);
        }
    }
    // f(key, block) for each of this thread's keys
    auto each = [&](auto f) {
        if constexpr (K > 0) {
#pragma unroll
            for (int i = 0; i < K; i += 4)
                if (i < n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) f(reg[i + j], b0 + i + j);
                }
        } else {
            for (int i = 0; i < n && b0 + i < nb; ++i) f(masked(keys[b0 + i], b0 + i), b0 + i);
        }
    };
    uint32_t want = (uint32_t)(p.top_k - p.sink - p.recent);  // of the keys that compete, fewer than there are
    uint32_t cut = 0xffffffffu, ties_taken = 0;               // taken: keys above cut, the first ties_taken equal ones
    if (want > 0) {
        if (tid < kBins) s_bin[tid] = 0;
        if (tid == 0) s_count = 0;
        uint32_t lo = 0xffffffffu, hi = 0;
        each([&](uint32_t k, int) {
            if (k) lo = min(lo, k);
            hi = max(hi, k);
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) s_sum[warp] = make_uint2(lo, hi);
        __syncthreads();
        const uint2 v = lane < W ? s_sum[lane] : make_uint2(0xffffffffu, 0);
        lo = __reduce_min_sync(0xffffffffu, v.x);
        hi = __reduce_max_sync(0xffffffffu, v.y);
        // the keys that compete agree above their low `open` bits with `prefix`
        int open = 32 - __clz(lo ^ hi);
        uint32_t prefix = hi;
        while (true) {
            const int shift = max(0, open - kBits);
            each([&](uint32_t k, int) {
                if (agree(k, prefix, open)) atomicAdd(&s_bin[k >> shift & (kBins - 1)], 1u);
            });
            __syncthreads();
            // thread t: bin 255 - t, and the keys in higher bins
            uint32_t mine = 0, x = 0;
            if (tid < kBins) {
                mine = x = s_bin[kBins - 1 - tid];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (lane == 31) s_warp[warp] = x;
            }
            __syncthreads();
            if (tid < kBins) {
                const uint32_t below = lane < warp ? s_warp[lane] : 0u;
                const uint32_t above = x - mine + __reduce_add_sync(0xffffffffu, below);
                if (above < want && above + mine >= want) {
                    s_digit = kBins - 1 - tid;
                    s_above = above;
                    s_left = mine;
                }
            }
            __syncthreads();
            const uint32_t digit = s_digit, count = s_left;
            want -= s_above;
            prefix = (open == 32 ? 0u : prefix >> open << open) | digit << shift;
            if (count == want) {  // the whole bin
                cut = prefix ? prefix - 1 : 0;  // (a key that competes is above 0)
                break;
            }
            open = shift;
            if (shift == 0) {  // equal keys
                cut = prefix;
                ties_taken = want;
                break;
            }
            if (count <= kBins) {
                each([&](uint32_t k, int) {
                    if (agree(k, prefix, shift)) s_list[atomicAdd(&s_count, 1u)] = k;
                });
                __syncthreads();
                if (tid < (int)count) {
                    const uint32_t k = s_list[tid];
                    uint32_t above = 0, equal = 0;
                    for (uint32_t i = 0; i < count; ++i) {
                        above += s_list[i] > k;
                        equal += s_list[i] == k;
                    }
                    if (above < want && above + equal >= want) {  // (equal keys write the same)
                        s_cut = k;
                        s_above = want - above;
                    }
                }
                __syncthreads();
                cut = s_cut;
                ties_taken = s_above;
                break;
            }
            if (tid < kBins) s_bin[tid] = 0;
            __syncthreads();
        }
    }
    // places: blocks kept and keys above cut before this thread's, and equal ones, of which ties_taken count
    uint32_t sure = 0, ties = 0;
    each([&](uint32_t k, int b) {
        sure += b < p.sink || (b >= nb - p.recent && b < nb) || k > cut;
        ties += k == cut;
    });
    uint32_t a = sure, t = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) {
            a += x;
            t += y;
        }
    }
    if (lane == 31) s_sum[warp] = make_uint2(a, t);
    __syncthreads();
    const uint2 v = lane < warp ? s_sum[lane] : make_uint2(0, 0);
    a += __reduce_add_sync(0xffffffffu, v.x) - sure;
    t += __reduce_add_sync(0xffffffffu, v.y) - ties;
    each([&](uint32_t k, int b) {
        const bool is_sure = b < p.sink || (b >= nb - p.recent && b < nb) || k > cut, tie = k == cut;
        if (is_sure || (tie && t < ties_taken)) out[a + min(t, ties_taken)] = b;
        a += is_sure;
        t += tie;
    });
}

// The list of a row with no more blocks than top_k: all of them.  No score has looked at their block-table entries: the
// sequence's first row does.
__device__ __forceinline__ void all_blocks(const SelectParams& p, int s, int h, int nb, int32_t* out) {
    const int32_t* table = p.tables + (int64_t)s * p.MB;
    bool bad = false;
    for (int i = threadIdx.x; i < p.top_k; i += blockDim.x) {
        if (h == 0 && i < nb) bad = bad || (unsigned)table[i] >= (unsigned)p.NB;
        out[i] = i < nb ? i : -1;
    }
    if (bad) flag_error(p.err, PA_DEV_ERR_BLOCK);
}

// (Where the scores' kernel runs before this one, its CTAs let this one start only once every kernel before them has
// finished: the lengths are read without waiting for the scores.)
template <int THREADS, int K>
__global__ void __launch_bounds__(THREADS) top_blocks_kernel(const SelectParams p, int early) {
    const int h = blockIdx.x, s = blockIdx.y;
    int nb = early ? context_blocks(p, s) : 0;
    griddep_wait();
    griddep_launch_dependents();
    if (!early) nb = context_blocks(p, s);
    const int64_t r = (int64_t)s * p.H_kv + h;
    if (nb == 0 && h == 0 && threadIdx.x == 0) flag_error(p.err, PA_DEV_ERR_CTX);
    if (nb <= p.top_k)
        all_blocks(p, s, h, nb, p.selected + r * p.top_k);
    else
        top_blocks<THREADS, K>(p, nb, p.keys + r * p.stride, p.selected + r * p.top_k);
}

// Rows whose clusters the device holds at once: a cluster of up to 8 CTAs per row, whose warps score the row's tiles in
// turn and leave the keys in the first CTA's shared memory, which then lists the row's blocks.  Against two kernels, 8
// rows of 1024 blocks take 4.7 us instead of 5.6, 64 rows 9.0 instead of 11.3, 304 rows (one CTA each) 21 instead of
// 25; 320 rows, which no longer fit, 35 instead of 27.  Half the cluster size serves better as long as a warp has no
// more than two tiles: 64 rows of 256 blocks 5.0 us with 2 CTAs, 5.3 with 4. Twice as many rows fit as CTAs of half the
// threads, which serve short rows: 512 rows of 256 blocks 12.8 us against 17.3 with two kernels, 512 rows of up to 1024
// blocks 31 against 25.
constexpr int kRowCluster = 8;
constexpr int kRowThreads = 256, kRowBlocks = kRowThreads * 8;    // (eight keys to a thread of the first CTA)
constexpr int kShortThreads = 128, kShortBlocks = kShortThreads * 4;
constexpr int kShortMax = 256;  // blocks of a row that still is a short one

template <typename T, int D, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) select_row_kernel(const SelectParams p) {
    __shared__ __align__(16) uint32_t s_keys[BLOCKS];
    cluster_arrive();
    griddep_wait();
    griddep_launch_dependents();
    const int rank = blockIdx.x % p.cluster, r = blockIdx.x / p.cluster;
    Tile x;
    x.s = r / p.H_kv;
    x.h = r - x.s * p.H_kv;
    x.nb = context_blocks(p, x.s);
    int32_t* out = p.selected + (int64_t)r * p.top_k;
    cluster_wait();
    if (x.nb <= p.top_k) {  // (the whole cluster returns)
        if (x.nb == 0 && x.h == 0 && rank == 0 && threadIdx.x == 0) flag_error(p.err, PA_DEV_ERR_CTX);
        if (rank == 0) all_blocks(p, x.s, x.h, x.nb, out);
        return;
    }
    const int warps = p.cluster * (THREADS / 32);
    x.tiles = (x.nb + 15) / 16;
    x.t = (int)(threadIdx.x >> 5) * p.cluster + rank;
    if (x.t < x.tiles) {
        const uint32_t keys = map_cluster(smem_addr(s_keys), 0);
        Scorer<T, D> scorer(p);
        scorer.run(x, (x.tiles - x.t + warps - 1) / warps, [&](Tile& y) { y.t += warps; },
                   [&](const Tile&, int b, uint32_t key) { st_cluster(keys + 4 * b, key); });
    }
    __syncwarp();
    cluster_sync();
    if (rank == 0) top_blocks<THREADS, BLOCKS / THREADS>(p, x.nb, s_keys, out);
}

// Keys of a row, in whole vectors of four.
static int64_t key_stride(int max_ctx, int B) { return (((int64_t)max_ctx + B - 1) / B + 3) & ~int64_t(3); }

static int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        sms = 1;
    return sms;
}

size_t select_workspace_bytes(int N, int H_kv, int max_ctx, int B) {
    if (N <= 0 || N > 65535 || H_kv <= 0 || H_kv > 65535 || max_ctx <= 0 || (B != 8 && B != 16 && B != 32)) return 0;
    return (size_t)N * H_kv * (size_t)key_stride(max_ctx, B) * sizeof(uint32_t);
}

pa_status launch_select(const SelectArgs& a) {
    SelectParams p;
    p.selected = a.selected;
    p.q = a.q;
    p.boxes = static_cast<const int8_t*>(a.summaries);
    p.box_scales = static_cast<const uint8_t*>(a.sum_scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.keys = static_cast<uint32_t*>(a.workspace);
    p.stride = key_stride(a.max_ctx, a.B);
    p.N = a.N;
    p.H_kv = a.H_kv;
    p.G = a.H_q / a.H_kv;
    p.lgB = a.B == 8 ? 3 : a.B == 16 ? 4 : 5;
    p.MB = a.MB;
    p.NB = a.NB;
    p.max_ctx = a.max_ctx;
    p.top_k = a.top_k;
    p.sink = a.sink;
    p.recent = a.recent;
    p.err = a.dev_err;
    const int64_t nb = std::min<int64_t>(((int64_t)a.max_ctx + a.B - 1) / a.B, a.MB);  // the longest context's
    const int64_t rows = (int64_t)a.N * a.H_kv;
    if (nb > a.top_k && nb <= kRowBlocks) {
        void (*kern)(SelectParams);
        void (*shorter)(SelectParams);
        ClusterRoom *room, *shorter_room;
        auto pick = [&](auto q, auto d) {
            static ClusterRoom of_kern, of_shorter;
            kern = select_row_kernel<decltype(q), decltype(d)::value, kRowThreads, kRowBlocks>;
            shorter = select_row_kernel<decltype(q), decltype(d)::value, kShortThreads, kShortBlocks>;
            room = &of_kern;
            shorter_room = &of_shorter;
        };
        auto by_dim = [&](auto q) {
            if (a.D == 128)
                pick(q, std::integral_constant<int, 128>());
            else
                pick(q, std::integral_constant<int, 64>());
        };
        if (a.q_dtype == PA_BF16)
            by_dim(__nv_bfloat16());
        else
            by_dim(__half());
        p.cluster = 0;
        for (int size = kRowCluster; size > 0; size /= 2) {
            int held = 0;
            const cudaError_t e = room->get(kern, size, kRowThreads, 0, &held);
            if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters(select_row)");
            const bool enough = size == 1 || nb > 2 * 16 * (kRowThreads / 32) * (size / 2);
            // (half the room where half the size would do)
            if (rows <= (enough ? held : held / 2)) {
                p.cluster = size;
                break;
            }
        }
        int threads = kRowThreads;
        if (!p.cluster && nb <= kShortMax) {
            int held = 0;
            const cudaError_t e = shorter_room->get(shorter, 1, kShortThreads, 0, &held);
            if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters(select_row)");
            if (rows <= held) {
                p.cluster = 1;
                kern = shorter;
                threads = kShortThreads;
            }
        }
        if (p.cluster) {
            const cudaError_t e = launch_clusters(kern, p.cluster, dim3((unsigned)(rows * p.cluster)),
                                                  dim3((unsigned)threads), 0, a.stream, p);
            count_launch();
            return e == cudaSuccess ? PA_OK : cuda_fail(e, "select_row launch");
        }
    }
    if (nb > a.top_k) {
        const int64_t tiles = (nb + 15) / 16 * a.N * a.H_kv;
        if (tiles >= 1LL << 31) return fail(PA_ERR_UNSUPPORTED, "too many blocks to score");
        const unsigned grid = (unsigned)std::min<int64_t>((tiles + kScoreWarps - 1) / kScoreWarps,
                                                          (int64_t)sm_count() * kScoreCtas);
        auto kern = a.q_dtype == PA_BF16
                        ? (a.D == 128 ? score_kernel<__nv_bfloat16, 128> : score_kernel<__nv_bfloat16, 64>)
                        : (a.D == 128 ? score_kernel<__half, 128> : score_kernel<__half, 64>);
        const cudaError_t e = launch_kernel(kern, dim3(grid), dim3(kScoreWarps * 32), 0, a.stream, p);
        count_launch();
        if (e != cudaSuccess) return cuda_fail(e, "score launch");
    }
    // keys in registers up to 16 per thread (32 spill)
    void (*top)(SelectParams, int) = top_blocks_kernel<1024, 0>;
    int threads = 1024;
    if (nb <= 256 * 8) {
        top = top_blocks_kernel<256, 8>;
        threads = 256;
    } else if (nb <= 1024 * 8) {
        top = top_blocks_kernel<1024, 8>;
    } else if (nb <= 1024 * 16) {
        top = top_blocks_kernel<1024, 16>;
    }
    const cudaError_t e =
        launch_kernel(top, dim3((unsigned)a.H_kv, (unsigned)a.N), dim3((unsigned)threads), 0, a.stream, p,
                      nb > a.top_k ? 1 : 0);
    count_launch();
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "top_blocks launch");
}

}  // namespace pa
