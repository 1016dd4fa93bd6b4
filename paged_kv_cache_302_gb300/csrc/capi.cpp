// capi.cpp -- argument validation and dispatch for the device entry points of pa.h.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include <nvtx3/nvToolsExt.h>

#include "pa_internal.h"

namespace pa {

static thread_local char g_msg[512] = "";
static std::atomic<uint64_t> g_launches{0};

pa_status fail(pa_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return st;
}

pa_status cuda_fail(cudaError_t e, const char* what) {
    return fail(PA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

static std::atomic<uint64_t> g_wait_ns{0};  // 0: the built-in limit

uint64_t wait_limit_ns() {
    const uint64_t ns = g_wait_ns.load(std::memory_order_relaxed);
    return ns ? ns : 1000000000ull;
}

// NVTX ranges around every device call, for profiler timelines; off unless PA_NVTX is set to a non-zero value
// (read once), so a call costs one predictable branch when they are off.
static bool nvtx_enabled() {
    static const bool on = [] {
        const char* v = std::getenv("PA_NVTX");
        return v && *v && *v != '0';
    }();
    return on;
}

struct NvtxRange {
    bool on;
    explicit NvtxRange(const char* name) : on(nvtx_enabled()) {
        if (on) nvtxRangePushA(name);
    }
    ~NvtxRange() {
        if (on) nvtxRangePop();
    }
};

bool pdl_enabled() {
    static const bool on = [] {
        const char* v = std::getenv("PA_NO_PDL");
        return !(v && *v && *v != '0');
    }();
    return on;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static bool kv_dtype_ok(int dt) { return dt == PA_F16 || dt == PA_BF16; }

static pa_status check_decode_common(pa_dtype out_dtype, pa_dtype kv_dtype, const void* out, const void* q,
                                     const int32_t* ctx_lens, int N, int H_q, int H_kv, int D, int max_ctx,
                                     int partition_tokens, const void* ws, size_t ws_bytes) {
    if (!kv_dtype_ok(kv_dtype)) return fail(PA_ERR_UNSUPPORTED, "kv_dtype must be F16 or BF16");
    if (out_dtype != PA_F32 && out_dtype != kv_dtype)
        return fail(PA_ERR_UNSUPPORTED, "out_dtype must be F32 or the kv dtype");
    if (N <= 0 || H_q <= 0 || H_kv <= 0 || max_ctx <= 0) return fail(PA_ERR_INVALID, "sizes must be positive");
    if (H_q % H_kv) return fail(PA_ERR_INVALID, "H_q (%d) must be a multiple of H_kv (%d)", H_q, H_kv);
    if (H_q / H_kv > kMaxGroup) return fail(PA_ERR_UNSUPPORTED, "H_q / H_kv must be <= %d", kMaxGroup);
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", D);
    if (!out || !q || !ctx_lens || !ws) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(out) || !aligned16(q) || !aligned16(ws))
        return fail(PA_ERR_INVALID, "out, q and workspace must be 16-byte aligned");
    WorkspaceLayout L;
    if (!workspace_layout(N, H_q, H_kv, D, max_ctx, partition_tokens, &L))
        return fail(PA_ERR_INVALID, "partition_tokens must be 0, -1 or a positive multiple of %d", kStageTok);
    if (ws_bytes < L.total) return fail(PA_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, L.total);
    if ((long)N * L.P * H_kv >= (1L << 30)) return fail(PA_ERR_UNSUPPORTED, "too many work records");
    return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" {

const char* pa_last_error(void) { return g_msg; }

const char* pa_version(void) { return "pa 0.1.0 (sm_103a)"; }

uint64_t pa_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

void pa_set_wait_limit_ns(uint64_t ns) { g_wait_ns.store(ns, std::memory_order_relaxed); }

pa_status pa_reshape_and_cache(const void* k, const void* v, void* pool, const int64_t* slot_mapping, int T, int NB,
                               int B, int H_kv, int D, pa_dtype dtype, int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_reshape_and_cache");
    g_msg[0] = 0;
    if (!kv_dtype_ok(dtype)) return fail(PA_ERR_UNSUPPORTED, "dtype must be F16 or BF16");
    if (T < 0 || NB <= 0 || B <= 0 || H_kv <= 0 || D <= 0) return fail(PA_ERR_INVALID, "bad sizes");
    if ((H_kv * D) % 8) return fail(PA_ERR_UNSUPPORTED, "H_kv * D must be a multiple of 8");
    if ((long long)NB * B >= (1LL << 62)) return fail(PA_ERR_INVALID, "pool too large");
    if (T == 0) return PA_OK;
    if (!k || !v || !pool || !slot_mapping) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(k) || !aligned16(v) || !aligned16(pool))
        return fail(PA_ERR_INVALID, "k, v and pool must be 16-byte aligned");
    return launch_reshape_and_cache(k, v, pool, slot_mapping, T, NB, B, H_kv, D, dev_err,
                                    static_cast<cudaStream_t>(stream));
}

pa_status pa_copy_blocks(void* pool, const int64_t* pairs, int n, int NB, int B, int H_kv, int D, pa_dtype dtype,
                         int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_copy_blocks");
    g_msg[0] = 0;
    if (!kv_dtype_ok(dtype) && dtype != PA_E4M3) return fail(PA_ERR_UNSUPPORTED, "dtype must be F16, BF16 or E4M3");
    if (n < 0 || NB <= 0 || B <= 0 || H_kv <= 0 || D <= 0) return fail(PA_ERR_INVALID, "bad sizes");
    const long long blk_bytes = (long long)B * 2 * H_kv * D * (dtype == PA_E4M3 ? 1 : 2);
    if (blk_bytes % 16) return fail(PA_ERR_UNSUPPORTED, "block bytes must be a multiple of 16");
    if (n > (1 << 30)) return fail(PA_ERR_INVALID, "too many pairs");
    if (n == 0) return PA_OK;
    if (!pool || !pairs) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(pool)) return fail(PA_ERR_INVALID, "pool must be 16-byte aligned");
    return launch_copy_blocks(pool, pairs, n, NB, blk_bytes, dev_err, static_cast<cudaStream_t>(stream));
}

// A pointer the GPU may dereference: device memory, managed memory, or page-locked host memory.
static pa_status check_device_accessible(const void* p, const char* what) {
    cudaPointerAttributes attr;
    cudaError_t e = cudaPointerGetAttributes(&attr, p);
    if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes");
    if (attr.type == cudaMemoryTypeUnregistered)
        return fail(PA_ERR_INVALID, "%s is pageable host memory; pin it (cudaHostAlloc / cudaHostRegister)", what);
    if (attr.type == cudaMemoryTypeHost && !attr.devicePointer)
        return fail(PA_ERR_INVALID, "%s is page-locked but not mapped into the device address space", what);
    return PA_OK;
}

pa_status pa_swap_blocks(void* dst_pool, int NB_dst, const void* src_pool, int NB_src, const int64_t* pairs, int n,
                         int B, int H_kv, int D, pa_dtype dtype, int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_swap_blocks");
    g_msg[0] = 0;
    if (!kv_dtype_ok(dtype) && dtype != PA_E4M3) return fail(PA_ERR_UNSUPPORTED, "dtype must be F16, BF16 or E4M3");
    if (n < 0 || NB_dst <= 0 || NB_src <= 0 || B <= 0 || H_kv <= 0 || D <= 0) return fail(PA_ERR_INVALID, "bad sizes");
    const long long blk_bytes = (long long)B * 2 * H_kv * D * (dtype == PA_E4M3 ? 1 : 2);
    if (blk_bytes % 16) return fail(PA_ERR_UNSUPPORTED, "block bytes must be a multiple of 16");
    if (n > (1 << 30)) return fail(PA_ERR_INVALID, "too many pairs");
    if (n == 0) return PA_OK;
    if (!dst_pool || !src_pool || !pairs) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(dst_pool) || !aligned16(src_pool)) return fail(PA_ERR_INVALID, "pools must be 16-byte aligned");
    pa_status st = check_device_accessible(dst_pool, "dst_pool");
    if (st == PA_OK) st = check_device_accessible(src_pool, "src_pool");
    if (st == PA_OK) st = check_device_accessible(pairs, "pairs");
    if (st != PA_OK) return st;
    return launch_swap_blocks(dst_pool, NB_dst, src_pool, NB_src, pairs, n, blk_bytes, dev_err,
                              static_cast<cudaStream_t>(stream));
}

pa_status pa_write_contiguous(const void* k, const void* v, void* k_buf, void* v_buf, const int32_t* req_ids,
                              const int32_t* positions, int T, int N_max, int S_max, int H_kv, int D, pa_dtype dtype,
                              int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_write_contiguous");
    g_msg[0] = 0;
    if (!kv_dtype_ok(dtype)) return fail(PA_ERR_UNSUPPORTED, "dtype must be F16 or BF16");
    if (T < 0 || N_max <= 0 || S_max <= 0 || H_kv <= 0 || D <= 0) return fail(PA_ERR_INVALID, "bad sizes");
    if ((H_kv * D) % 8) return fail(PA_ERR_UNSUPPORTED, "H_kv * D must be a multiple of 8");
    if (T == 0) return PA_OK;
    if (!k || !v || !k_buf || !v_buf || !req_ids || !positions) return fail(PA_ERR_INVALID, "null pointer");
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_buf) || !aligned16(v_buf))
        return fail(PA_ERR_INVALID, "k, v and the buffers must be 16-byte aligned");
    return launch_write_contiguous(k, v, k_buf, v_buf, req_ids, positions, T, N_max, S_max, H_kv, D, dev_err,
                                   static_cast<cudaStream_t>(stream));
}

pa_status pa_update_block_tables(int32_t* tables, int N, int MB, const int32_t* updates, int n, int* dev_err,
                                 void* stream) {
    const NvtxRange nvtx_range("pa_update_block_tables");
    g_msg[0] = 0;
    if (N <= 0 || MB <= 0 || n < 0) return fail(PA_ERR_INVALID, "bad sizes");
    if (n == 0) return PA_OK;
    if (!tables || !updates) return fail(PA_ERR_INVALID, "null pointer argument");
    if ((reinterpret_cast<uintptr_t>(updates) & 3u) || (reinterpret_cast<uintptr_t>(tables) & 3u))
        return fail(PA_ERR_INVALID, "tables and updates must be 4-byte aligned");
    return launch_update_tables(tables, N, MB, updates, n, dev_err, static_cast<cudaStream_t>(stream));
}

size_t pa_decode_workspace_bytes(int N, int H_q, int H_kv, int D, int max_ctx, int partition_tokens) {
    WorkspaceLayout L;
    if (!workspace_layout(N, H_q, H_kv, D, max_ctx, partition_tokens, &L)) return 0;
    size_t total = L.total;
    // a small batch's quantised decode takes shorter partitions, hence more of them
    if (partition_tokens == 0 && workspace_layout(N, H_q, H_kv, D, max_ctx, quant_partition(N, H_kv, max_ctx), &L))
        total = total > L.total ? total : L.total;
    return total;
}

pa_status pa_decode(void* out, pa_dtype out_dtype, const void* q, const void* pool, const int32_t* block_tables,
                    const int32_t* ctx_lens, int N, int H_q, int H_kv, int D, int B, int MB, int NB, int max_ctx,
                    float scale, int partition_tokens, void* workspace, size_t ws_bytes, pa_dtype kv_dtype,
                    int* dev_err, void* const* attend_events, void* stream) {
    const NvtxRange nvtx_range("pa_decode");
    g_msg[0] = 0;
    pa_status st = check_decode_common(out_dtype, kv_dtype, out, q, ctx_lens, N, H_q, H_kv, D, max_ctx,
                                       partition_tokens, workspace, ws_bytes);
    if (st != PA_OK) return st;
    if (B != 4 && B != 8 && B != 16 && B != 32) return fail(PA_ERR_UNSUPPORTED, "B must be 4, 8, 16 or 32");
    if (NB <= 0 || MB <= 0) return fail(PA_ERR_INVALID, "NB and MB must be positive");
    if ((long long)NB * B >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "NB * B must be < 2^31");
    if (!pool || !block_tables) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(pool)) return fail(PA_ERR_INVALID, "pool must be 16-byte aligned");
    DecodeArgs a;
    std::memset(&a, 0, sizeof a);
    a.out = out;
    a.out_dtype = out_dtype;
    a.q = q;
    a.kv_dtype = kv_dtype;
    a.pool = pool;
    a.tables = block_tables;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.paged = true;
    a.ctx_lens = ctx_lens;
    a.N = N;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.max_ctx = max_ctx;
    a.scale = scale;
    a.partition_tokens = partition_tokens;
    a.workspace = workspace;
    a.ws_bytes = ws_bytes;
    a.dev_err = dev_err;
    a.attend_events = attend_events;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_decode(a);
}

pa_status pa_decode_contiguous(void* out, pa_dtype out_dtype, const void* q, const void* k_buf, const void* v_buf,
                               const int32_t* req_ids, const int32_t* ctx_lens, int N, int H_q, int H_kv, int D,
                               int N_max, int S_max, int max_ctx, float scale, int partition_tokens, void* workspace,
                               size_t ws_bytes, pa_dtype kv_dtype, int* dev_err, void* const* attend_events,
                               void* stream) {
    const NvtxRange nvtx_range("pa_decode_contiguous");
    g_msg[0] = 0;
    pa_status st = check_decode_common(out_dtype, kv_dtype, out, q, ctx_lens, N, H_q, H_kv, D, max_ctx,
                                       partition_tokens, workspace, ws_bytes);
    if (st != PA_OK) return st;
    if (N_max <= 0 || S_max <= 0) return fail(PA_ERR_INVALID, "N_max and S_max must be positive");
    if ((long long)N_max * S_max >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "N_max * S_max must be < 2^31");
    if (!k_buf || !v_buf || !req_ids) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(k_buf) || !aligned16(v_buf)) return fail(PA_ERR_INVALID, "k_buf and v_buf must be 16-byte aligned");
    DecodeArgs a;
    std::memset(&a, 0, sizeof a);
    a.out = out;
    a.out_dtype = out_dtype;
    a.q = q;
    a.kv_dtype = kv_dtype;
    a.k_buf = k_buf;
    a.v_buf = v_buf;
    a.req_ids = req_ids;
    a.N_max = N_max;
    a.S_max = S_max;
    a.paged = false;
    a.ctx_lens = ctx_lens;
    a.N = N;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.max_ctx = max_ctx;
    a.scale = scale;
    a.partition_tokens = partition_tokens;
    a.workspace = workspace;
    a.ws_bytes = ws_bytes;
    a.dev_err = dev_err;
    a.attend_events = attend_events;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_decode(a);
}

// ----------------------------------------------------------------------------- quantised cache, tree attention

// Sizes of a quantised cache's calls: head dim, block size, and slots an int counts.
static pa_status check_quant_shape(int NB, int B, int H_kv, int D) {
    if (NB <= 0 || H_kv <= 0 || H_kv > 65535) return fail(PA_ERR_INVALID, "bad sizes");
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", D);
    if (B != 8 && B != 16 && B != 32) return fail(PA_ERR_UNSUPPORTED, "B must be 8, 16 or 32 (got %d)", B);
    if ((long long)NB * B >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "NB * B must be < 2^31");
    if ((long long)NB * H_kv >= (1LL << 31) - 1) return fail(PA_ERR_UNSUPPORTED, "NB * H_kv must be < 2^31 - 1");
    return PA_OK;
}

pa_status pa_reshape_and_cache_quant(const void* k, const void* v, void* qpool, void* scales,
                                     const int64_t* slot_mapping, int T, int NB, int B, int H_kv, int D,
                                     pa_dtype dtype, int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_reshape_and_cache_quant");
    g_msg[0] = 0;
    if (!kv_dtype_ok(dtype)) return fail(PA_ERR_UNSUPPORTED, "dtype must be F16 or BF16");
    if (T < 0) return fail(PA_ERR_INVALID, "bad sizes");
    const pa_status st = check_quant_shape(NB, B, H_kv, D);
    if (st != PA_OK) return st;
    if (T == 0) return PA_OK;
    if (!k || !v || !qpool || !scales || !slot_mapping) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(k) || !aligned16(v) || !aligned16(qpool) || !aligned16(scales))
        return fail(PA_ERR_INVALID, "k, v, qpool and scales must be 16-byte aligned");
    return launch_quant_cache(k, v, qpool, scales, slot_mapping, T, NB, B, H_kv, D, dtype, dev_err,
                              static_cast<cudaStream_t>(stream));
}

pa_status pa_dequant_blocks(void* dst_pool, int NB_dst, const void* qpool, const void* scales, int NB_src,
                            const int64_t* pairs, int n, int B, int H_kv, int D, pa_dtype dtype, int* dev_err,
                            void* stream) {
    const NvtxRange nvtx_range("pa_dequant_blocks");
    g_msg[0] = 0;
    if (!kv_dtype_ok(dtype)) return fail(PA_ERR_UNSUPPORTED, "dtype must be F16 or BF16");
    if (n < 0 || NB_dst <= 0) return fail(PA_ERR_INVALID, "bad sizes");
    const pa_status st = check_quant_shape(NB_src, B, H_kv, D);
    if (st != PA_OK) return st;
    if (n > (1 << 30)) return fail(PA_ERR_INVALID, "too many pairs");
    if (n == 0) return PA_OK;
    if (!dst_pool || !qpool || !scales || !pairs) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(dst_pool) || !aligned16(qpool) || !aligned16(scales))
        return fail(PA_ERR_INVALID, "dst_pool, qpool and scales must be 16-byte aligned");
    return launch_dequant_blocks(dst_pool, NB_dst, qpool, scales, NB_src, pairs, n, B, H_kv, D, dtype, dev_err,
                                 static_cast<cudaStream_t>(stream));
}

pa_status pa_decode_quant(void* out, pa_dtype out_dtype, const void* q, pa_dtype q_dtype, const void* qpool,
                          const void* scales, const int32_t* block_tables, const int32_t* ctx_lens, int N, int H_q,
                          int H_kv, int D, int B, int MB, int NB, int max_ctx, float scale, int partition_tokens,
                          void* workspace, size_t ws_bytes, int* dev_err, void* const* attend_events, void* stream) {
    const NvtxRange nvtx_range("pa_decode_quant");
    g_msg[0] = 0;
    pa_status st = check_decode_common(out_dtype, q_dtype, out, q, ctx_lens, N, H_q, H_kv, D, max_ctx,
                                       partition_tokens, workspace, ws_bytes);
    if (st != PA_OK) return st;
    st = check_quant_shape(NB, B, H_kv, D);
    if (st != PA_OK) return st;
    if (MB <= 0) return fail(PA_ERR_INVALID, "MB must be positive");
    if (!qpool || !scales || !block_tables) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(qpool) || !aligned16(scales)) return fail(PA_ERR_INVALID, "qpool and scales must be 16-byte aligned");
    DecodeQuantArgs a;
    a.out = out;
    a.out_dtype = out_dtype;
    a.q = q;
    a.q_dtype = q_dtype;
    a.qpool = qpool;
    a.scales = scales;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.N = N;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.max_ctx = max_ctx;
    a.scale = scale;
    a.partition_tokens = partition_tokens;
    a.workspace = workspace;
    a.ws_bytes = ws_bytes;
    a.dev_err = dev_err;
    a.attend_events = attend_events;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_decode_quant(a);
}

size_t pa_decode_tree_workspace_bytes(int N, int H_q, int H_kv, int D, int max_q_len) {
    return tree_workspace_bytes(N, H_q, H_kv, D, max_q_len);
}

pa_status pa_decode_tree(void* out, pa_dtype out_dtype, const void* q, pa_dtype q_dtype, const void* pool,
                         const void* scales, pa_dtype kv_dtype, const int32_t* block_tables, const int32_t* ctx_lens,
                         const int32_t* q_start, const int32_t* tree_mask, int mask_words, int N, int T, int H_q,
                         int H_kv, int D, int B, int MB, int NB, int max_q_len, float scale, void* workspace,
                         size_t ws_bytes, int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_decode_tree");
    g_msg[0] = 0;
    if (!kv_dtype_ok(q_dtype)) return fail(PA_ERR_UNSUPPORTED, "q_dtype must be F16 or BF16");
    if (kv_dtype != PA_E4M3 && kv_dtype != q_dtype)
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype must be q_dtype or E4M3");
    if (out_dtype != PA_F32 && out_dtype != q_dtype)
        return fail(PA_ERR_UNSUPPORTED, "out_dtype must be F32 or the query dtype");
    if (N <= 0 || N > 65535 || T < 0 || H_q <= 0 || MB <= 0 || max_q_len < 0 || mask_words <= 0)
        return fail(PA_ERR_INVALID, "bad sizes");
    pa_status st = check_quant_shape(NB, B, H_kv, D);
    if (st != PA_OK) return st;
    if (H_q % H_kv) return fail(PA_ERR_INVALID, "H_q (%d) must be a multiple of H_kv (%d)", H_q, H_kv);
    if (H_q / H_kv > 128) return fail(PA_ERR_UNSUPPORTED, "H_q / H_kv must be <= 128");
    if ((long long)MB * B >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "MB * B must be < 2^31");
    if (max_q_len > 32LL * mask_words)
        return fail(PA_ERR_INVALID, "a mask of %d words per row holds %lld drafted tokens, max_q_len is %d", mask_words,
                    32LL * mask_words, max_q_len);
    if (!(scale > 0.f && scale < HUGE_VALF)) return fail(PA_ERR_INVALID, "scale must be positive and finite");
    if (T == 0 || max_q_len == 0) return PA_OK;
    if (!out || !q || !pool || !block_tables || !ctx_lens || !q_start || !tree_mask || !workspace)
        return fail(PA_ERR_INVALID, "null pointer argument");
    if ((kv_dtype == PA_E4M3) != (scales != nullptr))
        return fail(PA_ERR_INVALID, "an E4M3 pool needs its scales, another pool has none");
    if (!aligned16(out) || !aligned16(q) || !aligned16(pool) || !aligned16(scales) || !aligned16(workspace))
        return fail(PA_ERR_INVALID, "out, q, pool, scales and workspace must be 16-byte aligned");
    const size_t need = tree_workspace_bytes(N, H_q, H_kv, D, max_q_len);
    if (ws_bytes < need) return fail(PA_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    TreeArgs a;
    a.out = out;
    a.out_dtype = out_dtype;
    a.q = q;
    a.q_dtype = q_dtype;
    a.pool = pool;
    a.scales = scales;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.q_start = q_start;
    a.mask = reinterpret_cast<const uint32_t*>(tree_mask);
    a.mask_words = mask_words;
    a.N = N;
    a.T = T;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.max_q_len = max_q_len;
    a.scale = scale;
    a.workspace = workspace;
    a.ws_bytes = ws_bytes;
    a.dev_err = dev_err;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_tree(a);
}

// ----------------------------------------------------------------------------- block-sparse decode, compaction

// Sizes that the calls over a cache of either kind and its block tables share.
static pa_status check_paged_cache(pa_dtype kv_dtype, const void* pool, const void* scales, int N, int H_kv, int D,
                                   int B, int MB, int NB) {
    if (!kv_dtype_ok(kv_dtype) && kv_dtype != PA_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype must be F16, BF16 or E4M3");
    if (N <= 0 || N > 65535 || MB <= 0) return fail(PA_ERR_INVALID, "bad sizes");
    const pa_status st = check_quant_shape(NB, B, H_kv, D);
    if (st != PA_OK) return st;
    if ((long long)MB * B >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "MB * B must be < 2^31");
    if ((kv_dtype == PA_E4M3) != (scales != nullptr))
        return fail(PA_ERR_INVALID, "an E4M3 pool needs its scales, another pool has none");
    if (!aligned16(pool) || !aligned16(scales)) return fail(PA_ERR_INVALID, "pool and scales must be 16-byte aligned");
    return PA_OK;
}

// Query heads of the calls that share a KV head's work among its group.
static pa_status check_group(int H_q, int H_kv) {
    if (H_q <= 0 || H_q % H_kv) return fail(PA_ERR_INVALID, "H_q (%d) must be a multiple of H_kv (%d)", H_q, H_kv);
    if (H_q / H_kv > kMaxGroup) return fail(PA_ERR_UNSUPPORTED, "H_q / H_kv must be <= %d", kMaxGroup);
    return PA_OK;
}

pa_status pa_summarize_blocks(void* summaries, void* sum_scales, const void* pool, const void* scales,
                              pa_dtype kv_dtype, const int32_t* block_tables, const int32_t* ctx_lens,
                              const int32_t* q_start, int N, int H_kv, int D, int B, int MB, int NB, int max_q_len,
                              int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_summarize_blocks");
    g_msg[0] = 0;
    const pa_status st = check_paged_cache(kv_dtype, pool, scales, N, H_kv, D, B, MB, NB);
    if (st != PA_OK) return st;
    if (max_q_len < 0) return fail(PA_ERR_INVALID, "bad sizes");
    if (max_q_len == 0) return PA_OK;
    if (!summaries || !sum_scales || !pool || !block_tables || !ctx_lens)
        return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(summaries)) return fail(PA_ERR_INVALID, "summaries must be 16-byte aligned");
    SummarizeArgs a;
    a.summaries = summaries;
    a.sum_scales = sum_scales;
    a.pool = pool;
    a.scales = scales;
    a.kv_dtype = kv_dtype;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.q_start = q_start;
    a.N = N;
    a.H_kv = H_kv;
    a.D = D;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.max_q_len = max_q_len;
    a.dev_err = dev_err;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_summarize(a);
}

size_t pa_select_workspace_bytes(int N, int H_kv, int max_ctx, int B) {
    return select_workspace_bytes(N, H_kv, max_ctx, B);
}

pa_status pa_select_blocks(int32_t* selected, const void* q, pa_dtype q_dtype, const void* summaries,
                           const void* sum_scales, const int32_t* block_tables, const int32_t* ctx_lens, int N, int H_q,
                           int H_kv, int D, int B, int MB, int NB, int max_ctx, int top_k, int sink_blocks,
                           int recent_blocks, void* workspace, size_t ws_bytes, int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_select_blocks");
    g_msg[0] = 0;
    if (!kv_dtype_ok(q_dtype)) return fail(PA_ERR_UNSUPPORTED, "q_dtype must be F16 or BF16");
    pa_status st = check_paged_cache(q_dtype, nullptr, nullptr, N, H_kv, D, B, MB, NB);
    if (st == PA_OK) st = check_group(H_q, H_kv);
    if (st != PA_OK) return st;
    if (max_ctx <= 0 || top_k <= 0) return fail(PA_ERR_INVALID, "max_ctx and top_k must be positive");
    if (top_k > kMaxTopK) return fail(PA_ERR_UNSUPPORTED, "top_k must be <= %d", kMaxTopK);
    if (sink_blocks < 0 || recent_blocks < 0 || (long long)sink_blocks + recent_blocks > top_k)
        return fail(PA_ERR_INVALID, "sink_blocks and recent_blocks must not be negative, nor more than top_k together");
    if (!selected || !q || !summaries || !sum_scales || !block_tables || !ctx_lens || !workspace)
        return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(q) || !aligned16(summaries) || !aligned16(workspace))
        return fail(PA_ERR_INVALID, "q, summaries and workspace must be 16-byte aligned");
    const size_t need = select_workspace_bytes(N, H_kv, max_ctx, B);
    if (ws_bytes < need) return fail(PA_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    SelectArgs a;
    a.selected = selected;
    a.q = q;
    a.q_dtype = q_dtype;
    a.summaries = summaries;
    a.sum_scales = sum_scales;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.N = N;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.max_ctx = max_ctx;
    a.top_k = top_k;
    a.sink = sink_blocks;
    a.recent = recent_blocks;
    a.workspace = workspace;
    a.dev_err = dev_err;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_select(a);
}

size_t pa_decode_sparse_workspace_bytes(int N, int H_q, int H_kv, int D, int B, int top_k) {
    return decode_sparse_workspace_bytes(N, H_q, H_kv, D, B, top_k);
}

pa_status pa_decode_sparse(void* out, pa_dtype out_dtype, const void* q, pa_dtype q_dtype, const void* pool,
                           const void* scales, pa_dtype kv_dtype, const int32_t* block_tables, const int32_t* ctx_lens,
                           const int32_t* selected, int top_k, int N, int H_q, int H_kv, int D, int B, int MB, int NB,
                           float scale, void* workspace, size_t ws_bytes, int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_decode_sparse");
    g_msg[0] = 0;
    if (!kv_dtype_ok(q_dtype)) return fail(PA_ERR_UNSUPPORTED, "q_dtype must be F16 or BF16");
    if (kv_dtype != PA_E4M3 && kv_dtype != q_dtype)
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype must be q_dtype or E4M3");
    if (out_dtype != PA_F32 && out_dtype != q_dtype)
        return fail(PA_ERR_UNSUPPORTED, "out_dtype must be F32 or the query dtype");
    pa_status st = check_paged_cache(kv_dtype, pool, scales, N, H_kv, D, B, MB, NB);
    if (st == PA_OK) st = check_group(H_q, H_kv);
    if (st != PA_OK) return st;
    if (top_k <= 0) return fail(PA_ERR_INVALID, "top_k must be positive");
    if (top_k > kMaxTopK) return fail(PA_ERR_UNSUPPORTED, "top_k must be <= %d", kMaxTopK);
    if (!(scale > 0.f && scale < HUGE_VALF)) return fail(PA_ERR_INVALID, "scale must be positive and finite");
    if (!out || !q || !pool || !block_tables || !ctx_lens || !selected || !workspace)
        return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(out) || !aligned16(q) || !aligned16(workspace))
        return fail(PA_ERR_INVALID, "out, q and workspace must be 16-byte aligned");
    const size_t need = decode_sparse_workspace_bytes(N, H_q, H_kv, D, B, top_k);
    if (need == 0) return fail(PA_ERR_UNSUPPORTED, "too many work records");
    if (ws_bytes < need) return fail(PA_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    DecodeSparseArgs a;
    a.out = out;
    a.out_dtype = out_dtype;
    a.q = q;
    a.q_dtype = q_dtype;
    a.pool = pool;
    a.scales = scales;
    a.kv_dtype = kv_dtype;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.selected = selected;
    a.top_k = top_k;
    a.N = N;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.scale = scale;
    a.workspace = workspace;
    a.dev_err = dev_err;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_decode_sparse(a);
}

pa_status pa_compact_tokens(void* pool, void* scales, pa_dtype kv_dtype, const int32_t* block_tables,
                            const int32_t* ctx_lens, const int32_t* base, const int32_t* keep,
                            const int32_t* keep_start, int N, int T, int H_kv, int D, int B, int MB, int NB,
                            int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_compact_tokens");
    g_msg[0] = 0;
    const pa_status st = check_paged_cache(kv_dtype, pool, scales, N, H_kv, D, B, MB, NB);
    if (st != PA_OK) return st;
    if (T < 0) return fail(PA_ERR_INVALID, "bad sizes");
    if (T == 0) return PA_OK;
    if (!pool || !block_tables || !ctx_lens || !base || !keep || !keep_start)
        return fail(PA_ERR_INVALID, "null pointer argument");
    CompactArgs a;
    a.pool = pool;
    a.scales = scales;
    a.kv_dtype = kv_dtype;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.base = base;
    a.keep = keep;
    a.keep_start = keep_start;
    a.N = N;
    a.T = T;
    a.H_kv = H_kv;
    a.D = D;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.dev_err = dev_err;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_compact(a);
}

size_t pa_prefill_workspace_bytes(int N, int H_kv, int D, int B, int MB) {
    PrefillWorkspace L;
    return prefill_workspace_layout(N, H_kv, D, B, MB, &L) ? L.total : 0;
}

pa_status pa_prefill(void* out, pa_dtype out_dtype, const void* q, const void* pool, const int32_t* block_tables,
                     const int32_t* ctx_lens, const int32_t* q_start, int N, int T, int H_q, int H_kv, int D, int B,
                     int MB, int NB, int max_q_len, float scale, pa_dtype kv_dtype, void* workspace, size_t ws_bytes,
                     int* dev_err, void* stream) {
    const NvtxRange nvtx_range("pa_prefill");
    g_msg[0] = 0;
    if (!kv_dtype_ok(kv_dtype)) return fail(PA_ERR_UNSUPPORTED, "kv_dtype must be F16 or BF16");
    if (out_dtype != PA_F32 && out_dtype != kv_dtype)
        return fail(PA_ERR_UNSUPPORTED, "out_dtype must be F32 or the kv dtype");
    if (N <= 0 || N > 65535 || T < 0 || H_q <= 0 || H_kv <= 0 || H_kv > 65535 || MB <= 0 || NB <= 0 ||
        max_q_len < 0)
        return fail(PA_ERR_INVALID, "bad sizes");
    if (H_q % H_kv) return fail(PA_ERR_INVALID, "H_q must be a multiple of H_kv");
    if (H_q / H_kv > 128) return fail(PA_ERR_UNSUPPORTED, "H_q / H_kv must be <= 128");
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "D must be 64 or 128");
    if (B != 8 && B != 16 && B != 32) return fail(PA_ERR_UNSUPPORTED, "prefill supports B in {8, 16, 32}");
    if (!(scale > 0.f)) return fail(PA_ERR_INVALID, "scale must be positive");
    if ((long long)NB * B >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "NB * B must be < 2^31");
    if (T == 0 || max_q_len == 0) return PA_OK;
    if (!out || !q || !pool || !block_tables || !ctx_lens || !q_start) return fail(PA_ERR_INVALID, "null pointer");
    if (!aligned16(out) || !aligned16(q) || !aligned16(pool) || !aligned16(workspace))
        return fail(PA_ERR_INVALID, "16-byte alignment");
    if (out_dtype == PA_F32 && (reinterpret_cast<uintptr_t>(out) & 31u))
        return fail(PA_ERR_INVALID, "an fp32 out must be 32-byte aligned");
    PrefillArgs a;
    a.out = out;
    a.out_dtype = out_dtype;
    a.q = q;
    a.pool = pool;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.q_start = q_start;
    a.N = N;
    a.T = T;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.B = B;
    a.MB = MB;
    a.NB = NB;
    a.max_q_len = max_q_len;
    a.scale = scale;
    a.kv_dtype = kv_dtype;
    a.workspace = workspace;
    a.ws_bytes = workspace ? ws_bytes : 0;
    a.dev_err = dev_err;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_prefill(a);
}

pa_status pa_partition_reduce(void* out, pa_dtype out_dtype, const float* part_m2, const float* part_l,
                              const float* part_acc, const int32_t* nparts, int R, int P, int D, int* dev_err,
                              void* stream) {
    const NvtxRange nvtx_range("pa_partition_reduce");
    g_msg[0] = 0;
    if (out_dtype != PA_F32 && out_dtype != PA_F16 && out_dtype != PA_BF16)
        return fail(PA_ERR_UNSUPPORTED, "bad out_dtype");
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "D must be 64 or 128");
    if (R < 0 || P <= 0) return fail(PA_ERR_INVALID, "bad sizes");
    if (R == 0) return PA_OK;
    if (!out || !part_m2 || !part_l || !part_acc || !nparts) return fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned16(part_acc)) return fail(PA_ERR_INVALID, "part_acc must be 16-byte aligned");
    return launch_partition_reduce(out, out_dtype, part_m2, part_l, part_acc, nparts, 1, R, P, D, false, dev_err,
                                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
