// tree.cu -- attention of drafted tokens over a paged cache under a tree mask.
#include "attend_rows.cuh"

namespace pa {

size_t tree_workspace_bytes(int N, int H_q, int H_kv, int D, int max_q_len) {
    if (N <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || (D != 64 && D != 128) || max_q_len <= 0) return 0;
    return 256;
}

pa_status launch_tree(const TreeArgs& a) {
    RowsParams p = {};
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.q = a.q;
    p.pool = a.pool;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.q_start = a.q_start;
    p.mask = a.mask;
    p.mask_words = a.mask_words;
    p.N = a.N;
    p.T = a.T;
    p.H_q = a.H_q;
    p.H_kv = a.H_kv;
    p.G = a.H_q / a.H_kv;
    p.lgB = a.B == 8 ? 3 : a.B == 16 ? 4 : 5;
    p.MB = a.MB;
    p.NB = a.NB;
    p.max_ctx = 0x7fffffff;
    p.max_q_len = a.max_q_len;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.err = a.dev_err;
    return launch_attend_rows(p, a.T, a.q_dtype, a.D, a.stream);
}

}  // namespace pa
