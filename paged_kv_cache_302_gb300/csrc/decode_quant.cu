// decode_quant.cu -- single-token decode attention over the quantised cache (quant.cuh).
#include "attend_rows.cuh"

namespace pa {

pa_status launch_decode_quant(const DecodeQuantArgs& a) {
    RowsParams p = {};
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.q = a.q;
    p.pool = a.qpool;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.tables = a.tables;
    p.ctx_lens = a.ctx_lens;
    p.N = a.N;
    p.H_q = a.H_q;
    p.H_kv = a.H_kv;
    p.G = a.H_q / a.H_kv;
    p.lgB = a.B == 8 ? 3 : a.B == 16 ? 4 : 5;
    p.MB = a.MB;
    p.NB = a.NB;
    p.max_ctx = a.max_ctx;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.err = a.dev_err;
    return launch_attend_rows(p, a.N, a.q_dtype, a.D, a.stream);
}

}  // namespace pa
