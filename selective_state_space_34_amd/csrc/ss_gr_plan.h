// Plans and workspace layout of the gated recurrence, layer norm and microscaled product entry
// points.  Host-only, HIP-free: everything here depends on the dims alone.
#pragma once

#include "ss_la_plan.h"

namespace ss {

struct GrPlan {
    int64_t B, T, D;
    int64_t nckpt;              // checkpoints of a row
    int64_t parts;              // rows of partial sums behind dlam
    // backward: off_ckpt [B, nckpt, D] where none are given, off_part [parts, D]
    size_t off_ckpt, off_part, total;
};

inline bool gr_strides_ok(const int64_t* s) {
    const int64_t lim = int64_t(1) << 40;
    return s[0] >= 0 && s[0] <= lim && s[1] >= 0 && s[1] <= lim;
}

inline int make_gr_plan(const ss_gr_dims& d, bool backward, bool given_ckpt, GrPlan* out) {
    if (d.batch <= 0 || d.seqlen <= 0 || d.dim <= 0 || d.dim > (int64_t(1) << 28)) return SS_ERR_DIMS;
    if (d.in_dtype != SS_F32 && d.in_dtype != SS_BF16) return SS_ERR_DTYPE;
    if (!(d.c > 0.0f) || !(d.c - d.c == 0.0f)) return SS_ERR_DIMS;
    if (!gr_strides_ok(d.x_stride) || !gr_strides_ok(d.r_stride) || !gr_strides_ok(d.i_stride))
        return SS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 40;   // elements of any tensor
    if (!mul_ok(d.batch, d.seqlen, lim) || !mul_ok(d.batch * d.seqlen, d.dim, lim)) return SS_ERR_DIMS;
    if (d.batch > kMaxGridYZ) return SS_ERR_DIMS;
    GrPlan p{};
    p.B = d.batch; p.T = d.seqlen; p.D = d.dim;
    if (!launch_ok((p.D + 127) / 128 * p.B, 512)) return SS_ERR_DIMS;
    p.nckpt = (p.T + SS_GR_CKPT - 1) / SS_GR_CKPT;
    size_t off = 0;
    if (backward) {
        p.parts = p.B;
        p.off_ckpt = off;
        if (!given_ckpt) off = align256(off + size_t(p.B * p.nckpt) * size_t(p.D) * sizeof(float));
        p.off_part = off;
        off = align256(off + size_t(p.parts) * size_t(p.D) * sizeof(float));
    }
    p.total = off;
    *out = p;
    return SS_OK;
}

// The layer norm shares the norm's split of a row; the gradient keeps two rows of partial sums.
inline int make_ln_plan(const ss_ln_dims& d, bool backward, RmsPlan* out) {
    ss_rms_dims r{d.rows, d.dim, d.in_dtype, d.res_dtype, d.q8, d.eps};
    if (d.q8 == SS_Q4_MX && !backward) {
        if (d.dim % 32 != 0) return SS_ERR_DIMS;
        r.q8 = SS_Q8_NONE;
    }
    const int rc = make_rms_plan(r, backward, out);
    if (rc == SS_OK && backward)
        out->total = align256(size_t(out->grid) * size_t(2 * out->D) * sizeof(float));
    return rc;
}

inline int check_mx4(const ss_mx4_dims& d, bool product) {
    if (d.rows <= 0 || d.k <= 0 || d.k % 32 != 0 || (product && d.n <= 0)) return SS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 38;
    if (!mul_ok(d.rows, d.k, lim)) return SS_ERR_DIMS;
    if (!product) return d.in_dtype == SS_F32 || d.in_dtype == SS_BF16 ? SS_OK : SS_ERR_DTYPE;
    if (!mul_ok(d.n, d.k, lim) || !mul_ok(d.rows, d.n, lim)) return SS_ERR_DIMS;
    if (d.x_q8 != SS_Q4_MX && d.x_q8 != SS_Q8_FP8) return SS_ERR_DTYPE;
    if (d.y_dtype != SS_F32 && d.y_dtype != SS_BF16) return SS_ERR_DTYPE;
    if ((d.rows + 63) / 64 > kMaxGridYZ || !launch_ok((d.n + 15) / 16 * ((d.rows + 63) / 64), 512))
        return SS_ERR_DIMS;
    return SS_OK;
}

}  // namespace ss
