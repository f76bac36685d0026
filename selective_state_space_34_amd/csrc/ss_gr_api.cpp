// C ABI of the gated recurrence, the layer norm and the microscaled 4-bit products: validation,
// workspace carving and launches on the caller's stream.  Declared in include/ss.h; nothing is
// launched before every argument is checked.
#include "ss.h"

#include <hip/hip_runtime.h>

#include "ss_gr_plan.h"
#include "ss_kernels.h"

namespace {

using ss::GrLaunch;
using ss::GrPlan;
using ss::GrRows;
using ss::hip_fail;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

GrRows rows(const void* p, const int64_t* stride, int64_t T, int64_t D) {
    if (stride[0] || stride[1]) return GrRows{p, stride[0], T == 1 ? D : stride[1]};
    return GrRows{p, T * D, D};
}

int check(const ss_gr_dims* d, bool backward, bool given_ckpt, const void* x, const void* r,
          const void* i, const float* lam, const int32_t* lengths, GrPlan* p) {
    const int rc = ss::make_gr_plan(*d, backward, given_ckpt, p);
    if (rc != SS_OK) return rc;
    if (!x || !r || !i || !lam) return SS_ERR_NULL;
    const size_t el = d->in_dtype == SS_BF16 ? 2 : 4;
    if (!aligned(x, el) || !aligned(r, el) || !aligned(i, el) || !aligned(lam, 16) ||
        !aligned(lengths, 4))
        return SS_ERR_ALIGN;
    return SS_OK;
}

// How neighbouring channels are taken (GrLaunch::vec).
int pairs(int64_t D) { return D == 1 ? 0 : D % 2 ? 2 : 1; }

GrLaunch launch(const ss_gr_dims* d, const GrPlan& p, const void* x, const void* r, const void* i,
                const float* lam, const float* h0, const int32_t* lengths, const void* reset) {
    GrLaunch l{};
    l.x = rows(x, d->x_stride, p.T, p.D);
    l.r = rows(r, d->r_stride, p.T, p.D);
    l.i = rows(i, d->i_stride, p.T, p.D);
    l.lam = lam; l.h0 = h0; l.lengths = lengths; l.reset = static_cast<const uint8_t*>(reset);
    l.B = p.B; l.T = p.T; l.D = p.D; l.c = d->c; l.in_dtype = d->in_dtype;
    l.vec = pairs(p.D);
    return l;
}

void chain(GrLaunch* l, const ss::GrChain& c, char* ws) {
    l->tiles = int(c.tiles);
    l->group = int(c.group);
    l->maps = l->ends = l->ticket = nullptr;
    if (c.tiles <= 1) return;
    l->ticket = reinterpret_cast<uint64_t*>(ws + c.off_ticket);
    l->maps = reinterpret_cast<uint64_t*>(ws + c.off_maps);
    l->ends = reinterpret_cast<uint64_t*>(ws + c.off_ends);
}

// Sets the chains' counters and words.
hipError_t begin(const GrPlan& p, char* ws, hipStream_t stream) {
    if (p.words == 0) return hipSuccess;
    return ss::launch_gr_chains(reinterpret_cast<uint64_t*>(ws),
                                reinterpret_cast<uint64_t*>(ws + p.off_words), p.words, stream);
}

ss::LnLaunch ln_launch(const ss_ln_dims& d, const ss::RmsPlan& p) {
    ss::LnLaunch l{};
    l.M = p.M; l.D = p.D; l.eps = d.eps; l.inv_d = float(1.0 / double(p.D));
    l.in_dtype = d.in_dtype; l.res_dtype = d.res_dtype;
    l.threads = p.threads; l.pieces = p.pieces; l.grid = p.grid;
    return l;
}

}  // namespace

extern "C" {

int ss_gr_fwd_workspace_size(const ss_gr_dims* dims, size_t* bytes) {
    if (!dims || !bytes) return SS_ERR_NULL;
    GrPlan p;
    const int rc = ss::make_gr_plan(*dims, false, false, &p);
    if (rc == SS_OK) *bytes = p.total;
    return rc;
}

int ss_gr_bwd_workspace_size(const ss_gr_dims* dims, int given_ckpt, size_t* bytes) {
    if (!dims || !bytes) return SS_ERR_NULL;
    GrPlan p;
    const int rc = ss::make_gr_plan(*dims, true, given_ckpt != 0, &p);
    if (rc == SS_OK) *bytes = p.total;
    return rc;
}

int ss_gr_fwd(const ss_gr_dims* dims, const void* x, const void* r, const void* i, const float* lam,
              const float* h0, const int32_t* lengths, const void* reset, void* y, float* h_final,
              float* h_ckpt, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    GrPlan p;
    const int rc = check(dims, false, false, x, r, i, lam, lengths, &p);
    if (rc != SS_OK) return rc;
    if (!y) return SS_ERR_NULL;
    if (!aligned(h0, 16) || !aligned(y, 16) || !aligned(h_final, 16) || !aligned(h_ckpt, 16))
        return SS_ERR_ALIGN;
    if (p.total > 0 && (!workspace || workspace_bytes < p.total)) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SS_ERR_ALIGN;
    GrLaunch l = launch(dims, p, x, r, i, lam, h0, lengths, reset);
    l.y = y; l.h_final = h_final; l.h_ckpt = h_ckpt;
    char* ws = static_cast<char*>(workspace);
    hipError_t e = begin(p, ws, stream);
    if (e != hipSuccess) return hip_fail(e);
    chain(&l, p.fwd, ws);
    e = ss::launch_gr_fwd(l, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_gr_bwd(const ss_gr_dims* dims, const void* x, const void* r, const void* i, const float* lam,
              const float* h0, const int32_t* lengths, const void* reset, const void* dy,
              const float* dh_final, const float* h_ckpt, void* dx, void* dr, void* di, float* dlam,
              float* dh0, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    GrPlan p;
    const int rc = check(dims, true, h_ckpt != nullptr, x, r, i, lam, lengths, &p);
    if (rc != SS_OK) return rc;
    if (!dy || !dx || !dr || !di || !dlam || ((h0 != nullptr) != (dh0 != nullptr))) return SS_ERR_NULL;
    const void* ptrs[] = {h0, dy, dh_final, h_ckpt, dx, dr, di, dlam, dh0};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return SS_ERR_ALIGN;
    if (!workspace || workspace_bytes < p.total) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SS_ERR_ALIGN;
    char* ws = static_cast<char*>(workspace);
    GrLaunch l = launch(dims, p, x, r, i, lam, h0, lengths, reset);
    hipError_t e = begin(p, ws, stream);
    if (e != hipSuccess) return hip_fail(e);
    if (h_ckpt) {
        l.h_ckpt = const_cast<float*>(h_ckpt);   // read only
    } else {
        l.h_ckpt = reinterpret_cast<float*>(ws + p.off_ckpt);
        chain(&l, p.fwd, ws);
        e = ss::launch_gr_fwd(l, stream);
        if (e != hipSuccess) return hip_fail(e);
    }
    l.dy = dy; l.dh_final = dh_final; l.dx = dx; l.dr = dr; l.di = di; l.dlam = dlam; l.dh0 = dh0;
    l.part = reinterpret_cast<float*>(ws + p.off_part);
    chain(&l, p.rev, ws);
    e = ss::launch_gr_bwd(l, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_gr_step(const ss_gr_dims* dims, const void* x, const void* r, const void* i, const float* lam,
               const float* h_in, float* h_out, void* y, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    if (dims->seqlen != 1) return SS_ERR_DIMS;
    GrPlan p;
    const int rc = check(dims, false, false, x, r, i, lam, nullptr, &p);
    if (rc != SS_OK) return rc;
    if (!h_in || !h_out || !y) return SS_ERR_NULL;
    if (!aligned(h_in, 16) || !aligned(h_out, 16) || !aligned(y, 16)) return SS_ERR_ALIGN;
    ss::GrStep s{};
    s.x = rows(x, dims->x_stride, 1, p.D);
    s.r = rows(r, dims->r_stride, 1, p.D);
    s.i = rows(i, dims->i_stride, 1, p.D);
    s.lam = lam; s.h_in = h_in; s.h_out = h_out; s.y = y;
    s.B = p.B; s.D = p.D; s.c = dims->c; s.in_dtype = dims->in_dtype;
    s.vec = pairs(p.D);
    const hipError_t e = ss::launch_gr_step(s, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_ln_fwd(const ss_ln_dims* dims, const void* x, const void* res, const float* w, const float* b,
              void* r, void* y, void* y_scale, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    ss::RmsPlan p;
    const int rc = ss::make_ln_plan(*dims, false, &p);
    if (rc != SS_OK) return rc;
    if (!x || !w || !y || ((res != nullptr) != (r != nullptr)) ||
        ((dims->q8 != SS_Q8_NONE) != (y_scale != nullptr)))
        return SS_ERR_NULL;
    const void* ptrs[] = {x, res, w, b, r, y, y_scale};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return SS_ERR_ALIGN;
    ss::LnLaunch l = ln_launch(*dims, p);
    l.x = x; l.res = res; l.w = w; l.b = b; l.r = r; l.y = y;
    l.y_scale = static_cast<float*>(y_scale); l.q8 = dims->q8;
    const hipError_t e = ss::launch_ln_fwd(l, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_ln_bwd_workspace_size(const ss_ln_dims* dims, size_t* bytes) {
    if (!dims || !bytes) return SS_ERR_NULL;
    ss::RmsPlan p;
    const int rc = ss::make_ln_plan(*dims, true, &p);
    if (rc == SS_OK) *bytes = p.total;
    return rc;
}

int ss_ln_bwd(const ss_ln_dims* dims, const void* dy, const void* r, const float* w, const void* dr,
              void* dx, float* dw, float* db, void* workspace, size_t workspace_bytes,
              hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    ss::RmsPlan p;
    const int rc = ss::make_ln_plan(*dims, true, &p);
    if (rc != SS_OK) return rc;
    if (!dy || !r || !w || !dx || !dw) return SS_ERR_NULL;
    const void* ptrs[] = {dy, r, w, dr, dx, dw, db};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return SS_ERR_ALIGN;
    if (!workspace || workspace_bytes < p.total) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SS_ERR_ALIGN;
    ss::LnLaunch l = ln_launch(*dims, p);
    l.x = dy; l.res = r; l.w = w; l.dr = dr; l.r = dx; l.part = static_cast<float*>(workspace);
    const hipError_t e = ss::launch_ln_bwd(l, dw, db, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_mx4_quant(const ss_mx4_dims* dims, const void* x, void* codes, void* exps, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    const int rc = ss::check_mx4(*dims, false);
    if (rc != SS_OK) return rc;
    if (!x || !codes || !exps) return SS_ERR_NULL;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(exps, 16)) return SS_ERR_ALIGN;
    ss::Mx4Quant q{};
    q.x = x; q.codes = static_cast<uint8_t*>(codes); q.exps = static_cast<uint8_t*>(exps);
    q.blocks = dims->rows * (dims->k / 32); q.in_dtype = dims->in_dtype;
    const hipError_t e = ss::launch_mx4_quant(q, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_mx4_mm(const ss_mx4_dims* dims, const void* x, const void* x_scale, const void* wq,
              const void* w_exps, void* y, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    const int rc = ss::check_mx4(*dims, true);
    if (rc != SS_OK) return rc;
    if (!x || !x_scale || !wq || !w_exps || !y) return SS_ERR_NULL;
    const void* ptrs[] = {x, x_scale, wq, w_exps, y};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return SS_ERR_ALIGN;
    ss::Mx4Launch l{};
    l.x = static_cast<const uint8_t*>(x); l.x_scale = x_scale;
    l.wq = static_cast<const uint8_t*>(wq); l.w_exps = static_cast<const uint8_t*>(w_exps);
    l.y = y; l.M = dims->rows; l.N = dims->n; l.K = dims->k;
    l.fp8 = dims->x_q8 == SS_Q8_FP8; l.y_dtype = dims->y_dtype;
    const hipError_t e = ss::launch_mx4_mm(l, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

}  // extern "C"
