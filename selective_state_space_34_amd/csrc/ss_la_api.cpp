// C ABI of the linear attention, the norm and the 4-bit products: validation, workspace carving and launches on the caller's
// stream.  Declared in include/ss.h; nothing is launched before every argument is checked.
#include "ss.h"

#include <hip/hip_runtime.h>

#include "ss_kernels.h"
#include "ss_la_plan.h"

namespace {

using ss::hip_fail;
using ss::LaOperand;
using ss::LaPlan;
using ss::LaSweep;
using ss::LaSweeps;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Row layout of a [B, T, heads, dim] tensor, dense where no stride is given.  full: every chunk
// holds as many tokens as it has room for.
LaOperand operand(const LaPlan& p, const void* ptr, const int64_t* stride, int64_t heads,
                  int64_t dim, bool full) {
    LaOperand o{};
    o.p = ptr;
    o.sb = p.T * heads * dim; o.st = heads * dim; o.sh = dim;
    if (stride && (stride[0] || stride[1] || stride[2])) {
        o.sb = stride[0]; o.st = stride[1]; o.sh = stride[2];
    }
    if (p.T == 1) o.st = dim;   // a single token's stride says nothing
    o.rep = p.H / heads;
    o.dim = int(dim);
    // Tokens that share memory (an expanded or overlapping operand) take, unless all chunks are
    // full, the loads that ask for each token whether it exists: the others take their bounds from
    // the end of the chunk's last row, behind which the next tokens begin only where a row is no
    // longer than its stride.  (k and v expanded, B = 4, H = 16, 128 x 128, bf16: T = 2048 80 us
    // with the bounds, 96 without.)
    const int64_t v = p.in_dtype == SS_BF16 ? 8 : 4;
    o.vec = aligned(ptr, 16) && o.sb % v == 0 && o.st % v == 0 && o.sh % v == 0 && dim % v == 0 &&
            (full || o.st >= dim) && o.st < (int64_t(1) << 22);
    return o;
}

struct Inputs {
    LaOperand q, k, v;
};

// Checks what the three entry points share.
int check(const ss_la_dims* d, bool backward, const void* q, const void* k, const void* v,
          const float* g, const int32_t* lengths, LaPlan* p) {
    const int rc = ss::make_la_plan(*d, backward, p);
    if (rc != SS_OK) return rc;
    if (!q || !k || !v || ((p->decay != SS_LA_DECAY_NONE) != (g != nullptr))) return SS_ERR_NULL;
    const size_t el = p->in_dtype == SS_BF16 ? 2 : 4;
    if (!aligned(q, el) || !aligned(k, el) || !aligned(v, el) || !aligned(g, 4) ||
        !aligned(lengths, 4))
        return SS_ERR_ALIGN;
    return SS_OK;
}

Inputs inputs(const ss_la_dims* d, const LaPlan& p, const void* q, const void* k, const void* v,
              const int32_t* lengths) {
    const bool full = !lengths && p.T % ss::la_chunk(p.in_dtype) == 0;
    return Inputs{operand(p, q, d->q_stride, p.Hk, p.dk, full),
                  operand(p, k, d->k_stride, p.Hk, p.dk, full),
                  operand(p, v, d->v_stride, p.H, p.dv, full)};
}

hipError_t sweep(const LaPlan& p, const LaSweeps& s, hipStream_t stream) {
    bool vec = true;
    for (int i = 0; i < s.n; ++i)
        vec = vec && s.p[i].a.vec && s.p[i].b.vec && s.p[i].c.vec && s.p[i].e.vec;
    if (p.in_dtype == SS_BF16)
        return vec ? ss::launch_la_sweep_bf16(s, stream) : ss::launch_la_sweep_bf16_any(s, stream);
    return vec ? ss::launch_la_sweep_f32(s, stream) : ss::launch_la_sweep_f32_any(s, stream);
}

LaSweep base(const LaPlan& p, const float* g, const int32_t* lengths, int reverse) {
    LaSweep s{};
    s.g = g; s.decay_token = p.decay == SS_LA_DECAY_TOKEN; s.lengths = lengths;
    s.B = p.B; s.T = p.T; s.H = p.H;
    s.nseg = int(p.nseg); s.seg_chunks = p.seg_chunks;
    s.reverse = reverse;
    // forward: the scale goes into out; reverse: the state collects scale·q doᵀ, so that dS_T
    // enters it as it is
    s.alpha = p.scale;
    s.in_scale = reverse ? 1.0f : p.scale;
    s.up_scale = reverse ? p.scale : 1.0f;
    return s;
}

void shape(LaSweep* s, const ss::LaShape& f) {
    s->pad_a = f.pad_a; s->waves = f.waves; s->tiles = f.tiles;
}

// States entering every segment, [B, H, nseg, dA, dC] from where[i].state on, from the operands
// b, c of each sweep and the state that enters the whole sequence (element (i, j) at
// i·f_i + j·f_j; nullable).
struct Entering {
    float* state;
    float* decay;
    const float* first;
    int64_t f_i, f_j;
};
hipError_t segment_states(const LaPlan& p, LaSweeps w, const ss::LaShape& f, const Entering* where,
                          hipStream_t stream) {
    const int64_t sz = p.dk * p.dv;
    ss::LaCarries c{};
    c.n = w.n;
    for (int i = 0; i < w.n; ++i) {
        LaSweep& s = w.p[i];
        const Entering& e = where[i];
        shape(&s, f);
        s.state_only = 1;
        s.a = s.b; s.e = s.b;
        s.grid_seg = s.nseg - 1; s.seg0 = s.reverse ? 1 : 0;
        s.s_in = nullptr; s.in_seg = 1; s.s_in_sz = sz;
        s.s_out = e.state;
        s.seg_decay = e.decay;
        s.dots = nullptr; s.out = nullptr;
        ss::LaCarry& t = c.p[i];
        t.state = e.state; t.decay = e.decay; t.first = e.first; t.BH = p.B * p.H; t.sz = sz;
        t.dC = s.c.dim; t.f_i = e.f_i; t.f_j = e.f_j; t.nseg = s.nseg; t.reverse = s.reverse;
    }
    const hipError_t e = sweep(p, w, stream);
    return e == hipSuccess ? ss::launch_la_carry(c, stream) : e;
}

// What is common to whole sweeps: the state [dA, dC] enters each segment from `state` (nseg > 1)
// or from `first`; strides as element (i, j).
void whole(const LaPlan& p, LaSweep* s, const ss::LaShape& f, const float* first, int64_t f_i,
           int64_t f_j, const float* state, int64_t s_i, int64_t s_j) {
    shape(s, f);
    s->grid_seg = s->nseg; s->seg0 = 0;
    s->s_in_sz = p.dk * p.dv;
    if (s->nseg > 1) {
        s->s_in = state; s->in_seg = s->nseg; s->s_in_i = s_i; s->s_in_j = s_j;
    } else {
        s->s_in = first; s->in_seg = 1; s->s_in_i = f_i; s->s_in_j = f_j;
    }
}

int workspace_size(const ss_la_dims* dims, bool backward, size_t* bytes) {
    if (!dims || !bytes) return SS_ERR_NULL;
    LaPlan p;
    const int rc = ss::make_la_plan(*dims, backward, &p);
    if (rc != SS_OK) return rc;
    *bytes = p.total;
    return SS_OK;
}

ss::RmsLaunch rms_launch(const ss_rms_dims& d, const ss::RmsPlan& p) {
    ss::RmsLaunch l{};
    l.M = p.M; l.D = p.D; l.eps = d.eps; l.inv_d = float(1.0 / double(p.D));
    l.in_dtype = d.in_dtype; l.res_dtype = d.res_dtype;
    l.threads = p.threads; l.pieces = p.pieces; l.grid = p.grid;
    return l;
}

}  // namespace

extern "C" {

int ss_la_fwd_workspace_size(const ss_la_dims* dims, size_t* bytes) {
    return workspace_size(dims, false, bytes);
}

int ss_la_bwd_workspace_size(const ss_la_dims* dims, size_t* bytes) {
    return workspace_size(dims, true, bytes);
}

int ss_la_fwd(const ss_la_dims* dims, const void* q, const void* k, const void* v, const float* g,
              const float* s0, const int32_t* lengths, void* o, float* s_final,
              void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    LaPlan p;
    const int rc = check(dims, false, q, k, v, g, lengths, &p);
    if (rc != SS_OK) return rc;
    if (!o) return SS_ERR_NULL;
    if (!aligned(o, 16) || !aligned(s0, 16) || !aligned(s_final, 16)) return SS_ERR_ALIGN;
    if (p.total > 0 && (!workspace || workspace_bytes < p.total)) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SS_ERR_ALIGN;
    char* ws = static_cast<char*>(workspace);
    float* state = reinterpret_cast<float*>(ws + p.off_state);
    const Inputs in = inputs(dims, p, q, k, v, lengths);
    LaSweeps w{};
    w.n = 1;
    LaSweep& s = w.p[0];
    s = base(p, g, lengths, 0);
    s.a = in.q; s.b = in.k; s.c = in.v; s.e = in.v;
    hipError_t e;
    if (p.nseg > 1) {
        const Entering where{state, reinterpret_cast<float*>(ws + p.off_decay), s0, p.dv, 1};
        e = segment_states(p, w, p.fwd, &where, stream);
        if (e != hipSuccess) return hip_fail(e);
    }
    s.out = o; s.s_out = s_final;
    whole(p, &s, p.fwd, s0, p.dv, 1, state, p.dv, 1);
    e = sweep(p, w, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_la_bwd(const ss_la_dims* dims, const void* q, const void* k, const void* v, const float* g,
              const float* s0, const int32_t* lengths, const void* dO, const float* ds_final,
              void* dq, void* dk, void* dv, float* dg, float* ds0,
              void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    LaPlan p;
    const int rc = check(dims, true, q, k, v, g, lengths, &p);
    if (rc != SS_OK) return rc;
    if (!dO || !dq || !dk || !dv) return SS_ERR_NULL;
    if ((g != nullptr) != (dg != nullptr) || (s0 != nullptr) != (ds0 != nullptr)) return SS_ERR_NULL;
    const void* ptrs[] = {s0, dO, ds_final, dq, dk, dv, dg, ds0};
    for (const void* x : ptrs)
        if (!aligned(x, 16)) return SS_ERR_ALIGN;
    if (p.total > 0 && (!workspace || workspace_bytes < p.total)) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SS_ERR_ALIGN;
    char* ws = static_cast<char*>(workspace);
    auto at = [ws](size_t off) { return reinterpret_cast<float*>(ws + off); };
    float* state = at(p.off_state);
    float* decay = at(p.off_decay);
    float* part = p.Hk < p.H ? at(p.off_part) : nullptr;
    auto dots = [ws](size_t off) { return reinterpret_cast<double*>(ws + off); };
    float* s_final = g && ds_final ? at(p.off_final) : nullptr;
    const int bf16 = p.in_dtype == SS_BF16;
    const Inputs in = inputs(dims, p, q, k, v, lengths);
    const LaOperand od = operand(p, dO, nullptr, p.H, p.dv, true);
    float* part2 = p.Hk < p.H ? at(p.off_part2) : nullptr;
    float* rstate = at(p.off_rstate);
    hipError_t e;

    // 1. the segments' states, S_tᵀ forward and dS_tᵀ reverse, both [dv, dk]
    LaSweeps w{};
    w.n = 2;
    LaSweep &f = w.p[0], &r = w.p[1];
    f = base(p, g, lengths, 0);
    f.a = od; f.b = in.v; f.c = in.k; f.e = in.q;
    r = base(p, g, lengths, 1);
    r.a = in.v; r.b = od; r.c = in.q; r.e = in.k;
    if (p.nseg > 1) {
        const Entering where[2] = {{state, decay, s0, 1, p.dv},
                                   {rstate, at(p.off_rdecay), ds_final, 1, p.dv}};
        e = segment_states(p, w, p.rev, where, stream);
        if (e != hipSuccess) return hip_fail(e);
    }

    // 2. dq: forward sweep of (dO, v, k); dk: reverse sweep of (v, dO, q)
    f.out = part ? static_cast<void*>(part) : dq; f.out_f32 = part != nullptr;
    f.dots = g ? dots(p.off_row) : nullptr;
    f.s_out = s_final; f.s_out_t = 1;
    whole(p, &f, p.rev, s0, 1, p.dv, state, p.dk, 1);
    r.out = part2 ? static_cast<void*>(part2) : dk; r.out_f32 = part2 != nullptr;
    r.dots = g ? dots(p.off_col) : nullptr;
    whole(p, &r, p.rev, ds_final, 1, p.dv, rstate, p.dk, 1);
    e = sweep(p, w, stream);
    if (e != hipSuccess) return hip_fail(e);
    if (part) {
        const ss::LaGroupSum gs{{part, part2}, {dq, dk}, p.B * p.T * p.Hk * p.dk, p.H / p.Hk, p.dk};
        e = ss::launch_la_group_sum(bf16, gs, stream);
        if (e != hipSuccess) return hip_fail(e);
    }

    // dg from the row and column sums and the states at the segments' borders
    ss::LaDecayGrad d{};
    d.row = dots(p.off_row); d.col = dots(p.off_col); d.tiles = p.rev.tiles;
    d.fwd_state = state; d.rev_state = rstate;
    d.s0 = s0; d.ds0 = ds0; d.ds = ds_final; d.s_final = s_final;
    d.border = dots(p.off_border); d.head_part = dots(p.off_head);
    d.lengths = lengths; d.dg = dg;
    d.B = p.B; d.T = p.T; d.H = p.H; d.dk = p.dk; d.dv = p.dv;
    d.nseg = int(p.nseg); d.seg_tokens = p.seg_chunks * ss::la_chunk(p.in_dtype);
    d.decay_token = p.decay == SS_LA_DECAY_TOKEN;
    d.borders = d.nseg + 1;
    if (s_final && ds0 == ds_final) {   // in place: the last border before dS_0 replaces dS_T
        d.border0 = d.nseg; d.borders = 1;
        e = ss::launch_la_borders(d, stream);
        if (e != hipSuccess) return hip_fail(e);
        d.border0 = 0; d.borders = d.nseg;
    }

    // 3. dv: reverse sweep of (k, q, dO) with the state transposed, dS_t [dk, dv]
    w.n = 1;
    LaSweep& s = w.p[0];
    s = base(p, g, lengths, 1);
    s.a = in.k; s.b = in.q; s.c = od; s.e = od;
    s.out = dv; s.s_out = ds0;
    whole(p, &s, p.fwd, ds_final, p.dv, 1, rstate, 1, p.dk);
    e = sweep(p, w, stream);
    if (e != hipSuccess) return hip_fail(e);

    // 4. dg
    if (g) {
        e = ss::launch_la_borders(d, stream);
        if (e != hipSuccess) return hip_fail(e);
        e = ss::launch_la_decay_grad(d, stream);
        if (e != hipSuccess) return hip_fail(e);
    }
    return SS_OK;
}

int ss_la_step(const ss_la_dims* dims, const void* q, const void* k, const void* v, const float* g,
               const float* s_in, float* s_out, void* o, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    if (dims->seqlen != 1) return SS_ERR_DIMS;
    LaPlan p;
    const int rc = check(dims, false, q, k, v, g, nullptr, &p);
    if (rc != SS_OK) return rc;
    const int columns = ss::la_step_columns(p.B * p.H, p.dv);
    if (!ss::launch_ok(p.B * p.H * ((p.dv + columns - 1) / columns), 256)) return SS_ERR_DIMS;
    if (!s_in || !s_out || !o) return SS_ERR_NULL;
    if (!aligned(s_in, 16) || !aligned(s_out, 16) || !aligned(o, 16)) return SS_ERR_ALIGN;
    const Inputs in = inputs(dims, p, q, k, v, nullptr);
    ss::LaStep s{};
    s.q = in.q; s.k = in.k; s.v = in.v; s.g = g; s.decay_token = p.decay == SS_LA_DECAY_TOKEN;
    s.s_in = s_in; s.s_out = s_out; s.o = o;
    s.B = p.B; s.H = p.H; s.dk = p.dk; s.dv = p.dv; s.columns = columns; s.scale = p.scale;
    const hipError_t e = ss::launch_la_step(p.in_dtype == SS_BF16, s, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_rms_fwd(const ss_rms_dims* dims, const void* x, const void* res, const float* w, void* r,
               void* y, float* y_scale, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    ss::RmsPlan p;
    const int rc = ss::make_rms_plan(*dims, false, &p);
    if (rc != SS_OK) return rc;
    if (!x || !w || !y || ((res != nullptr) != (r != nullptr)) ||
        ((dims->q8 != SS_Q8_NONE) != (y_scale != nullptr)))
        return SS_ERR_NULL;
    const void* ptrs[] = {x, res, w, r, y, y_scale};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return SS_ERR_ALIGN;
    ss::RmsLaunch l = rms_launch(*dims, p);
    l.x = x; l.res = res; l.w = w; l.r = r; l.y = y; l.y_scale = y_scale; l.q8 = dims->q8;
    const hipError_t e = ss::launch_rms_fwd(l, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_rms_bwd_workspace_size(const ss_rms_dims* dims, size_t* bytes) {
    if (!dims || !bytes) return SS_ERR_NULL;
    ss::RmsPlan p;
    const int rc = ss::make_rms_plan(*dims, true, &p);
    if (rc != SS_OK) return rc;
    *bytes = p.total;
    return SS_OK;
}

int ss_rms_bwd(const ss_rms_dims* dims, const void* dy, const void* r, const float* w,
               const void* dr, void* dx, float* dw, void* workspace, size_t workspace_bytes,
               hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    ss::RmsPlan p;
    const int rc = ss::make_rms_plan(*dims, true, &p);
    if (rc != SS_OK) return rc;
    if (!dy || !r || !w || !dx || !dw) return SS_ERR_NULL;
    const void* ptrs[] = {dy, r, w, dr, dx, dw};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return SS_ERR_ALIGN;
    if (!workspace || workspace_bytes < p.total) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SS_ERR_ALIGN;
    ss::RmsLaunch l = rms_launch(*dims, p);
    l.x = dy; l.res = r; l.w = w; l.dr = dr; l.r = dx; l.part = static_cast<float*>(workspace);
    const hipError_t e = ss::launch_rms_bwd(l, dw, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

int ss_q4_mv(const ss_q4_dims* dims, const void* x, const float* x_scale, const void* wq,
             const void* scales, const void* zeros, void* y, hipStream_t stream) {
    if (!dims) return SS_ERR_NULL;
    ss::Q4Plan p;
    const int rc = ss::make_q4_plan(*dims, &p);
    if (rc != SS_OK) return rc;
    if (!x || !wq || !scales || !y || ((dims->x_q8 != SS_Q8_NONE) != (x_scale != nullptr)))
        return SS_ERR_NULL;
    const void* ptrs[] = {x, x_scale, wq, scales, zeros, y};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return SS_ERR_ALIGN;
    ss::Q4Launch l{};
    l.x = x; l.x_scale = x_scale; l.wq = static_cast<const uint8_t*>(wq);
    l.scales = static_cast<const uint16_t*>(scales); l.zeros = static_cast<const uint8_t*>(zeros);
    l.y = y; l.M = dims->rows; l.N = dims->n; l.K = dims->k;
    l.groups = p.groups; l.mb = p.mb; l.tiles = p.tiles; l.group = dims->group;
    l.in_dtype = dims->in_dtype; l.x_q8 = dims->x_q8; l.y_dtype = dims->y_dtype;
    const hipError_t e = ss::launch_q4(l, stream);
    return e == hipSuccess ? SS_OK : hip_fail(e);
}

}  // extern "C"
