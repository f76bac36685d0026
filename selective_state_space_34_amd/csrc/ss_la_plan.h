// Plans and workspace layout of the linear-attention, norm and 4-bit product entry points.
// Host-only, HIP-free: everything here depends on the dims alone.
#pragma once

#include "ss_plan.h"

namespace ss {

// Whether one launch takes the workgroups: the runtime counts its threads in 32 bits, and more of
// them are cut off without an error.
inline bool launch_ok(int64_t blocks, int threads) {
    return blocks <= int64_t(0xffffffffu) / threads;
}

// Tiling of one sweep (ss_la_sweep.h) over rows of width dA (contracted, and the state's rows)
// and dC (the output's columns, and the state's).
struct LaShape {
    int pad_a;   // dA padded to the kernel's 64, 128 or 256
    int waves;   // of a workgroup, 16 columns each: 4 or 8
    int tiles;   // workgroups over dC
};

inline LaShape la_shape(int64_t dA, int64_t dC) {
    LaShape s;
    s.pad_a = dA <= 64 ? 64 : dA <= 128 ? 128 : 256;
    s.waves = dC <= 64 ? 4 : 8;
    s.tiles = int((dC + 16 * s.waves - 1) / (16 * s.waves));
    return s;
}

constexpr int64_t kLaMaxDim = 256;
inline int64_t la_chunk(int in_dtype) { return in_dtype == SS_BF16 ? 64 : 32; }

// Workgroups of a sweep that the 256 CUs hold at once, by the waves a SIMD that its registers
// and LDS allow (four workgroups of four waves would need 188 KB of it in bf16); dots: the
// sweeps that also give the sums behind dg.
inline int64_t la_round(const LaShape& s, bool dots, int in_dtype) {
    const int small = in_dtype == SS_BF16 && s.waves == 4 ? 3 : 4;
    const int waves = s.pad_a == 64 && !dots ? small : s.pad_a == 256 && s.waves == 4 ? 1 : 2;
    return 256 * (4 * waves / s.waves);
}

// Segments of a sequence that are swept side by side: as many as are resident at once (a few
// more would take a second round as long as the first: a sweep over 13 segments of 40 heads
// measured 369 us, over 12 it measured 281), none shorter than `least` chunks.
inline int64_t la_segments(int64_t n, int64_t nchunk, int64_t least) {
    if (n > nchunk / least) n = nchunk / least;
    if (n < 1) n = 1;
    const int64_t len = (nchunk + n - 1) / n;
    return (nchunk + len - 1) / len;
}

struct LaPlan {
    int64_t B, T, H, Hk, dk, dv;
    int in_dtype, decay;
    float scale;
    int64_t nchunk;
    LaShape fwd, rev;           // sweeps whose state is [dk, dv]; [dv, dk]
    int64_t nseg, seg_chunks;
    // forward: off_state [B, H, nseg, dk·dv], off_decay [B, H, nseg] (nseg > 1)
    // backward: the same for the forward direction, and
    //   off_rstate, off_rdecay   the same of the reverse direction (nseg > 1)
    //   off_row, off_col   [rev.tiles, B, H, T] row and column sums behind dg (64 bits)
    //   off_final          [B, H, dk, dv] S_T
    //   off_border         [B, H, nseg + 1] (64 bits) <adjoint, state> at the segments' borders
    //   off_head           [B, H, nseg] (64 bits) dg summed over a segment (one decay a head)
    //   off_part, off_part2      [B, T, H, dk] float32 dq and dk of each value head (Hk < H)
    size_t off_state, off_decay, off_rstate, off_rdecay, off_row, off_col, off_final, off_border,
        off_head, off_part, off_part2, total;
};

// q, k, v strides: all zero means dense; otherwise each must be >= 0.
inline bool la_strides_ok(const int64_t* s) {
    const int64_t lim = int64_t(1) << 40;
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] > lim) return false;
    return true;
}

inline int make_la_plan(const ss_la_dims& d, bool backward, LaPlan* out) {
    if (d.batch <= 0 || d.seqlen <= 0 || d.heads <= 0 || d.kheads <= 0 || d.dk <= 0 || d.dv <= 0)
        return SS_ERR_DIMS;
    if (d.dk > kLaMaxDim || d.dv > kLaMaxDim || d.heads % d.kheads != 0) return SS_ERR_DIMS;
    if (d.in_dtype != SS_F32 && d.in_dtype != SS_BF16) return SS_ERR_DTYPE;
    if (d.decay < SS_LA_DECAY_NONE || d.decay > SS_LA_DECAY_TOKEN) return SS_ERR_DTYPE;
    // a chunk's rows of an output lie within 2^30 bytes
    if (d.heads >= (int64_t(1) << 22) / (d.dk > d.dv ? d.dk : d.dv)) return SS_ERR_DIMS;
    if (!(d.scale - d.scale == 0.0f)) return SS_ERR_DIMS;   // not finite
    if (!la_strides_ok(d.q_stride) || !la_strides_ok(d.k_stride) || !la_strides_ok(d.v_stride))
        return SS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 38;   // elements of any tensor
    if (!mul_ok(d.batch, d.seqlen, lim) || !mul_ok(d.batch * d.seqlen, d.heads, lim / kLaMaxDim))
        return SS_ERR_DIMS;
    if (!mul_ok(d.batch, d.heads, lim / (kLaMaxDim * kLaMaxDim))) return SS_ERR_DIMS;
    LaPlan p{};
    p.B = d.batch; p.T = d.seqlen; p.H = d.heads; p.Hk = d.kheads; p.dk = d.dk; p.dv = d.dv;
    p.in_dtype = d.in_dtype; p.decay = d.decay; p.scale = d.scale;
    const int64_t C = la_chunk(d.in_dtype);
    p.nchunk = (p.T + C - 1) / C;
    p.fwd = la_shape(p.dk, p.dv);
    p.rev = la_shape(p.dv, p.dk);
    const int64_t bh = p.B * p.H;
    int64_t n = la_round(p.fwd, false, p.in_dtype) / (bh * p.fwd.tiles);
    if (backward) {
        const int64_t r = la_round(p.rev, p.decay != SS_LA_DECAY_NONE, p.in_dtype) / (bh * p.rev.tiles);
        n = r < n ? r : n;
    }
    // the gradient's borders are exact, so there short segments are a gain in themselves
    p.nseg = la_segments(n, p.nchunk, backward ? 1 : 2);
    p.seg_chunks = (p.nchunk + p.nseg - 1) / p.nseg;
    // one workgroup for each (column tile, row, head, segment), and for each border of a segment
    if (!launch_ok(bh * p.nseg * p.fwd.tiles, 64 * p.fwd.waves)) return SS_ERR_DIMS;
    if (backward && (!launch_ok(bh * p.nseg * p.rev.tiles, 64 * p.rev.waves) ||
                     !launch_ok(bh * (p.nseg + 1), 256)))
        return SS_ERR_DIMS;
    const size_t f = sizeof(float);
    const size_t state = size_t(bh) * size_t(p.dk * p.dv) * f;
    size_t off = 0;
    p.off_state = off;
    if (p.nseg > 1) off = align256(off + size_t(p.nseg) * state);
    p.off_decay = off;
    if (p.nseg > 1) off = align256(off + size_t(bh * p.nseg) * f);
    if (backward) {
        p.off_rstate = off;
        if (p.nseg > 1) off = align256(off + size_t(p.nseg) * state);
        p.off_rdecay = off;
        if (p.nseg > 1) off = align256(off + size_t(bh * p.nseg) * f);
        const size_t dots = size_t(p.rev.tiles) * size_t(bh) * size_t(p.T) * sizeof(double);
        p.off_row = off; off = align256(off + dots);
        p.off_col = off; off = align256(off + dots);
        p.off_final = off; off = align256(off + state);
        p.off_border = off; off = align256(off + size_t(bh * (p.nseg + 1)) * sizeof(double));
        p.off_head = off; off = align256(off + size_t(bh * p.nseg) * sizeof(double));
        const size_t part = p.Hk < p.H ? size_t(bh) * size_t(p.T) * size_t(p.dk) * f : 0;
        p.off_part = off; off = align256(off + part);
        p.off_part2 = off; off = align256(off + part);
    }
    p.total = off;
    *out = p;
    return SS_OK;
}

// Single-token step: columns of a head's state that a workgroup of 256 threads takes, four a
// thread where rows keep 16-byte alignment.  Few heads are spread over more workgroups by narrow
// strips, many keep whole rows together (us with 32 columns and with 128: 64 heads of 128 x 128 6.5 and
// 10.7, 256 heads 12.4 and 17.5, 512 23.0 and 22.1, 1024 39.6 and 35.2; 64 x 128: 1280 heads 32
// and 23, 10240 207 and 147).
inline int la_step_columns(int64_t bh, int64_t dv) {
    if (dv % 4 == 0) return bh >= 512 ? 128 : 32;
    return 32;
}

// Norm: how many threads share a row and how many eight-element pieces each holds.
struct RmsPlan {
    int64_t M, D;
    int threads, pieces, grid;
    size_t total;                // backward: part [grid, D] float32
};

constexpr int64_t kRmsMaxDim = 32768;

inline int make_rms_plan(const ss_rms_dims& d, bool backward, RmsPlan* out) {
    if (d.rows <= 0 || d.dim <= 0 || d.dim > kRmsMaxDim) return SS_ERR_DIMS;
    if (!mul_ok(d.rows, d.dim, int64_t(1) << 40)) return SS_ERR_DIMS;
    if (d.in_dtype != SS_F32 && d.in_dtype != SS_BF16) return SS_ERR_DTYPE;
    if (d.res_dtype != SS_F32 && d.res_dtype != SS_BF16) return SS_ERR_DTYPE;
    if (d.in_dtype == SS_F32 && d.res_dtype != SS_F32) return SS_ERR_DTYPE;
    if (d.q8 < SS_Q8_NONE || d.q8 > SS_Q8_INT8 || (backward && d.q8 != SS_Q8_NONE))
        return SS_ERR_DTYPE;
    if (!(d.eps >= 0.0f) || !(d.eps - d.eps == 0.0f)) return SS_ERR_DIMS;
    RmsPlan p{};
    p.M = d.rows; p.D = d.dim;
    const int64_t D = d.dim;
    // The fewest threads that hold a row in one or two pieces each, so that many rows are in
    // flight on a CU.  In between, 2048 < D <= 64·8·6, the forward over many rows is faster with
    // a wave a row and no barrier (D = 2560, 16384 rows, bf16, 8-bit output: 56 us against 61;
    // odd width 2563: 75 against 96), the gradient, with three rows and dw to hold, is not
    // (97 us against 83).
    if (D <= 64 * 8 * 2) {
        p.threads = D <= 8 * 8 ? 8 : D <= 32 * 8 ? 32 : 64;
        p.pieces = D <= 64 * 8 ? 1 : 2;
    } else if (!backward && D > 256 * 8 && D <= 64 * 8 * 6 && d.rows >= 1024) {
        p.threads = 64;
        p.pieces = 6;
    } else if (D <= 256 * 8 * 2) {
        p.threads = 256;
        p.pieces = D <= 256 * 8 ? 1 : 2;
    } else if (D <= 512 * 8 * 2) {
        p.threads = 512;
        p.pieces = 2;
    } else {
        p.threads = 1024;
        p.pieces = D <= 1024 * 8 * 2 ? 2 : 4;
    }
    const int64_t wg_rows = p.threads >= 256 ? 1 : 256 / p.threads;
    const int64_t need = (d.rows + wg_rows - 1) / wg_rows;
    // Workgroups take rows in turn.  Two on each CU where one holds much, four where each leaves
    // a row of partial sums (gradient, D = 2560: 1024 workgroups 81 us, 2048 86; D = 5120: 512
    // 146 us, 1024 153), else eight.
    const int64_t most = p.threads >= 512 || p.pieces == 6 ? 512 : backward ? 1024 : 2048;
    p.grid = int(need < most ? need : most);
    p.total = backward ? align256(size_t(p.grid) * size_t(D) * sizeof(float)) : 0;
    *out = p;
    return SS_OK;
}

// 4-bit products: rows of x a workgroup takes, and its 16-row tiles of weights.
struct Q4Plan {
    int64_t groups;
    int mb, tiles;
};

inline int make_q4_plan(const ss_q4_dims& d, Q4Plan* out) {
    if (d.rows <= 0 || d.n <= 0 || d.k <= 0 || d.k % 32 != 0) return SS_ERR_DIMS;
    if (d.group != 32 && d.group != 64 && d.group != 128) return SS_ERR_DIMS;
    if (d.in_dtype != SS_F32 && d.in_dtype != SS_BF16) return SS_ERR_DTYPE;
    if (d.y_dtype != SS_F32 && d.y_dtype != SS_BF16) return SS_ERR_DTYPE;
    if (d.x_q8 < SS_Q8_NONE || d.x_q8 > SS_Q8_INT8) return SS_ERR_DTYPE;
    const int64_t lim = int64_t(1) << 38;
    if (!mul_ok(d.rows, d.k, lim) || !mul_ok(d.n, d.k, lim) || !mul_ok(d.rows, d.n, lim))
        return SS_ERR_DIMS;
    Q4Plan p{};
    const int terms = d.x_q8 == SS_Q8_NONE && d.in_dtype == SS_F32 ? 3 : 1;
    p.mb = 16 / terms;
    if (d.rows < p.mb) p.mb = int(d.rows);
    if ((d.rows + p.mb - 1) / p.mb > kMaxGridYZ) return SS_ERR_DIMS;
    p.groups = (d.k + d.group - 1) / d.group;
    // A workgroup's eight waves share the groups of its rows of weights.  Two tiles of rows share the
    // work on x where that leaves a workgroup for every CU (bf16, us: 16 x 2560 by 10240 11 with
    // two tiles, 12.5 with one; 1 x 8192 by 16384 24 against 27); with fewer, one tile keeps
    // more CUs busy (16 x 5120 in 8 bits by 2560 11 against 17).
    const int64_t wgs = (d.n + 15) / 16 * ((d.rows + p.mb - 1) / p.mb);
    p.tiles = wgs >= 512 ? 2 : 1;
    if (!launch_ok((d.n + 16 * p.tiles - 1) / (16 * p.tiles), 512)) return SS_ERR_DIMS;
    *out = p;
    return SS_OK;
}

}  // namespace ss
