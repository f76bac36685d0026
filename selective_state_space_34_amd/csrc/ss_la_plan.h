// Plans and workspace layout of the linear-attention, norm and 4-bit product entry points.
// Host-only, HIP-free: everything here depends on the dims alone.
#pragma once

#include "ss_plan.h"

namespace ss {

// Tiling of one sweep (ss_la_sweep.h) over rows of width dA (contracted, and the state's rows)
// and dC (the output's columns, and the state's).
struct LaShape {
    int pad_a;   // dA padded to the kernel's 64, 128 or 256
    int nt;      // 16-column tiles of each of a workgroup's four waves
    int tiles;   // workgroups over dC
};

inline LaShape la_shape(int64_t dA, int64_t dC) {
    LaShape s;
    s.pad_a = dA <= 64 ? 64 : dA <= 128 ? 128 : 256;
    // 256 state rows leave registers for one 16-column tile a wave
    s.nt = dC <= 64 || s.pad_a == 256 ? 1 : 2;
    s.tiles = int((dC + 64 * s.nt - 1) / (64 * s.nt));
    return s;
}

constexpr int64_t kLaMaxDim = 256;
inline int64_t la_chunk(int in_dtype) { return in_dtype == SS_BF16 ? 64 : 32; }

// Segments of a sequence that are swept side by side: enough for two workgroups on each of
// the 256 CUs, none shorter than two chunks.
inline int64_t la_segments(int64_t rows, int64_t nchunk) {
    int64_t n = (512 + rows - 1) / rows;
    if (n > nchunk / 2) n = nchunk / 2;
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
    // backward: the same (used by one direction after the other), and
    //   off_row, off_col   [rev.tiles, B, H, T] row and column sums behind dg
    //   off_final          [B, H, dv·dk] S_Tᵀ
    //   off_head           [B, H] dg of each (row, head) summed over tokens (one decay a head)
    //   off_part           [B, T, H, dk] float32 dq, then dk, of each value head (Hk < H)
    size_t off_state, off_decay, off_row, off_col, off_final, off_head, off_part, total;
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
    const int tiles = backward && p.rev.tiles < p.fwd.tiles ? p.rev.tiles : p.fwd.tiles;
    const int most = p.rev.tiles > p.fwd.tiles ? p.rev.tiles : p.fwd.tiles;
    p.nseg = la_segments(bh * tiles, p.nchunk);
    p.seg_chunks = (p.nchunk + p.nseg - 1) / p.nseg;
    // one workgroup for each (column tile, row, head, segment), and the row-wise kernels
    const int64_t grid = int64_t(1) << 31;
    if (!mul_ok(bh, p.nseg * most, grid - 1)) return SS_ERR_DIMS;
    const size_t f = sizeof(float);
    const size_t state = size_t(bh) * size_t(p.dk * p.dv) * f;
    size_t off = 0;
    p.off_state = off;
    if (p.nseg > 1) off = align256(off + size_t(p.nseg) * state);
    p.off_decay = off;
    if (p.nseg > 1) off = align256(off + size_t(bh * p.nseg) * f);
    if (backward) {
        const size_t dots = size_t(p.rev.tiles) * size_t(bh) * size_t(p.T) * f;
        p.off_row = off; off = align256(off + dots);
        p.off_col = off; off = align256(off + dots);
        p.off_final = off; off = align256(off + state);
        p.off_head = off; off = align256(off + size_t(bh) * f);
        p.off_part = off;
        if (p.Hk < p.H) off = align256(off + size_t(bh) * size_t(p.T) * size_t(p.dk) * f);
    }
    p.total = off;
    *out = p;
    return SS_OK;
}

}  // namespace ss
