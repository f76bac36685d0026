// Plans and workspace layout of the gated recurrence, layer norm and microscaled product entry
// points.  Host-only, HIP-free: everything here depends on the dims alone.
#pragma once

#include "ss_la_plan.h"

namespace ss {

constexpr int64_t kGrMaxStep = int64_t(1) << 25;   // elements from token to token: 16 tokens' rows
                                                   // stay within a descriptor's 2^31 bytes
constexpr int kGrFwdTile = 128;                    // tokens of a workgroup, forward
// Tiles of a group.  us with 16, 24, 32 and 48: forward 8 x 2048 x 5120 (16 tiles a row) 153, 152, 147, 147,
// 1 x 262144 x 256 160, 148, 149, 154; a training step of 4 x 4096 x 2048 with the same in both
// directions 202, 204, 210, 214.
// In the gradient, twice as many tiles make twice as many links of a row's chain, which one or two
// workgroups at a time (for 128 channels each) wait for: 1 x 262144 x 256 322 and 285 with 16 and 32, x 128 252 and 179; where there
// are more, 2 x 131072 x 256 268 and 277.
constexpr int kGrFwdGroup = 32, kGrBwdGroup = 16, kGrBwdLong = 32;

// Whether rows are walked by a wave for each 128 channels (`waves` of them in all) rather than taken by a
// workgroup each: 4 us and 0.22 a token against 10, or, where there are many, what their bytes take against
// 75 ns each.  us by walk and by workgroups, 2560 channels, bfloat16: 4 rows of 32 tokens 11.1 and 10.2, of
// 48 14 and 10; 64 rows of 48 22 and 31, of 96 37 and 34; 256 of 128 138 and 137.  (A few rows of up to 32
// tokens would gain up to a microsecond from workgroups; they walk, as the more usual many do.)  st: the widest step
// from token to token; all tokens of a row, and eight more, stay within a descriptor's 2^31 bytes.
inline bool gr_walks(int64_t T, int64_t waves, int64_t st) {
    return T <= kGrFwdTile && (T <= 32 || waves >= 16 * T) && (T + 8) * st < (int64_t(1) << 28);
}

// What links the tiles of a row: the tiles' maps and, right behind them, the groups' ends (words of
// 8 bytes), and a counter (tiles > 1).
struct GrChain {
    int64_t tiles, groups, group;
    size_t off_ticket, off_maps, off_ends;
};

// The chains' counters come first (256 bytes), then the words of the forward's, then those of the
// gradient's: one launch sets them all.  words: how many.
struct GrPlan {
    int64_t B, T, D;
    GrChain fwd, rev;
    size_t off_words;
    int64_t words;
    // backward: off_ckpt [B, rev.tiles, D] where none are given, off_part [B, rev.tiles, D]
    size_t off_ckpt, off_part, total;
};

// (with one token its stride says nothing)
inline bool gr_strides_ok(const int64_t* s, int64_t T) {
    const int64_t lim = int64_t(1) << 40;
    return s[0] >= 0 && s[0] <= lim && s[1] >= 0 && s[1] <= (T == 1 ? lim : kGrMaxStep);
}

inline void gr_chain(GrPlan* p, int64_t tokens, int64_t group, size_t ticket, GrChain* c) {
    c->tiles = (p->T + tokens - 1) / tokens;
    c->group = group;
    c->groups = (c->tiles + group - 1) / group;
    if (c->tiles <= 1) return;
    c->off_ticket = ticket;
    c->off_maps = p->off_words + size_t(p->words) * sizeof(uint64_t);
    c->off_ends = c->off_maps + size_t(p->B * c->tiles) * size_t(p->D) * sizeof(uint64_t);
    p->words += p->B * (c->tiles + c->groups) * p->D;
}

inline int make_gr_plan(const ss_gr_dims& d, bool backward, bool given_ckpt, GrPlan* out) {
    if (d.batch <= 0 || d.seqlen <= 0 || d.dim <= 0 || d.dim > (int64_t(1) << 24)) return SS_ERR_DIMS;
    if (d.in_dtype != SS_F32 && d.in_dtype != SS_BF16) return SS_ERR_DTYPE;
    if (!(d.c > 0.0f) || !(d.c - d.c == 0.0f)) return SS_ERR_DIMS;
    if (!gr_strides_ok(d.x_stride, d.seqlen) || !gr_strides_ok(d.r_stride, d.seqlen) ||
        !gr_strides_ok(d.i_stride, d.seqlen))
        return SS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 40;   // elements of any tensor
    if (!mul_ok(d.batch, d.seqlen, lim) || !mul_ok(d.batch * d.seqlen, d.dim, lim)) return SS_ERR_DIMS;
    if (d.batch > kMaxGridYZ) return SS_ERR_DIMS;
    GrPlan p{};
    p.B = d.batch; p.T = d.seqlen; p.D = d.dim;
    p.off_words = 256;
    if (!backward || !given_ckpt) gr_chain(&p, kGrFwdTile, kGrFwdGroup, 0, &p.fwd);
    const int64_t cols = (p.D + 127) / 128 * p.B;
    if (backward) gr_chain(&p, SS_GR_CKPT, cols <= 2 ? kGrBwdLong : kGrBwdGroup, 128, &p.rev);
    if (!mul_ok(cols, p.fwd.tiles + p.rev.tiles, lim) || !launch_ok(cols * p.fwd.tiles, 512) ||
        !launch_ok(cols * p.rev.tiles, 512))
        return SS_ERR_DIMS;
    size_t off = p.words ? align256(p.off_words + size_t(p.words) * sizeof(uint64_t)) : 0;
    if (backward) {
        const size_t row = size_t(p.B * p.rev.tiles) * size_t(p.D) * sizeof(float);
        p.off_ckpt = off;
        if (!given_ckpt) off = align256(off + row);
        p.off_part = off;
        off = align256(off + row);
    }
    p.total = off;
    *out = p;
    return SS_OK;
}

// The layer norm: its own split of a row over threads; the gradient keeps two rows of partial sums.
inline int make_ln_plan(const ss_ln_dims& d, bool backward, RmsPlan* out) {
    ss_rms_dims r{d.rows, d.dim, d.in_dtype, d.res_dtype, d.q8, d.eps};
    if (d.q8 == SS_Q4_MX && !backward) {
        if (d.dim % 32 != 0) return SS_ERR_DIMS;
        r.q8 = SS_Q8_NONE;
    }
    RmsPlan p;
    const int rc = make_rms_plan(r, backward, &p);
    if (rc != SS_OK) return rc;
    const int64_t pieces = (p.D + 7) / 8;
    const bool many = p.M >= 1024;
    // Whole waves of threads, a piece each; 448 have no step of their own (3584 wide with 512: 11702 rows
    // forward 69 us, as many bytes 2560 wide 70; gradient 87, 4096 wide 77).
    if (pieces <= 128) {
        p.threads = pieces <= 8 ? 8 : pieces <= 32 ? 32 : 64;
        p.pieces = pieces <= 64 ? 1 : 2;
    } else if (!backward && many && pieces <= 64 * 6) {
        p.threads = 64;
        p.pieces = int((pieces + 63) / 64);
    } else if (pieces <= 512) {
        p.threads = pieces <= 256 ? 256 : pieces <= 320 ? 320 : pieces <= 384 ? 384 : 512;
        p.pieces = 1;
    } else {
        p.threads = pieces <= 1024 ? 512 : 1024;
        p.pieces = pieces <= 2048 ? 2 : 4;
    }
    const int64_t wg_rows = p.threads >= 256 ? 1 : 256 / p.threads;
    const int64_t need = (p.M + wg_rows - 1) / wg_rows;
    // A gradient's workgroups each write two rows of sums; as many as run at once.  us, bfloat16 / float32
    // (rows times width 2^25 / 2^24), of 768, 1024, 1280, 1536 and 2048 of them:
    //   512 wide 67 58 53 51 64 / 46 44 45 47 51    1472  92 76 66 62 81 / 57 51 51 50 59
    //   1471    116 103 91 121 109 / 65 60 58 75 68  1024  55 51 67 62 57 / 43 46 50 49 51
    //   2560     66 57 77 70 76 / 49 48 61 58 61     3000  63 77 74 82 78 / 65 59 62 61 64
    // 256 and 512 of them: 8192 wide 68 and 73 / 94 and 99, 16384 96 and 109 / 182 and 196.
    int64_t most = p.threads >= 512 ? 512 : 2048;
    if (backward) {
        if (p.pieces * p.threads >= 768) most = 256;
        else if (p.pieces == 1 && p.threads <= 256) most = p.D % 8 == 0 ? 1536 : 1280;
        else if (p.threads == 384 && p.D % 8 == 0 && d.in_dtype == SS_BF16) most = 768;
        else if (p.threads < 512) most = 1024;
    }
    p.grid = int(need < most ? need : most);
    p.total = backward ? align256(size_t(p.grid) * size_t(2 * p.D) * sizeof(float)) : 0;
    *out = p;
    return SS_OK;
}

// Products of microscaled weights.  Either 16 rows of weights by 16·high of x go to a workgroup of
// `waves` waves, which share the columns (rows), or 128 by 64·high (tiles).
struct Mx4Plan {
    bool tiled;
    int high, waves;
};

// us, x in 4 bits / in 8 (which takes two matrix instructions where 4 bits take one):
// Tiles take a time of their own for a walk over K however few they are, rows a time for every 64 of
// them and every 16 of the weights.  N x K, rows of x: with rows and with tiles.
//   2560 x 2560,  128: 7.0 and 8.0 / 8.4 and 14.1,      192: 8.2 and 8.1 / 10.3 and 14.3
//   10240 x 2560, 64:  10.3 and 9.3 / 14.4 and 15.0,    128: 14.9 and 9.0 / 20.6 and 15.4
//   2560 x 10240, 128: 18.2 and 22.5 / 24.2 and 44.0,   192: 24.2 and 24.3 / 30.0 and 44.1
//   5120 x 5120,  64:  11.1 and 13.8 / 14.9 and 24.7,   128: 17.1 and 13.2 / 22.8 and 24.7
//   in 8 bits:    2560 x 2560, 256: 13.7 and 14.5, 384: 17.0 and 14.9; 5120 x 5120, 192: 28.1 and 25.0
// Tiles of 64 and of 128 rows of x, up to 256 of them (a compute unit one), in 8 bits up to 768, and more:
//   2560 x 2560,  768 rows of x: 9.3 and 10.1 / 15.8 and 22.6, 1024: 12.1 and 10.4 / 20.9 and 23.1
//   10240 x 2560, 192: 9.4 and 10.7 / 16.0 and 22.3,           256: 13.0 and 10.8 / 21.1 and 22.9
//   in 8 bits:    2560 x 2560, 2048: 30.5 and 35.2, 2500: 38.7 and 34.9; 10240 x 2560, 512: 28.5 and 32.5,
//                 768: 38.1 and 34.8, 16384: 669 and 622
// and of 128 and 256, in 4 bits: 10240 x 2560, 384: 11.9 and 15.4, 512: 16.9 and 15.9, 4096: 80 and 67
// But none taller than the rows there are, nor, in 8 bits, where a tile of 128 rows, by 5 % the cheaper, would be half
// empty; weights of 33000 and 151936 by 2560, tiles of 64, 128 and 256 (8 bits: 64 and 128):
//   64 rows: 18.5, 19.4, 24.7 and 62, 59, 69 / 23.3, 32.9 and 66, 88      128: 22.3, 21.8, 27.0 and 87, 66, 75 /
//   30.9, 35.6 and 103, 99      192: 25.7, 26.9, 28.1 and 108, 94, 81 / 39.9, 51.3 and 134, 172
//   513: 55, 46, 48 and 264, 193, 181 / 88, 95 and 371, 386
// Rows: as high as leaves two workgroups to a compute unit, else lower; 64 rows of x, high 4, 2, 1:
//   2560 x 5120:  7.0, 6.8, 7.0 / 10.2, 10.2, 10.0     640 x 1024: 3.5, 3.0, 2.7 / 5.0, 4.2, 3.8
// 8 and 16 waves where each compute unit has one workgroup: 2560 x 5120, 1 row of x, 4.4 and 3.9 / 5.2
// and 5.0; 2560 x 10240, 7.0 and 5.4 / 10.3 and 7.7.
// (A tile's rows of y stay within a descriptor's 2^31 bytes.)
inline Mx4Plan mx4_plan(int64_t rows, int64_t n, int64_t k, bool fp8) {
    if (rows > 32 && n * ((rows + 63) / 64) >= (fp8 ? 12800 : 7680) && n < (int64_t(1) << 20)) {
        auto tiles = [&](int64_t high) { return (rows + 64 * high - 1) / (64 * high) * ((n + 127) / 128); };
        if (fp8) {
            const bool tall = tiles(1) > 768 && 19 * ((rows + 127) / 128) < 10 * ((rows + 63) / 64);
            return {true, tall ? 2 : 1, 4};
        }
        const int high = tiles(1) <= 256 ? 1 : tiles(2) <= 256 ? 2 : 4;
        return {true, rows <= 64 ? 1 : rows <= 128 && high > 2 ? 2 : high, 4};
    }
    auto groups = [&](int64_t high) { return (rows + 16 * high - 1) / (16 * high) * ((n + 15) / 16); };
    if (rows > 32 && groups(4) >= 512) return {false, 4, 8};
    const int high = rows > 16 && groups(2) >= 512 ? 2 : 1;
    return {false, high, groups(high) <= 256 && k >= 2048 ? 16 : 8};
}

inline int check_mx4(const ss_mx4_dims& d, bool product) {
    if (d.rows <= 0 || d.k <= 0 || d.k % 32 != 0 || (product && d.n <= 0)) return SS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 38;
    if (!mul_ok(d.rows, d.k, lim)) return SS_ERR_DIMS;
    if (!product) return d.in_dtype == SS_F32 || d.in_dtype == SS_BF16 ? SS_OK : SS_ERR_DTYPE;
    if (!mul_ok(d.n, d.k, lim) || !mul_ok(d.rows, d.n, lim)) return SS_ERR_DIMS;
    if (d.k >= (int64_t(1) << 23)) return SS_ERR_DIMS;   // 256 rows stay within a descriptor
    if (d.x_q8 != SS_Q4_MX && d.x_q8 != SS_Q8_FP8) return SS_ERR_DTYPE;
    if (d.y_dtype != SS_F32 && d.y_dtype != SS_BF16) return SS_ERR_DTYPE;
    const Mx4Plan p = mx4_plan(d.rows, d.n, d.k, d.x_q8 == SS_Q8_FP8);
    const int64_t m = (p.tiled ? 64 : 16) * p.high, high = (d.rows + m - 1) / m;
    if (p.tiled ? !launch_ok((d.n + 127) / 128 * high + 7, 256)
                : !launch_ok((d.n + 15) / 16 * high, 64 * p.waves))
        return SS_ERR_DIMS;
    return SS_OK;
}

}  // namespace ss
