// Internal launch interface between the C-ABI layer (ss_api.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ss.h"

namespace ss {

// Steps between the forward's state checkpoints (the backward's tile length).
constexpr int kCkptSteps = 16;

// Where channel (b, d)'s Δraw values lie: element t at dt_raw[b·sb + d·sd + t·ts].
//   [B, D, L]: (D·L, L, 1);  [B, L, D]: (L·D, 1, D);  one value per token [B, L]: (L, 0, 1).
struct DtRows {
    int64_t sb, sd, ts;
};

// Calls f(std::integral_constant<bool, v>): a runtime flag as a template argument.
template <typename F>
inline hipError_t with_bool(bool v, F&& f) {
    return v ? f(std::true_type{}) : f(std::false_type{});
}

struct ScanLaunch {
    const void* x;
    const void* dt_raw;
    const void* z;          // nullable (no gate); ignored in AGG mode
    const float* dt_bias;
    const float* A;
    const float* Dskip;
    const float* BC;        // [B, L, 2N] float32 staging copy of B and C (one-lane kernel)
    const void* Bm;         // [B, N, L] inputs (group kernel)
    const void* Cm;
    const float* h_init;    // nullable; [B, D, K, N]
    float* y;               // OUT mode
    float* h_last;          // OUT: h_final (nullable); AGG: h_end [B, D, K, N]
    float* h_ckpt;          // OUT: nullable; [B, D, ceil(L / kCkptSteps), N]: state entering
                            // every kCkptSteps-th step
    float* dsum;            // AGG: Σδ per chunk [B, D, K]
    int64_t B, L, D, chunk;
    int K;
    int vec;                // 1: L % 8 == 0, 8-step vector loads
    int agg;                // 1: AGG mode
    int64_t d4;             // mixed layout: channels [0, d4) on four lanes, [d4, D) on eight
    int nb4;                //               four-lane workgroups per batch row (d4 / 64)
    int zoh;                // 1: exact zero-order-hold B̄
    int tok;                // 1: token-major x, z, y [B, L, D] and B, C [B, L, N]
    DtRows dtr;             // Δraw rows
};

// Affine-pair carry across chunks (one workgroup per channel).  Chunk c's pair is
// (exp(A Σδ_c), h_end_c); h_start_c is the state entering chunk c in scan order
// (reverse = 1 scans chunks from last to first, for the adjoint), h_out the state
// after the last one.  h_in, h_out nullable.
struct CarryLaunch {
    const float* h_end;     // [B, D, K, N]
    const float* dsum;      // [B, D, K]
    const float* A;         // [D, N]
    const float* h_in;      // [B, D, N]
    float* h_start;         // [B, D, K, N]
    float* h_out;           // [B, D, N]
    int64_t B, D;
    int K;
    int reverse;
    // optional second set, carried in the same launch when dual = 1
    int dual;
    const float* h_end2;
    const float* h_in2;
    float* h_start2;
    float* h_out2;
    int reverse2;
};

// Backward launches (four lanes per channel).  stage 0: chunk aggregates (h_end, rev_end, dsum);
// stage 1: final pass (h_end holds chunk start states on entry and dA partials on exit,
// rev_end holds the adjoints entering each chunk from the right).
struct BwdLaunch {
    const void* x;
    const void* dt_raw;
    const void* z;
    const float* dy;
    const float* dt_bias;
    const float* A;
    const float* Dskip;
    const void* Bm;    // [B, N, L] inputs
    const void* Cm;
    const float* h_ckpt;  // nullable: the forward's checkpoints; then h_end holds only dA
    float* h_end;      // [B, D, K, N]
    float* rev_end;    // [B, D, K, N]
    float* dsum;       // [B, D, K]
    float* dbc_part;   // [B, ceil(D/64), L, 2N]
    float* ddt_part;   // [B, D, K, 2]
    float* dx;
    float* ddt_raw;
    float* dz;
    float* dA;
    float* dB;
    float* dC;
    float* dD;
    float* ddt_bias;
    int64_t B, L, D, N, chunk;
    int K;
    int vec;
    int stage;
    int tok;           // 1: token-major x, z, dy, dx, dz [B, L, D] and B, C, dB, dC [B, L, N]
    DtRows dtr;        // Δraw rows
    DtRows gdr;        // rows the per-channel Δraw gradient is written to (ddt_raw)
    int zoh;           // 1: gradients of the exact zero-order hold
    float* ddt_shared; // nullable: Δraw shared by the channels; its gradient [B, L]
    float* ddt_blk;    // with ddt_shared: per-64-channel-block sums [B, ceil(D/64), L]
};

// Single-token step: x, dt_raw, z [B, D]; Bm, Cm [B, N]; h_in, h_out [B, D, N] (may be equal).
struct StepLaunch {
    const void* x;
    const void* dt_raw;
    const void* z;          // nullable
    const float* dt_bias;
    const float* A;
    const void* Bm;
    const void* Cm;
    const float* Dskip;
    const float* h_in;
    float* h_out;
    float* y;
    int64_t B, D;
    int N;
    int zoh;                // 1: exact zero-order-hold B̄
    int dt_shared;          // 1: dt_raw [B], one value per token
};

hipError_t launch_bc_stage(int bf16, int N, const void* Bm, const void* Cm, float* BC, int64_t B,
                           int64_t L, int tok, hipStream_t s);
hipError_t launch_scan(int bf16, int N, const ScanLaunch& p, hipStream_t s);
// group-split layout: G = 4 (N in {4, 8, 16, 32}) or G = 8 (N in {8, 16, 32}); L % 8 == 0
// for channel-major inputs
hipError_t launch_scang(int bf16, int N, int G, const ScanLaunch& p, hipStream_t s);
// single pass, N in {8, 16, 32}: four lanes for channels [0, d4), eight for [d4, D)
hipError_t launch_scang_mixed(int bf16, int N, const ScanLaunch& p, hipStream_t s);
hipError_t launch_carry(int N, const CarryLaunch& p, hipStream_t s);
hipError_t launch_step(int bf16, const StepLaunch& p, hipStream_t s);
hipError_t launch_bwd(int bf16, const BwdLaunch& p, hipStream_t s);
hipError_t launch_bwd_reduce(const BwdLaunch& p, hipStream_t s);

// Block projections (ss_block.hip).  C0 | C1 = A [M, K] · W [Nc, K]ᵀ (bf16 in, fp32 out),
// split at column nsplit; K % 8 == 0, 16-byte aligned rows.
hipError_t launch_gemm_bf16_nt(const void* A, const void* W, float* C0, float* C1, int64_t M,
                               int64_t Nc, int64_t K, int64_t nsplit, int64_t ld0, int64_t ld1,
                               hipStream_t s);
// [Δ | B | C] = x [M, D] · Wx [1 + 2N, D]ᵀ (fp32) through split-K partials part
// [S, M, 1 + 2N] (S = xproj_splits, ss_plan.h); D % 4 == 0.
hipError_t launch_xproj(const float* x, const float* Wx, float* part, float* dt, float* Bm,
                        float* Cm, int64_t M, int64_t D, int N, hipStream_t s);

// ---- linear attention with a decay for each head (ss_la*.hip) -----------------------------------

// Rows of one operand: element (b, t, head, i) at p + b·sb + t·st + (head / rep)·sh + i elements.
struct LaOperand {
    const void* p;
    int64_t sb, st, sh;
    int64_t rep;       // value heads that share a row
    int dim;           // width
    int vec;           // every row starts on 16 bytes and holds whole 16-byte pieces, a token's
                       // row ends before the next one's begins or all chunks are full, and a
                       // chunk's rows lie within 2^30 bytes
};

// One sweep (ss_la_sweep.h).
struct LaSweep {
    LaOperand a, b, c, e;      // e: with dots
    const float* g;            // nullable; log decays [B, T, H] or [H]
    int decay_token;
    const int32_t* lengths;    // nullable [B]
    void* out;                 // [B, T, H, dC]; the operands' type, or float32 with out_f32
    int out_f32;
    const float* s_in;         // nullable; element (i, j) of row-head bh, segment s at
    int64_t s_in_sz, s_in_i, s_in_j;   // (bh·in_seg + s)·s_in_sz + i·s_in_i + j·s_in_j
    int64_t in_seg;
    float* s_out;              // nullable [B, H, dA, dC] (s_out_t, with dots: [B, H, dC, dA]);
    int s_out_t;               // state_only: [B, H, nseg, dA, dC]
    double* dots;              // nullable [tiles, B, H, T]
    float* seg_decay;          // state_only: [B, H, nseg]
    int64_t B, T, H;
    int tiles, nseg, grid_seg, seg0;   // the grid covers segments [seg0, seg0 + grid_seg)
    int64_t seg_chunks;
    int reverse, state_only;
    float alpha, in_scale, up_scale;   // of a·b; of the entering state in out; of c in the state
    int pad_a, waves;
};
// n = 1 or 2 sweeps in one launch; two differ in operands, results and direction only, and
// neither reads what the other writes.
struct LaSweeps {
    LaSweep p[2];
    int n;
};
// all operands of aligned rows; any rows
hipError_t launch_la_sweep_bf16(const LaSweeps& p, hipStream_t s);
hipError_t launch_la_sweep_bf16_any(const LaSweeps& p, hipStream_t s);
hipError_t launch_la_sweep_f32(const LaSweeps& p, hipStream_t s);
hipError_t launch_la_sweep_f32_any(const LaSweeps& p, hipStream_t s);

// State entering each segment, in place over what each segment adds: state [BH, nseg, sz].
// first: nullable, element i·dC + j of row-head bh at bh·sz + i·f_i + j·f_j.
struct LaCarry {
    float* state;
    const float* decay;        // [BH, nseg]
    const float* first;
    int64_t BH, sz, dC, f_i, f_j;
    int nseg, reverse;
};
struct LaCarries {             // n = 1 or 2 of the same sizes
    LaCarry p[2];
    int n;
};
hipError_t launch_la_carry(const LaCarries& p, hipStream_t s);

// dg from the row and column sums and the states at the segments' borders: token [B, T, H]
// (dg), or one value a head [H] through head_part [B, H, nseg].
struct LaDecayGrad {
    const double *row, *col;   // [tiles, B, H, T]
    int tiles;
    const float *fwd_state, *rev_state;   // [B, H, nseg, dv, dk]: the states that enter each
                                          // segment from the left, from the right
    const float *s0, *ds0, *ds, *s_final; // nullable [B, H, dk, dv]
    double* border;            // [B, H, nseg + 1]
    int border0, borders;      // launch_la_borders forms borders border0 .. border0 + borders - 1
    const int32_t* lengths;
    float* dg;
    double* head_part;
    int64_t B, T, H, dk, dv;
    int nseg;
    int64_t seg_tokens;
    int decay_token;
};
hipError_t launch_la_borders(const LaDecayGrad& p, hipStream_t s);
hipError_t launch_la_decay_grad(const LaDecayGrad& p, hipStream_t s);   // after all the borders

// Gradients of the shared key heads, dq and dk in turn: sums over the value heads of each,
// part[x] [tokens, key heads, rep, d] float32 into out[x], n = tokens·key heads·d elements.
struct LaGroupSum {
    const float* part[2];
    void* out[2];
    int64_t n, rep, d;
};
hipError_t launch_la_group_sum(int bf16, const LaGroupSum& p, hipStream_t s);

// One token: state [B, H, dk, dv] float32, s_out may be s_in.
struct LaStep {
    LaOperand q, k, v;         // st unused
    const float* g;            // nullable; [B, H] or [H]
    int decay_token;
    const float* s_in;
    float* s_out;
    void* o;                   // [B, H, dv], the operands' type
    int64_t B, H, dk, dv;
    int columns;               // of a workgroup: 128, 32
    float scale;
};
hipError_t launch_la_step(int bf16, const LaStep& p, hipStream_t s);

// ---- norm (ss_norm.hip) --------------------------------------------------------------------------

// Forward: x [M, D] (in_dtype), res (nullable) and r [M, D] (res_dtype), y in in_dtype or 8-bit
// codes with y_scale [M].  Backward: x is dy, res is r, r is dx; dr nullable; part [grid, D].
struct RmsLaunch {
    const void *x, *res, *dr;
    const float* w;
    void *r, *y;
    float *y_scale, *part;
    int64_t M, D;
    float eps, inv_d;
    int in_dtype, res_dtype, q8;
    int threads, pieces, grid;   // threads of a row, eight-element pieces of each, workgroups
};
hipError_t launch_rms_fwd(const RmsLaunch& p, hipStream_t s);
hipError_t launch_rms_bwd(const RmsLaunch& p, float* dw, hipStream_t s);

// Layer norm: as above, with the bias b (nullable); backward: part [grid, 2 D], the sums behind dw
// and db.  q8 may be SS_Q4_MX: y holds 4-bit codes and y_scale the blocks' exponents, in bytes.
struct LnLaunch : RmsLaunch {
    const float* b;
};
hipError_t launch_ln_fwd(const LnLaunch& p, hipStream_t s);
hipError_t launch_ln_bwd(const LnLaunch& p, float* dw, float* db, hipStream_t s);

// ---- products with 4-bit weights (ss_q4.hip) -----------------------------------------------------

struct Q4Launch {
    const void* x;               // [M, K]
    const float* x_scale;        // nullable [M]
    const uint8_t* wq;           // [N, K / 2]
    const uint16_t* scales;      // bf16 [N, groups]
    const uint8_t* zeros;        // nullable [N, groups]
    void* y;                     // [M, N]
    int64_t M, N, K, groups;
    int mb, tiles;               // of a workgroup: rows of x, 16-row tiles of weights
    int group, in_dtype, x_q8, y_dtype;
};
hipError_t launch_q4(const Q4Launch& p, hipStream_t s);

// ---- gated recurrence (ss_gr.hip) ----------------------------------------------------------------

// Rows of a [B, T, D] operand with a contiguous last axis.
struct GrRows {
    const void* p;
    int64_t sb, st;            // elements from batch row to batch row, token to token
};

struct GrLaunch {
    GrRows x, r, i;
    const float *lam, *h0;     // [D]; nullable [B, D]
    const int32_t* lengths;    // nullable [B]
    const uint8_t* reset;      // nullable [B, T]
    int64_t B, T, D;
    float c;
    int in_dtype, vec;         // vec: two neighbouring channels load as one (2: their number is odd)
    int tiles, group;          // of a row: kGrFwdTile tokens (forward, ss_gr_plan.h), SS_GR_CKPT (backward)
    // where there are more than one: the tiles' maps [B, tiles, D] and, right behind them, the ends of
    // groups of `group` of them [B, ceil(tiles / group), D]; the workgroups' counter
    uint64_t *maps, *ends, *ticket;
    // forward
    void* y;                   // nullable
    float *h_final, *h_ckpt;   // nullable
    // backward (h_ckpt is read)
    const void* dy;
    const float* dh_final;     // nullable
    void *dx, *dr, *di;
    float *dh0, *part, *dlam;  // nullable; [parts, D]; [D]
};
// Before them: `words` words from maps on say that nothing is there yet, and the two counters (at
// `tickets` and 128 bytes behind) begin at 0.
hipError_t launch_gr_chains(uint64_t* tickets, uint64_t* maps, int64_t words, hipStream_t s);
hipError_t launch_gr_fwd(const GrLaunch& p, hipStream_t s);
hipError_t launch_gr_bwd(const GrLaunch& p, hipStream_t s);

struct GrStep {
    GrRows x, r, i;            // st unused
    const float *lam, *h_in;
    float* h_out;
    void* y;
    int64_t B, D;
    float c;
    int in_dtype, vec;
};
hipError_t launch_gr_step(const GrStep& p, hipStream_t s);

// ---- microscaled 4-bit values (ss_mx4.hip) -------------------------------------------------------

struct Mx4Quant {
    const void* x;               // [M, K]
    uint8_t *codes, *exps;       // [M, K / 2], [M, K / 32]
    int64_t blocks;              // M·K / 32
    int in_dtype;
};
hipError_t launch_mx4_quant(const Mx4Quant& p, hipStream_t s);

struct Mx4Launch {
    const uint8_t* x;            // [M, K / 2] codes, or [M, K] e4m3
    const void* x_scale;         // [M, K / 32] exponents, or [M] float32
    const uint8_t *wq, *w_exps;  // [N, K / 2], [N, K / 32]
    void* y;                     // [M, N]
    int64_t M, N, K;
    int fp8, y_dtype;
};
hipError_t launch_mx4_mm(const Mx4Launch& p, hipStream_t s);

// Records a failed HIP call for ss_last_hip_error; returns SS_ERR_HIP.
int hip_fail(hipError_t e);

}  // namespace ss
