// Chunked linear attention with a decay for each head, for gfx950: the sweep that the forward
// and all three gradients are instances of.
//
// A sweep takes rows a_t, b_t (width dA) and c_t (width dC) of every (batch row, head) and
// gives, with G the running sum of the log decays,
//   forward direction   out_t = α·(Σ_{s<=t} e^{G_t-G_s} (a_t·b_s) c_s + e^{G_t} Sᵀa_t)
//   reverse direction   out_t = α·Σ_{s>=t} e^{G_s-G_t} (a_t·b_s) c_s + e^{G_end-G_t} Sᵀa_t
// where S is the dA x dC state that enters from the side the sweep starts at.  With
// S_t = e^{g_t} S_{t-1} + k_t v_tᵀ and o_t = α S_tᵀ q_t,
//   o  is the forward sweep of (q, k, v) from S_0,
//   dq is the forward sweep of (do, v, k) from S_0ᵀ,
//   dk is the reverse sweep of (v, do, q) from dS_Tᵀ,
//   dv is the reverse sweep of (k, q, do) from dS_T, and its last state is dS_0.
// The log decays' gradient needs only the products A_ts = α e^{G_t-G_s} (q_t·k_s)(do_t·v_s):
//   dg_t = Σ_{u>=t} (row_u - col_u) + <dS_T, S_T>, row_u = Σ_{s<u} A_us + (S_0's part),
// and likewise col_u = Σ_{t>u} A_tu + (dS_T's part): row_u is e_u·out_u of the dq sweep with
// e = q and the diagonal left out, col_u that of the dk sweep with e = k (kDot).  (The running
// sum starts anew at every segment, ss_la.hip.)
//
// A workgroup of four or eight waves takes one head's rows chunk by chunk (64 tokens of bf16,
// 32 of float32) with the state in registers: a wave holds all dA rows of 16 columns, in the
// accumulator layout of v_mfma_f32_16x16x32_bf16 (lane l: column l % 16, rows 4·(l/16) + r).
// Inside a chunk:
//   P  = (a bᵀ) ⊙ decay: 16 x 16 tiles dealt to the waves, only those the mask leaves, through LDS
//   out = Sᵀaᵀ (state as an operand straight from the accumulators: the rows of S are dealt to
//         accumulators so that a lane's eight values are the eight consecutive k it must feed)
//         scaled by each token's entering decay, plus cᵀPᵀ
//   S  = e^{G_C} S + bᵀ(w ⊙ c)   (transposed operands: ds_read_b64_tr_b16)
// The next chunk's rows are loaded into registers meanwhile.
//
// Numerics.  Log decays are summed as 64-bit integers with 44 fraction bits, in base 2, so a
// weight is ldexp(2^fraction, integer) of an exact difference, however far the sum has come, and a
// token that decays by e^{-inf} cuts the sequence exactly.  Over n tokens a sum is at most n·2^-45
// off.  The state itself is float32: it takes one rounding of its decay and one of its product a
// chunk (and a segment), as any recurrence in float32 does.  P, and S where it
// feeds out, go to the matrix cores as two bf16 terms, 16 bits: with one, out was 2.0e-3 off
// (root mean square against 64 bits) where its own rounding to bf16 is 1.7e-3.
// The state's own sums are float32: c's weight w is not a bf16 value, so w·c is fed as three
// bf16 terms (24 bits, all of it).  The products behind dg (P, e·c, e·(Sᵀa)) are kept in float32 the same
// way, since dg is float32.  With float32 rows the matrix cores' float32 form runs on the same
// layouts and nothing is rounded.
//
// What bounds it.  By its traffic a sweep is bound by memory, but with the state in registers a
// CU holds eight or sixteen waves, and their chunk is a chain of barriers and dependent products:
// at 128 x 128 vector ALUs are busy for 43% of the time, LDS for 33%, the matrix cores for 25%, and
// 40% of the waves' time is waiting (64 x 128: 59, 43, 29 and 37%; dq and dk: 39, 34, 25 and 43%).
// Measured, bf16, token decays: B = 4, T = 2048, H = 16, 128 x 128 the states of 4 segments
// (kState) 23 us, the carry 7, the sweep 53 (2.9 TB/s); B = 1, T = 32768, H = 40 on 8, 64 x 128 130, 9
// and 290 us; gradient at B = 4, T = 4096, H = 16, 128 x 128 states of both directions 61, carries
// 12, dq and dk 233, dv 97.  Float32, B = 4, T = 2048, H = 16, 64 x 128: 113 us for all three, the
// gradient 312.  A sequence that is
// swept once instead, without segments, leaves most CUs idle where B·H is small; two chunks of rows
// in flight instead of one cost more registers than they hid (59 us became 68), and out by way
// of LDS in whole rows another barrier (235 us became 279).  (Both at one term of S.)
#pragma once

#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {
namespace la {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// One k step of the products: 16 rows x 32 k of either operand, lane l holding row l % 16 and
// k = 8·(l / 16) .. + 7.
template <typename T>
struct Mma;

template <>
struct Mma<bf16_t> {
    using Frag = bf16x8;
    using Elem = __bf16;
    static constexpr int kChunk = 64;  // tokens of a chunk
    static constexpr int kVec = 8;     // elements of a 16-byte load
    static constexpr int kTerms = 3;   // bf16 terms of a float32 operand
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // eight consecutive elements of a row in LDS
    static __device__ __forceinline__ Frag row(const Elem* p) {
        return *reinterpret_cast<const Frag*>(p);
    }
    // Transposed: one column of eight tokens, 4·(l / 16) .. + 3 and the same 16 tokens on (the
    // order of tokens along k is free; in this one the eight rows that 32 lanes read together
    // lie next to each other, in different banks).  In a group of 16 lanes, lane λ of
    // ds_read_b64_tr_b16 names four consecutive elements (row λ / 4, piece λ % 4 of 16 columns)
    // and receives column λ of the four rows.  p: row 0 of the 32 tokens; piece_col: the first
    // column of piece λ % 4.
    static __device__ __forceinline__ Frag col(const Elem* p, int ld, int lane, int piece_col) {
        const Elem* q = p + (4 * (lane >> 4) + ((lane >> 2) & 3)) * ld + piece_col;
        typedef __attribute__((address_space(3))) s16x4* Lds;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(q));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(q + 16 * ld));
        union { s16x4 h[2]; Frag f; } u;
        u.h[0] = lo;
        u.h[1] = hi;
        return u.f;
    }
    static __device__ __forceinline__ float get(Frag f, int e) { return float(f[e]); }
    static __device__ __forceinline__ Elem from(float v) { return Elem(v); }
    // v as two bf16 terms, to 2^-16 of it; an infinity is its first term alone
    static __device__ __forceinline__ void two(const float (&v)[8], Frag (&f)[2]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[0][e] = Elem(v[e]);
            const float left = v[e] - float(f[0][e]);
            f[1][e] = Elem(__builtin_isfinite(left) ? left : 0.0f);
        }
    }
    // v as kTerms bf16 terms that sum to it exactly: each takes the upper eight significant bits
    // of what is left.  keep 0 (else all ones) where v may hold an infinity, which is then its
    // first term alone.
    static __device__ __forceinline__ void split(const float (&v)[8], unsigned keep, Frag (&f)[kTerms]) {
        const unsigned upper = 0x07060302u, rest = keep ? upper : 0x0c0c0c0cu;
        union { Frag f; unsigned w[4]; } t[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            unsigned x[2][3];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float a = v[2 * i + y];
                x[y][0] = __float_as_uint(a);
                const float b = a - __uint_as_float(x[y][0] & 0xffff0000u);
                x[y][1] = __float_as_uint(b);
                x[y][2] = __float_as_uint(b - __uint_as_float(x[y][1] & 0xffff0000u));
            }
            t[0].w[i] = __builtin_amdgcn_perm(x[1][0], x[0][0], upper);
            t[1].w[i] = __builtin_amdgcn_perm(x[1][1], x[0][1], rest);
            t[2].w[i] = __builtin_amdgcn_perm(x[1][2], x[0][2], rest);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) f[q] = t[q].f;
    }
};

template <>
struct Mma<float> {
    using Frag = f32x8;
    using Elem = float;
    static constexpr int kChunk = 32;
    static constexpr int kVec = 4;
    static constexpr int kTerms = 1;
    // eight v_mfma_f32_16x16x4_f32, one for each of a lane's k values: both operands hold the
    // same k in the same lane and place, which is all a product needs
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag row(const Elem* p) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(p);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(p + 4);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // piece_col as above: lane λ's own column is that of piece λ / 4, element λ % 4, which the
    // caller's formula gives for the lane whose λ % 4 is that piece
    static __device__ __forceinline__ Frag col_at(const Elem* p, int ld, int lane, int column) {
        const Elem* q = p + 4 * (lane >> 4) * ld + column;
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = q[(e < 4 ? e : 12 + e) * ld];
        return f;
    }
    static __device__ __forceinline__ float get(Frag f, int e) { return f[e]; }
    static __device__ __forceinline__ Elem from(float v) { return v; }
    static __device__ __forceinline__ void two(const float (&v)[8], Frag (&f)[1]) { split(v, ~0u, f); }
    static __device__ __forceinline__ void split(const float (&v)[8], unsigned, Frag (&f)[kTerms]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[0][e] = v[e];
    }
};

// Transposed operand of 16 columns: column of MFMA row ρ is base + step·(ρ / 4) + ρ % 4.
template <typename T>
__device__ __forceinline__ typename Mma<T>::Frag col_frag(const typename Mma<T>::Elem* p, int ld,
                                                          int lane, int base, int step) {
    if constexpr (sizeof(T) == 2) {
        return Mma<T>::col(p, ld, lane, base + step * (lane & 3));
    } else {
        const int rho = lane & 15;
        return Mma<T>::col_at(p, ld, lane, base + step * (rho >> 2) + (rho & 3));
    }
}

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// Rows of one operand of one (batch row, head), and this thread's place in them: the same
// columns in every one of its 16-byte pieces.
template <typename T>
struct Rows {
    const T* p;
    int64_t st;       // elements from token to token
    int dim;
    int tok, col;     // of the thread's first piece
    unsigned at;      // its byte offset from a chunk's first row; beyond any row where col >= dim
};

constexpr unsigned kNowhere = 0x80000000u;
constexpr int kRsrcFlags = 0x00020000;   // raw buffer, 32-bit elements

template <typename T>
__device__ __forceinline__ Rows<T> rows_of(const LaOperand& o, int64_t b, int64_t h, int tok,
                                           int col) {
    Rows<T> r{static_cast<const T*>(o.p) + b * o.sb + (h / o.rep) * o.sh, o.st, o.dim, tok, col,
              kNowhere};
    if (col < o.dim) r.at = unsigned((tok * int(o.st) + col) * int(sizeof(T)));
    return r;
}

// A 16-byte load that needs only the elements' alignment.
template <typename T>
__device__ __forceinline__ u32x4 load_unaligned(const T* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// N pieces of a chunk (nv of its tokens exist), STEP tokens apart; zeros outside the tokens and
// the width.  Aligned rows (kVec) go through a buffer descriptor that ends with the chunk's last
// row, so the bounds cost nothing; tokens behind it are outside because a row is no longer than the
// stride (or there are none).  For others a piece that would pass the row's end starts
// earlier, at the row's last 16 bytes, and is shifted into place; rows shorter than a piece are
// put together element by element.
template <typename T, bool kVec, int N, int STEP>
__device__ __forceinline__ void load_pieces(const Rows<T>& r, int64_t t0, int nv, u32x4 (&v)[N]) {
    constexpr int V = Mma<T>::kVec, kBits = 8 * int(sizeof(T));
    const T* base = r.p + t0 * r.st;
    if constexpr (kVec) {
        const int bytes = nv > 0 ? (int(r.st) * (nv - 1) + r.dim) * int(sizeof(T)) : 0;
        const __amdgpu_buffer_rsrc_t d =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0, bytes, kRsrcFlags);
#pragma unroll
        for (int x = 0; x < N; ++x)
            v[x] = __builtin_amdgcn_raw_buffer_load_b128(d, int(r.at), x * STEP * int(r.st) * int(sizeof(T)), 0);
    } else {
        const bool some = r.col < r.dim;
        const int back = r.col + V > r.dim ? r.col + V - r.dim : 0;   // elements it starts early
#pragma unroll
        for (int x = 0; x < N; ++x) {
            v[x] = u32x4{0, 0, 0, 0};
            const int t = r.tok + x * STEP;
            if (!some || t >= nv) continue;
            const T* q = base + int64_t(t) * r.st + r.col;
            uint64_t lo = 0, hi = 0;
            if (r.dim >= V) {
                union { u32x4 v; uint64_t w[2]; } u;
                u.v = load_unaligned(q - back);
                const int bits = back * kBits;
                lo = bits >= 64 ? u.w[1] >> (bits - 64)
                   : bits > 0 ? (u.w[0] >> bits) | (u.w[1] << (64 - bits)) : u.w[0];
                hi = bits >= 64 ? 0 : u.w[1] >> bits;
            } else {
                for (int i = r.dim - 1; i >= 0; --i) {
                    uint64_t e;
                    if constexpr (sizeof(T) == 2) e = reinterpret_cast<const uint16_t*>(q)[i];
                    else e = reinterpret_cast<const uint32_t*>(q)[i];
                    hi = (hi << kBits) | (lo >> (64 - kBits));
                    lo = (lo << kBits) | e;
                }
            }
            v[x] = u32x4{unsigned(lo), unsigned(lo >> 32), unsigned(hi), unsigned(hi >> 32)};
        }
    }
}

// The log decays of a chunk in base 2 and the weights made of them.
template <int C>
struct Decay {
    float frac[C];   // G_t = whole + frac
    int whole[C];
    float in[C];     // weight of the entering state in token t's output
    float up[C];     // weight of token t in the state that leaves the chunk
    float all;       // decay of the state over the chunk
};

// 2^x for x given as whole + frac
__device__ __forceinline__ float exp2_parts(float frac, int whole) {
    return __builtin_amdgcn_ldexpf(exp2_hw(frac), whole);
}

// A log decay (natural) in base 2 with 44 fraction bits, rounded to the nearest, and bounded so that
// sums of 64 and their differences fit 64 bits: 2^±1024 is 0 or inf in float32 either way.  (NaN is
// kept apart, by its lane.)  With 32 bits a segment of 2^18 tokens could be off by 4e-5.
constexpr int kFracBits = 44;
__device__ __forceinline__ int64_t decay_fixed(float g) {
    double x = double(g) * 1.4426950408889634074;
    x = fmin(fmax(x, -1024.0), 1024.0);
    return int64_t(__builtin_rint(x * double(int64_t(1) << kFracBits)));
}

__device__ __forceinline__ int whole_of(int64_t v) { return int(v >> kFracBits); }
// the upper 32 of the fraction bits, in [0, 1]
__device__ __forceinline__ float fraction_of(int64_t v) {
    return float(uint32_t(v >> (kFracBits - 32))) * 2.3283064365386963e-10f;
}
__device__ __forceinline__ float exp2_fixed(int64_t v) { return exp2_parts(fraction_of(v), whole_of(v)); }

template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t add_moved(int64_t v) {
    const int lo = __builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xf, true);
    const int hi = __builtin_amdgcn_update_dpp(0, int(v >> 32), CTRL, ROWS, 0xf, true);
    return v + ((int64_t(hi) << 32) | uint32_t(lo));
}

// One wave: lane t holds token t's log decay (0 beyond the rows' end and for lanes >= C).
// Running sums by lane moves inside 16 lanes, then across.  Returns the chunk's sum.
template <int C>
__device__ __forceinline__ int64_t decay_prepare(float g, int lane, int reverse, float in_scale,
                                                 float up_scale, Decay<C>& d) {
    int64_t sum = decay_fixed(g);
    sum = add_moved<0x111, 0xf>(sum);
    sum = add_moved<0x112, 0xf>(sum);
    sum = add_moved<0x114, 0xf>(sum);
    sum = add_moved<0x118, 0xf>(sum);
    sum = add_moved<0x142, 0xa>(sum);   // row 0's last lane to row 1, row 2's to row 3
    sum = add_moved<0x143, 0xc>(sum);   // lane 31 to rows 2 and 3
    const int64_t total = (int64_t(__builtin_amdgcn_readlane(int(sum >> 32), 63)) << 32) |
                          uint32_t(__builtin_amdgcn_readlane(int(sum), 63));
    // from the first NaN on every sum is one
    const uint64_t bad = __ballot(g != g);
    const float mark = (bad << (63 - lane)) ? __builtin_nanf("") : 0.0f;
    const float mark_all = bad ? __builtin_nanf("") : 0.0f;
    if (lane < C) {
        d.whole[lane] = whole_of(sum);
        d.frac[lane] = fraction_of(sum) + mark;
        const float fwd = exp2_fixed(sum) + mark, bwd = exp2_fixed(total - sum) + mark_all;
        d.in[lane] = in_scale * (reverse ? bwd : fwd);
        d.up[lane] = up_scale * (reverse ? fwd : bwd);
        if (lane == 0) d.all = exp2_fixed(total) + mark_all;
    }
    return bad ? INT64_MIN : total;
}

// Whether a fragment holds an infinity or NaN: bit 31 of the result, or bit 15 for bf16.
__device__ __forceinline__ uint32_t not_finite(bf16x8 f, uint32_t seen) {
    union { bf16x8 f; uint32_t w[4]; } u;
    u.f = f;
#pragma unroll
    for (int i = 0; i < 4; ++i) seen |= (u.w[i] & 0x7f807f80u) + 0x00800080u;
    return seen;
}
__device__ __forceinline__ uint32_t not_finite(f32x8 f, uint32_t seen) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        seen |= ((__float_as_uint(f[i]) & 0x7fffffffu) + 0x00800000u) & 0x80000000u;
    return seen;
}

// Waves a SIMD that the registers are to allow (la_round in ss_la_plan.h counts on them).  Four
// where the state, the rows in flight and the products fit 128 registers; at 128 state rows they
// would spill 18 of them, and two workgroups a CU were no faster than one after the other
// (B = 4, T = 2048, H = 16, 128 x 128: 47 us with four waves, 44 with two on half the segments).
constexpr int sweep_occupancy(int el, bool vec, int DA, int NW, bool dot, bool state) {
    if (DA == 256 && NW == 4 && !state) return 1;
    if (state) return DA == 256 ? 2 : 4;
    return DA > 64 || dot || !vec ? 2 : el == 2 && NW == 4 ? 3 : 4;
}

// kState: only the state that a segment adds from zero, and the segment's decay (the first of
// the two passes over a sequence that is split into segments).  kDot: also e_t·out_t without
// the diagonal.  Its pairs are summed in 64 bits: a pair's value has the same bits in the row
// sums and in the column sums, so what enters one and leaves the other cancels exactly in the
// running sum of dg.
template <typename T, bool kVec, int DA, int NW, bool kDot, bool kState, bool kPair>
__global__ __launch_bounds__(64 * NW, sweep_occupancy(int(sizeof(T)), kVec, DA, NW, kDot, kState)) void sweep_kernel(const LaSweeps sweeps) {
    const LaSweep& p = sweeps.p[kPair ? blockIdx.y : 0];
    using M = Mma<T>;
    using Frag = typename M::Frag;
    using Elem = typename M::Elem;
    constexpr int C = M::kChunk, V = M::kVec, KT = M::kTerms;
    constexpr int NT = 64 * NW;                     // threads
    constexpr int DC = 16 * NW;                     // columns of a workgroup
    constexpr int kPad = 16 / int(sizeof(Elem));    // rows start 16 bytes (four banks) apart
    constexpr int LA = DA + kPad;                   // read by rows of 16 bytes
    constexpr int LB = DA + 2 * kPad, LC = DC + 2 * kPad;   // read transposed, 32 bytes a row
    constexpr int NA = C * DA / V / NT, NC = C * DC / V / NT;    // 16-byte pieces of a thread
    constexpr int SA = NT * V / DA, SC = NT * V / DC;            // tokens between them
    constexpr int TB = C / 16, KS = C / 32, IB = DA / 32;
    constexpr int kTiles = TB * (TB + 1) / 2;
    constexpr int PT = sizeof(T) == 2 ? 2 : 1;      // terms of P
    constexpr int ST = kDot ? KT : PT;              // terms of S where it feeds out

    __shared__ __attribute__((aligned(16))) Elem lb[C * LB];
    __shared__ __attribute__((aligned(16))) Elem lc[C * LC];
    __shared__ __attribute__((aligned(16))) Elem la_[kState ? 8 : C * LA];
    __shared__ __attribute__((aligned(16))) Elem lp[kState ? 8 : PT * C * C];
    __shared__ __attribute__((aligned(16))) Elem le[kDot ? C * DC : 8];
    __shared__ __attribute__((aligned(16))) Decay<C> dec[2];
    __shared__ double dot_tile[kDot ? kTiles * 16 : 1];
    __shared__ float dot_wave[kDot ? NW * C : 1];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, lg = lane >> 4;
    // P and e lie in LDS without padding, their 16-byte pieces exchanged by row instead; P with
    // the tokens s of each 32 in the order of the transposed operands
    auto p_at = [](int t, int s) { return t * C + (((s / V) ^ ((t >> 1) & (C / V - 1))) * V) + s % V; };
    auto e_at = [](int t, int j) { return t * DC + (((j / V) ^ (t & (DC / V - 1))) * V) + j % V; };
    auto p_row = [&](int t, int s, int term) {   // eight consecutive values
        if constexpr (sizeof(T) == 2) return M::row(&lp[term * C * C + p_at(t, s)]);
        else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(&lp[p_at(t, s)]);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(&lp[p_at(t, s + 4)]);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    auto e_row = [&](int t, int j) {
        if constexpr (sizeof(T) == 2) return M::row(&le[e_at(t, j)]);
        else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(&le[e_at(t, j)]);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(&le[e_at(t, j + 4)]);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    // Work items: column tile fastest, then head, then segment, then batch row.  Workgroups go
    // round the eight XCDs in turn, so each XCD is given a run of consecutive items: the tiles
    // of a head, and the heads that share q and k, find each other's rows in their L2.
    const unsigned xcd = blockIdx.x % 8, each = gridDim.x / 8, more = gridDim.x % 8;
    unsigned blk = xcd * each + (xcd < more ? xcd : more) + blockIdx.x / 8;
    const int tile = int(blk % unsigned(p.tiles));
    blk /= unsigned(p.tiles);
    const int64_t h = blk % unsigned(p.H);
    blk /= unsigned(p.H);
    const int seg = int(blk % unsigned(p.grid_seg)) + p.seg0;
    const int64_t b = blk / unsigned(p.grid_seg);
    const int64_t bh = b * p.H + h;
    const int c0 = tile * DC;                       // first column
    const int jw = wave * 16;                       // the wave's first column in the tile

    const int tok_a = tid / (DA / V), col_a = (tid % (DA / V)) * V;
    const int tok_c = tid / (DC / V), col_c = (tid % (DC / V)) * V;
    const Rows<T> rb = rows_of<T>(p.b, b, h, tok_a, col_a);
    const Rows<T> rc = rows_of<T>(p.c, b, h, tok_c, c0 + col_c);
    const Rows<T> ra = kState ? rb : rows_of<T>(p.a, b, h, tok_a, col_a);
    const Rows<T> re = kDot ? rows_of<T>(p.e, b, h, tok_c, c0 + col_c) : rc;
    int64_t len = p.T;
    if (p.lengths) {
        len = p.lengths[b];
        len = len < 0 ? 0 : len > p.T ? p.T : len;
    }
    const int64_t nchunk = (p.T + C - 1) / C;
    const int64_t ch_lo = int64_t(seg) * p.seg_chunks;
    int64_t ch_hi = ch_lo + p.seg_chunks;
    ch_hi = ch_hi < nchunk ? ch_hi : nchunk;
    const int n = int(ch_hi > ch_lo ? ch_hi - ch_lo : 0);
    const int rev = p.reverse;

    // ---- the state this segment starts from --------------------------------------------------
    f32x4 S[IB][2];
#pragma unroll
    for (int ib = 0; ib < IB; ++ib)
#pragma unroll
        for (int u = 0; u < 2; ++u) S[ib][u] = f32x4{0, 0, 0, 0};
    // element (i, j) of a lane's register r; descriptors again stand for the bounds, so that all
    // of a lane's accesses are in flight at once
    const int state_bytes = int(p.s_in_sz) * 4;
    auto state_at = [&](int ib, int u, int r, int sti, int stj) {
        const int i = 32 * ib + 8 * lg + 4 * u + r, j = c0 + jw + l16;
        return i < p.b.dim && j < p.c.dim ? (i * sti + j * stj) * 4 : int(kNowhere);
    };
    if (!kState && p.s_in) {
        const float* si = p.s_in + (bh * p.in_seg + (p.in_seg > 1 ? seg : 0)) * p.s_in_sz;
        const __amdgpu_buffer_rsrc_t d =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(si), 0, state_bytes, kRsrcFlags);
#pragma unroll
        for (int ib = 0; ib < IB; ++ib)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[ib][u][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                        d, state_at(ib, u, r, int(p.s_in_i), int(p.s_in_j)), 0, 0));
    }

    u32x4 va[kState ? 1 : NA], vb[NA], vc[NC], ve[kDot ? NC : 1];
    float vg = 0.0f;
    // first token of step i, in the sweep's direction, and how many tokens its chunk has
    auto first_of = [&](int i) { return (rev ? ch_hi - 1 - i : ch_lo + i) * C; };
    auto tokens_at = [](int64_t t0, int64_t end) {
        const int64_t m = end - t0;
        return int(m < 0 ? 0 : m < C ? m : C);
    };
    auto load_rows = [&](int i) {
        const int64_t t0 = first_of(i);
        const int nv = tokens_at(t0, len);
        load_pieces<T, kVec, NA, SA>(rb, t0, nv, vb);
        if constexpr (!kState) load_pieces<T, kVec, NA, SA>(ra, t0, nv, va);
        load_pieces<T, kVec, NC, SC>(rc, t0, nv, vc);
        if constexpr (kDot) load_pieces<T, kVec, NC, SC>(re, t0, nv, ve);
    };
    auto load_g = [&](int i) {  // the last wave prepares the decays
        if (wave != NW - 1) return;
        vg = 0.0f;
        const int64_t t0 = first_of(i);
        if (p.g && lane < tokens_at(t0, len))
            vg = p.decay_token ? p.g[(b * p.T + t0 + lane) * p.H + h] : p.g[h];
    };
    int64_t seg_sum = 0;
    bool seg_nan = false;
    auto prepare = [&](int i) {
        if (wave != NW - 1) return;
        const int64_t sum = decay_prepare<C>(vg, lane, rev, p.in_scale, p.up_scale, dec[i & 1]);
        if (sum == INT64_MIN) {
            seg_nan = true;
        } else {
            // beyond ±2^17 the decay is 0 or inf in any case, and the sum must not wrap
            const int64_t most = int64_t(1) << (17 + kFracBits);
            seg_sum += sum;
            seg_sum = seg_sum < -most ? -most : seg_sum > most ? most : seg_sum;
        }
    };

    if constexpr (!kState)
        // tiles of P that the mask empties are read but never written again
        for (int i = tid; i < PT * C * C; i += NT) lp[i] = M::from(0.0f);
    if (n > 0) {
        load_g(0);
        load_rows(0);
        prepare(0);
        if (n > 1) load_g(1);
    }
    for (int it = 0; it < n; ++it) {
        const int64_t t0 = first_of(it);
        const int nv = tokens_at(t0, len);
        __syncthreads();  // the last chunk's readers are done
#pragma unroll
        for (int x = 0; x < NA; ++x) {
            const int t = tok_a + x * SA;
            *reinterpret_cast<u32x4*>(&lb[t * LB + col_a]) = vb[x];
            if constexpr (!kState) *reinterpret_cast<u32x4*>(&la_[t * LA + col_a]) = va[x];
        }
#pragma unroll
        for (int x = 0; x < NC; ++x) {
            *reinterpret_cast<u32x4*>(&lc[(tok_c + x * SC) * LC + col_c]) = vc[x];
            if constexpr (kDot) *reinterpret_cast<u32x4*>(&le[e_at(tok_c + x * SC, col_c)]) = ve[x];
        }
        __syncthreads();
        if (it + 1 < n) {
            load_rows(it + 1);
            prepare(it + 1);
            if (it + 2 < n) load_g(it + 2);
        }
        const Decay<C>& d = dec[it & 1];

        // columns of c, transposed: the operand of out and of the state
        Frag cf[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) cf[ks] = col_frag<T>(&lc[32 * ks * LC], LC, lane, jw, 4);

        // whether something in the wave's columns of c is not finite
        uint32_t seen = 0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) seen = not_finite(cf[ks], seen);
        const unsigned keep = (seen & 0x80008000u) ? 0u : ~0u;
        const bool bad = __any(keep == 0);
        if constexpr (!kState) {
            // ---- P, transposed tiles: lane's column is token t, its rows four tokens s ----------
            for (int x = wave; x < kTiles; x += NW) {
                const int hi = (x >= 1) + (x >= 3) + (x >= 6), lo = x - hi * (hi + 1) / 2;
                const int tb = rev ? lo : hi, sb = rev ? hi : lo;
                f32x4 acc = {0, 0, 0, 0}, ec = {0, 0, 0, 0};
                const Elem* brow = &lb[(16 * sb + l16) * LB + 8 * lg];
                const Elem* arow = &la_[(16 * tb + l16) * LA + 8 * lg];
#pragma unroll
                for (int k = 0; k < IB; ++k) acc = M::mma(M::row(brow + 32 * k), M::row(arow + 32 * k), acc);
                if constexpr (kDot) {
                    const Elem* crow = &lc[(16 * sb + l16) * LC + 8 * lg];
#pragma unroll
                    for (int k = 0; k < DC / 32; ++k)
                        ec = M::mma(M::row(crow + 32 * k), e_row(16 * tb + l16, 32 * k + 8 * lg), ec);
                }
                const int t = 16 * tb + l16, s0 = 16 * sb + 4 * lg;
                const int sp = 32 * (sb / 2) + 8 * lg + 4 * (sb & 1);   // s0's place in P
                const float ft = d.frac[t];
                const int wt = d.whole[t];
                const f32x4 fs = *reinterpret_cast<const f32x4*>(&d.frac[s0]);
                const int4 ws = *reinterpret_cast<const int4*>(&d.whole[s0]);
                const int wsa[4] = {ws.x, ws.y, ws.z, ws.w};
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float df = ft - fs[r];
                    const int dw = wt - wsa[r];
                    v[r] = acc[r] * (p.alpha * exp2_parts(rev ? -df : df, rev ? -dw : dw));
                }
                if (tb == sb || nv < C) {
                    // the mask selects: what a masked place holds reaches nothing
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int s = s0 + r;
                        v[r] = (rev ? s >= t : s <= t) && s < nv ? v[r] : 0.0f;
                    }
                }
                if constexpr (kDot) {
                    double dot = 0.0;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int s = s0 + r;
                        const bool off = (rev ? s > t : s < t) && s < nv;
                        dot += off ? double(v[r]) * double(ec[r]) : 0.0;
                    }
                    dot += __shfl_xor(dot, 16, 64);
                    dot += __shfl_xor(dot, 32, 64);
                    if (lg == 0) dot_tile[x * 16 + l16] = dot;
                }
                if constexpr (sizeof(T) == 2) {
                    bf16x4 o[PT];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        o[0][r] = __bf16(v[r]);
                        const float left = v[r] - float(o[0][r]);
                        o[1][r] = __bf16(left == left ? left : 0.0f);
                    }
#pragma unroll
                    for (int q = 0; q < PT; ++q)
                        *reinterpret_cast<bf16x4*>(&lp[q * C * C + p_at(t, sp)]) = o[q];
                } else {
                    *reinterpret_cast<f32x4*>(&lp[p_at(t, sp)]) = f32x4{v[0], v[1], v[2], v[3]};
                }
            }
            // ---- out, transposed: the entering state's part ---------------------------------------
            f32x4 O[TB];
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) O[tb] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int ib = 0; ib < IB; ++ib) {
                Frag sf[ST];
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = S[ib][e >> 2][e & 3];
                if constexpr (kDot) M::split(v, ~0u, sf);
                else M::two(v, sf);
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    const Frag af = M::row(&la_[(16 * tb + l16) * LA + 32 * ib + 8 * lg]);
#pragma unroll
                    for (int q = 0; q < ST; ++q) O[tb] = M::mma(sf[q], af, O[tb]);
                }
            }
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) O[tb] *= d.in[16 * tb + l16];
            if constexpr (kDot) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    float dot = 0.0f;
                    const Elem* q = &le[e_at(16 * tb + l16, jw + 4 * lg)];
#pragma unroll
                    for (int r = 0; r < 4; ++r) dot = fmaf(float(q[r]), O[tb][r], dot);
                    dot += __shfl_xor(dot, 16, 64);
                    dot += __shfl_xor(dot, 32, 64);
                    if (lg == 0) dot_wave[wave * C + 16 * tb + l16] = dot;
                }
            }
            __syncthreads();  // P is whole
            if constexpr (kDot) {
                if (tid < C && t0 + tid < p.T) {
                    double dot = 0.0;
#pragma unroll
                    for (int w = 0; w < NW; ++w) dot += double(dot_wave[w * C + tid]);
                    const int tb = tid >> 4;
                    for (int x = 0; x < kTiles; ++x) {
                        const int hi = (x >= 1) + (x >= 3) + (x >= 6), lo = x - hi * (hi + 1) / 2;
                        if ((rev ? lo : hi) == tb) dot += dot_tile[x * 16 + (tid & 15)];
                    }
                    p.dots[(int64_t(tile) * p.B * p.H + bh) * p.T + t0 + tid] = tid < nv ? dot : 0.0;
                }
            }
            // ---- the chunk's own part ---------------------------------------------------------------
            // All of P, the tiles that the mask empties too (zeros).
            if (!bad) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int q = 0; q < PT; ++q)
                            O[tb] = M::mma(cf[ks], p_row(16 * tb + l16, 32 * ks + 8 * lg, q), O[tb]);
                settle();
            } else {
                // A masked weight is 0, and its product with an infinity would be NaN: the
                // allowed pairs alone, one by one.
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    const int t = 16 * tb + l16;
#pragma unroll 1
                    for (int s = 0; s < nv; ++s) {
                        if (rev ? s < t : s > t) continue;
                        const int sp = (s & ~31) + 8 * ((s >> 2) & 3) + 4 * ((s >> 4) & 1) + (s & 3);
                        float w = float(lp[p_at(t, sp)]);
                        if (PT == 2) w += float(lp[(PT - 1) * C * C + p_at(t, sp)]);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            O[tb][r] = fmaf(w, float(lc[s * LC + jw + 4 * lg + r]), O[tb][r]);
                    }
                }
            }
            // ---- store: four consecutive columns of one token a lane ------------------------------------
            if (nv < C) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
                    if (16 * tb + l16 >= nv) O[tb] = f32x4{0, 0, 0, 0};
            }
            const int rows = tokens_at(t0, p.T), dim = p.c.dim;
            const int64_t first = ((b * p.T + t0) * p.H + h) * dim;
            const bool wide = sizeof(T) == 4 || p.out_f32;
            const int st = int(p.H) * dim, el = wide ? 4 : 2;
            // the descriptor ends with the chunk's last row: tokens beyond are dropped
            const __amdgpu_buffer_rsrc_t od = __builtin_amdgcn_make_buffer_rsrc(
                static_cast<char*>(p.out) + first * el, 0, ((rows - 1) * st + dim) * el, kRsrcFlags);
            const int j = c0 + jw + 4 * lg;
            const unsigned at = j < dim ? unsigned((l16 * st + j) * el) : kNowhere;
            if (dim % 4 == 0) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    if (wide) {
                        union { f32x4 f; u32x4 u; } w;
                        w.f = O[tb];
                        __builtin_amdgcn_raw_buffer_store_b128(w.u, od, int(at), 16 * tb * st * el, 0);
                    } else {
                        union { bf16x4 f; u32x2 u; } w;
#pragma unroll
                        for (int r = 0; r < 4; ++r) w.f[r] = __bf16(O[tb][r]);
                        __builtin_amdgcn_raw_buffer_store_b64(w.u, od, int(at), 16 * tb * st * el, 0);
                    }
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const unsigned to = j + r < dim ? at + unsigned(r * el) : kNowhere;
#pragma unroll
                    for (int tb = 0; tb < TB; ++tb) {
                        union { float f; unsigned u; } w;
                        union { __bf16 f; unsigned short u; } x;
                        w.f = O[tb][r];
                        x.f = __bf16(O[tb][r]);
                        if (wide) __builtin_amdgcn_raw_buffer_store_b32(w.u, od, int(to), 16 * tb * st * el, 0);
                        else __builtin_amdgcn_raw_buffer_store_b16(x.u, od, int(to), 16 * tb * st * el, 0);
                    }
                }
            }
        }

        // ---- the state: S = all·S + bᵀ(up ⊙ c) --------------------------------------------------------
        const float all = d.all;
#pragma unroll
        for (int ib = 0; ib < IB; ++ib)
#pragma unroll
            for (int u = 0; u < 2; ++u) S[ib][u] *= all;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Frag wf[KT];
            const f32x4 u0 = *reinterpret_cast<const f32x4*>(&d.up[32 * ks + 4 * lg]);
            const f32x4 u1 = *reinterpret_cast<const f32x4*>(&d.up[32 * ks + 16 + 4 * lg]);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = M::get(cf[ks], e) * (e < 4 ? u0[e & 3] : u1[e & 3]);
            M::split(v, keep, wf);
#pragma unroll
            for (int ib = 0; ib < IB; ++ib)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const Frag bf = col_frag<T>(&lb[32 * ks * LB], LB, lane, 32 * ib + 4 * u, 8);
#pragma unroll
                    for (int q = KT - 1; q >= 0; --q) S[ib][u] = M::mma(bf, wf[q], S[ib][u]);
                }
        }
    }

    // ---- the state this segment leaves ---------------------------------------------------------------
    const bool last = kState || (rev ? seg == 0 : seg == p.nseg - 1);
    if (p.s_out && last) {
        const int out_i = kDot && p.s_out_t ? 1 : p.c.dim, out_j = kDot && p.s_out_t ? p.b.dim : 1;
        float* so = p.s_out + (bh * (kState ? p.nseg : 1) + (kState ? seg : 0)) * p.s_in_sz;
        const __amdgpu_buffer_rsrc_t d = __builtin_amdgcn_make_buffer_rsrc(so, 0, state_bytes, kRsrcFlags);
#pragma unroll
        for (int ib = 0; ib < IB; ++ib)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[ib][u][r]), d,
                                                          state_at(ib, u, r, out_i, out_j), 0, 0);
    }
    if (kState && tile == 0 && tid == NT - 64)
        p.seg_decay[bh * p.nseg + seg] = seg_nan ? __builtin_nanf("") : exp2_fixed(seg_sum);
}

template <typename T, bool kVec, int DA, int NW>
hipError_t launch_sweep_t(const LaSweeps& w, hipStream_t s) {
    const LaSweep& p = w.p[0];
    const int64_t blocks = int64_t(p.tiles) * p.H * p.grid_seg * p.B;
    if (blocks <= 0) return hipSuccess;
    if (w.n == 2 && !p.state_only && !p.dots) {   // no pair instance: gradients without decays
        LaSweeps one = w;
        one.n = 1;
        const hipError_t e = launch_sweep_t<T, kVec, DA, NW>(one, s);
        if (e != hipSuccess) return e;
        one.p[0] = w.p[1];
        return launch_sweep_t<T, kVec, DA, NW>(one, s);
    }
    const dim3 grid{unsigned(blocks), unsigned(w.n)}, block(64 * NW);
    if (p.state_only && w.n == 2)
        hipLaunchKernelGGL((sweep_kernel<T, kVec, DA, NW, false, true, true>), grid, block, 0, s, w);
    else if (p.state_only)
        hipLaunchKernelGGL((sweep_kernel<T, kVec, DA, NW, false, true, false>), grid, block, 0, s, w);
    else if (p.dots)
        hipLaunchKernelGGL((sweep_kernel<T, kVec, DA, NW, true, false, true>), grid, block, 0, s, w);
    else
        hipLaunchKernelGGL((sweep_kernel<T, kVec, DA, NW, false, false, false>), grid, block, 0, s, w);
    return hipGetLastError();
}

template <typename T, bool kVec>
hipError_t launch_sweep_type(const LaSweeps& w, hipStream_t s) {
    const int key = w.p[0].pad_a * 10 + w.p[0].waves;
    switch (key) {
        case 644: return launch_sweep_t<T, kVec, 64, 4>(w, s);
        case 648: return launch_sweep_t<T, kVec, 64, 8>(w, s);
        case 1284: return launch_sweep_t<T, kVec, 128, 4>(w, s);
        case 1288: return launch_sweep_t<T, kVec, 128, 8>(w, s);
        case 2564: return launch_sweep_t<T, kVec, 256, 4>(w, s);
        case 2568: return launch_sweep_t<T, kVec, 256, 8>(w, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace la
}  // namespace ss
