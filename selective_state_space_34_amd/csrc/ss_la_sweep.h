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
// e = q and the diagonal left out, col_u that of the dk sweep with e = k (kDot).  Every pair
// that a row or column sum holds is also held by some dg near it, so the running sum loses
// nothing to cancellation.
//
// A workgroup of four waves takes one head's rows chunk by chunk (64 tokens of bf16, 32 of
// float32) with the state in registers: wave w holds all dA rows of its 16·NT columns, in the
// accumulator layout of v_mfma_f32_16x16x32_bf16 (lane l: column l % 16, rows 4·(l/16) + r).
// Inside a chunk:
//   P  = (a bᵀ) ⊙ decay: 16 x 16 tiles dealt to the waves, only those the mask leaves, through LDS
//   out = Sᵀaᵀ (state as an operand straight from the accumulators: the rows of S are dealt to
//         accumulators so that a lane's eight values are the eight consecutive k it must feed)
//         scaled by each token's entering decay, plus cᵀPᵀ
//   S  = e^{G_C} S + bᵀ(w ⊙ c)   (transposed operands: ds_read_b64_tr_b16)
// The next chunk's rows are loaded into registers meanwhile.
//
// Numerics.  Log decays are summed in 64 bits and kept as an integer and a fraction in base 2,
// so a weight is ldexp(2^fraction, integer) of an exact difference: no error grows with the
// length, and a token that decays by e^{-inf} cuts the sequence exactly.  P, and S where it
// feeds out, are rounded to bf16 once (the operand the matrix cores take; out is bf16 too).
// The state's own sums are float32: c's weight w is not a bf16 value, so w·c is fed as three
// bf16 terms (24 bits).  The products behind dg (P, e·c, e·(Sᵀa)) are kept in float32 the same
// way, since dg is float32.  With float32 rows the matrix cores' float32 form runs on the same
// layouts and nothing is rounded.
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
    // Transposed: eight consecutive rows (tokens) of one column.  In a group of 16 lanes,
    // lane λ of ds_read_b64_tr_b16 names four consecutive elements (row λ / 4, piece λ % 4 of
    // 16 columns) and receives column λ of the four rows.  p: row 0 of the 32 tokens; col(q):
    // the first column of piece q.
    static __device__ __forceinline__ Frag col(const Elem* p, int ld, int lane, int piece_col) {
        const Elem* q = p + (8 * (lane >> 4) + ((lane >> 2) & 3)) * ld + piece_col;
        typedef __attribute__((address_space(3))) s16x4* Lds;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(q));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(q + 4 * ld));
        union { s16x4 h[2]; Frag f; } u;
        u.h[0] = lo;
        u.h[1] = hi;
        return u.f;
    }
    static __device__ __forceinline__ float get(Frag f, int e) { return float(f[e]); }
    static __device__ __forceinline__ Elem from(float v) { return Elem(v); }
    static __device__ __forceinline__ Frag round8(const float (&v)[8]) {
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = Elem(v[e]);
        return f;
    }
    // v as kTerms bf16 terms that sum to it (relative error below 2^-24).  An infinite value
    // is its first term alone.
    static __device__ __forceinline__ void split(const float (&v)[8], Frag (&f)[kTerms]) {
        float r[8], probe = 0.0f;
        f[0] = round8(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[e] = v[e] - float(f[0][e]);
            probe = fmaf(r[e], 0.0f, probe);
        }
        if (__any(probe != probe)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = r[e] != r[e] ? 0.0f : r[e];
        }
        f[1] = round8(r);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] -= float(f[1][e]);
        f[2] = round8(r);
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
        const Elem* q = p + 8 * (lane >> 4) * ld + column;
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = q[e * ld];
        return f;
    }
    static __device__ __forceinline__ float get(Frag f, int e) { return f[e]; }
    static __device__ __forceinline__ Elem from(float v) { return v; }
    static __device__ __forceinline__ Frag round8(const float (&v)[8]) {
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e];
        return f;
    }
    static __device__ __forceinline__ void split(const float (&v)[8], Frag (&f)[kTerms]) {
        f[0] = round8(v);
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

// Rows of one operand of one (batch row, head).
template <typename T>
struct Rows {
    const T* p;
    int64_t st;  // elements from token to token
    int dim, vec;
};

template <typename T>
__device__ __forceinline__ Rows<T> rows_of(const LaOperand& o, int64_t b, int64_t h) {
    return Rows<T>{static_cast<const T*>(o.p) + b * o.sb + (h / o.rep) * o.sh, o.st, o.dim, o.vec};
}

// 16 bytes of token t, elements [col, col + kVec); zeros outside the token range and the width.
template <typename T>
__device__ __forceinline__ uint4 load16(const Rows<T>& r, int64_t t, int64_t end, int col) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t >= end || col >= r.dim) return v;
    const T* q = r.p + t * r.st + col;
    if (r.vec) return *reinterpret_cast<const uint4*>(q);
    constexpr int kVec = Mma<T>::kVec;
    union { uint4 v; T e[kVec]; } u;
    u.v = v;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (col + i < r.dim) u.e[i] = q[i];
    return u.v;
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

// 2^d of a 64-bit exponent
__device__ __forceinline__ float exp2_wide(double d) {
    const double n = __builtin_rint(d);
    return exp2_parts(float(d - n), int(n));
}

// Per-token log decays (natural) to base 2, bounded so that sums stay exact: 2^±1024 is 0 or
// inf in float32 either way.  NaN stays NaN.
__device__ __forceinline__ double decay_log2(float g) {
    double x = double(g) * 1.4426950408889634074;
    x = x < -1024.0 ? -1024.0 : x;
    return x > 1024.0 ? 1024.0 : x;
}

// One wave: lane t holds token t's log decay (0 beyond the rows' end and for lanes >= C).
// Returns the chunk's sum.
template <int C>
__device__ __forceinline__ double decay_prepare(double x, int lane, int reverse, float in_scale,
                                                float up_scale, Decay<C>& d) {
    double sum = x;
#pragma unroll
    for (int m = 1; m < C; m <<= 1) {
        const double o = __shfl_up(sum, m, 64);
        if (lane >= m) sum += o;
    }
    const double total = __shfl(sum, C - 1, 64);
    if (lane < C) {
        const double n = __builtin_rint(sum);
        d.whole[lane] = int(n);
        d.frac[lane] = float(sum - n);
        const float fwd = exp2_wide(sum), bwd = exp2_wide(total - sum);
        d.in[lane] = in_scale * (reverse ? bwd : fwd);
        d.up[lane] = up_scale * (reverse ? fwd : bwd);
        if (lane == 0) d.all = exp2_wide(total);
    }
    return total;
}

// kState: only the state that a segment adds from zero, and the segment's decay (the first of
// the two passes over a sequence that is split into segments).  kDot: also e_t·out_t without
// the diagonal, in float32.
template <typename T, int DA, int NT, bool kDot, bool kState>
__global__ __launch_bounds__(256) void sweep_kernel(const LaSweep p) {
    using M = Mma<T>;
    using Frag = typename M::Frag;
    using Elem = typename M::Elem;
    constexpr int C = M::kChunk, V = M::kVec, KT = M::kTerms;
    constexpr int DC = 64 * NT;                     // columns of a workgroup
    constexpr int kPad = 16 / int(sizeof(Elem));    // rows start 16 bytes (four banks) apart
    constexpr int LA = DA + kPad, LC = DC + kPad, LP = C + kPad;
    constexpr int NA = C * DA / V / 256, NC = C * DC / V / 256;  // 16-byte loads of a thread
    constexpr int TB = C / 16, KS = C / 32, IB = DA / 32;
    constexpr int kTiles = TB * (TB + 1) / 2;

    __shared__ __attribute__((aligned(16))) Elem lb[C * LA];
    __shared__ __attribute__((aligned(16))) Elem lc[C * LC];
    __shared__ __attribute__((aligned(16))) Elem lall[kState ? 1 : C * LA];
    __shared__ __attribute__((aligned(16))) Elem lp[kState ? 1 : C * LP];
    __shared__ __attribute__((aligned(16))) Elem le[kDot ? C * LC : 1];
    __shared__ Decay<C> dec[2];
    __shared__ float dot_tile[kDot ? TB * TB * 16 : 1];
    __shared__ float dot_wave[kDot ? 4 * C : 1];
    Elem* const la_ = lall;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    // blocks: column tile fastest, then head, then segment, then batch row
    int64_t blk = blockIdx.x;
    const int tile = int(blk % p.tiles);
    blk /= p.tiles;
    const int64_t h = blk % p.H;
    blk /= p.H;
    const int seg = int(blk % p.grid_seg) + p.seg0;
    const int64_t b = blk / p.grid_seg;
    const int64_t bh = b * p.H + h;
    const int c0 = tile * DC;                       // first column
    const int jw = wave * 16 * NT;                  // the wave's first column in the tile

    const Rows<T> rb = rows_of<T>(p.b, b, h), rc = rows_of<T>(p.c, b, h);
    const Rows<T> ra = kState ? rb : rows_of<T>(p.a, b, h);
    const Rows<T> re = kDot ? rows_of<T>(p.e, b, h) : rb;
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
    f32x4 S[IB][2][NT];
#pragma unroll
    for (int ib = 0; ib < IB; ++ib)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                f32x4 s = {0, 0, 0, 0};
                if (!kState && p.s_in) {
                    const int j = c0 + jw + 16 * nt + l16;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = 32 * ib + 8 * lg + 4 * u + r;
                        if (i < p.b.dim && j < p.c.dim)
                            s[r] = p.s_in[(bh * p.in_seg + (p.in_seg > 1 ? seg : 0)) * p.s_in_sz +
                                          i * p.s_in_i + j * p.s_in_j];
                    }
                }
                S[ib][u][nt] = s;
            }

    uint4 va[kState ? 1 : NA], vb[NA], vc[NC], ve[kDot ? NC : 1];
    float vg = 0.0f;
    // chunk number of step i, in the sweep's direction
    auto chunk_of = [&](int i) { return rev ? ch_hi - 1 - i : ch_lo + i; };
    auto load_rows = [&](int i) {
        const int64_t t0 = chunk_of(i) * C;
#pragma unroll
        for (int x = 0; x < NA; ++x) {
            const int id = x * 256 + tid, t = id / (DA / V), col = (id % (DA / V)) * V;
            vb[x] = load16(rb, t0 + t, len, col);
            if constexpr (!kState) va[x] = load16(ra, t0 + t, len, col);
        }
#pragma unroll
        for (int x = 0; x < NC; ++x) {
            const int id = x * 256 + tid, t = id / (DC / V), col = c0 + (id % (DC / V)) * V;
            vc[x] = load16(rc, t0 + t, len, col);
            if constexpr (kDot) ve[x] = load16(re, t0 + t, len, col);
        }
    };
    auto load_g = [&](int i) {  // the last wave prepares the decays
        vg = 0.0f;
        const int64_t t = chunk_of(i) * C + lane;
        if (wave == 3 && p.g && lane < C && t < len)
            vg = p.g[p.decay_token ? (b * p.T + t) * p.H + h : h];
    };
    double seg_sum = 0.0;
    auto prepare = [&](int i) {
        if (wave == 3)
            seg_sum += decay_prepare<C>(decay_log2(vg), lane, rev, p.in_scale, p.up_scale, dec[i & 1]);
    };

    if constexpr (!kState) {
        // tiles of P that the mask empties are read in 32-wide steps but never written again
        for (int i = tid; i < C * LP; i += 256) lp[i] = M::from(0.0f);
        if constexpr (kDot)
            for (int i = tid; i < TB * TB * 16; i += 256) dot_tile[i] = 0.0f;
    }
    if (n > 0) {
        load_g(0);
        load_rows(0);
        prepare(0);
        if (n > 1) load_g(1);
    }
    for (int it = 0; it < n; ++it) {
        const int64_t t0 = chunk_of(it) * C;
        __syncthreads();  // the last chunk's readers are done
#pragma unroll
        for (int x = 0; x < NA; ++x) {
            const int id = x * 256 + tid, at = (id / (DA / V)) * LA + (id % (DA / V)) * V;
            *reinterpret_cast<uint4*>(&lb[at]) = vb[x];
            if constexpr (!kState) *reinterpret_cast<uint4*>(&la_[at]) = va[x];
        }
#pragma unroll
        for (int x = 0; x < NC; ++x) {
            const int id = x * 256 + tid, at = (id / (DC / V)) * LC + (id % (DC / V)) * V;
            *reinterpret_cast<uint4*>(&lc[at]) = vc[x];
            if constexpr (kDot) *reinterpret_cast<uint4*>(&le[at]) = ve[x];
        }
        __syncthreads();
        if (it + 1 < n) {
            load_rows(it + 1);
            prepare(it + 1);
            if (it + 2 < n) load_g(it + 2);
        }
        const Decay<C>& d = dec[it & 1];

        // columns of c, transposed: the operand of out and of the state
        Frag cf[KS][NT];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                cf[ks][nt] = col_frag<T>(&lc[32 * ks * LC], LC, lane, jw + 16 * nt, 4);

        if constexpr (!kState) {
            // ---- P, transposed tiles: lane's column is token t, its rows four tokens s ----------
            for (int x = wave; x < kTiles; x += 4) {
                int hi = 0, lo = x;
                while (lo > hi) lo -= ++hi;  // row hi of the triangle, 0 <= lo <= hi
                const int tb = rev ? lo : hi, sb = rev ? hi : lo;
                f32x4 acc = {0, 0, 0, 0}, ec = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < IB; ++k)
                    acc = M::mma(M::row(&lb[(16 * sb + l16) * LA + 32 * k + 8 * lg]),
                                 M::row(&la_[(16 * tb + l16) * LA + 32 * k + 8 * lg]), acc);
                if constexpr (kDot) {
#pragma unroll
                    for (int k = 0; k < DC / 32; ++k)
                        ec = M::mma(M::row(&lc[(16 * sb + l16) * LC + 32 * k + 8 * lg]),
                                    M::row(&le[(16 * tb + l16) * LC + 32 * k + 8 * lg]), ec);
                }
                const int t = 16 * tb + l16, s0 = 16 * sb + 4 * lg;
                const float ft = d.frac[t];
                const int wt = d.whole[t];
                float dot = 0.0f;
                Elem out[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int s = s0 + r;
                    const float df = rev ? d.frac[s] - ft : ft - d.frac[s];
                    const int dw = rev ? d.whole[s] - wt : wt - d.whole[s];
                    float v = acc[r] * (p.alpha * exp2_parts(df, dw));
                    // the mask selects: what a masked place holds reaches nothing
                    v = ((rev ? s >= t : s <= t) && t0 + s < len) ? v : 0.0f;
                    if (kDot && s != t && (rev ? s >= t : s <= t) && t0 + s < len)
                        dot = fmaf(v, ec[r], dot);
                    out[r] = M::from(v);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) lp[t * LP + s0 + r] = out[r];
                if constexpr (kDot) {
                    dot += __shfl_xor(dot, 16, 64);
                    dot += __shfl_xor(dot, 32, 64);
                    if (lg == 0) dot_tile[(tb * TB + sb) * 16 + l16] = dot;
                }
            }
            // ---- out, transposed: the entering state's part ---------------------------------------
            f32x4 O[TB][NT];
            auto entering = [&]() {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) O[tb][nt] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int ib = 0; ib < IB; ++ib) {
                    Frag sf[NT][kDot ? KT : 1];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = S[ib][e >> 2][nt][e & 3];
                        if constexpr (kDot) M::split(v, sf[nt]);
                        else sf[nt][0] = M::round8(v);
                    }
#pragma unroll
                    for (int tb = 0; tb < TB; ++tb) {
                        const Frag af = M::row(&la_[(16 * tb + l16) * LA + 32 * ib + 8 * lg]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int q = 0; q < (kDot ? KT : 1); ++q)
                                O[tb][nt] = M::mma(sf[nt][q], af, O[tb][nt]);
                    }
                }
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) O[tb][nt] *= d.in[16 * tb + l16];
            };
            entering();
            if constexpr (kDot) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    float dot = 0.0f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            dot = fmaf(float(le[(16 * tb + l16) * LC + jw + 16 * nt + 4 * lg + r]),
                                       O[tb][nt][r], dot);
                    dot += __shfl_xor(dot, 16, 64);
                    dot += __shfl_xor(dot, 32, 64);
                    if (lg == 0) dot_wave[wave * C + 16 * tb + l16] = dot;
                }
            }
            __syncthreads();  // P is whole
            if constexpr (kDot) {
                if (tid < C && t0 + tid < p.T) {
                    float dot = 0.0f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) dot += dot_wave[w * C + tid];
#pragma unroll
                    for (int sb = 0; sb < TB; ++sb) dot += dot_tile[((tid >> 4) * TB + sb) * 16 + (tid & 15)];
                    p.dots[(int64_t(tile) * p.B * p.H + bh) * p.T + t0 + tid] = t0 + tid < len ? dot : 0.0f;
                }
            }
            // ---- the chunk's own part ---------------------------------------------------------------
            float probe = 0.0f;
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    if (rev ? ks < tb / 2 : ks > tb / 2) continue;
                    const Frag pf = M::row(&lp[(16 * tb + l16) * LP + 32 * ks + 8 * lg]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) O[tb][nt] = M::mma(cf[ks][nt], pf, O[tb][nt]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) probe = fmaf(O[tb][nt][r], 0.0f, probe);
            }
            // A masked weight is 0, and 0·inf in the product above is NaN: where something not
            // finite came out, the products are formed again from the allowed pairs alone.
            if (__any(probe != probe)) {
                entering();
                for (int tb = 0; tb < TB; ++tb) {
                    const int t = 16 * tb + l16;
                    for (int s = 0; s < C; ++s) {
                        if ((rev ? s < t : s > t) || t0 + s >= len) continue;
                        const float w = float(lp[t * LP + s]);
#pragma unroll
                        for (int q = 0; q < TB; ++q)
                            if (q == tb)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int r = 0; r < 4; ++r)
                                        O[q][nt][r] = fmaf(w, float(lc[s * LC + jw + 16 * nt + 4 * lg + r]), O[q][nt][r]);
                    }
                }
            }
            // ---- store: four consecutive columns of one token a lane ------------------------------------
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                const int64_t t = t0 + 16 * tb + l16;
                if (t >= p.T) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int j = c0 + jw + 16 * nt + 4 * lg;
                    const int left = p.c.dim - j;
                    if (left <= 0) continue;
                    f32x4 v = O[tb][nt];
                    if (t >= len) v = f32x4{0, 0, 0, 0};
                    const int64_t at = ((b * p.T + t) * p.H + h) * p.c.dim + j;
                    if (sizeof(T) == 4 || p.out_f32) {
                        float* o = static_cast<float*>(p.out) + at;
                        if (left >= 4 && p.c.dim % 4 == 0) {
                            *reinterpret_cast<f32x4*>(o) = v;
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (r < left) o[r] = v[r];
                        }
                    } else {
                        __bf16* o = static_cast<__bf16*>(p.out) + at;
                        bf16x4 w;
#pragma unroll
                        for (int r = 0; r < 4; ++r) w[r] = __bf16(v[r]);
                        if (left >= 4 && p.c.dim % 4 == 0) {
                            *reinterpret_cast<bf16x4*>(o) = w;
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (r < left) o[r] = w[r];
                        }
                    }
                }
            }
        }

        // ---- the state: S = all·S + bᵀ(up ⊙ c) --------------------------------------------------------
        const float all = d.all;
#pragma unroll
        for (int ib = 0; ib < IB; ++ib)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) S[ib][u][nt] *= all;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Frag wf[NT][KT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = M::get(cf[ks][nt], e) * d.up[32 * ks + 8 * lg + e];
                M::split(v, wf[nt]);
            }
#pragma unroll
            for (int ib = 0; ib < IB; ++ib)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const Frag bf = col_frag<T>(&lb[32 * ks * LA], LA, lane, 32 * ib + 4 * u, 8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int q = KT - 1; q >= 0; --q) S[ib][u][nt] = M::mma(bf, wf[nt][q], S[ib][u][nt]);
                }
        }
    }

    // ---- the state this segment leaves ---------------------------------------------------------------
    const bool last = kState || (rev ? seg == 0 : seg == p.nseg - 1);
    if (p.s_out && last) {
        float* so = p.s_out + (bh * (kState ? p.nseg : 1) + (kState ? seg : 0)) * p.s_out_sz;
#pragma unroll
        for (int ib = 0; ib < IB; ++ib)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int j = c0 + jw + 16 * nt + l16;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = 32 * ib + 8 * lg + 4 * u + r;
                        if (i < p.b.dim && j < p.c.dim) so[int64_t(i) * p.c.dim + j] = S[ib][u][nt][r];
                    }
                }
    }
    if (kState && tile == 0 && tid == 192) p.seg_decay[bh * p.nseg + seg] = exp2_wide(seg_sum);
}

template <typename T, int DA, int NT>
hipError_t launch_sweep_t(const LaSweep& p, hipStream_t s) {
    const int64_t blocks = int64_t(p.tiles) * p.H * p.grid_seg * p.B;
    if (blocks <= 0) return hipSuccess;
    const dim3 grid{unsigned(blocks)}, block(256);
    if (p.state_only) hipLaunchKernelGGL((sweep_kernel<T, DA, NT, false, true>), grid, block, 0, s, p);
    else if (p.dots) hipLaunchKernelGGL((sweep_kernel<T, DA, NT, true, false>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((sweep_kernel<T, DA, NT, false, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_sweep_type(const LaSweep& p, hipStream_t s) {
    const int key = p.pad_a * 10 + p.nt;
    switch (key) {
        case 641: return launch_sweep_t<T, 64, 1>(p, s);
        case 642: return launch_sweep_t<T, 64, 2>(p, s);
        case 1281: return launch_sweep_t<T, 128, 1>(p, s);
        case 1282: return launch_sweep_t<T, 128, 2>(p, s);
        case 2561: return launch_sweep_t<T, 256, 1>(p, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace la
}  // namespace ss
