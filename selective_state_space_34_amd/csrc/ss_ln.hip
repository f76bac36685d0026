// Layer norm with the residual's addition, its 8- and 4-bit outputs and its gradients, for gfx950.
//
//   r = x + res                  d = r - mean(r)      c = 1/sqrt(mean(d²) + eps)     n = d·c
//   y = n·w + b                  8 bits as the RMS norm's; 4 bits: e2m1 blocks of 32 columns
//   dx = dr + c·(w·dy - mean(w·dy) - n·mean(w·dy·n))      dw = Σ_rows dy·n      db = Σ_rows dy
//
// A row stays in its threads' registers from its one reading on, up to a width of 16384 forward and 8192 in the
// gradient: the mean, the sum of squares about it (so that a row far from 0 keeps its digits) and the result
// are three walks over registers.  (Beyond, 1024 threads leave a thread 128 registers, and some of the row and of
// the columns' sums is kept in scratch: of the gradient 20 to 45 up to 16384 and 112 to 204 above, in rows
// that are no multiple of 8 wide 81 to 163 and 307 to 487; forward, above 16384, 2 to 18 and 35 to 63.  bfloat16,
// 67 MB of rows, forward and gradient: 8192 wide 49 and 68 us, 16384 55 and 97, 32768 63 and 281, where
// scratch writes 335 MB.)  Memory
// bounds both directions: 16384 rows of 2560 bfloat16, r = x + res, 335 MB, 71 us (4.7 TB/s; a copy
// 5.06); gradient, with dr, 335 MB, 76 us (4.4 TB/s), 6 of them the sum of the workgroups' partial dw and db.
// One row takes 3.3 us, a launch's own time and two rounds of memory latency.
// Rows of odd widths start anywhere and end inside a piece: 26155 x 1471 76 us, gradient 102 (1472: 59 and
// 71; waves wait for memory 76 % of their time: pieces of a row that starts between lines touch one line more for
// every eight, and a wave's last pieces are read twice); 181 and 185 with the last elements one by one.
#include "ss_norm_rows.h"

namespace ss {

namespace {

// Rows whose width is a multiple of 8 (kWhole) end with a piece, which is in the row or not as a
// whole: it needs no element accesses, and no element of it has to be left out of a sum.
template <typename T, bool kWhole>
__device__ __forceinline__ Piece<T> take(const T* row, int64_t col, int64_t dim) {
    if constexpr (kWhole) {
        Piece<T> o;
        if (col < dim) o.load(row + col);
        else o.clear();
        return o;
    } else {
        return get8(row, col, dim);
    }
}
template <typename T, bool kWhole>
__device__ __forceinline__ void give(T* row, int64_t col, int64_t dim, const float (&v)[8]) {
    if constexpr (kWhole) {
        if (col < dim) put8(row, col, int64_t(1) << 40, v);
    } else {
        put8(row, col, dim, v);
    }
}
// Where the piece at col is taken from: other rows' last pieces are their last eight elements, and
// `twice` of those, the piece before has them too, are left out of the sums.  (A row's loads all come
// before the barrier of its first sum, and its stores behind it, so this holds in place as well.)
template <bool kWhole>
__device__ __forceinline__ Span place(int64_t col, int64_t dim) {
    if (!kWhole && dim >= 8 && col < dim && col + 8 > dim) return Span{dim - 8, int(col + 8 - dim)};
    return Span{col, 0};
}

// v less m in the elements of the piece at c that are the row's own, 0 in the others.
template <bool kWhole>
__device__ __forceinline__ float less(float v, float m, const Span& c, int e, int64_t dim) {
    if constexpr (kWhole) return v - m;          // (m is 0 for a piece behind the row's end)
    return e >= c.twice && c.at + e < dim ? v - m : 0.0f;
}

// Eight e2m1 codes of v / 2^(e - 127) and, with them, the exponent e of the block of 32 columns
// that four neighbouring lanes hold.
__device__ __forceinline__ uint32_t block_codes8(const float (&v)[8], int& e) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m = __float_as_uint(v[i]) & 0x7fffffffu;
        top = top > m ? top : m;
    }
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        const uint32_t o = uint32_t(__shfl_xor(int(top), m, 64));
        top = top > o ? top : o;
    }
    return mx4_codes8(v, top, e);
}

template <typename Tx, typename Tr, int P, int NV, bool kWhole>
__global__ __launch_bounds__(P > 256 ? P : 256) void ln_fwd_kernel(const LnLaunch p) {
    constexpr int kRowsWG = P >= 256 ? 1 : 256 / P;
    __shared__ float slots[64];
    RowSum<P> rs{slots};
    const int tid = threadIdx.x % P;
    const int64_t D = p.D, step = int64_t(gridDim.x) * kRowsWG;
    for (int64_t row = int64_t(blockIdx.x) * kRowsWG + threadIdx.x / P; row < p.M; row += step) {
        const Tx* x = static_cast<const Tx*>(p.x) + row * D;
        const Tr* res = static_cast<const Tr*>(p.res) + (p.res ? row * D : 0);
        Piece<Tx> px[NV];
        Piece<Tr> pr[NV];
        float v[NV][8], m = 0.0f, sq = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = place<kWhole>((int64_t(j) * P + tid) * 8, D);
            px[j] = take<Tx, kWhole>(x, c.at, D);
            if (p.res) pr[j] = take<Tr, kWhole>(res, c.at, D);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = place<kWhole>((int64_t(j) * P + tid) * 8, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = px[j].get(e);
            if (p.res) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] += pr[j].get(e);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) m += kWhole || e >= c.twice ? v[j][e] : 0.0f;
        }
        m = rs.sum(m) * p.inv_d;
        // (elements that two threads hold keep their value: both store them)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = place<kWhole>((int64_t(j) * P + tid) * 8, D);
            const float own = kWhole && c.at >= D ? 0.0f : m;
            if (p.res) give<Tr, kWhole>(static_cast<Tr*>(p.r) + row * D, c.at, D, v[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = less<kWhole>(v[j][e], own, c, e, D);
                sq = fmaf(d, d, sq);
                // (0 behind the row's end: -m·c there may be infinite, and has no part in the row's scale)
                v[j][e] = kWhole || c.at + e < D ? v[j][e] - own : 0.0f;
            }
        }
        sq = rs.sum(sq);
        const float c = rsqrtf(sq * p.inv_d + p.eps);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t at = place<kWhole>((int64_t(j) * P + tid) * 8, D).at;
            const Piece<float> w = take<float, kWhole>(p.w, at, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * c * w.get(e);
            if (p.b) {
                const Piece<float> b = take<float, kWhole>(p.b, at, D);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] += b.get(e);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // bit patterns of magnitudes order like the magnitudes, NaN above all
                const uint32_t u = __float_as_uint(v[j][e]) & 0x7fffffffu;
                top = top > u ? top : u;
            }
        }
        if (p.q8 == SS_Q8_NONE) {
            Tx* y = static_cast<Tx*>(p.y) + row * D;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                give<Tx, kWhole>(y, place<kWhole>((int64_t(j) * P + tid) * 8, D).at, D, v[j]);
        } else if (p.q8 == SS_Q4_MX) {
            // D is a multiple of 32: four lanes hold a block
            uint8_t* y = static_cast<uint8_t*>(p.y) + row * (D / 2);
            uint8_t* es = reinterpret_cast<uint8_t*>(p.y_scale) + row * (D / 32);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int64_t col = (int64_t(j) * P + tid) * 8;
                int e;
                const uint32_t q = block_codes8(v[j], e);
                if (col < D) {
                    *reinterpret_cast<uint32_t*>(y + col / 2) = q;
                    if (tid % 4 == 0) es[col / 32] = uint8_t(e);
                }
            }
        } else {
            const float amax = __uint_as_float(rs.max(top));
            const float full = p.q8 == SS_Q8_FP8 ? 448.0f : 127.0f;
            // below 1e-35 the reciprocal would leave float32: such a row is all zero codes
            const float inv = amax > 1e-35f ? full / amax : 0.0f;
            uint8_t* y = static_cast<uint8_t*>(p.y) + row * D;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int64_t col = place<kWhole>((int64_t(j) * P + tid) * 8, D).at;
                // a row that is not finite keeps NaN codes where e4m3 has them
                const uint2 q = codes8(v[j], amax != amax ? amax : inv, p.q8);
                if (col + 8 <= D) {
                    __builtin_memcpy(y + col, &q, 8);
                } else if (!kWhole && col < D) {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (col + e < D) y[col + e] = uint8_t((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
                }
            }
            if (tid == 0) p.y_scale[row] = amax / full;
        }
    }
}

// dx of each row; the workgroup's sums of dy·n and of dy over its rows go to part [gridDim.x, 2 D].
template <typename Tx, typename Tr, int P, int NV, bool kWhole>
__global__ __launch_bounds__(P > 256 ? P : 256) void ln_bwd_kernel(const LnLaunch p) {
    constexpr int kRowsWG = P >= 256 ? 1 : 256 / P;
    __shared__ float slots[96];
    __shared__ float fold[kRowsWG > 1 ? P * 8 : 1];
    RowSum<P> rs{slots};
    const int tid = threadIdx.x % P, sub = threadIdx.x / P;
    const int64_t D = p.D, step = int64_t(gridDim.x) * kRowsWG;
    float dw[2][NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[0][j][e] = dw[1][j][e] = 0.0f;
    for (int64_t row = int64_t(blockIdx.x) * kRowsWG + sub; row < p.M; row += step) {
        const Tr* rr = static_cast<const Tr*>(p.res) + row * D;
        const Tx* dyr = static_cast<const Tx*>(p.x) + row * D;
        Piece<Tr> r[NV], g[NV];
        Piece<Tx> dy[NV];
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = place<kWhole>((int64_t(j) * P + tid) * 8, D).at;
            r[j] = take<Tr, kWhole>(rr, col, D);
            dy[j] = take<Tx, kWhole>(dyr, col, D);
            if (p.dr) g[j] = take<Tr, kWhole>(static_cast<const Tr*>(p.dr) + row * D, col, D);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = place<kWhole>((int64_t(j) * P + tid) * 8, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) m += kWhole || e >= c.twice ? r[j].get(e) : 0.0f;
        }
        // sum and sum3 have slots of their own; the other's barrier lies between two uses of one
        rs.at = 0;
        m = rs.sum(m) * p.inv_d;
        float sq = 0.0f, dot = 0.0f, all = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = place<kWhole>((int64_t(j) * P + tid) * 8, D);
            const Piece<float> w = take<float, kWhole>(p.w, c.at, D);
            const float own = kWhole && c.at >= D ? 0.0f : m;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = less<kWhole>(r[j].get(e), own, c, e, D);
                float y = dy[j].get(e) * w.get(e);
                if (!kWhole) y = e >= c.twice && c.at + e < D ? y : 0.0f;
                sq = fmaf(d, d, sq);
                dot = fmaf(y, d, dot);
                all += y;
            }
        }
        rs.at = 1;
        rs.sum3(sq, dot, all);
        const float c = rsqrtf(sq * p.inv_d + p.eps);
        // c²·(dot/D) first meets one c, then n: c³ would leave float32 for rows of small size
        const float k = c * (c * (dot * p.inv_d)), mean_y = all * p.inv_d;
        Tr* dx = static_cast<Tr*>(p.r) + row * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span at = place<kWhole>((int64_t(j) * P + tid) * 8, D);
            const Piece<float> w = take<float, kWhole>(p.w, at.at, D);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = dy[j].get(e), n = (r[j].get(e) - m) * c;
                o[e] = fmaf(c, fmaf(w.get(e), y, -mean_y), -k * n);
                const float own = kWhole || e >= at.twice ? y : 0.0f;
                dw[0][j][e] = fmaf(own, n, dw[0][j][e]);
                dw[1][j][e] += own;
                if (p.dr) o[e] += g[j].get(e);
            }
            give<Tr, kWhole>(dx, at.at, D, o);
        }
    }
    float* part = p.part + int64_t(blockIdx.x) * 2 * D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = place<kWhole>((int64_t(j) * P + tid) * 8, D);
            if constexpr (kRowsWG > 1) {
                // the workgroup's row slots one after the other
                for (int s = 0; s < kRowsWG; ++s) {
                    __syncthreads();
                    if (sub == s)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            fold[e * P + tid] = (s ? fold[e * P + tid] : 0.0f) + dw[which][j][e];
                }
                __syncthreads();
                if (sub == 0)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[which][j][e] = fold[e * P + tid];
            }
            if (kRowsWG == 1 || sub == 0) {
                if (kWhole || c.twice == 0) {
                    give<float, kWhole>(part + which * D, c.at, D, dw[which][j]);
                } else {
#pragma unroll
                    for (int e = 1; e < 8; ++e)
                        if (e >= c.twice) part[which * D + c.at + e] = dw[which][j][e];
                }
            }
        }
    }
}

// dw and db: sums over the workgroups' partial sums [n, 2 D], 64 columns a workgroup, 16 groups of
// partials.  The first D columns are dw's, the others db's (nullable).
__global__ __launch_bounds__(1024) void ln_dw_kernel(const float* __restrict__ part,
                                                     float* __restrict__ dw,
                                                     float* __restrict__ db, int64_t D, int n) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int64_t col = int64_t(blockIdx.x) * 64 + lane;
    float v = 0.0f;
    if (col < 2 * D)
#pragma unroll 8
        for (int i = grp; i < n; i += 16) v += part[int64_t(i) * 2 * D + col];
    red[grp][lane] = v;
    __syncthreads();
    if (grp == 0 && col < 2 * D) {
        v = 0.0f;
#pragma unroll
        for (int g = 0; g < 16; ++g) v += red[g][lane];
        if (col < D) dw[col] = v;
        else if (db) db[col - D] = v;
    }
}

template <typename Tx, typename Tr, int P, int NV, bool kWhole>
hipError_t launch_t(const LnLaunch& p, bool backward, hipStream_t s) {
    const dim3 block(P > 256 ? P : 256), grid{unsigned(p.grid)};
    if (!backward)
        hipLaunchKernelGGL((ln_fwd_kernel<Tx, Tr, P, NV, kWhole>), grid, block, 0, s, p);
    else if constexpr (NV <= 2 || P == 1024)
        hipLaunchKernelGGL((ln_bwd_kernel<Tx, Tr, P, NV, kWhole>), grid, block, 0, s, p);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

// The shapes that make_ln_plan gives.
template <typename Tx, typename Tr, bool kWhole>
hipError_t launch_of(const LnLaunch& p, bool backward, hipStream_t s) {
    switch (p.threads * 10 + p.pieces) {
        case 81: return launch_t<Tx, Tr, 8, 1, kWhole>(p, backward, s);
        case 321: return launch_t<Tx, Tr, 32, 1, kWhole>(p, backward, s);
        case 641: return launch_t<Tx, Tr, 64, 1, kWhole>(p, backward, s);
        case 642: return launch_t<Tx, Tr, 64, 2, kWhole>(p, backward, s);
        case 643: return launch_t<Tx, Tr, 64, 3, kWhole>(p, backward, s);
        case 644: return launch_t<Tx, Tr, 64, 4, kWhole>(p, backward, s);
        case 645: return launch_t<Tx, Tr, 64, 5, kWhole>(p, backward, s);
        case 646: return launch_t<Tx, Tr, 64, 6, kWhole>(p, backward, s);
        case 2561: return launch_t<Tx, Tr, 256, 1, kWhole>(p, backward, s);
        case 3201: return launch_t<Tx, Tr, 320, 1, kWhole>(p, backward, s);
        case 3841: return launch_t<Tx, Tr, 384, 1, kWhole>(p, backward, s);
        case 5121: return launch_t<Tx, Tr, 512, 1, kWhole>(p, backward, s);
        case 5122: return launch_t<Tx, Tr, 512, 2, kWhole>(p, backward, s);
        case 10242: return launch_t<Tx, Tr, 1024, 2, kWhole>(p, backward, s);
        case 10244: return launch_t<Tx, Tr, 1024, 4, kWhole>(p, backward, s);
        default: return hipErrorInvalidValue;
    }
}

template <typename Tx, typename Tr>
hipError_t launch_shape(const LnLaunch& p, bool backward, hipStream_t s) {
    return p.D % 8 == 0 ? launch_of<Tx, Tr, true>(p, backward, s) : launch_of<Tx, Tr, false>(p, backward, s);
}

hipError_t launch(const LnLaunch& p, bool backward, hipStream_t s) {
    if (p.in_dtype == SS_F32) return launch_shape<float, float>(p, backward, s);
    return p.res_dtype == SS_F32 ? launch_shape<bf16_t, float>(p, backward, s)
                                 : launch_shape<bf16_t, bf16_t>(p, backward, s);
}

}  // namespace

hipError_t launch_ln_fwd(const LnLaunch& p, hipStream_t s) { return launch(p, false, s); }

hipError_t launch_ln_bwd(const LnLaunch& p, float* dw, float* db, hipStream_t s) {
    const hipError_t e = launch(p, true, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ln_dw_kernel, dim3(unsigned((2 * p.D + 63) / 64)), dim3(1024), 0, s, p.part, dw,
                       db, p.D, p.grid);
    return hipGetLastError();
}

}  // namespace ss
