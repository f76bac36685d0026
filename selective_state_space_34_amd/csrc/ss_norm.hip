// Root-mean-square norm with the residual's addition, its 8-bit output and its gradients, for
// gfx950.
//
//   r = x + res                      (kept unrounded for y; stored in the residual's type)
//   y = r·c·w,  c = 1/sqrt(mean(r²) + eps)
//   8 bits: scale = max|y| / top, codes = y·(top / max|y|), top 448 (e4m3) or 127 (int8)
//   dx = dr + c·(w·dy) - (r·c)·(c·(c·Σ(w·dy·r)/D))        dw = Σ_rows dy·r·c
//
// The work is traffic: every element is read once and written once, a row staying in registers
// between the sums and the result.  (Up to a width of 16384 forward and 8192 in the gradient, that
// is.  Beyond, 1024 threads leave a thread 128 registers, and some of the row is kept in scratch:
// 6 to 12 registers of the gradient up to 16384, above it 53 to 76 forward and 195 to 410 in the
// gradient.  bf16, 67 MB of rows, forward and gradient: width 8192 44 and 59 us, 16384 48 and 71,
// 32768 70 and 185.)  A row belongs to P threads (8 to 1024, by its length
// and by how many rows there are), eight consecutive elements of it to each thread at a time,
// NV such pieces a thread; sums meet by shuffles, across waves through LDS.  Workgroups take
// rows in turn, so that in the gradient the columns' sums stay in registers over a workgroup's
// rows; the sums of dw over workgroups are added by a second kernel in a fixed order.  w is
// read for every row (it stays in the CU's cache): holding it too would cost 8·NV registers
// and with them the waves that keep loads in flight.  All loads of a row are issued before the
// first is used, and kept as they lie until then: bf16, D = 2560, 16384 rows with a residual and
// 8-bit output 89 us became 57 (5.2 TB/s, the rate of a copy).  The gradient of the same rows
// takes 75 us and the sum of dw over workgroups 6; at 26155 rows of 1472, where 184 of a row's 256
// threads have work, 97 us for 308 MB.
#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight consecutive elements as they lie in memory; 16-byte accesses that need only the
// elements' alignment (rows of odd widths start anywhere).
template <typename T> struct Piece;
template <> struct Piece<bf16_t> {
    u32x4 w;
    __device__ __forceinline__ float get(int e) const {
        return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
    __device__ __forceinline__ void load(const bf16_t* p) { __builtin_memcpy(&w, p, 16); }
    __device__ __forceinline__ void clear() { w = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void set(int e, bf16_t v) { w[e / 2] |= uint32_t(v.bits) << (16 * (e & 1)); }
};
template <> struct Piece<float> {
    f32x4 v[2];
    __device__ __forceinline__ float get(int e) const { return v[e / 4][e & 3]; }
    __device__ __forceinline__ void load(const float* p) { __builtin_memcpy(&v, p, 32); }
    __device__ __forceinline__ void clear() { v[0] = v[1] = f32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void set(int e, float x) { v[e / 4][e & 3] = x; }
};

// The row's piece at col, zeros beyond the width.
template <typename T>
__device__ __forceinline__ Piece<T> get8(const T* row, int64_t col, int64_t dim) {
    Piece<T> o;
    if (col + 8 <= dim) {
        o.load(row + col);
        return o;
    }
    o.clear();
    if (col < dim) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (col + e < dim) o.set(e, row[col + e]);
    }
    return o;
}

__device__ __forceinline__ void put8(float* row, int64_t col, int64_t dim, const float (&v)[8]) {
    if (col + 8 <= dim) {
        __builtin_memcpy(row + col, v, 32);
    } else if (col < dim) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (col + e < dim) row[col + e] = v[e];
    }
}
__device__ __forceinline__ void put8(bf16_t* row, int64_t col, int64_t dim, const float (&v)[8]) {
    bf16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __bf16(v[e]);
    if (col + 8 <= dim) {
        __builtin_memcpy(row + col, &h, 16);
    } else if (col < dim) {
        __bf16* p = reinterpret_cast<__bf16*>(row);
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (col + e < dim) p[col + e] = h[e];
    }
}

// Where the piece at col is taken from.  A row that ends inside a piece would be read and written
// there element by element; where one wave holds a row, the last piece is the row's last eight
// elements instead, and `twice` of them, its neighbour's too, are left out of the sums.  (All
// loads of a wave come before its stores, so this holds in place as well; between waves it would
// not.)
struct Span {
    int64_t at;
    int twice;
};
template <int P>
__device__ __forceinline__ Span span_of(int64_t col, int64_t dim) {
    if (P <= 64 && dim >= 8 && col < dim && col + 8 > dim) return Span{dim - 8, int(col + 8 - dim)};
    return Span{col, 0};
}

// Eight codes of v·inv: e4m3 (round to nearest even; |v·inv| <= 448, so none overflows) or
// int8 in [-127, 127].
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv, int q8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = v[4 * i + e] * inv;
        if (q8 == SS_Q8_FP8) {
            int x = __builtin_amdgcn_cvt_pk_fp8_f32(a[0], a[1], 0, false);
            w[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(a[2], a[3], x, true));
        } else {
            w[i] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = int(rintf(fminf(fmaxf(a[e], -127.0f), 127.0f)));
                w[i] |= uint32_t(c & 255) << (8 * e);
            }
        }
    }
    return make_uint2(w[0], w[1]);
}

// Sums (or maxima of bit patterns) over the P threads of a row.  P > 64: one row a workgroup;
// two slots alternate so that one barrier a call is enough.
template <int P>
struct RowSum {
    float* slots;   // [2][32], LDS
    int at = 0;
    static constexpr int kLanes = P < 64 ? P : 64;
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) v += __shfl_xor(v, m, 64);
        if constexpr (P > 64) {
            float* s = slots + 32 * at;
            at ^= 1;
            if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int w = 0; w < P / 64; ++w) v += s[w];
        }
        return v;
    }
    __device__ __forceinline__ void sum2(float& a, float& b) {
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) {
            a += __shfl_xor(a, m, 64);
            b += __shfl_xor(b, m, 64);
        }
        if constexpr (P > 64) {
            float* s = slots + 32 * at;
            at ^= 1;
            if ((threadIdx.x & 63) == 0) {
                s[threadIdx.x >> 6] = a;
                s[16 + (threadIdx.x >> 6)] = b;
            }
            __syncthreads();
            a = b = 0.0f;
#pragma unroll
            for (int w = 0; w < P / 64; ++w) {
                a += s[w];
                b += s[16 + w];
            }
        }
    }
    // (slots: [2][48] where this is used)
    __device__ __forceinline__ void sum3(float& a, float& b, float& c) {
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) {
            a += __shfl_xor(a, m, 64);
            b += __shfl_xor(b, m, 64);
            c += __shfl_xor(c, m, 64);
        }
        if constexpr (P > 64) {
            float* s = slots + 48 * at;
            at ^= 1;
            if ((threadIdx.x & 63) == 0) {
                s[threadIdx.x >> 6] = a;
                s[16 + (threadIdx.x >> 6)] = b;
                s[32 + (threadIdx.x >> 6)] = c;
            }
            __syncthreads();
            a = b = c = 0.0f;
#pragma unroll
            for (int w = 0; w < P / 64; ++w) {
                a += s[w];
                b += s[16 + w];
                c += s[32 + w];
            }
        }
    }
    __device__ __forceinline__ uint32_t max(uint32_t v) {
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) {
            const uint32_t o = uint32_t(__shfl_xor(int(v), m, 64));
            v = v > o ? v : o;
        }
        if constexpr (P > 64) {
            uint32_t* s = reinterpret_cast<uint32_t*>(slots) + 32 * at;
            at ^= 1;
            if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
            __syncthreads();
            v = 0;
#pragma unroll
            for (int w = 0; w < P / 64; ++w) v = v > s[w] ? v : s[w];
        }
        return v;
    }
};

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

// Mean and deviation of a row of the layer norm: v less its mean; the columns behind the row's end
// stay out of the sums.
template <int P, int NV>
__device__ __forceinline__ void centre(RowSum<P>& rs, float (&v)[NV][8], int tid, int64_t D,
                                       float inv_d, float& sq) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
#pragma unroll
        for (int e = 0; e < 8; ++e) m += e >= c.twice ? v[j][e] : 0.0f;
    }
    m = rs.sum(m) * inv_d;
    sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
        const int n = int(c.at < D ? D - c.at : 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[j][e] -= m;
            const float x = e >= c.twice && e < n ? v[j][e] : 0.0f;
            sq = fmaf(x, x, sq);
        }
    }
}

template <typename Tx, typename Tr, int P, int NV, typename L>
__global__ __launch_bounds__(P > 256 ? P : 256) void rms_fwd_kernel(const L p) {
    constexpr int kRowsWG = P >= 256 ? 1 : 256 / P;
    constexpr bool kMean = std::is_same<L, LnLaunch>::value;
    __shared__ float slots[64];
    RowSum<P> rs{slots};
    const int tid = threadIdx.x % P;
    const int64_t D = p.D, step = int64_t(gridDim.x) * kRowsWG;
    for (int64_t row = int64_t(blockIdx.x) * kRowsWG + threadIdx.x / P; row < p.M; row += step) {
        const Tx* x = static_cast<const Tx*>(p.x) + row * D;
        const Tr* res = static_cast<const Tr*>(p.res) + (p.res ? row * D : 0);
        Piece<Tx> px[NV];
        Piece<Tr> pr[NV];
        float v[NV][8], sq = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
            px[j] = get8(x, c.at, D);
            if (p.res) pr[j] = get8(res, c.at, D);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = px[j].get(e);
            if (p.res) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] += pr[j].get(e);
                put8(static_cast<Tr*>(p.r) + row * D, c.at, D, v[j]);
            }
            if constexpr (!kMean) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = e >= c.twice ? v[j][e] : 0.0f;
                    sq = fmaf(x, x, sq);
                }
            }
        }
        if constexpr (kMean) centre<P, NV>(rs, v, tid, D, p.inv_d, sq);
        sq = rs.sum(sq);
        const float c = rsqrtf(sq * p.inv_d + p.eps);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t at = span_of<P>((int64_t(j) * P + tid) * 8, D).at;
            const Piece<float> w = get8(p.w, at, D);
            Piece<float> b;
            b.clear();
            if constexpr (kMean) {
                if (p.b) b = get8(p.b, at, D);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[j][e] = v[j][e] * c * w.get(e);
                if constexpr (kMean) v[j][e] += b.get(e);
                // bit patterns of magnitudes order like the magnitudes, NaN above all
                const uint32_t m = __float_as_uint(v[j][e]) & 0x7fffffffu;
                top = top > m ? top : m;
            }
        }
        if (p.q8 == SS_Q8_NONE) {
            Tx* y = static_cast<Tx*>(p.y) + row * D;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                put8(y, span_of<P>((int64_t(j) * P + tid) * 8, D).at, D, v[j]);
        } else if (kMean && p.q8 == SS_Q4_MX) {
            // D is a multiple of 32: four lanes hold a block, and none ends inside a piece
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
                const int64_t col = span_of<P>((int64_t(j) * P + tid) * 8, D).at;
                // a row that is not finite keeps NaN codes where e4m3 has them
                const uint2 q = codes8(v[j], amax != amax ? amax : inv, p.q8);
                if (col + 8 <= D) {
                    __builtin_memcpy(y + col, &q, 8);
                } else if (col < D) {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (col + e < D) y[col + e] = uint8_t((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
                }
            }
            if (tid == 0) p.y_scale[row] = amax / full;
        }
    }
}

// dx of each row; the workgroup's sum of dy·r·c over its rows goes to part [gridDim.x, D].
template <typename Tx, typename Tr, int P, int NV, typename L>
__global__ __launch_bounds__(P > 256 ? P : 256) void rms_bwd_kernel(const L p) {
    constexpr int kRowsWG = P >= 256 ? 1 : 256 / P;
    __shared__ float slots[64];
    __shared__ float fold[kRowsWG > 1 ? P * 8 : 1];
    RowSum<P> rs{slots};
    const int tid = threadIdx.x % P, sub = threadIdx.x / P;
    const int64_t D = p.D, step = int64_t(gridDim.x) * kRowsWG;
    float dw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    for (int64_t row = int64_t(blockIdx.x) * kRowsWG + sub; row < p.M; row += step) {
        const Tr* rr = static_cast<const Tr*>(p.res) + row * D;
        const Tx* dyr = static_cast<const Tx*>(p.x) + row * D;
        Piece<Tr> r[NV], g[NV];
        Piece<Tx> dy[NV];
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = span_of<P>((int64_t(j) * P + tid) * 8, D).at;
            r[j] = get8(rr, col, D);
            dy[j] = get8(dyr, col, D);
            if (p.dr) g[j] = get8(static_cast<const Tr*>(p.dr) + row * D, col, D);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
            const Piece<float> w = get8(p.w, c.at, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = e >= c.twice ? r[j].get(e) : 0.0f;
                sq = fmaf(x, x, sq);
                dot = fmaf(dy[j].get(e) * w.get(e), x, dot);
            }
        }
        rs.sum2(sq, dot);
        const float c = rsqrtf(sq * p.inv_d + p.eps);
        // c²·(dot/D) first meets one c, then c·x: c³ would leave float32 for rows whose size is
        // below 1e-13 or above 1e12, where each of these is of dx's own size or of 1
        const float k = c * (c * (dot * p.inv_d));
        Tr* dx = static_cast<Tr*>(p.r) + row * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span at = span_of<P>((int64_t(j) * P + tid) * 8, D);
            const Piece<float> w = get8(p.w, at.at, D);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = r[j].get(e), y = dy[j].get(e);
                const float n = x * c;
                o[e] = fmaf(c * w.get(e), y, -k * n);
                dw[j][e] = fmaf(y, e >= at.twice ? n : 0.0f, dw[j][e]);
                if (p.dr) o[e] += g[j].get(e);
            }
            put8(dx, at.at, D, o);
        }
    }
    float* part = p.part + int64_t(blockIdx.x) * D;
    auto put_own = [&](const Span& c, const float (&v)[8]) {
        if (c.twice == 0) {
            put8(part, c.at, D, v);
        } else {
#pragma unroll
            for (int e = 1; e < 8; ++e)
                if (e >= c.twice) part[c.at + e] = v[e];
        }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
        if constexpr (kRowsWG > 1) {
            // the workgroup's row slots one after the other
            for (int s = 0; s < kRowsWG; ++s) {
                __syncthreads();
                if (sub == s)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        fold[e * P + tid] = (s ? fold[e * P + tid] : 0.0f) + dw[j][e];
            }
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[j][e] = fold[e * P + tid];
                put_own(c, dw[j]);
            }
        } else {
            put_own(c, dw[j]);
        }
    }
}

// The layer norm's: dx of each row, and the workgroup's sums of dy·n (n = d·c) and of dy over its
// rows to part [gridDim.x, 2 D].
template <typename Tx, typename Tr, int P, int NV>
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
            const int64_t col = span_of<P>((int64_t(j) * P + tid) * 8, D).at;
            r[j] = get8(rr, col, D);
            dy[j] = get8(dyr, col, D);
            if (p.dr) g[j] = get8(static_cast<const Tr*>(p.dr) + row * D, col, D);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) m += e >= c.twice ? r[j].get(e) : 0.0f;
        }
        // (every thread is through the last row's sums before it comes here: sum3's barrier)
        rs.at = 0;
        m = rs.sum(m) * p.inv_d;
        float sq = 0.0f, dot = 0.0f, all = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
            const int n = int(c.at < D ? D - c.at : 0);
            const Piece<float> w = get8(p.w, c.at, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool own = e >= c.twice && e < n;
                const float x = own ? r[j].get(e) - m : 0.0f;
                const float y = own ? dy[j].get(e) * w.get(e) : 0.0f;
                sq = fmaf(x, x, sq);
                dot = fmaf(y, x, dot);
                all += y;
            }
        }
        rs.at = 1;
        rs.sum3(sq, dot, all);
        const float c = rsqrtf(sq * p.inv_d + p.eps);
        const float k = c * (c * (dot * p.inv_d)), mean_y = all * p.inv_d;
        Tr* dx = static_cast<Tr*>(p.r) + row * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span at = span_of<P>((int64_t(j) * P + tid) * 8, D);
            const Piece<float> w = get8(p.w, at.at, D);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = dy[j].get(e), n = (r[j].get(e) - m) * c;
                o[e] = fmaf(c, fmaf(w.get(e), y, -mean_y), -k * n);
                const float own = e >= at.twice ? y : 0.0f;
                dw[0][j][e] = fmaf(own, n, dw[0][j][e]);
                dw[1][j][e] += own;
                if (p.dr) o[e] += g[j].get(e);
            }
            put8(dx, at.at, D, o);
        }
    }
    float* part = p.part + int64_t(blockIdx.x) * 2 * D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Span c = span_of<P>((int64_t(j) * P + tid) * 8, D);
            if constexpr (kRowsWG > 1) {
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
                if (c.twice == 0) {
                    put8(part + which * D, c.at, D, dw[which][j]);
                } else {
#pragma unroll
                    for (int e = 1; e < 8; ++e)
                        if (e >= c.twice) part[which * D + c.at + e] = dw[which][j][e];
                }
            }
        }
    }
}

// dw = Σ over the workgroups' partial sums: 64 columns a workgroup, 16 groups of partials.
__global__ __launch_bounds__(1024) void rms_dw_kernel(const float* __restrict__ part,
                                                      float* __restrict__ dw, int64_t D, int n) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int64_t col = int64_t(blockIdx.x) * 64 + lane;
    float v = 0.0f;
    if (col < D)
#pragma unroll 8
        for (int i = grp; i < n; i += 16) v += part[int64_t(i) * D + col];
    red[grp][lane] = v;
    __syncthreads();
    if (grp == 0 && col < D) {
        v = 0.0f;
#pragma unroll
        for (int g = 0; g < 16; ++g) v += red[g][lane];
        dw[col] = v;
    }
}

// The same for [n, 2 D] of the layer norm: the first D columns are dw's, the others db's.
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

template <typename Tx, typename Tr, int P, int NV, typename L>
hipError_t launch_t(const L& p, bool backward, hipStream_t s) {
    const dim3 block(P > 256 ? P : 256), grid{unsigned(p.grid)};
    if (!backward) {
        hipLaunchKernelGGL((rms_fwd_kernel<Tx, Tr, P, NV, L>), grid, block, 0, s, p);
    } else if constexpr (NV < 6) {
        if constexpr (std::is_same<L, LnLaunch>::value)
            hipLaunchKernelGGL((ln_bwd_kernel<Tx, Tr, P, NV>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((rms_bwd_kernel<Tx, Tr, P, NV, L>), grid, block, 0, s, p);
    }
    return hipGetLastError();
}

template <typename Tx, typename Tr, typename L>
hipError_t launch_shape(const L& p, bool backward, hipStream_t s) {
    switch (p.threads * 10 + p.pieces) {
        case 81: return launch_t<Tx, Tr, 8, 1, L>(p, backward, s);
        case 321: return launch_t<Tx, Tr, 32, 1, L>(p, backward, s);
        case 641: return launch_t<Tx, Tr, 64, 1, L>(p, backward, s);
        case 642: return launch_t<Tx, Tr, 64, 2, L>(p, backward, s);
        case 646: return launch_t<Tx, Tr, 64, 6, L>(p, backward, s);
        case 2561: return launch_t<Tx, Tr, 256, 1, L>(p, backward, s);
        case 2562: return launch_t<Tx, Tr, 256, 2, L>(p, backward, s);
        case 5122: return launch_t<Tx, Tr, 512, 2, L>(p, backward, s);
        case 10242: return launch_t<Tx, Tr, 1024, 2, L>(p, backward, s);
        case 10244: return launch_t<Tx, Tr, 1024, 4, L>(p, backward, s);
        default: return hipErrorInvalidValue;
    }
}

template <typename L>
hipError_t launch(const L& p, bool backward, hipStream_t s) {
    if (p.in_dtype == SS_F32) return launch_shape<float, float, L>(p, backward, s);
    return p.res_dtype == SS_F32 ? launch_shape<bf16_t, float, L>(p, backward, s)
                                 : launch_shape<bf16_t, bf16_t, L>(p, backward, s);
}

}  // namespace

hipError_t launch_rms_fwd(const RmsLaunch& p, hipStream_t s) { return launch(p, false, s); }

hipError_t launch_rms_bwd(const RmsLaunch& p, float* dw, hipStream_t s) {
    hipError_t e = launch(p, true, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(rms_dw_kernel, dim3(unsigned((p.D + 63) / 64)), dim3(1024), 0, s, p.part, dw,
                       p.D, p.grid);
    return hipGetLastError();
}

hipError_t launch_ln_fwd(const LnLaunch& p, hipStream_t s) { return launch(p, false, s); }

hipError_t launch_ln_bwd(const LnLaunch& p, float* dw, float* db, hipStream_t s) {
    hipError_t e = launch(p, true, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ln_dw_kernel, dim3(unsigned((2 * p.D + 63) / 64)), dim3(1024), 0, s, p.part, dw,
                       db, p.D, p.grid);
    return hipGetLastError();
}

}  // namespace ss
