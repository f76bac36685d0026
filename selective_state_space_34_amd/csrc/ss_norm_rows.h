// Rows of the norms in registers: eight-element pieces, sums over the threads of a row, 8-bit codes.
#pragma once

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

}  // namespace

}  // namespace ss
