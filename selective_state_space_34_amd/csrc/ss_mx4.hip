// Microscaled 4-bit values for gfx950: rounding to them, and products with weights held in them.
//
//   value = e2m1(code)·2^(exponent - 127), one exponent for 32 consecutive columns
//   y[m, n] = Σ_k x[m, k]·w[n, k]        x the same, or e4m3 with a float32 scale for each row
//
// The matrix cores take both formats as they lie in memory: v_mfma_scale_f32_16x16x128_f8f6f4 reads
// 32 codes of a block (16 bytes) and the block's exponent from a lane, lane l row l % 16 and block
// l / 16 of the 128 columns; of e4m3 two runs of 16, at 16·(l / 16) and at 64 more.
#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// ---- rounding --------------------------------------------------------------------------------

// Eight elements a thread and turn, a block to four neighbouring lanes.
template <typename T>
__global__ __launch_bounds__(256) void mx4_quant_kernel(const Mx4Quant p) {
    const int64_t n = p.blocks * 4, step = int64_t(gridDim.x) * 256;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
        float v[8];
        load8(static_cast<const T*>(p.x) + i * 8, v);
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = __float_as_uint(v[e]) & 0x7fffffffu;
            top = top > m ? top : m;
        }
#pragma unroll
        for (int m = 1; m < 4; m <<= 1) {
            const uint32_t o = uint32_t(__shfl_xor(int(top), m, 64));
            top = top > o ? top : o;
        }
        int e;
        const uint32_t q = mx4_codes8(v, top, e);
        reinterpret_cast<uint32_t*>(p.codes)[i] = q;
        if (i % 4 == 0) p.exps[i / 4] = uint8_t(e);
    }
}

// ---- few rows --------------------------------------------------------------------------------

__device__ __forceinline__ void load16(i32x8& f, int at, const uint8_t* p) {
    const int4 w = *reinterpret_cast<const int4*>(p);
    f[at] = w.x; f[at + 1] = w.y; f[at + 2] = w.z; f[at + 3] = w.w;
}

// Eight e2m1 codes times 2^(e - 127) and four e4m3 values as bfloat16, exact (where the product is
// a normal number).
__device__ __forceinline__ bf16x8 widen4(uint32_t q, int e) {
    const float scale = __uint_as_float(uint32_t(e) << 23);
    union { bf16x2 h[4]; bf16x8 f; uint32_t w[4]; } o;
    o.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
    o.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
    o.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
    o.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = e == 255 ? 0x7fc07fc0u : o.w[i];
    return o.f;
}
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
    union { bf16x2 h[4]; bf16x8 f; } o;
    o.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    o.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    o.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    o.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return o.f;
}

// What x is: in 4 bits; e4m3; e4m3 where y is float32.  The matrix cores align the products of e4m3
// with one another before they add them, and lose what is below 2^-14 of the largest (against 64
// bits, random rows are 4.4e-6 off, at any K).  That is far below a bfloat16 result's own rounding;
// for a float32 result both operands go in as bfloat16, exactly (2.5e-8 off).
enum { kX4, kX8, kX8Wide };

// 16 rows of weights and 16·kTiles rows of x a workgroup; its waves take the columns, 128 at a time,
// in turn and meet in LDS.
template <int kTiles, int kX, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void mx4_rows_kernel(const Mx4Launch p) {
    __shared__ float red[kWaves][kTiles][64][4];
    constexpr bool kFp8 = kX != kX4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane & 15, g = lane >> 4;
    const int64_t K = p.K, kb = K / 32, n0 = int64_t(blockIdx.x) * 16;
    const int64_t m0 = int64_t(blockIdx.y) * 16 * kTiles;
    const int64_t wr = n0 + row < p.N ? n0 + row : p.N - 1;
    const uint8_t* w = p.wq + wr * (K / 2);
    const uint8_t* we = p.w_exps + wr * kb;
    const uint8_t* xs[kTiles];
    const uint8_t* xe[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int64_t m = m0 + 16 * t + row, mr = m < p.M ? m : p.M - 1;
        xs[t] = p.x + mr * (kFp8 ? K : K / 2);
        xe[t] = static_cast<const uint8_t*>(p.x_scale) + mr * kb;
    }
    f32x4 acc[kTiles] = {};
    for (int64_t k0 = int64_t(wave) * 128; k0 < K; k0 += kWaves * 128) {
        const int blocks = int(K - k0 < 128 ? (K - k0) / 32 : 4);
        i32x8 a = {};
        int sa = 127;
        if (g < blocks) {
            load16(a, 0, w + k0 / 2 + 16 * g);
            sa = we[k0 / 32 + g];
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            i32x8 b = {};
            int sb = 127;
            if constexpr (kX == kX8Wide) {
                if (g < blocks) {
                    load16(b, 0, xs[t] + k0 + 32 * g);
                    load16(b, 4, xs[t] + k0 + 32 * g + 16);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        widen4(uint32_t(a[q]), sa), widen8(uint32_t(b[2 * q]), uint32_t(b[2 * q + 1])),
                        acc[t], 0, 0, 0);
                continue;
            }
            if constexpr (kFp8) {
                if (g / 2 < blocks) load16(b, 0, xs[t] + k0 + 16 * g);
                if (2 + g / 2 < blocks) load16(b, 4, xs[t] + k0 + 64 + 16 * g);
            } else if (g < blocks) {
                load16(b, 0, xs[t] + k0 / 2 + 16 * g);
                sb = xe[t][k0 / 32 + g];
            }
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[t], 4, kFp8 ? 0 : 4,
                                                                      0, sa, 0, sb);
        }
        settle();   // the sums may change registers where the loop ends
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[wave][t][lane][j] = acc[t][j];
    __syncthreads();
    for (int o = threadIdx.x; o < kTiles * 256; o += 64 * kWaves) {
        // weights' row o % 16, x's row o / 16 of the workgroup's
        const int t = o >> 8, from = (o >> 4 & 15) + 16 * ((o & 15) >> 2), j = o & 3;
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < kWaves; ++s) v += red[s][t][from][j];
        const int64_t n = n0 + (o & 15), m = m0 + (o >> 4);
        if (n < p.N && m < p.M) {
            if constexpr (kFp8) v *= static_cast<const float*>(p.x_scale)[m];
            if (p.y_dtype == SS_F32) static_cast<float*>(p.y)[m * p.N + n] = v;
            else static_cast<__bf16*>(p.y)[m * p.N + n] = __bf16(v);
        }
    }
}

template <int kTiles, int kX>
hipError_t launch_rows(const Mx4Launch& p, hipStream_t s) {
    const dim3 grid(unsigned((p.N + 15) / 16), unsigned((p.M + 16 * kTiles - 1) / (16 * kTiles)));
    hipLaunchKernelGGL((mx4_rows_kernel<kTiles, kX, 8>), grid, dim3(512), 0, s, p);
    return hipGetLastError();
}

template <int kX>
hipError_t launch_mm(const Mx4Launch& p, hipStream_t s) {
    if (p.M <= 16) return launch_rows<1, kX>(p, s);
    if (p.M <= 32) return launch_rows<2, kX>(p, s);
    return launch_rows<4, kX>(p, s);
}

}  // namespace

hipError_t launch_mx4_quant(const Mx4Quant& p, hipStream_t s) {
    const int64_t need = (p.blocks * 4 + 255) / 256, most = 1 << 16;
    const dim3 grid(unsigned(need < most ? need : most));
    if (p.in_dtype == SS_BF16) hipLaunchKernelGGL(mx4_quant_kernel<bf16_t>, grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(mx4_quant_kernel<float>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_mx4_mm(const Mx4Launch& p, hipStream_t s) {
    if (!p.fp8) return launch_mm<kX4>(p, s);
    return p.y_dtype == SS_F32 ? launch_mm<kX8Wide>(p, s) : launch_mm<kX8>(p, s);
}

}  // namespace ss
