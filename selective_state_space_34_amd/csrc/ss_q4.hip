// Products of a few rows with 4-bit weights, for gfx950:
//   y[m, n] = xs[m]·Σ_k x[m, k]·s[n, k / G]·(u[n, k] - z[n, k / G])
// u the 4-bit codes of row n, two a byte, low half first; z 8 where no zeros are given; xs the
// rows' scales where x is in 8 bits, else 1.
//
// What bounds it is reading the codes, so they go from memory to the matrix cores with the
// fewest instructions.  A lane reads G/8 bytes of one row (16 rows a wave, the four 16-lane
// groups side by side: one group of G codes a row), and turns eight codes of 32 bits into the
// eight bf16 values of one v_mfma_f32_16x16x32_bf16 operand with four shifts and four
// and-ors: a code in the upper mantissa bits of 16.0 is exactly 16 + u.  The products of one
// group are summed on the matrix cores, Σ x of the group by one more product with ones, and
//   acc += s·(Σ x(16 + u) - (16 + z)·Σ x)
// in float32, so every scale is applied exactly.  The codes of a word come out in the order
// 0 4 1 5 2 6 3 7; x is put into LDS in that order, as bf16.  Float32 rows are three bf16 rows
// there (24 bits), which the products' unused rows hold for nothing; 8-bit rows are bf16
// exactly.  A workgroup's four waves take the groups of 16 rows in turn and meet in LDS.
#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int W> struct Words;
template <> struct Words<1> { using type = uint32_t; };
template <> struct Words<2> { using type = uint2; };
template <> struct Words<4> { using type = uint4; };

// eight codes of a word as 16 + u, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ bf16x8 widen(uint32_t d) {
    const uint32_t mask = 0x00780078u, one = 0x41804180u;
    union { uint32_t w[4]; bf16x8 f; } o;
    o.w[0] = ((d << 3) & mask) | one;
    o.w[1] = ((d >> 1) & mask) | one;
    o.w[2] = ((d >> 5) & mask) | one;
    o.w[3] = ((d >> 9) & mask) | one;
    return o.f;
}

// eight elements of x as float32
__device__ __forceinline__ void read8(const float* p, float (&o)[8]) { load8(p, o); }
__device__ __forceinline__ void read8(const bf16_t* p, float (&o)[8]) { load8(p, o); }
struct fp8_t { uint8_t b; };
struct int8_q { int8_t b; };
__device__ __forceinline__ void read8(const fp8_t* p, float (&o)[8]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int w = int(i ? v.y : v.x);
        o[4 * i] = __builtin_amdgcn_cvt_f32_fp8(w, 0);
        o[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1);
        o[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2);
        o[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3);
    }
}
__device__ __forceinline__ void read8(const int8_q* p, float (&o)[8]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = float(int8_t((e < 4 ? v.x : v.y) >> (8 * (e & 3))));
}

// W: 32-bit words of codes a lane reads of each group (G = 32·W codes).
template <typename Tx, int W>
__global__ __launch_bounds__(256) void q4_kernel(const Q4Launch p) {
    constexpr int G = 32 * W;
    constexpr int kTerms = sizeof(Tx) == 4 ? 3 : 1;  // bf16 rows of one row of x
    constexpr int kAhead = 4;                        // groups whose loads are in flight
    extern __shared__ __attribute__((aligned(16))) char lds[];
    __bf16* const xl = reinterpret_cast<__bf16*>(lds);
    __shared__ float red[4][16][17];
    using Word = typename Words<W>::type;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    const int64_t m0 = int64_t(blockIdx.y) * p.mb;
    const int rows = int(p.M - m0 < p.mb ? p.M - m0 : p.mb), xrows = rows * kTerms;
    const int64_t n = int64_t(blockIdx.x) * 16 + l16;
    const int64_t nr = n < p.N ? n : p.N - 1;        // rows behind the end repeat the last one
    const uint8_t* wq = p.wq + nr * (p.K / 2) + lg * 4 * W;
    const uint16_t* sc = p.scales + nr * p.groups;
    const uint8_t* zr = p.zeros ? p.zeros + nr * p.groups : nullptr;
    const int ld = int(p.slab) + 8;                  // rows of x in LDS start 4 banks apart
    const int xrow = (l16 < xrows ? l16 : xrows - 1) * ld + lg * 8 * W;

    f32x4 acc = {0, 0, 0, 0};
    for (int64_t k0 = 0; k0 < p.K; k0 += p.slab) {
        const int64_t kn = p.K - k0 < p.slab ? p.K - k0 : p.slab;
        const int64_t kpad = (kn + G - 1) / G * G;
        if (k0) __syncthreads();
        for (int64_t i = tid; i < rows * (kpad / 8); i += 256) {
            const int r = int(i / (kpad / 8));
            const int64_t k = (i - r * (kpad / 8)) * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            if (k < kn) read8(static_cast<const Tx*>(p.x) + (m0 + r) * p.K + k0 + k, v);
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
                bf16x8 o;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __bf16 h = __bf16(v[e]);
                    o[(e & 3) * 2 + (e >> 2)] = h;
                    // an infinite value is its first term alone
                    const float left = v[e] - float(h);
                    v[e] = left == left ? left : 0.0f;
                }
                *reinterpret_cast<bf16x8*>(&xl[(r * kTerms + t) * ld + k]) = o;
            }
        }
        __syncthreads();
        const int64_t g0 = k0 / G, gn = kpad / G;
        for (int64_t gb = wave; gb < gn; gb += 4 * kAhead) {
            Word d[kAhead];
            uint32_t s[kAhead], z[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int64_t g = gb + 4 * a;
                if (g >= gn) break;
                d[a] = Word{};
                // a short last group ends between lanes: 8·W codes divide 32, which divides K
                if (g * G + lg * 8 * W < kn) d[a] = *reinterpret_cast<const Word*>(wq + (k0 + g * G) / 2);
                s[a] = sc[g0 + g];
                z[a] = zr ? zr[g0 + g] : 8;
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int64_t g = gb + 4 * a;
                if (g >= gn) break;
                const uint32_t* q = reinterpret_cast<const uint32_t*>(&d[a]);
                f32x4 t = {0, 0, 0, 0}, u = {0, 0, 0, 0};
                bf16x8 ones;
#pragma unroll
                for (int e = 0; e < 8; ++e) ones[e] = __bf16(1.0f);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const bf16x8 xf = *reinterpret_cast<const bf16x8*>(&xl[xrow + g * G + 8 * i]);
                    t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, widen(q[i]), t, 0, 0, 0);
                    u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, ones, u, 0, 0, 0);
                }
                const float sf = __uint_as_float(s[a] << 16), zf = 16.0f + float(z[a]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = fmaf(sf, fmaf(-zf, u[r], t[r]), acc[r]);
            }
        }
    }
    // lane: column n = l16, rows 4·lg + r of x in LDS
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][4 * lg + r][l16] = acc[r];
    __syncthreads();
    const int m = tid >> 4, c = tid & 15;
    const int64_t col = int64_t(blockIdx.x) * 16 + c;
    if (m < rows && col < p.N) {
        float v = 0.0f;
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
#pragma unroll
            for (int w = 0; w < 4; ++w) v += red[w][m * kTerms + (kTerms - 1 - t)][c];
        if (p.x_scale) v *= p.x_scale[m0 + m];
        const int64_t at = (m0 + m) * p.N + col;
        if (p.y_dtype == SS_BF16) static_cast<__bf16*>(p.y)[at] = __bf16(v);
        else static_cast<float*>(p.y)[at] = v;
    }
}

template <typename Tx>
hipError_t launch_x(const Q4Launch& p, hipStream_t s) {
    const dim3 grid{unsigned((p.N + 15) / 16), unsigned((p.M + p.mb - 1) / p.mb)};
    const unsigned lds = unsigned(p.mb * (sizeof(Tx) == 4 ? 3 : 1) * (p.slab + 8) * 2);
    switch (p.group) {
        case 32: hipLaunchKernelGGL((q4_kernel<Tx, 1>), grid, dim3(256), lds, s, p); break;
        case 64: hipLaunchKernelGGL((q4_kernel<Tx, 2>), grid, dim3(256), lds, s, p); break;
        case 128: hipLaunchKernelGGL((q4_kernel<Tx, 4>), grid, dim3(256), lds, s, p); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_q4(const Q4Launch& p, hipStream_t s) {
    if (p.x_q8 == SS_Q8_FP8) return launch_x<fp8_t>(p, s);
    if (p.x_q8 == SS_Q8_INT8) return launch_x<int8_q>(p, s);
    return p.in_dtype == SS_BF16 ? launch_x<bf16_t>(p, s) : launch_x<float>(p, s);
}

}  // namespace ss
