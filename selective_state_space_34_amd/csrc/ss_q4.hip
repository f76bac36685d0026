// Products of a few rows with 4-bit weights, for gfx950:
//   y[m, n] = xs[m]·Σ_k x[m, k]·s[n, k / G]·(u[n, k] - z[n, k / G])
// u the 4-bit codes of row n, two a byte, low half first; z 8 where no zeros are given; xs the
// rows' scales where x is in 8 bits, else 1.
//
// What bounds it is reading the codes (a decode step's matrices are a few MB: mostly the time
// until the first of them arrive), so all loads of a wave are in flight at once and the codes go
// from registers to the matrix cores with the fewest instructions.  A lane reads G/8 bytes of
// one row (16 rows a wave, the four 16-lane groups side by side: one group of G codes a row),
// and turns eight codes of 32 bits into the eight bf16 values of one v_mfma_f32_16x16x32_bf16
// operand with four shifts and four and-ors: a code in the upper mantissa bits of 16.0 is
// exactly 16 + u.  The products of one group are summed on the matrix cores, Σ x of the group by
// one more product with ones, and
//   acc += s·(Σ x(16 + u) - (16 + z)·Σ x)
// in float32, so every scale is applied exactly.  The codes of a word come out in the order
// 0 4 1 5 2 6 3 7, and x, read by its lane straight from memory (each wave needs other k, so
// LDS would be a detour: with it 27 us at 16 x 5120 in 8 bits by 2560, without 11), is put
// into that order.  A float32 row takes three of the product's 16 rows, one for each bf16 term
// (exact: eight significant bits each); 8-bit values are bf16 exactly.  The waves of a workgroup
// take the groups of 16 rows in turn and meet in LDS.  Measured, bf16: 1 x 2560 by 10240 8.3 us
// (13.5 MB: 2.7 us at a copy's rate, the rest a launch, the first loads and the join), 1 x 8192 by
// 16384 24 us (2.9 TB/s).  Every 16 rows read and widen all weights again: 2560 by 10240 takes 11 us
// for 16 rows, 23 for 64, 76 for 256 and 292 for 1024, where a bf16 product of dense weights takes
// 14, 14, 29 and 51.
//
// The sum is formed from terms of up to (32 + z)/|u - z| of the result's own; against 64 bits, float32 x
// and y at K = 5120 are 1.5e-7 off (root mean square; a float32 product of dense weights 6.2e-7).
#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

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

// the same less by, exact where by is 16 and a zero
__device__ __forceinline__ bf16x8 less(bf16x8 f, float by) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __bf16(float(f[e]) - by);
    return f;
}

struct fp8_t { uint8_t b; };
struct int8_q { int8_t b; };

// eight values, exact in bf16, in the codes' order
__device__ __forceinline__ bf16x8 ordered(const float (&v)[8]) {
    bf16x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[(e & 3) * 2 + (e >> 2)] = __bf16(v[e]);
    return o;
}

// Eight elements of x as they lie in memory, and as an operand; term: which bf16 term of
// float32 values.  get: for finite values (others give values that are not finite); get_any: for
// any, as the product takes them.
template <typename T> struct Eight;
template <> struct Eight<bf16_t> {
    u32x4 w = {0, 0, 0, 0};
    __device__ __forceinline__ void load(const bf16_t* p) { w = *reinterpret_cast<const u32x4*>(p); }
    __device__ __forceinline__ bf16x8 get(int) const {
        union { uint32_t w[4]; bf16x8 f; } o;
        o.w[0] = __builtin_amdgcn_perm(w[2], w[0], 0x05040100u);
        o.w[1] = __builtin_amdgcn_perm(w[2], w[0], 0x07060302u);
        o.w[2] = __builtin_amdgcn_perm(w[3], w[1], 0x05040100u);
        o.w[3] = __builtin_amdgcn_perm(w[3], w[1], 0x07060302u);
        return o.f;
    }
    __device__ __forceinline__ bf16x8 get_any(int) const { return get(0); }
};
template <> struct Eight<fp8_t> {
    uint2 w = {0, 0};
    __device__ __forceinline__ void load(const fp8_t* p) { w = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ bf16x8 get(int) const {
        float v[8];
        v[0] = __builtin_amdgcn_cvt_f32_fp8(int(w.x), 0);
        v[1] = __builtin_amdgcn_cvt_f32_fp8(int(w.x), 1);
        v[2] = __builtin_amdgcn_cvt_f32_fp8(int(w.x), 2);
        v[3] = __builtin_amdgcn_cvt_f32_fp8(int(w.x), 3);
        v[4] = __builtin_amdgcn_cvt_f32_fp8(int(w.y), 0);
        v[5] = __builtin_amdgcn_cvt_f32_fp8(int(w.y), 1);
        v[6] = __builtin_amdgcn_cvt_f32_fp8(int(w.y), 2);
        v[7] = __builtin_amdgcn_cvt_f32_fp8(int(w.y), 3);
        return ordered(v);
    }
    __device__ __forceinline__ bf16x8 get_any(int) const { return get(0); }
};
template <> struct Eight<int8_q> {
    uint2 w = {0, 0};
    __device__ __forceinline__ void load(const int8_q* p) { w = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ bf16x8 get(int) const {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = float(int8_t((e < 4 ? w.x : w.y) >> (8 * (e & 3))));
        return ordered(v);
    }
    __device__ __forceinline__ bf16x8 get_any(int) const { return get(0); }
};
template <> struct Eight<float> {
    f32x4 v[2] = {};
    __device__ __forceinline__ void load(const float* p) {
        v[0] = *reinterpret_cast<const f32x4*>(p);
        v[1] = *reinterpret_cast<const f32x4*>(p + 4);
    }
    // the upper eight significant bits, the next eight of what is left, or the rest
    __device__ __forceinline__ uint32_t part(float a, int term) const {
        const uint32_t first = term >= 1 ? 0xffff0000u : 0u, second = term == 2 ? 0xffff0000u : 0u;
        a -= __uint_as_float(__float_as_uint(a) & first);
        a -= __uint_as_float(__float_as_uint(a) & second);
        return __float_as_uint(a);
    }
    __device__ __forceinline__ bf16x8 get(int term) const {
        union { uint32_t w[4]; bf16x8 f; } o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o.w[i] = __builtin_amdgcn_perm(part(v[1][i], term), part(v[0][i], term), 0x07060302u);
        return o.f;
    }
    // an infinity is its first term alone (what is left of it would be NaN), a NaN is one in each
    __device__ __forceinline__ bf16x8 get_any(int term) const {
        Eight<float> f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a = v[e / 4][e & 3];
            if (__builtin_isinf(a) && term > 0) a = 0.0f;
            if (a != a) a = __uint_as_float(0x7fc00000u);
            f.v[e / 4][e & 3] = a;
        }
        return f.get(term);
    }
};

// W: 32-bit words of codes a lane reads of each group (G = 32·W codes); NW: waves; NT: tiles of
// 16 rows of weights of a workgroup, which share what is done to x.
template <typename Tx, int W, int NW, int NT>
__global__ __launch_bounds__(64 * NW) void q4_kernel(const Q4Launch p) {
    constexpr int G = 32 * W;
    constexpr int kTerms = sizeof(Tx) == 4 ? 3 : 1;       // product rows of one row of x
    // groups whose loads are in flight, by the registers that one takes
    constexpr int kRegs = W * (NT + int(sizeof(Eight<Tx>)) / 4) + 2 * NT;
    constexpr int kAhead = 72 / kRegs < 2 ? 2 : 72 / kRegs > 6 ? 6 : 72 / kRegs;
    __shared__ float red[NW][16][16 * NT + 1];
    using Word = typename Words<W>::type;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, lg = lane >> 4;
    const int64_t m0 = int64_t(blockIdx.y) * p.mb;
    const int rows = int(p.M - m0 < p.mb ? p.M - m0 : p.mb);
    const int xm = l16 / kTerms, term = l16 - xm * kTerms;
    const bool has_x = xm < rows;                         // else a row of zeros
    const int64_t kl = lg * 8 * W;                        // the lane's first code of a group
    const uint8_t* wq[NT];
    const uint16_t* sc[NT];
    const uint8_t* zr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t n = int64_t(blockIdx.x) * 16 * NT + 16 * t + l16;
        const int64_t nr = n < p.N ? n : p.N - 1;         // rows behind the end repeat the last one
        wq[t] = p.wq + nr * (p.K / 2) + kl / 2;
        sc[t] = p.scales + nr * p.groups;
        zr[t] = p.zeros ? p.zeros + nr * p.groups : nullptr;
    }
    const Tx* xp = static_cast<const Tx*>(p.x) + (m0 + (has_x ? xm : 0)) * p.K + kl;
    bf16x8 ones;
#pragma unroll
    for (int e = 0; e < 8; ++e) ones[e] = __bf16(1.0f);

    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    Word d[kAhead][NT];
    Eight<Tx> x[kAhead][W];
    uint32_t s[kAhead][NT], z[kAhead][NT];
    auto load = [&](int a, int64_t g) {
        const int64_t k = g * G;
        // a short last group ends between lanes: 8·W codes divide 32, which divides K
        const bool on = k + kl < p.K;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            d[a][t] = Word{};
            if (on) d[a][t] = *reinterpret_cast<const Word*>(wq[t] + k / 2);
            s[a][t] = sc[t][g];
            z[a][t] = p.zeros ? zr[t][g] : 8;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            x[a][i] = Eight<Tx>{};
            if (on && has_x) x[a][i].load(xp + k + 8 * i);
        }
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
        if (wave + NW * a < p.groups) load(a, wave + NW * a);
    for (int64_t gb = wave; gb < p.groups; gb += NW * kAhead) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int64_t g = gb + NW * a;
            if (g >= p.groups) break;
            f32x4 v[NT], u = {0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < NT; ++t) v[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const bf16x8 xf = x[a][i].get(term);
                u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, ones, u, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t* q = reinterpret_cast<const uint32_t*>(&d[a][t]);
                    v[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, widen(q[i]), v[t], 0, 0, 0);
                }
            }
            // The sums before the next loads: between a product and the use of its result stands no
            // branch (see settle() in ss_device.h).
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float sf = __uint_as_float(s[a][t] << 16), zf = 16.0f + float(z[a][t]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(sf, fmaf(-zf, u[r], v[t][r]), acc[t][r]);
            }
            if (g + NW * kAhead < p.groups) load(a, g + NW * kAhead);
        }
    }
    // An infinity in x, or values whose sum with 16 added to the codes leaves float32, end in an acc
    // that is not finite and stays so: those are formed once more, from weights u - z themselves
    // (whole numbers of at most eight bits, exact in bf16).
    bool finite = true;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) finite = finite && __builtin_isfinite(acc[t][r]);
    if (__any(!finite)) {
        int own = lane;
        asm volatile("" : "+v"(own));   // nothing of what follows is kept in registers until here
        const int c16 = own & 15, m = c16 / kTerms, part = c16 - m * kTerms;
        const int64_t first = (own >> 4) * 8 * W;
        const Tx* xr = static_cast<const Tx*>(p.x) + (m0 + (m < rows ? m : 0)) * p.K + first;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t n = int64_t(blockIdx.x) * 16 * NT + 16 * t + c16, nr = n < p.N ? n : p.N - 1;
            f32x4 again = {0, 0, 0, 0};
#pragma unroll 1
            for (int64_t g = wave; g < p.groups; g += NW) {
                const bool on = g * G + first < p.K;
                Word code{};
                if (on) code = *reinterpret_cast<const Word*>(p.wq + nr * (p.K / 2) + (g * G + first) / 2);
                const uint32_t* q = reinterpret_cast<const uint32_t*>(&code);
                const float sf = __uint_as_float(uint32_t(p.scales[nr * p.groups + g]) << 16);
                const float zf = 16.0f + (p.zeros ? float(p.zeros[nr * p.groups + g]) : 8.0f);
                f32x4 v = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    Eight<Tx> e;
                    if (on && m < rows) e.load(xr + g * G + 8 * i);
                    v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e.get_any(part), less(widen(q[i]), zf), v, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) again[r] = fmaf(sf, v[r], again[r]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (!__builtin_isfinite(acc[t][r])) acc[t][r] = again[r];
        }
    }
    // lane: column l16 of each tile, product rows 4·lg + r
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][4 * lg + r][16 * t + l16] = acc[t][r];
    __syncthreads();
    for (int i = tid; i < rows * 16 * NT; i += 64 * NW) {
        const int m = i / (16 * NT), c = i % (16 * NT);
        const int64_t col = int64_t(blockIdx.x) * 16 * NT + c;
        if (col >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
#pragma unroll
            for (int w = 0; w < NW; ++w) v += red[w][m * kTerms + (kTerms - 1 - t)][c];
        if (p.x_scale) v *= p.x_scale[m0 + m];
        const int64_t at = (m0 + m) * p.N + col;
        if (p.y_dtype == SS_BF16) static_cast<__bf16*>(p.y)[at] = __bf16(v);
        else static_cast<float*>(p.y)[at] = v;
    }
}

template <typename Tx, int W, int NW, int NT>
hipError_t launch_tiles(const Q4Launch& p, hipStream_t s) {
    const dim3 grid{unsigned((p.N + 16 * NT - 1) / (16 * NT)), unsigned((p.M + p.mb - 1) / p.mb)};
    hipLaunchKernelGGL((q4_kernel<Tx, W, NW, NT>), grid, dim3(64 * NW), 0, s, p);
    return hipGetLastError();
}

template <typename Tx, int W>
hipError_t launch_words(const Q4Launch& p, hipStream_t s) {
    return p.tiles == 2 ? launch_tiles<Tx, W, 8, 2>(p, s) : launch_tiles<Tx, W, 8, 1>(p, s);
}

template <typename Tx>
hipError_t launch_x(const Q4Launch& p, hipStream_t s) {
    switch (p.group) {
        case 32: return launch_words<Tx, 1>(p, s);
        case 64: return launch_words<Tx, 2>(p, s);
        case 128: return launch_words<Tx, 4>(p, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_q4(const Q4Launch& p, hipStream_t s) {
    if (p.x_q8 == SS_Q8_FP8) return launch_x<fp8_t>(p, s);
    if (p.x_q8 == SS_Q8_INT8) return launch_x<int8_q>(p, s);
    return p.in_dtype == SS_BF16 ? launch_x<bf16_t>(p, s) : launch_x<float>(p, s);
}

}  // namespace ss
