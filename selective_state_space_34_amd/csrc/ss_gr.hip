// Gated linear recurrence of one number a channel, for gfx950: forward, gradients, single token.
//
//   log a_t = -c·softplus(lam)·σ(r_t)     s_t = sqrt(1 - a_t²)     v_t = σ(i_t)·x_t
//   h_t = a_t h_{t-1} + s_t v_t           y_t = h_t
// and with c_t = a_{t+1} g_{t+1} (dh_final behind the last token)
//   g_t = dy_t + c_t
//   dx = g s σ(i)      di = g s x σ(i)(1 - σ(i))
//   ∂/∂log a = g (a h_{t-1} - a²/s v)     dr = ∂/∂log a · log a·(1 - σ(r))
//   dlam = -c σ(lam) Σ ∂/∂log a · σ(r)
#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {

namespace {

constexpr int kCols = 128;     // channels of a workgroup, two a lane

// s² = 1 - a² = -(e^u - 1), u = 2 log a = 2 ln2·t2: the series of e^u - 1 for |u| < 1/4 (its rest is
// below 5e-8 of the sum), where the difference would lose the small ones' digits.
constexpr float kS1 = 1.3862943611198906f;    // (2 ln2)^n / n!
constexpr float kS2 = 0.9609060278364028f;
constexpr float kS3 = 0.4440328693185726f;
constexpr float kS4 = 0.15389006572205563f;
constexpr float kS5 = 0.04266738606857101f;
constexpr float kS6 = 0.009858259451764228f;
constexpr float kSSwitch = 0.18033688011112042f;   // |u| = 1/4 in units of t2

__device__ __forceinline__ float one_less_square(float t2, float a) {
    float p = fmaf(t2, kS6, kS5);
    p = fmaf(t2, p, kS4);
    p = fmaf(t2, p, kS3);
    p = fmaf(t2, p, kS2);
    p = fmaf(t2, p, kS1);
    return fabsf(t2) < kSSwitch ? -t2 * p : fmaf(-a, a, 1.0f);
}

// Two channels of a token as they lie in memory.  kVec: neighbours c0 + 2·lane + {0, 1}, one
// load; else c0 + lane and c0 + 64 + lane.  Channels behind the last one load that one's value.
template <typename T> struct Two;
template <> struct Two<float> {
    float a, b;
    __device__ __forceinline__ float get(int j) const { return j ? b : a; }
    template <bool kVec> __device__ __forceinline__ void load(const float* p, const int (&ch)[2]) {
        if constexpr (kVec) {
            const float2 v = *reinterpret_cast<const float2*>(p + ch[0]);
            a = v.x; b = v.y;
        } else {
            a = p[ch[0]]; b = p[ch[1]];
        }
    }
};
template <> struct Two<bf16_t> {
    uint32_t w;
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float(j ? w & 0xffff0000u : w << 16);
    }
    template <bool kVec> __device__ __forceinline__ void load(const bf16_t* p, const int (&ch)[2]) {
        if constexpr (kVec) w = *reinterpret_cast<const uint32_t*>(p + ch[0]);
        else w = uint32_t(p[ch[0]].bits) | uint32_t(p[ch[1]].bits) << 16;
    }
};

// What a lane knows of its two channels.
struct Cols {
    int load[2];         // clamped to the last channel
    bool on[2];
};
template <bool kVec>
__device__ __forceinline__ Cols columns(int64_t c0, int lane, int64_t D) {
    Cols c;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t ch = c0 + (kVec ? 2 * lane + j : lane + 64 * j);
        c.on[j] = ch < D;
        // with kVec D is even: a pair is in or out as a whole
        c.load[j] = int(ch < D ? ch : kVec ? D - 2 + j : D - 1);
    }
    return c;
}

template <bool kVec>
__device__ __forceinline__ void store2(float* row, const Cols& c, float a, float b) {
    if constexpr (kVec) {
        if (c.on[0]) *reinterpret_cast<float2*>(row + c.load[0]) = make_float2(a, b);
    } else {
        if (c.on[0]) row[c.load[0]] = a;
        if (c.on[1]) row[c.load[1]] = b;
    }
}
template <bool kVec>
__device__ __forceinline__ void store2(bf16_t* row, const Cols& c, float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 h;
    h[0] = __bf16(a); h[1] = __bf16(b);
    uint32_t w;
    __builtin_memcpy(&w, &h, 4);
    if constexpr (kVec) {
        if (c.on[0]) *reinterpret_cast<uint32_t*>(row + c.load[0]) = w;
    } else {
        if (c.on[0]) row[c.load[0]].bits = uint16_t(w);
        if (c.on[1]) row[c.load[1]].bits = uint16_t(w >> 16);
    }
}

// -c·softplus(lam) in units of log2
__device__ __forceinline__ float rate2(float lam, float c) { return -c * softplus(lam) * kLog2e; }

// Affine maps h -> A h + H of consecutive stretches, one after the other; an A of 0 cuts off what
// came before, NaN and infinities included.
__device__ __forceinline__ float through(float A, float H, float h) {
    return A == 0.0f ? H : fmaf(A, h, H);
}

// Which of the kS tokens from t0 on begin a document: bit s for token t0 + s.
template <int kS>
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* reset, int64_t b, int64_t T,
                                               int64_t t0, int lane) {
    if (!reset) return 0;
    bool set = false;
    if (lane < kS && t0 + lane < T) set = reset[b * T + t0 + lane] != 0;
    return uint32_t(__ballot(set));
}

__device__ __forceinline__ int64_t live_tokens(const int32_t* lengths, int64_t b, int64_t T) {
    if (!lengths) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < T ? n : T;
}

// ---- forward ---------------------------------------------------------------------------------

template <typename T, bool kVec, int kWaves, int kS>
__global__ __launch_bounds__(64 * kWaves) void gr_fwd_kernel(const GrLaunch p) {
    __shared__ float sh[2][2][kWaves][kCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.y, D = p.D;
    const Cols col = columns<kVec>(int64_t(blockIdx.x) * kCols, lane, D);
    const T* x = static_cast<const T*>(p.x.p) + b * p.x.sb;
    const T* r = static_cast<const T*>(p.r.p) + b * p.r.sb;
    const T* g = static_cast<const T*>(p.i.p) + b * p.i.sb;
    const int64_t live = live_tokens(p.lengths, b, p.T);
    float k2[2], h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        k2[j] = rate2(p.lam[col.load[j]], p.c);
        h[j] = p.h0 ? p.h0[b * D + col.load[j]] : 0.0f;
    }
    int slot = 0;
    for (int64_t tile = 0; tile < p.T; tile += kWaves * kS, slot ^= 1) {
        const int64_t t0 = tile + wave * kS;
        Two<T> wx[kS], wr[kS], wi[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const int64_t t = t0 + s < p.T ? t0 + s : p.T - 1;
            wx[s].template load<kVec>(x + t * p.x.st, col.load);
            wr[s].template load<kVec>(r + t * p.r.st, col.load);
            wi[s].template load<kVec>(g + t * p.i.st, col.load);
        }
        const uint32_t first = reset_bits<kS>(p.reset, b, p.T, t0, lane);
        float a[kS][2], u[kS][2], A[2] = {1.0f, 1.0f}, H[2] = {0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const bool cut = first >> s & 1, on = t0 + s < live;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float t2 = k2[j] * sigmoid(wr[s].get(j));
                const float e = exp2_hw(t2);
                const float q = __builtin_amdgcn_sqrtf(one_less_square(t2, e));
                const float v = sigmoid(wi[s].get(j)) * wx[s].get(j);
                a[s][j] = !on ? 1.0f : cut ? 0.0f : e;
                u[s][j] = !on ? 0.0f : cut ? v : q * v;
                H[j] = through(a[s][j], u[s][j], H[j]);
                A[j] *= a[s][j];
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sh[slot][0][wave][lane + 64 * j] = A[j];
            sh[slot][1][wave][lane + 64 * j] = H[j];
        }
        __syncthreads();
        float in[2] = {h[0], h[1]};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (w == wave) in[j] = h[j];
                h[j] = through(sh[slot][0][w][lane + 64 * j], sh[slot][1][w][lane + 64 * j], h[j]);
            }
        }
        if (p.h_ckpt && t0 % SS_GR_CKPT == 0 && t0 < p.T) {
            const int64_t n = (p.T + SS_GR_CKPT - 1) / SS_GR_CKPT;
            store2<kVec>(p.h_ckpt + (b * n + t0 / SS_GR_CKPT) * D, col, in[0], in[1]);
        }
        if (p.y) {
            T* y = static_cast<T*>(p.y) + b * p.T * D;
#pragma unroll
            for (int s = 0; s < kS; ++s) {
#pragma unroll
                for (int j = 0; j < 2; ++j) in[j] = through(a[s][j], u[s][j], in[j]);
                const bool on = t0 + s < live;
                if (t0 + s < p.T)
                    store2<kVec>(y + (t0 + s) * D, col, on ? in[0] : 0.0f, on ? in[1] : 0.0f);
            }
        }
    }
    if (p.h_final && wave == 0) store2<kVec>(p.h_final + b * D, col, h[0], h[1]);
}

// ---- backward --------------------------------------------------------------------------------

// The states before a wave's tokens come from the checkpoint that its workgroup's tile starts
// with; the adjoint c comes from the right.
template <typename T, bool kVec, int kWaves, int kS>
__global__ __launch_bounds__(64 * kWaves) void gr_bwd_kernel(const GrLaunch p) {
    static_assert(kWaves * kS == SS_GR_CKPT, "a tile is what one checkpoint starts");
    __shared__ float sh[2][3][kWaves][kCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.y, D = p.D, n = (p.T + SS_GR_CKPT - 1) / SS_GR_CKPT;
    const Cols col = columns<kVec>(int64_t(blockIdx.x) * kCols, lane, D);
    const T* x = static_cast<const T*>(p.x.p) + b * p.x.sb;
    const T* r = static_cast<const T*>(p.r.p) + b * p.r.sb;
    const T* g = static_cast<const T*>(p.i.p) + b * p.i.sb;
    const T* dy = static_cast<const T*>(p.dy) + b * p.T * D;
    T* dx = static_cast<T*>(p.dx) + b * p.T * D;
    T* dr = static_cast<T*>(p.dr) + b * p.T * D;
    T* di = static_cast<T*>(p.di) + b * p.T * D;
    const int64_t live = live_tokens(p.lengths, b, p.T);
    float k2[2], c[2], dl[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        k2[j] = rate2(p.lam[col.load[j]], p.c);
        c[j] = p.dh_final ? p.dh_final[b * D + col.load[j]] : 0.0f;
    }
    int slot = 0;
    for (int64_t tile = n - 1; tile >= 0; --tile, slot ^= 1) {
        const int64_t t0 = tile * SS_GR_CKPT + wave * kS;
        Two<T> wx[kS], wr[kS], wi[kS], wd[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const int64_t t = t0 + s < p.T ? t0 + s : p.T - 1;
            wx[s].template load<kVec>(x + t * p.x.st, col.load);
            wr[s].template load<kVec>(r + t * p.r.st, col.load);
            wi[s].template load<kVec>(g + t * p.i.st, col.load);
            wd[s].template load<kVec>(dy + t * D, col.load);
        }
        float hin[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) hin[j] = p.h_ckpt[(b * n + tile) * D + col.load[j]];
        const uint32_t first = reset_bits<kS>(p.reset, b, p.T, t0, lane);
        float a[kS][2], q[kS][2], sr[kS][2], si[kS][2];
        float A[2] = {1.0f, 1.0f}, H[2] = {0.0f, 0.0f}, G[2] = {0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const bool cut = first >> s & 1, on = t0 + s < live;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sr[s][j] = sigmoid(wr[s].get(j));
                si[s][j] = on ? sigmoid(wi[s].get(j)) : 0.0f;
                const float t2 = k2[j] * sr[s][j];
                const float e = exp2_hw(t2);
                a[s][j] = !on ? 1.0f : cut ? 0.0f : e;
                q[s][j] = !on ? 0.0f : cut ? 1.0f : __builtin_amdgcn_sqrtf(one_less_square(t2, e));
                const float v = on ? si[s][j] * wx[s].get(j) : 0.0f;
                H[j] = through(a[s][j], q[s][j] * v, H[j]);
                A[j] *= a[s][j];
            }
        }
#pragma unroll
        for (int s = kS - 1; s >= 0; --s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float d = (t0 + s < live ? wd[s].get(j) : 0.0f) + G[j];
                G[j] = a[s][j] == 0.0f ? 0.0f : a[s][j] * d;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sh[slot][0][wave][lane + 64 * j] = A[j];
            sh[slot][1][wave][lane + 64 * j] = H[j];
            sh[slot][2][wave][lane + 64 * j] = G[j];
        }
        __syncthreads();
        float cin[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float hh = hin[j];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (w == wave) hin[j] = hh;
                hh = through(sh[slot][0][w][lane + 64 * j], sh[slot][1][w][lane + 64 * j], hh);
            }
#pragma unroll
            for (int w = kWaves - 1; w >= 0; --w) {
                if (w == wave) cin[j] = c[j];
                c[j] = through(sh[slot][0][w][lane + 64 * j], sh[slot][2][w][lane + 64 * j], c[j]);
            }
        }
        float before[kS][2];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                before[s][j] = hin[j];
                const float v = t0 + s < live ? si[s][j] * wx[s].get(j) : 0.0f;
                hin[j] = through(a[s][j], q[s][j] * v, hin[j]);
            }
        }
#pragma unroll
        for (int s = kS - 1; s >= 0; --s) {
            const bool cut = first >> s & 1, on = t0 + s < live;
            float ox[2], orr[2], oi[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float as = a[s][j], qs = q[s][j], xv = wx[s].get(j);
                const float gt = (on ? wd[s].get(j) : 0.0f) + cin[j];
                cin[j] = as == 0.0f ? 0.0f : as * gt;
                const float gs = gt * qs;
                ox[j] = on ? gs * si[s][j] : 0.0f;
                oi[j] = on ? gs * xv * si[s][j] * (1.0f - si[s][j]) : 0.0f;
                // below 1e-15 the root's slope would leave float32; its share is below 1e-15 too
                const float slope = qs > 1e-15f ? as * rcp_hw(qs) : 0.0f;
                const float v = si[s][j] * xv;
                const float dla = on && !cut ? gt * as * fmaf(-slope, v, before[s][j]) : 0.0f;
                orr[j] = dla * (k2[j] * kLn2) * sr[s][j] * (1.0f - sr[s][j]);
                if (!on || cut) orr[j] = 0.0f;
                else dl[j] = fmaf(dla, sr[s][j], dl[j]);
            }
            if (t0 + s < p.T) {
                store2<kVec>(dx + (t0 + s) * D, col, ox[0], ox[1]);
                store2<kVec>(dr + (t0 + s) * D, col, orr[0], orr[1]);
                store2<kVec>(di + (t0 + s) * D, col, oi[0], oi[1]);
            }
        }
    }
    if (p.dh0 && wave == 0) store2<kVec>(p.dh0 + b * D, col, c[0], c[1]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) sh[0][0][wave][lane + 64 * j] = dl[j];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
#pragma unroll
            for (int j = 0; j < 2; ++j) dl[j] += sh[0][0][w][lane + 64 * j];
        store2<kVec>(p.part + b * D, col, dl[0], dl[1]);
    }
}

// dlam = -c·σ(lam)·Σ over the partial sums: 64 columns a workgroup, 16 groups of partials.
__global__ __launch_bounds__(1024) void gr_dlam_kernel(const float* __restrict__ part,
                                                       const float* __restrict__ lam,
                                                       float* __restrict__ dlam, float c, int64_t D,
                                                       int64_t n) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int64_t col = int64_t(blockIdx.x) * 64 + lane;
    float v = 0.0f;
    if (col < D)
#pragma unroll 8
        for (int64_t i = grp; i < n; i += 16) v += part[i * D + col];
    red[grp][lane] = v;
    __syncthreads();
    if (grp == 0 && col < D) {
        v = 0.0f;
#pragma unroll
        for (int g = 0; g < 16; ++g) v += red[g][lane];
        dlam[col] = -c * sigmoid(lam[col]) * v;
    }
}

// ---- one token -------------------------------------------------------------------------------

template <typename T, bool kVec>
__global__ __launch_bounds__(256) void gr_step_kernel(const GrStep p) {
    const int lane = threadIdx.x & 63;
    const int64_t b = int64_t(blockIdx.y) * 4 + (threadIdx.x >> 6), D = p.D;
    if (b >= p.B) return;
    const Cols col = columns<kVec>(int64_t(blockIdx.x) * kCols, lane, D);
    Two<T> x, r, i;
    x.template load<kVec>(static_cast<const T*>(p.x.p) + b * p.x.sb, col.load);
    r.template load<kVec>(static_cast<const T*>(p.r.p) + b * p.r.sb, col.load);
    i.template load<kVec>(static_cast<const T*>(p.i.p) + b * p.i.sb, col.load);
    float h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float t2 = rate2(p.lam[col.load[j]], p.c) * sigmoid(r.get(j));
        const float a = exp2_hw(t2);
        const float q = __builtin_amdgcn_sqrtf(one_less_square(t2, a));
        h[j] = fmaf(a, p.h_in[b * D + col.load[j]], q * (sigmoid(i.get(j)) * x.get(j)));
    }
    store2<kVec>(p.h_out + b * D, col, h[0], h[1]);
    store2<kVec>(static_cast<T*>(p.y) + b * D, col, h[0], h[1]);
}

template <typename F>
hipError_t with_type(int in_dtype, int vec, F&& f) {
    if (in_dtype == SS_BF16) return vec ? f(bf16_t{}, std::true_type{}) : f(bf16_t{}, std::false_type{});
    return vec ? f(0.0f, std::true_type{}) : f(0.0f, std::false_type{});
}

unsigned groups(int64_t D) { return unsigned((D + kCols - 1) / kCols); }

}  // namespace

hipError_t launch_gr_fwd(const GrLaunch& p, hipStream_t s) {
    return with_type(p.in_dtype, p.vec, [&](auto t, auto v) {
        hipLaunchKernelGGL((gr_fwd_kernel<decltype(t), decltype(v)::value, 8, 16>),
                           dim3(groups(p.D), unsigned(p.B)), dim3(512), 0, s, p);
        return hipGetLastError();
    });
}

hipError_t launch_gr_bwd(const GrLaunch& p, hipStream_t s) {
    const hipError_t e = with_type(p.in_dtype, p.vec, [&](auto t, auto v) {
        hipLaunchKernelGGL((gr_bwd_kernel<decltype(t), decltype(v)::value, 8, 8>),
                           dim3(groups(p.D), unsigned(p.B)), dim3(512), 0, s, p);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gr_dlam_kernel, dim3(unsigned((p.D + 63) / 64)), dim3(1024), 0, s, p.part,
                       p.lam, p.dlam, p.c, p.D, p.B);
    return hipGetLastError();
}

hipError_t launch_gr_step(const GrStep& p, hipStream_t s) {
    return with_type(p.in_dtype, p.vec, [&](auto t, auto v) {
        hipLaunchKernelGGL((gr_step_kernel<decltype(t), decltype(v)::value>),
                           dim3(groups(p.D), unsigned((p.B + 3) / 4)), dim3(256), 0, s, p);
        return hipGetLastError();
    });
}

}  // namespace ss
