// Linear attention with a decay for each head, beside the sweep (ss_la_sweep.h): the state
// carried across segments, the log decays' gradient, the sum of shared heads' gradients and
// the single-token step.
#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16_t round_bf16(float v) {
    union { __bf16 h; bf16_t b; } u;
    u.h = __bf16(v);
    return u.b;
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = round_bf16(v); }

// S_{s+1} = decay_s·S_s + U_s over the segments, element by element: state holds U and gets S.
// The next segment's load is in flight meanwhile; 7 us for 64 heads' 4 segments of 128 x 128.
__global__ __launch_bounds__(256) void la_carry_kernel(const LaCarries carries) {
    const LaCarry& p = carries.p[blockIdx.y];
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t bh = id / p.sz, x = id - bh * p.sz;
    if (bh >= p.BH) return;
    float s = 0.0f;
    if (p.first) s = p.first[bh * p.sz + (x / p.dC) * p.f_i + (x % p.dC) * p.f_j];
    float* st = p.state + bh * p.nseg * p.sz + x;
    const float* dec = p.decay + bh * p.nseg;
    const int step = p.reverse ? -1 : 1;
    int seg = p.reverse ? p.nseg - 1 : 0;
    float u = st[seg * p.sz];
    for (int i = 0; i < p.nseg - 1; ++i, seg += step) {
        const float next = i + 2 < p.nseg ? st[(seg + step) * p.sz] : 0.0f;
        st[seg * p.sz] = s;
        s = fmaf(dec[seg], s, u);
        u = next;
    }
    st[seg * p.sz] = s;
}

// Sum over the 256 threads of a workgroup; part: four doubles in LDS.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

// E at the segments' borders: <adjoint of the state, state> there, which is dg of the first
// token behind the border.  Border 0: dS_0 and S_0; border nseg: dS_T and S_T (0 where either is
// not given); between them the states that enter the segments from either side.  All loads of a
// thread are in flight at once; 8 us for 64 heads' 4 segments of 128 x 128.
__global__ __launch_bounds__(256) void la_border_kernel(const LaDecayGrad p) {
    __shared__ double part[4];
    const int64_t bh = blockIdx.x / p.borders;
    const int k = p.border0 + int(blockIdx.x - bh * p.borders);
    const int sz = int(p.dk * p.dv), tid = threadIdx.x;
    const float *r = p.ds0, *s = p.s0;
    int64_t at_r = bh, at_s = bh;
    if (k > 0 && k < p.nseg) {
        r = p.rev_state; at_r = bh * p.nseg + k - 1;
        s = p.fwd_state; at_s = bh * p.nseg + k;
    } else if (k > 0) {
        r = p.ds; s = p.s_final;
    }
    double v = 0.0;
    if (r && s) {
        r += at_r * sz; s += at_s * sz;
        for (int x0 = tid; x0 < sz; x0 += 16 * 256) {
            float a[16], c[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {       // all in flight; what is outside is not used
                const int x = min(x0 + i * 256, sz - 1);
                a[i] = s[x];
                c[i] = r[x];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v += x0 + i * 256 < sz ? double(a[i]) * double(c[i]) : 0.0;
        }
    }
    v = block_sum(v, part);
    if (tid == 0) p.border[bh * (p.nseg + 1) + k] = v;
}

// dg_t = Σ_{u>=t} (row_u - col_u) + E at the segment's end, u inside the segment.  A sum over the
// whole sequence would hold the rounding of every row and column sum behind t, which grows with
// the length and, summed again for one decay a head, is all that is left where dg is small; so
// each segment starts from the exact value at its end, and what it misses at its beginning,
// where the exact value is known too, is taken off in proportion to the way.  One workgroup a
// segment, 1024 tokens at a time from its end, in 64 bits.
__global__ __launch_bounds__(256) void la_decay_grad_kernel(const LaDecayGrad p) {
    __shared__ double part[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t bh = blockIdx.x / p.nseg, b = bh / p.H, h = bh - b * p.H;
    const int seg = int(blockIdx.x - bh * p.nseg);
    int64_t len = p.T;
    if (p.lengths) {
        len = p.lengths[b];
        len = len < 0 ? 0 : len > p.T ? p.T : len;
    }
    const int64_t lo = seg * p.seg_tokens;
    const int64_t hi = lo + p.seg_tokens < p.T ? lo + p.seg_tokens : p.T;
    const int64_t plane = p.B * p.H * p.T;
    auto diff = [&](int64_t t) {
        double x = 0.0;
        if (t < hi && t < len)
            for (int q = 0; q < p.tiles; ++q) {
                const int64_t at = q * plane + bh * p.T + t;
                x += p.row[at] - p.col[at];
            }
        return x;
    };
    double miss = 0.0, run = p.border[bh * (p.nseg + 1) + seg + 1], total = 0.0;
    for (int64_t t = lo + tid; t < hi; t += 256) miss += diff(t);
    miss = run + block_sum(miss, part) - p.border[bh * (p.nseg + 1) + seg];
    const double slope = miss / double(hi - lo);
    for (int64_t w = (hi - lo + 1023) / 1024 - 1; w >= 0; --w) {
        const int64_t t0 = lo + w * 1024 + tid * 4;
        double v[4];
#pragma unroll
        for (int i = 3; i >= 0; --i) v[i] = diff(t0 + i) + (i < 3 ? v[i + 1] : 0.0);
        double s = v[0];                          // suffix sum over the lanes behind this one
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double o = __shfl_down(s, m, 64);
            if (lane + m < 64) s += o;
        }
        const double wave_sum = __shfl(s, 0, 64);
        __syncthreads();
        if (lane == 0) part[wave] = wave_sum;
        __syncthreads();
        double behind = run + (s - v[0]), all = 0.0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q > wave) behind += part[q];
            all += part[q];
        }
        run += all;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + i;
            if (t >= hi) continue;
            const double dg = t < len ? v[i] + behind - slope * double(hi - t) : 0.0;
            if (p.decay_token) p.dg[(b * p.T + t) * p.H + h] = float(dg);
            else total += dg;
        }
    }
    if (!p.decay_token) {
        total = block_sum(total, part);
        if (tid == 0) p.head_part[blockIdx.x] = total;
    }
}

// One wave a head: the sums of its rows and segments.
__global__ __launch_bounds__(64) void la_head_sum_kernel(const LaDecayGrad p) {
    const int64_t h = blockIdx.x, n = p.B * p.nseg;
    double v = 0.0;
    for (int64_t x = threadIdx.x; x < n; x += 64) {
        const int64_t b = x / p.nseg, seg = x - b * p.nseg;
        v += p.head_part[(b * p.H + h) * p.nseg + seg];
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    if (threadIdx.x == 0) p.dg[h] = float(v);
}

template <typename T>
__global__ __launch_bounds__(256) void la_group_sum_kernel(const LaGroupSum p) {
    const int64_t step = int64_t(gridDim.x) * 256;
    for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < p.n; id += step) {   // (token, key head, i)
        const int64_t g = id / p.d, i = id - g * p.d;
        const float* q = p.part[blockIdx.y] + g * p.rep * p.d + i;
        float v = 0.0f;
        for (int64_t r = 0; r < p.rep; ++r) v += q[r * p.d];
        put(static_cast<T*>(p.out[blockIdx.y]) + id, v);
    }
}

// One token.  S ← e^g S + k vᵀ, o = α Sᵀ q: every element of the state is read and written
// once, and that traffic is all of the cost.  A workgroup takes CW·VW columns of one head's
// state: CW threads across them, 256 / CW row groups, each thread its rows in batches of kRows
// loads in flight.  Row groups meet in LDS for o.  B = 256, H = 40, 64 x 128: 145 us, 4.7 TB/s of
// the 5.1 that a copy reaches; B = 1, H = 16, 128 x 128, one round of loads' latency: 5.4 us.
template <typename T, int CW, int VW>
__global__ __launch_bounds__(256) void la_step_kernel(const LaStep p) {
    constexpr int RG = 256 / CW, kRows = 8;
    __shared__ float ql[256], kl[256];
    __shared__ float red[RG][CW * VW];
    const int tid = threadIdx.x, cw = tid % CW, rg = tid / CW;
    const int64_t slabs = (p.dv + CW * VW - 1) / (CW * VW);
    const int64_t bh = blockIdx.x / slabs, slab = blockIdx.x - bh * slabs;
    const int64_t b = bh / p.H, h = bh - b * p.H;
    const int64_t j = (slab * CW + cw) * VW;
    const bool on = j < p.dv;                       // VW divides dv
    const float* sp = p.s_in + bh * p.dk * p.dv + j;
    float* so = p.s_out + bh * p.dk * p.dv + j;
    auto row = [](const LaOperand& o, int64_t b, int64_t h) {
        return static_cast<const T*>(o.p) + b * o.sb + (h / o.rep) * o.sh;
    };
    if (tid < p.dk) {
        ql[tid] = p.scale * to_f32(row(p.q, b, h)[tid]);
        kl[tid] = to_f32(row(p.k, b, h)[tid]);
    }
    float v[VW], acc[VW];
#pragma unroll
    for (int c = 0; c < VW; ++c) {
        v[c] = on ? to_f32(row(p.v, b, h)[j + c]) : 0.0f;
        acc[c] = 0.0f;
    }
    float a = 1.0f;
    if (p.g) a = expf(p.g[p.decay_token ? bh : h]);
    __syncthreads();
    for (int64_t i0 = rg; i0 < p.dk; i0 += RG * kRows) {
        float s[kRows][VW];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t i = i0 + r * RG;
            if (!on || i >= p.dk) continue;
            if constexpr (VW == 4) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(sp + i * p.dv);
#pragma unroll
                for (int c = 0; c < VW; ++c) s[r][c] = x[c];
            } else {
                s[r][0] = sp[i * p.dv];
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t i = i0 + r * RG;
            if (!on || i >= p.dk) continue;
            const float kk = kl[i], qq = ql[i];
#pragma unroll
            for (int c = 0; c < VW; ++c) {
                s[r][c] = fmaf(a, s[r][c], kk * v[c]);
                acc[c] = fmaf(qq, s[r][c], acc[c]);
            }
            if constexpr (VW == 4) {
                *reinterpret_cast<f32x4*>(so + i * p.dv) = f32x4{s[r][0], s[r][1], s[r][2], s[r][3]};
            } else {
                so[i * p.dv] = s[r][0];
            }
        }
    }
#pragma unroll
    for (int c = 0; c < VW; ++c) red[rg][cw * VW + c] = acc[c];
    __syncthreads();
    if (tid < CW * VW) {
        const int64_t col = slab * CW * VW + tid;
        float o = 0.0f;
#pragma unroll
        for (int g = 0; g < RG; ++g) o += red[g][tid];
        if (col < p.dv) put(static_cast<T*>(p.o) + bh * p.dv + col, o);
    }
}

template <typename T, int CW, int VW>
hipError_t launch_step_slab(const LaStep& p, hipStream_t s) {
    const int64_t slabs = (p.dv + CW * VW - 1) / (CW * VW);
    const dim3 grid{unsigned(p.B * p.H * slabs)};
    hipLaunchKernelGGL((la_step_kernel<T, CW, VW>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_step_type(const LaStep& p, hipStream_t s) {
    if (p.columns == 128) return launch_step_slab<T, 32, 4>(p, s);
    return p.dv % 4 == 0 ? launch_step_slab<T, 8, 4>(p, s) : launch_step_slab<T, 32, 1>(p, s);
}

}  // namespace

hipError_t launch_la_carry(const LaCarries& p, hipStream_t s) {
    const dim3 grid{unsigned((p.p[0].BH * p.p[0].sz + 255) / 256), unsigned(p.n)};
    hipLaunchKernelGGL(la_carry_kernel, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_la_borders(const LaDecayGrad& p, hipStream_t s) {
    hipLaunchKernelGGL(la_border_kernel, dim3(unsigned(p.B * p.H * p.borders)), dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_la_decay_grad(const LaDecayGrad& p, hipStream_t s) {
    hipLaunchKernelGGL(la_decay_grad_kernel, dim3(unsigned(p.B * p.H * p.nseg)), dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.decay_token) return e;
    hipLaunchKernelGGL(la_head_sum_kernel, dim3(unsigned(p.H)), dim3(64), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_la_group_sum(int bf16, const LaGroupSum& p, hipStream_t s) {
    // a launch takes fewer than 2^32 threads: beyond 2^31 elements each takes several
    const int64_t need = (p.n + 255) / 256, most = int64_t(1) << 23;
    const dim3 grid{unsigned(need < most ? need : most), 2};
    if (bf16) hipLaunchKernelGGL(la_group_sum_kernel<bf16_t>, grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(la_group_sum_kernel<float>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_la_step(int bf16, const LaStep& p, hipStream_t s) {
    return bf16 ? launch_step_type<bf16_t>(p, s) : launch_step_type<float>(p, s);
}

}  // namespace ss
