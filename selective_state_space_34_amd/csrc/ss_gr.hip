// Gated linear recurrence of one number a channel, for gfx950: forward, gradients, single token.
//
//   log a_t = -c·softplus(lam)·σ(r_t)     s_t = sqrt(1 - a_t²)     v_t = σ(i_t)·x_t
//   h_t = a_t h_{t-1} + s_t v_t           y_t = h_t
// and with c_t = a_{t+1} g_{t+1} (dh_final behind the last token)
//   g_t = dy_t + c_t
//   dx = g s σ(i)      di = g s x σ(i)(1 - σ(i))
//   ∂/∂log a = g (a h_{t-1} - a²/s v)     dr = ∂/∂log a · log a·(1 - σ(r))
//   dlam = -c σ(lam) Σ ∂/∂log a · σ(r)
//
// Everything is read once and written once: a workgroup's tile stays in registers while it waits for
// the state that enters it ("states from tile to tile" below).  Bound by memory, then by the vector
// ALUs (37 instructions an element, six of them transcendental; the gradient 78, nine): bfloat16, forward
// 8 x 2048 x 5120, 671 MB, 148 us (4.6 TB/s; a copy 5.06), 4 x 4096 x 2048 with documents, forward 268 MB in
// 78 us, gradient 470 MB in 131 (3.6 TB/s, ALUs 58 % busy), 10 of them the words' launch and dlam's sums.
// A long sequence of few channels waits for its chain, a link for each group of 32 tiles: 1 x 262144 x 256, 537 MB,
// 151 us (3.6 TB/s; waves wait 57 % of their time, of the prompts' 43), gradient 288, of 128 channels 181,
// 1.4 us for each of 128 links; dlam's 4096 rows of partial sums take 20 us of it on four workgroups.
// Tiles: forward 8 waves of 16 tokens (of 8 tokens, one and a half times the waves in flight:
// 169 and 191 us for the first two); gradient 8 of 8, a checkpoint's 64.  Workgroups that took one tile
// after the other and asked for the next one's number ahead needed more registers: 165 to 185 us.
#include "ss_device.h"
#include "ss_gr_plan.h"
#include "ss_kernels.h"

#include <algorithm>
#include <cfloat>

namespace ss {

namespace {

constexpr int kCols = 128;     // channels of a workgroup, two a lane

// s² = 1 - a² = -(e^u - 1), u = 2 log a = 2 ln2·t2: the series of e^u - 1 for |u| < 1/4 (its rest is
// below 6e-8 of the sum), where the difference would lose the small ones' digits.
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

// σ(x) and 1 - σ(x), each relative to itself (a subtraction from 1 would lose the digits of an open gate's
// rest), in one number: the smaller of the two, with a minus where it is the rest.  (Of a rest at least
// 2^-126 stays, so that the sign does.)  What is left above a number's floor unfolds it.  s: σ(x).
__device__ __forceinline__ float folded(float x, float& s) {
    const float e = exp2_hw(-x * kLog2e);
    s = rcp_hw(1.0f + e);
    return x < 0.0f ? s : fmaf(-e, s, -0x1p-126f);
}
__device__ __forceinline__ float gate_of(float f) { return __builtin_amdgcn_fractf(f); }
__device__ __forceinline__ float rest_of(float f) { return __builtin_amdgcn_fractf(-f); }

// Two channels of a token as they lie in memory, through a buffer descriptor over a wave's rows:
// what lies behind the last token loads as 0 and is not stored.  kVec: neighbours c0 + 2·lane +
// {0, 1}, one access, which needs the elements' alignment only (8 x 2048 x 2561, bfloat16: 121 us, gradient
// 219, with two accesses, 96 and 183 so).  2: the number of channels is odd; the lane of the last one
// loads it as the second of a pair.  0 (a single channel): c0 + lane and c0 + 64 + lane.
constexpr int kRsrcFlags = 0x00020000;   // raw buffer, 32-bit elements
constexpr int kNowhere = int(0x80000000u);   // behind every descriptor's end

struct Cols {
    int ch[2];           // clamped to the last channel, so that loads have a place
    bool on[2];
    bool tail;           // kVec 2: the last channel is among the workgroup's
};
template <int kVec>
__device__ __forceinline__ Cols columns(int64_t c0, int lane, int64_t D) {
    Cols c;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int ch = int(c0) + (kVec ? 2 * lane + j : lane + 64 * j), n = int(D);
        c.on[j] = ch < n;
        // with kVec 1 a pair is in or out as a whole
        c.ch[j] = ch < n ? ch : kVec == 1 ? n - 2 + j : n - 1;
    }
    c.tail = kVec == 2 && c0 + kCols > D;
    return c;
}

// The wave's place in its workgroup, known to be the same in all its lanes: descriptors stay in
// scalar registers.
__device__ __forceinline__ int wave_number() {
    return __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
}

// Rows of n tokens (any number, also none) from p on, st elements apart, D wide.
template <typename T, int kVec>
struct Rows {
    __amdgpu_buffer_rsrc_t d;
    int step, at[2];      // kVec 2, to store: of a pair, and of a last channel alone
    int low;              // kVec 2, to load: bits before a last channel alone
    bool tail;
    __device__ __forceinline__ Rows(const void* p, int64_t st, int64_t n, int64_t D, const Cols& c,
                                    bool store) {
        const int bytes = n > 0 ? int(((n - 1) * st + D) * int64_t(sizeof(T))) : 0;
        d = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, kRsrcFlags);
        step = int(st) * int(sizeof(T));
        tail = c.tail;
        if constexpr (kVec == 2) {
            low = c.on[0] && !c.on[1] ? 8 * int(sizeof(T)) : 0;
            at[0] = c.on[1] ? c.ch[0] * int(sizeof(T)) : store ? kNowhere : (int(D) - 2) * int(sizeof(T));
            at[1] = c.on[0] && !c.on[1] ? c.ch[0] * int(sizeof(T)) : kNowhere;
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                at[j] = store && !c.on[j] ? kNowhere : c.ch[j] * int(sizeof(T));
        }
    }
};

template <typename T> struct Two;
template <> struct Two<float> {
    float v[2];
    __device__ __forceinline__ float get(int j) const { return v[j]; }
    __device__ __forceinline__ void anew() { asm volatile("" : "+v"(v[0]), "+v"(v[1])); }
    template <int kVec> __device__ __forceinline__ void load(const Rows<float, kVec>& r, int s) {
        if constexpr (kVec) {
            typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(r.d, r.at[0], s * r.step, 0);
            v[0] = __uint_as_float(kVec == 2 && r.low ? w[1] : w[0]); v[1] = __uint_as_float(w[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                v[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r.d, r.at[j], s * r.step, 0));
        }
    }
};
template <> struct Two<bf16_t> {
    uint32_t w;
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float(j ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ void anew() { asm volatile("" : "+v"(w)); }
    template <int kVec> __device__ __forceinline__ void load(const Rows<bf16_t, kVec>& r, int s) {
        if constexpr (kVec) {
            w = __builtin_amdgcn_raw_buffer_load_b32(r.d, r.at[0], s * r.step, 0);
            if constexpr (kVec == 2) w >>= r.low;
        } else {
            const uint32_t a = __builtin_amdgcn_raw_buffer_load_b16(r.d, r.at[0], s * r.step, 0);
            const uint32_t b = __builtin_amdgcn_raw_buffer_load_b16(r.d, r.at[1], s * r.step, 0);
            w = a | b << 16;
        }
    }
};

template <int kVec>
__device__ __forceinline__ void store2(const Rows<float, kVec>& r, int s, float a, float b) {
    if constexpr (kVec) {
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(a), __float_as_uint(b)}, r.d,
                                              r.at[0], s * r.step, 0);
        if (r.tail) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(a), r.d, r.at[1], s * r.step, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(a), r.d, r.at[0], s * r.step, 0);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(b), r.d, r.at[1], s * r.step, 0);
    }
}
template <int kVec>
__device__ __forceinline__ void store2(const Rows<bf16_t, kVec>& r, int s, float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 h;
    h[0] = __bf16(a); h[1] = __bf16(b);
    uint32_t w;
    __builtin_memcpy(&w, &h, 4);
    if constexpr (kVec) {
        __builtin_amdgcn_raw_buffer_store_b32(w, r.d, r.at[0], s * r.step, 0);
        if (r.tail) __builtin_amdgcn_raw_buffer_store_b16(uint16_t(w), r.d, r.at[1], s * r.step, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b16(uint16_t(w), r.d, r.at[0], s * r.step, 0);
        __builtin_amdgcn_raw_buffer_store_b16(uint16_t(w >> 16), r.d, r.at[1], s * r.step, 0);
    }
}

// One row of float32 (states, partial sums): p + row·D.
template <int kVec>
__device__ __forceinline__ void store_row(float* row, const Cols& c, float a, float b) {
    if constexpr (kVec == 1) {
        if (c.on[0]) *reinterpret_cast<float2*>(row + c.ch[0]) = make_float2(a, b);
    } else {
        if (c.on[0]) row[c.ch[0]] = a;
        if (c.on[1]) row[c.ch[1]] = b;
    }
}

// -c·softplus(lam) in units of log2
__device__ __forceinline__ float rate2(float lam, float c) { return -c * softplus(lam) * kLog2e; }

// Affine maps h -> A h + H of consecutive stretches, one after the other.  An A of -0 cuts off what
// it meets, NaN and infinities included: a document begins there.  Of a product of decays that has left
// float32 the least number stays, which takes finite states to nothing (2^-149 of them) and leaves NaN and
// infinities as they are, as they would be token after token.  (Exactly nothing, by a second factor in
// through(), made the gradient of 1 x 262144 x 128 6 % slower, the others 1 to 3.)
struct Map {
    float A, H;
};
constexpr float kCut = -0.0f;
__device__ __forceinline__ bool cuts(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float held(float A) { return __float_as_uint(A) == 0 ? 0x1p-149f : A; }
__device__ __forceinline__ float through(float A, float H, float h) {
    return cuts(A) ? H : fmaf(A, h, H);
}
// (the A of several, one after the other, is held() at the end)
__device__ __forceinline__ Map after(const Map& second, const Map& first) {
    return Map{cuts(first.A) || cuts(second.A) ? kCut : second.A * first.A,
               through(second.A, second.H, first.H)};
}

// ---- states from tile to tile ----------------------------------------------------------------
//
// A workgroup reads its tile once, keeps it in registers, and needs the state that enters it.  It
// publishes the map of its own tile, then takes those of the tiles before it in its group (of
// kGroup), and what the group before ended with, which that group's last tile publishes.  Maps are
// joined in the order of the tiles, whoever came first, so results do not depend on timing.
//
// A word of 64 bits holds a channel's map (or state, with A = 1) and is stored and loaded in one
// piece, past the caches of the eight dies (device scope); all ones, which no map has (NaN is
// stored as 0x7fc00000), means not yet.  So no other memory has to be ordered with it.  Every wait
// ends: workgroups take their tiles from a counter in the order in which they start to run, and
// wait for tiles of lower numbers only, whose workgroups run already and publish their maps before
// they wait themselves.
constexpr uint64_t kNotYet = ~uint64_t(0);

__device__ __forceinline__ uint64_t word_of(const Map& m) {
    const uint32_t a = m.A != m.A ? 0x7fc00000u : __float_as_uint(m.A);
    return uint64_t(a) << 32 | __float_as_uint(m.H);
}
__device__ __forceinline__ Map map_of(uint64_t w) {
    return Map{__uint_as_float(uint32_t(w >> 32)), __uint_as_float(uint32_t(w))};
}
__device__ __forceinline__ void publish(uint64_t* p, const Map& m) {
    __hip_atomic_store(p, word_of(m), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The maps of tiles [from, from + n) of a row (n <= kMost), joined, for channels ch[0 .. kCh - 1].
template <int kMost, int kCh>
__device__ __forceinline__ void joined(const uint64_t* tiles, int64_t D, const int (&ch)[kCh], int from,
                                       int n, Map (&m)[kCh]) {
    uint64_t w[kMost][kCh];
#pragma unroll
    for (int q = 0; q < kMost; ++q)
#pragma unroll
        for (int j = 0; j < kCh; ++j)
            w[q][j] = q < n ? peek(tiles + int64_t(from + q) * D + ch[j]) : 0;
#pragma unroll
    for (int q = 0; q < kMost; ++q) {
        if (q < n) {
#pragma unroll
            for (int j = 0; j < kCh; ++j) {
                while (w[q][j] == kNotYet) {
                    __builtin_amdgcn_s_sleep(1);
                    w[q][j] = peek(tiles + int64_t(from + q) * D + ch[j]);
                }
                m[j] = after(map_of(w[q][j]), m[j]);
            }
        }
    }
}

// Sets the counters and words (two at a time; the last may be padding) of a call's chains.
__global__ __launch_bounds__(256) void gr_chain_kernel(uint64_t* tickets, ulonglong2* words, int64_t n) {
    const int64_t step = int64_t(gridDim.x) * 256;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += step)
        words[i] = make_ulonglong2(kNotYet, kNotYet);
    if (blockIdx.x == 0 && threadIdx.x < 2) tickets[16 * threadIdx.x] = 0;
}

// Where a workgroup works: its tile in the chain's order, row and channels.
struct Place {
    int tile;
    int64_t b, c0;
};
__device__ __forceinline__ Place place(const GrLaunch& p, int& shared) {
    const unsigned groups = unsigned((p.D + kCols - 1) / kCols);
    unsigned n = blockIdx.x;
    if (p.ticket) {
        if (threadIdx.x == 0)
            shared = int(__hip_atomic_fetch_add(reinterpret_cast<unsigned*>(p.ticket), 1u,
                                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        __syncthreads();
        n = unsigned(__builtin_amdgcn_readfirstlane(shared));
    }
    const unsigned per = groups * unsigned(p.B), in = n % per;
    return Place{int(n / per), int64_t(in / groups), int64_t(in % groups) * kCols};
}

// What the waves of a workgroup share: their maps, by the channel's place in the workgroup's 128
// (a lane's two are neighbours or 64 apart), and the states that enter each of them.
template <int kWaves>
struct Shared {
    float A[kWaves][kCols], H[kWaves][kCols], in[kWaves][kCols];
    float lookA[kWaves - 2][kCols], lookH[kWaves - 2][kCols];
    int number;
};

template <int kVec> __device__ __forceinline__ int spot(int lane, int j) {
    return kVec ? 2 * lane + j : lane + 64 * j;
}

// Sets in[wave] to the states that enter the waves' stretches (kReverse: taken from the last wave to
// the first) from `first`, the state that enters the row (nullable: 0), and stores what leaves the
// row in `last` (nullable).  Two waves hold a channel a lane and walk over the waves' maps; the
// others meanwhile fetch the maps of the tiles before.  All maps are in place (a barrier) before.
template <int kVec, bool kReverse, int kGroup, int kWaves, typename Sh>
__device__ __forceinline__ void link(const GrLaunch& p, const Place& at, const Cols& col, int lane,
                                     int wave, Sh& sh, const float (&maps_h)[kWaves][kCols],
                                     const float* first, float* last) {
    constexpr int kFetch = kWaves - 2, kMost = (kGroup - 1 + kFetch - 1) / kFetch;
    const int groups = (p.tiles + kGroup - 1) / kGroup;
    const int n = at.tile % kGroup, group = at.tile / kGroup;
    uint64_t* maps = p.maps + at.b * p.tiles * p.D;
    uint64_t* ends = p.ends + at.b * groups * p.D;
    const int l = lane + 64 * wave;           // of the walking waves
    const int ch = int(at.c0) + l;
    const bool on = wave < 2 && ch < int(p.D);
    float h = 0.0f;
    Map own = {1.0f, 0.0f};
    if (wave < 2) {
        if (on && first && group == 0) h = first[at.b * p.D + ch];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int v = kReverse ? kWaves - 1 - w : w;
            own = after(Map{sh.A[v][l], maps_h[v][l]}, own);
        }
        own.A = held(own.A);
        if (p.ticket && n < kGroup - 1) {
            // the state that enters the row has come in before this map goes out: what leaves the row
            // may take its place (h_final over h0, dh0 over dh_final)
            asm volatile("" ::"v"(h));
            if (on) publish(maps + int64_t(at.tile) * p.D + ch, own);
        }
    } else if (p.ticket && n > 0) {
        Map m[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
        const int f = wave - 2, lo = n * f / kFetch, hi = n * (f + 1) / kFetch;
        if (hi > lo) joined<kMost, 2>(maps, p.D, col.ch, group * kGroup + lo, hi - lo, m);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sh.lookA[f][spot<kVec>(lane, j)] = held(m[j].A);
            sh.lookH[f][spot<kVec>(lane, j)] = m[j].H;
        }
    }
    if (p.ticket && (n > 0 || group > 0)) {
        if (on && group > 0) {
            Map e[1] = {{1.0f, 0.0f}};
            const int one[1] = {ch};
            joined<1, 1>(ends, p.D, one, group - 1, 1, e);
            h = e[0].H;
        }
        __syncthreads();
        if (wave < 2 && n > 0) {
#pragma unroll
            for (int f = 0; f < kFetch; ++f) h = through(sh.lookA[f][l], sh.lookH[f][l], h);
        }
    }
    if (wave < 2) {
        const float out = through(own.A, own.H, h);
        if (on && p.ticket && n == kGroup - 1 && at.tile + 1 < p.tiles)
            publish(ends + int64_t(group) * p.D + ch, Map{1.0f, out});
        if (on && last && at.tile + 1 == p.tiles) last[at.b * p.D + ch] = out;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int v = kReverse ? kWaves - 1 - w : w;
            sh.in[v][l] = h;
            h = through(sh.A[v][l], maps_h[v][l], h);
        }
    }
    __syncthreads();
}

// Which of the `live` tokens from t0 on begin a document: bit s for token t0 + s.
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* reset, int64_t b, int64_t T,
                                               int64_t t0, int lane, int live) {
    if (!reset) return 0;
    bool set = false;
    if (lane < live) set = reset[b * T + t0 + lane] != 0;
    return uint32_t(__ballot(set));
}

// How many of the kS tokens from t0 on exist in row b.
template <int kS>
__device__ __forceinline__ int live_tokens(const int32_t* lengths, int64_t b, int64_t t0, int64_t T) {
    int64_t n = T;
    if (lengths) n = lengths[b] < T ? lengths[b] : T;
    n -= t0;
    return n < 0 ? 0 : n < kS ? int(n) : kS;
}

// ---- forward ---------------------------------------------------------------------------------

template <typename T, int kVec, int kWaves, int kS>
__global__ __launch_bounds__(64 * kWaves) void gr_fwd_kernel(const GrLaunch p) {
    static_assert(SS_GR_CKPT % kS == 0, "checkpoints stand before a wave's first token");
    __shared__ Shared<kWaves> sh;
    const int lane = threadIdx.x & 63, wave = wave_number();
    const Place at = place(p, sh.number);
    const int64_t b = at.b, D = p.D;
    const Cols col = columns<kVec>(at.c0, lane, D);
    const int64_t t0 = (int64_t(at.tile) * kWaves + wave) * kS;
    const int64_t n = p.T - t0 < kS ? p.T - t0 : kS;
    Two<T> wx[kS], wr[kS], wi[kS];
    {
        const Rows<T, kVec> x(static_cast<const T*>(p.x.p) + b * p.x.sb + t0 * p.x.st, p.x.st, n, D, col, false);
        const Rows<T, kVec> r(static_cast<const T*>(p.r.p) + b * p.r.sb + t0 * p.r.st, p.r.st, n, D, col, false);
        const Rows<T, kVec> g(static_cast<const T*>(p.i.p) + b * p.i.sb + t0 * p.i.st, p.i.st, n, D, col, false);
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            wr[s].load(r, s);
            wi[s].load(g, s);
            wx[s].load(x, s);
        }
    }
    const int live = live_tokens<kS>(p.lengths, b, t0, p.T);
    const uint32_t first = reset_bits(p.reset, b, p.T, t0, lane, live);
    float k2[2], h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) k2[j] = rate2(p.lam[col.ch[j]], p.c);
    float a[kS][2], u[kS][2];
    Map own[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
    // the wave's map; all: every token exists and none begins a document
    const bool all = first == 0 && live == kS;
    auto tokens = [&](auto all) {
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const bool cut = !all && (first >> s & 1), on = all || s < live;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float t2 = k2[j] * sigmoid(wr[s].get(j));
                const float e = exp2_hw(t2);
                const float q = __builtin_amdgcn_sqrtf(one_less_square(t2, e));
                const float v = sigmoid(wi[s].get(j)) * wx[s].get(j);
                a[s][j] = !on ? 1.0f : cut ? 0.0f : e;
                u[s][j] = !on ? 0.0f : cut ? v : q * v;
                own[j].H = fmaf(a[s][j], cut ? 0.0f : own[j].H, u[s][j]);
                own[j].A *= a[s][j];
            }
        }
    };
    if (all) tokens(std::true_type{});
    else tokens(std::false_type{});
    for (int j = 0; j < 2; ++j) own[j].A = first ? kCut : held(own[j].A);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        sh.A[wave][spot<kVec>(lane, j)] = own[j].A;
        sh.H[wave][spot<kVec>(lane, j)] = own[j].H;
    }
    __syncthreads();
    link<kVec, false, kGrFwdGroup, kWaves>(p, at, col, lane, wave, sh, sh.H, p.h0, p.h_final);
#pragma unroll
    for (int j = 0; j < 2; ++j) h[j] = sh.in[wave][spot<kVec>(lane, j)];
    if (p.h_ckpt && t0 % SS_GR_CKPT == 0 && t0 < p.T) {
        const int64_t nc = (p.T + SS_GR_CKPT - 1) / SS_GR_CKPT;
        store_row<kVec>(p.h_ckpt + (b * nc + t0 / SS_GR_CKPT) * D, col, h[0], h[1]);
    }
    if (p.y) {
        const Rows<T, kVec> y(static_cast<T*>(p.y) + (b * p.T + t0) * D, D, n, D, col, true);
#pragma unroll
        for (int s = 0; s < kS; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) h[j] = fmaf(a[s][j], first >> s & 1 ? 0.0f : h[j], u[s][j]);
            const bool on = s < live;
            store2(y, s, on ? h[0] : 0.0f, on ? h[1] : 0.0f);
        }
    }
}

// Short rows: a wave takes 128 channels of a row from its first token to its last, kS at a time, the next
// ones on their way.  1024 rows of 1 token, 2560 channels, bfloat16: 15 us (a tile's workgroup for each 374),
// of 32 tokens, 671 MB, 135 us (374).
template <typename T, int kVec, int kS>
__global__ __launch_bounds__(256) void gr_walk_kernel(const GrLaunch p) {
    const int lane = threadIdx.x & 63;
    const unsigned groups = unsigned((p.D + kCols - 1) / kCols);
    const unsigned number = blockIdx.x * 4 + unsigned(wave_number());
    if (number >= groups * unsigned(p.B)) return;
    const int64_t b = number / groups, D = p.D, nc = (p.T + SS_GR_CKPT - 1) / SS_GR_CKPT;
    const Cols col = columns<kVec>(int64_t(number % groups) * kCols, lane, D);
    const Rows<T, kVec> x(static_cast<const T*>(p.x.p) + b * p.x.sb, p.x.st, p.T, D, col, false);
    const Rows<T, kVec> r(static_cast<const T*>(p.r.p) + b * p.r.sb, p.r.st, p.T, D, col, false);
    const Rows<T, kVec> g(static_cast<const T*>(p.i.p) + b * p.i.sb, p.i.st, p.T, D, col, false);
    const Rows<T, kVec> y(static_cast<T*>(p.y) + b * p.T * D, D, p.T, D, col, true);
    struct In {
        Two<T> x[kS], r[kS], i[kS];
    };
    auto load = [&](int t0, In& in) {
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            in.r[s].load(r, t0 + s);
            in.i[s].load(g, t0 + s);
            in.x[s].load(x, t0 + s);
        }
    };
    In now;
    load(0, now);
    float k2[2], h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        k2[j] = rate2(p.lam[col.ch[j]], p.c);
        h[j] = p.h0 ? p.h0[b * D + col.ch[j]] : 0.0f;
    }
    for (int64_t t0 = 0; t0 < p.T; t0 += kS) {
        In next;
        if (t0 + kS < p.T) load(int(t0) + kS, next);
        const int live = live_tokens<kS>(p.lengths, b, t0, p.T);
        const uint32_t first = reset_bits(p.reset, b, p.T, t0, lane, live);
        if (p.h_ckpt && t0 % SS_GR_CKPT == 0) store_row<kVec>(p.h_ckpt + (b * nc + t0 / SS_GR_CKPT) * D, col, h[0], h[1]);
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const bool cut = first >> s & 1, on = s < live;
            float o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float t2 = k2[j] * sigmoid(now.r[s].get(j));
                const float e = exp2_hw(t2);
                const float q = __builtin_amdgcn_sqrtf(one_less_square(t2, e));
                const float v = sigmoid(now.i[s].get(j)) * now.x[s].get(j);
                if (on) h[j] = cut ? v : fmaf(e, h[j], q * v);
                o[j] = on ? h[j] : 0.0f;
            }
            store2(y, int(t0) + s, o[0], o[1]);
        }
        now = next;
    }
    if (p.h_final) store_row<kVec>(p.h_final + b * D, col, h[0], h[1]);
}

// ---- backward --------------------------------------------------------------------------------

// The states before a wave's tokens come from the checkpoint that its workgroup's tile starts
// with; the adjoint c comes from the right: the chain's first tile is the row's last.  Two workgroups share a
// compute unit where a lane has 128 registers: 4 x 4096 x 2048, bfloat16, 132 us, 168 with the 138 that the
// compiler takes by itself (float32 has no room for two).
template <typename T, int kVec, int kWaves, int kS, int kGroup>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) == 2 && kVec ? 4 : 1) void gr_bwd_kernel(const GrLaunch p) {
    static_assert(kWaves * kS == SS_GR_CKPT, "a tile is what one checkpoint starts");
    __shared__ Shared<kWaves> sh;
    __shared__ float G[kWaves][kCols];
    const int lane = threadIdx.x & 63, wave = wave_number();
    const Place at = place(p, sh.number);
    const int64_t b = at.b, D = p.D;
    const Cols col = columns<kVec>(at.c0, lane, D);
    const int64_t tile = p.tiles - 1 - at.tile, t0 = tile * SS_GR_CKPT + wave * kS;
    const int64_t n = p.T - t0 < kS ? p.T - t0 : kS;
    Two<T> wx[kS], wr[kS], wi[kS], wd[kS];
    {
        const Rows<T, kVec> x(static_cast<const T*>(p.x.p) + b * p.x.sb + t0 * p.x.st, p.x.st, n, D, col, false);
        const Rows<T, kVec> r(static_cast<const T*>(p.r.p) + b * p.r.sb + t0 * p.r.st, p.r.st, n, D, col, false);
        const Rows<T, kVec> g(static_cast<const T*>(p.i.p) + b * p.i.sb + t0 * p.i.st, p.i.st, n, D, col, false);
        const Rows<T, kVec> dy(static_cast<const T*>(p.dy) + (b * p.T + t0) * D, D, n, D, col, false);
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            wr[s].load(r, s);
            wi[s].load(g, s);
            wx[s].load(x, s);
            wd[s].load(dy, s);
        }
    }
    const int live = live_tokens<kS>(p.lengths, b, t0, p.T);
    const uint32_t first = reset_bits(p.reset, b, p.T, t0, lane, live);
    float k2[2], c[2], h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        k2[j] = rate2(p.lam[col.ch[j]], p.c);
        h[j] = p.h_ckpt[(b * p.tiles + tile) * D + col.ch[j]];
    }
    float a[kS][2], q[kS][2], fi[kS][2];          // fi: the input's gate, folded
    Map fwd[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}}, rev[2];
    // What stands behind a text becomes 0 (and its a 1) before anything is formed from it; a token
    // that begins a document has a = 0 and s = 1.
    const bool all = first == 0 && live == kS;
    auto tokens = [&](auto all) {
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const bool cut = !all && (first >> s & 1), on = all || s < live;
            if (!on) wx[s] = wd[s] = Two<T>{};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float sx;
                const float f = folded(wi[s].get(j), sx);
                fi[s][j] = on ? f : 0.0f;
                asm volatile("" : "+v"(fi[s][j]));    // (formed here: its parts would live on)
                if (!on) sx = 0.0f;
                const float t2 = k2[j] * sigmoid(wr[s].get(j));
                const float e = exp2_hw(t2);
                a[s][j] = !on ? 1.0f : cut ? 0.0f : e;
                q[s][j] = !on ? 0.0f : cut ? 1.0f : __builtin_amdgcn_sqrtf(one_less_square(t2, e));
                fwd[j].H = fmaf(a[s][j], cut ? 0.0f : fwd[j].H, q[s][j] * (sx * wx[s].get(j)));
                fwd[j].A *= a[s][j];
            }
        }
        rev[0].H = rev[1].H = 0.0f;
#pragma unroll
        for (int s = kS - 1; s >= 0; --s) {
            const bool cut = !all && (first >> s & 1);
#pragma unroll
            for (int j = 0; j < 2; ++j)       // c -> a (dy + c)
                rev[j].H = cut ? 0.0f : a[s][j] * (wd[s].get(j) + rev[j].H);
        }
    };
    if (all) tokens(std::true_type{});
    else tokens(std::false_type{});
    for (int j = 0; j < 2; ++j) fwd[j].A = first ? kCut : held(fwd[j].A);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        sh.A[wave][spot<kVec>(lane, j)] = fwd[j].A;
        sh.H[wave][spot<kVec>(lane, j)] = fwd[j].H;
        G[wave][spot<kVec>(lane, j)] = rev[j].H;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int l = spot<kVec>(lane, j);
            h[j] = through(sh.A[w][l], sh.H[w][l], h[j]);
        }
    }
    link<kVec, true, kGroup, kWaves>(p, at, col, lane, wave, sh, G, p.dh_final, p.dh0);
#pragma unroll
    for (int j = 0; j < 2; ++j) c[j] = sh.in[wave][spot<kVec>(lane, j)];
    // From here on x, dy, both gates and their products are formed once more from the packed values: kept
    // from above, they would take 80 registers a lane.
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        wx[s].anew();
        wr[s].anew();
        wd[s].anew();
        asm volatile("" : "+v"(fi[s][0]), "+v"(fi[s][1]));
    }
    float old[kS][2], dl[2] = {0.0f, 0.0f};
    const Rows<T, kVec> dx(static_cast<T*>(p.dx) + (b * p.T + t0) * D, D, n, D, col, true);
    const Rows<T, kVec> dr(static_cast<T*>(p.dr) + (b * p.T + t0) * D, D, n, D, col, true);
    const Rows<T, kVec> di(static_cast<T*>(p.di) + (b * p.T + t0) * D, D, n, D, col, true);
    auto gradients = [&](auto all) {
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const bool cut = !all && (first >> s & 1);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                old[s][j] = h[j];
                h[j] = fmaf(a[s][j], cut ? 0.0f : h[j], q[s][j] * (gate_of(fi[s][j]) * wx[s].get(j)));
            }
        }
#pragma unroll
        for (int s = 0; s < kS; ++s) wx[s].anew();
#pragma unroll
        for (int s = kS - 1; s >= 0; --s) {
            const bool cut = !all && (first >> s & 1), on = all || s < live;
            float ox[2], orr[2], oi[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float as = a[s][j], qs = q[s][j], xv = wx[s].get(j), sx = gate_of(fi[s][j]);
                // σ(r), and σ(r)(1 - σ(r)) as its square times e^-r (0 where that is infinite)
                const float e = exp2_hw(-wr[s].get(j) * kLog2e), sg = rcp_hw(1.0f + e);
                const float both = fminf(e, FLT_MAX) * sg * sg;
                const float gt = wd[s].get(j) + c[j], ag = as * gt;
                c[j] = cut ? 0.0f : ag;
                ox[j] = gt * qs * sx;
                oi[j] = ox[j] * xv * rest_of(fi[s][j]);
                // a slope past 1e15 is taken as 0: its share of the gradient is below 1e-15
                const float slope = qs > 1e-15f ? as * rcp_hw(qs) : 0.0f;
                const float dla = ag * fmaf(-slope, sx * xv, old[s][j]);
                orr[j] = dla * (k2[j] * kLn2) * both;
                dl[j] = on && !cut ? fmaf(dla, sg, dl[j]) : dl[j];
                if (!on) ox[j] = oi[j] = 0.0f;
                if (!on || cut) orr[j] = 0.0f;
            }
            store2(dx, s, ox[0], ox[1]);
            store2(dr, s, orr[0], orr[1]);
            store2(di, s, oi[0], oi[1]);
        }
    };
    if (all) gradients(std::true_type{});
    else gradients(std::false_type{});
    // (A is no longer read: link ends with a barrier)
#pragma unroll
    for (int j = 0; j < 2; ++j) sh.A[wave][spot<kVec>(lane, j)] = dl[j];
    __syncthreads();
    const int64_t ch = at.c0 + threadIdx.x;
    if (threadIdx.x < kCols && ch < D) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += sh.A[w][threadIdx.x];
        p.part[(b * p.tiles + tile) * D + ch] = v;
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

template <typename T, int kVec>
__global__ __launch_bounds__(256) void gr_step_kernel(const GrStep p) {
    const int lane = threadIdx.x & 63;
    const int64_t b = int64_t(blockIdx.y) * 4 + wave_number(), D = p.D;
    if (b >= p.B) return;
    const Cols col = columns<kVec>(int64_t(blockIdx.x) * kCols, lane, D);
    Two<T> x, r, i;
    x.load(Rows<T, kVec>(static_cast<const T*>(p.x.p) + b * p.x.sb, 0, 1, D, col, false), 0);
    r.load(Rows<T, kVec>(static_cast<const T*>(p.r.p) + b * p.r.sb, 0, 1, D, col, false), 0);
    i.load(Rows<T, kVec>(static_cast<const T*>(p.i.p) + b * p.i.sb, 0, 1, D, col, false), 0);
    float h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float t2 = rate2(p.lam[col.ch[j]], p.c) * sigmoid(r.get(j));
        const float a = exp2_hw(t2);
        const float q = __builtin_amdgcn_sqrtf(one_less_square(t2, a));
        h[j] = fmaf(a, p.h_in[b * D + col.ch[j]], q * (sigmoid(i.get(j)) * x.get(j)));
    }
    store_row<kVec>(p.h_out + b * D, col, h[0], h[1]);
    store2(Rows<T, kVec>(static_cast<T*>(p.y) + b * D, 0, 1, D, col, true), 0, h[0], h[1]);
}

template <typename F>
hipError_t with_type(int in_dtype, int vec, F&& f) {
    auto typed = [&](auto t) {
        return vec == 1   ? f(t, std::integral_constant<int, 1>())
               : vec == 2 ? f(t, std::integral_constant<int, 2>())
                          : f(t, std::integral_constant<int, 0>());
    };
    return in_dtype == SS_BF16 ? typed(bf16_t{}) : typed(0.0f);
}

constexpr int kFwdWaves = 8, kBwdWaves = SS_GR_CKPT / 8;

unsigned groups(int64_t D) { return unsigned((D + kCols - 1) / kCols); }

}  // namespace

hipError_t launch_gr_chains(uint64_t* tickets, uint64_t* maps, int64_t words, hipStream_t s) {
    const int64_t n = (words + 1) / 2, need = (n + 255) / 256;
    hipLaunchKernelGGL(gr_chain_kernel, dim3(unsigned(need < 1024 ? need : 1024)), dim3(256), 0, s,
                       tickets, reinterpret_cast<ulonglong2*>(maps), n);
    return hipGetLastError();
}

hipError_t launch_gr_fwd(const GrLaunch& p, hipStream_t s) {
    return with_type(p.in_dtype, p.vec, [&](auto t, auto v) {
        if (p.y && gr_walks(p.T, int64_t(groups(p.D)) * p.B, std::max({p.x.st, p.r.st, p.i.st, p.D}))) {
            hipLaunchKernelGGL((gr_walk_kernel<decltype(t), decltype(v)::value, 8>),
                               dim3((groups(p.D) * unsigned(p.B) + 3) / 4), dim3(256), 0, s, p);
            return hipGetLastError();
        }
        hipLaunchKernelGGL((gr_fwd_kernel<decltype(t), decltype(v)::value, kFwdWaves, kGrFwdTile / kFwdWaves>),
                           dim3(groups(p.D) * unsigned(p.B) * unsigned(p.tiles)), dim3(64 * kFwdWaves), 0, s, p);
        return hipGetLastError();
    });
}

hipError_t launch_gr_bwd(const GrLaunch& p, hipStream_t s) {
    const hipError_t e = with_type(p.in_dtype, p.vec, [&](auto t, auto v) {
        constexpr int kS = SS_GR_CKPT / kBwdWaves;
        const dim3 grid(groups(p.D) * unsigned(p.B) * unsigned(p.tiles)), block(64 * kBwdWaves);
        if (p.group == kGrBwdLong)
            hipLaunchKernelGGL((gr_bwd_kernel<decltype(t), decltype(v)::value, kBwdWaves, kS, kGrBwdLong>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((gr_bwd_kernel<decltype(t), decltype(v)::value, kBwdWaves, kS, kGrBwdGroup>), grid, block, 0, s, p);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gr_dlam_kernel, dim3(unsigned((p.D + 63) / 64)), dim3(1024), 0, s, p.part,
                       p.lam, p.dlam, p.c, p.D, p.B * p.tiles);
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
