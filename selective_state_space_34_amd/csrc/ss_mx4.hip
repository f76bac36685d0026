// Microscaled 4-bit values for gfx950: rounding to them, and products with weights held in them.
//
//   value = e2m1(code)·2^(exponent - 127), one exponent for 32 consecutive columns
//   y[m, n] = Σ_k x[m, k]·w[n, k]        x the same, or e4m3 with a float32 scale for each row
//
// The matrix cores take both formats as they lie in memory: v_mfma_scale_f32_16x16x128_f8f6f4 reads
// 32 codes of a block (16 bytes) and the block's exponent from a lane, lane l row l % 16 and block
// l / 16 of the 128 columns; of e4m3 two runs of 16, at 16·(l / 16) and at 64 more.
//
// Few rows: the bytes of w bound it, and how fast a compute unit's cache takes accesses
// (mx4_rows_kernel).  Many rows: the matrix cores' rate (mx4_tile_kernel).  Rounding: the bytes of x
// (mx4_quant_kernel; 16384 x 2560 bfloat16, 106 MB, 25 us, 4.2 TB/s).
#include "ss_device.h"
#include "ss_gr_plan.h"
#include "ss_kernels.h"

namespace ss {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
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

// ---- buffers ---------------------------------------------------------------------------------

constexpr int kRsrcFlags = 0x00020000;       // raw buffer, 32-bit elements
constexpr int kNowhere = int(0x80000000u);   // behind every descriptor's end: loads 0, stores nothing

constexpr int kPast = 2;                     // a store that the caches do not keep (nt)

// Up to `most` rows, `bytes` each, from number r0 of `rows` on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const void* p, int64_t r0, int64_t rows,
                                                           int64_t most, int64_t bytes) {
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(static_cast<const uint8_t*>(p)) + r0 * bytes, 0, int(n * bytes), kRsrcFlags);
}

// ---- few rows --------------------------------------------------------------------------------

// What x is: in 4 bits, or e4m3.  The matrix cores add the products of e4m3 eight neighbouring columns at
// a time, and first align them with the largest: of a product whose operands' exponents sum to e, bits below
// 2^(E - 13) are cut, E the largest of the eight sums.  A product's last bit is 2^(e - 4), so none is lost
// where the exponents of x are within 7 of one another (those of w are within 2).  e4m3's go from -6 to 8:
// x is taken in two parts, of exponents up to 0 and from 1 on, a product each, and every bit counts; from
// there on sums are float32, as for two operands in 4 bits, whose products fit as they are.  In one part, rows
// whose largest columns cancel lost a fifth of the result.
enum { kX4, kX8 };

// The e4m3 values of w from 2 on (the exponent's first bit is set: bit 6), NaN with them, or 0; what is
// left of w is the rest.
__device__ __forceinline__ int from_two(int w) {
    // bytes of ones where the bit is set: the permutation's signs of bytes 1 and 3 of both operands
    const uint32_t b = uint32_t(w) << 1;
    return w & int(__builtin_amdgcn_perm(b << 8, b, 0x090b080a));
}

// 16 rows of weights and 16·kTiles rows of x a workgroup; its waves take the columns, 128 at a time,
// in turn and meet in LDS.  The matrix cores want 16 rows in neighbouring lanes; the cache takes four
// neighbouring lanes at a time if they share a line, else one.  So four lanes load a row's 64 bytes
// and exponents, and ds_bpermute brings them where they belong.  With loads straight into place the
// cache's one access a clock bound this kernel: 64 rows by 2560 x 5120, 14.2 us, now 7.0 (x in e4m3
// 8.4); 1 row by 10240 x 2560 5.9, now 5.0, of which 2.6 at the rate of a large copy and
// 2.4 the shortest launch of all.  Loading the next columns ahead made no case faster.
// What lies behind the last row or column loads as 0, exponents too.
template <int kTiles, int kX, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void mx4_rows_kernel(const Mx4Launch p) {
    __shared__ float red[kWaves][kTiles][64][4];
    constexpr bool kFp8 = kX != kX4;
    constexpr int kPieces = kFp8 ? 2 : 1;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane >> 2, g = lane & 3, from = ((lane & 15) * 4 + (lane >> 4)) * 4;
    const int K = int(p.K), kb = K / 32, row_x = kFp8 ? K : K / 2;
    const int64_t n0 = int64_t(blockIdx.x) * 16, m0 = int64_t(blockIdx.y) * 16 * kTiles;
    const __amdgpu_buffer_rsrc_t dw = rows_from(p.wq, n0, p.N, 16, K / 2);
    const __amdgpu_buffer_rsrc_t dwe = rows_from(p.w_exps, n0, p.N, 16, kb);
    const __amdgpu_buffer_rsrc_t dx = rows_from(p.x, m0, p.M, 16 * kTiles, row_x);
    const __amdgpu_buffer_rsrc_t dxe = rows_from(p.x_scale, m0, p.M, 16 * kTiles, kFp8 ? 0 : kb);
    struct Operands {
        u32x4 w, x[kTiles][kPieces];
        int we, xe[kTiles];
    };
    auto fetch = [&](int k0, Operands& s) {
        const bool in = k0 + 32 * g < K;
        s.w = __builtin_amdgcn_raw_buffer_load_b128(dw, in ? row * (K / 2) + 16 * g : kNowhere, k0 / 2, 0);
        s.we = __builtin_amdgcn_raw_buffer_load_b8(dwe, in ? row * kb + g : kNowhere, k0 / 32, 0);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int at = 16 * g + 64 * i;      // (e4m3: as the instruction takes them)
                s.x[t][i] = __builtin_amdgcn_raw_buffer_load_b128(
                    dx, (kFp8 ? k0 + at < K : in) ? (16 * t + row) * row_x + at : kNowhere,
                    kFp8 ? k0 : k0 / 2, 0);
            }
            if constexpr (!kFp8)
                s.xe[t] = __builtin_amdgcn_raw_buffer_load_b8(dxe, in ? (16 * t + row) * kb + g : kNowhere,
                                                              k0 / 32, 0);
        }
    };
    f32x4 acc[kTiles] = {};
    auto add = [&](const Operands& s) {
        i32x8 a = {};
#pragma unroll
        for (int c = 0; c < 4; ++c) a[c] = __builtin_amdgcn_ds_bpermute(from, int(s.w[c]));
        const int sa = __builtin_amdgcn_ds_bpermute(from, s.we);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            i32x8 b = {};
#pragma unroll
            for (int c = 0; c < 4 * kPieces; ++c)
                b[c] = __builtin_amdgcn_ds_bpermute(from, int(s.x[t][c / 4][c % 4]));
            if constexpr (kFp8) {
                i32x8 large;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    large[c] = from_two(b[c]);
                    b[c] ^= large[c];
                }
                acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, large, acc[t], 4, 0, 0, sa, 0, 127);
                acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[t], 4, 0, 0, sa, 0, 127);
            } else {
                const int sb = __builtin_amdgcn_ds_bpermute(from, s.xe[t]);
                acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[t], 4, 4, 0, sa, 0, sb);
            }
        }
        settle();   // the sums may change registers where the loop ends
    };
    for (int k0 = wave * 128; k0 < K; k0 += kWaves * 128) {
        Operands s;
        fetch(k0, s);
        add(s);
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

// ---- many rows -------------------------------------------------------------------------------

// A workgroup of four waves takes 128 rows of weights and 64·kM of x; a wave 64 by 32·kM of them, as
// products of 32 by 32 rows and 64 columns (v_mfma_scale_f32_32x32x64_f8f6f4: lane l row l % 32 and
// block l / 32; of e4m3 two runs of 16 columns, 32 apart; 7.3 PFLOP/s in a loop of nothing else, where
// 16x16x128 gives 6.0).  Both operands pass through LDS, 128 columns (a stage) at a time, in two
// buffers; two workgroups share a compute unit (128 sums and 108 other registers a lane).  A row's
// 16-byte pieces are placed by their number xor some bits of the row, so that the 16 lanes that read
// at once (0-3, 12-15, 20-23, 24-27; the others of 32; and so on) meet all banks.  Weights' rows are
// dealt to the two products of a wave so that a lane ends up with runs of eight of a row of y.
// Exponents come 16 to a row and four stages, and go to the instruction as one word a row and stage.
//
// 16384 x 10240 x 2560, x in 4 bits: 250 us, 3.4 PFLOP/s (8192 x 8192 x 8192: 284 us, 3.9).  Of the 250,
// 178 are left without the loads and stores of global memory, 205 without loads, 217 without stores:
// the matrix cores work 40 % of the time, at 1.9 GHz, and wait for LDS and at the stages' barriers.
// One workgroup of 256 by 256 rows a compute unit took 365 us, a third buffer does not fit two.
// x in e4m3: 622 us, with a float32 y 649 (in one instruction, which cuts bits, 387; both operands widened to
// bfloat16, float32 y, 802); matrix cores 65 % busy.
template <int kX, int kM>
struct Tile {
    static constexpr int kRowsN = 128, kRowsM = 64 * kM;
    static constexpr int kBytesX = kX == kX4 ? 64 : 128;      // a row of x, 128 columns
    static constexpr int kPiecesW = kRowsN * 4, kPiecesX = kRowsM * (kBytesX / 16);
    static constexpr int kUsed = kRowsN + (kX == kX4 ? kRowsM : 0);
    static constexpr int kScales = (kUsed + 255) / 256 * 256;
    u32x4 w[2][kPiecesW], x[2][kPiecesX];
    uint32_t e[2][4][kScales];
};

__device__ __forceinline__ int turn_w(int row) { return row >> 3 & 3; }
template <int kX> __device__ __forceinline__ int turn_x(int row) {
    return kX == kX4 ? row >> 2 & 3 : row >> 1 & 7;
}

// Row of weights, of a wave's 64, that product u takes as its row r.
__device__ __forceinline__ int dealt(int u, int r) {
    return 16 * (r >> 3) + 8 * (r >> 2 & 1) + 4 * u + (r & 3);
}

// Exponents 16·block .. of the row at `at` that has n of them.  kEven: n is a multiple of 4; others'
// rows start on any byte, and a row's last 16 are taken whole and shifted.  (Behind the row's end:
// anything.)
template <bool kEven>
__device__ __forceinline__ u32x4 exponents(__amdgpu_buffer_rsrc_t d, int at, int block, int n) {
    if constexpr (kEven) return __builtin_amdgcn_raw_buffer_load_b128(d, at, 16 * block, 0);
    const int from = 16 * block + 16 <= n ? 16 * block : n - 16;
    if (n < 16) {
        u32x4 w = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 15; ++i)
            w[i / 4] |= uint32_t(__builtin_amdgcn_raw_buffer_load_b8(
                            d, i < n && block == 0 ? at + i : kNowhere, 0, 0)) << (8 * (i % 4));
        return w;
    }
    return __builtin_amdgcn_raw_buffer_load_b128(d, at, from, 0);
}
// Exponents 16·block .. out of what came for them.
template <bool kEven>
__device__ __forceinline__ u32x4 in_place(u32x4 w, int block, int n) {
    if constexpr (!kEven) {
        const int left = n - 16 * block, off = n < 16 || left >= 16 ? 0 : 16 - left;   // bytes
        uint64_t lo = uint64_t(w[1]) << 32 | w[0], hi = uint64_t(w[3]) << 32 | w[2];
        if (off >= 8) {
            lo = off >= 16 ? 0 : hi >> (8 * (off - 8));
            hi = 0;
        } else if (off > 0) {
            lo = lo >> (8 * off) | hi << (64 - 8 * off);
            hi >>= 8 * off;
        }
        w = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
    }
    return w;
}

// A workgroup's tile.  Dies get consecutive tiles (blocks go to the eight of them in turn), eight row
// tiles of x by one of weights after the other, so that what they read stays in a die's L2.
__device__ __forceinline__ bool tile_of(int64_t tiles_m, int64_t tiles_n, int64_t& m, int64_t& n) {
    const int64_t total = tiles_m * tiles_n, each = (total + 7) / 8;
    const int64_t number = int64_t(blockIdx.x % 8) * each + blockIdx.x / 8;
    if (blockIdx.x / 8 >= each || number >= total) return false;
    const int64_t per = 8 * tiles_n, first = number / per * 8;
    const int64_t high = tiles_m - first < 8 ? tiles_m - first : 8;
    m = first + number % per % high;
    n = number % per / high;
    return true;
}

// Rows behind the last one are behind the descriptor's end.  A wave whose columns all exist turns 32 rows of 128 bytes at a time in LDS (`own`: 4 KB of the wave's, twice)
// and stores whole lines; where the lines are memory's own, past the caches, which keep x and w
// instead.  16384 x 10240 x 2560: 278 us with 16 bytes of a row to a lane, 257 so, 250 past the caches
// (which made the pieces of 16 bytes slower, 480).
template <int kX, int kM>
__device__ __forceinline__ void store_tile(const Mx4Launch& p, int64_t m0, int64_t n0, int wn, int wm,
                                           int lane, const f32x16 (&acc)[2][kM], u32x4* own) {
    const int row = lane & 31, g = lane >> 5;
    const int N = int(p.N), el = p.y_dtype == SS_F32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t dy = rows_from(p.y, m0, p.M, 64 * kM, int64_t(N) * el);
    char* rows = static_cast<char*>(p.y) + m0 * N * el;
    const int c0 = int(n0) + 64 * wn, n = c0 + 8 * g;
    const bool wide = c0 + 64 <= N, whole = N * el % 128 == 0, words = N * el % 4 == 0;
#pragma unroll
    for (int t = 0; t < kM; ++t) {
        const int top = 32 * kM * wm + 32 * t, m = top + row;
        float f = 1.0f;
        if constexpr (kX != kX4)
            f = static_cast<const float*>(p.x_scale)[m0 + m < p.M ? m0 + m : p.M - 1];
        // eight columns from n + 16 q on: four of each product
        auto eight = [&](int q, float (&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = acc[j / 4][t][4 * q + j % 4];
                if constexpr (kX != kX4) v[j] *= f;
            }
        };
        if (wide) {
            const int lines = el / 2;       // of 128 bytes in a row
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half >= lines) break;
                u32x4* at = own + 256 * ((t + half) & 1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[8];
                    if (el == 2) {
                        eight(q, v);
                        union { bf16x8 h; u32x4 w; } o;
#pragma unroll
                        for (int j = 0; j < 8; ++j) o.h[j] = __bf16(v[j]);
                        at[8 * row + ((2 * q + g) ^ (row & 7))] = o.w;
                    } else if (q < 2) {
                        eight(2 * half + q, v);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            at[8 * row + ((4 * q + 2 * g + i) ^ (row & 7))] =
                                u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                      __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * i + (lane >> 3), piece = lane & 7;
                    const u32x4 w = at[8 * r + (piece ^ (r & 7))];
                    const int to = ((top + r) * N + c0) * el + 128 * half + 16 * piece;
                    if (whole) __builtin_amdgcn_raw_buffer_store_b128(w, dy, to, 0, kPast);
                    else if (words) __builtin_amdgcn_raw_buffer_store_b128(w, dy, to, 0, 0);
                    else if (m0 + top + r < p.M) __builtin_memcpy(rows + to, &w, 16);   // (any 2 bytes)
                }
            }
            continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int at = n + 16 * q;
            float v[8];
            eight(q, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int to = at + j < N ? (m * N + at + j) * el : kNowhere;
                if (el == 4) {
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[j]), dy, to, 0, 0);
                } else {
                    union { __bf16 h; uint16_t w; } o;
                    o.h = __bf16(v[j]);
                    __builtin_amdgcn_raw_buffer_store_b16(o.w, dy, to, 0, 0);
                }
            }
        }
    }
}

// kEven: K is a multiple of 128.
template <int kX, int kM, bool kEven>
__global__ __launch_bounds__(256, 2) void mx4_tile_kernel(const Mx4Launch p, int64_t tiles_m,
                                                          int64_t tiles_n) {
    using L = Tile<kX, kM>;
    __shared__ L sh;
    int64_t m0, n0;
    if (!tile_of(tiles_m, tiles_n, m0, n0)) return;
    m0 *= L::kRowsM;
    n0 *= L::kRowsN;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave & 1, wm = wave >> 1;
    const int row = lane & 31, g = lane >> 5;
    const int K = int(p.K), kb = K / 32, row_w = K / 2, row_x = kX == kX4 ? K / 2 : K;
    const __amdgpu_buffer_rsrc_t dw = rows_from(p.wq, n0, p.N, L::kRowsN, row_w);
    const __amdgpu_buffer_rsrc_t dx = rows_from(p.x, m0, p.M, L::kRowsM, row_x);
    const __amdgpu_buffer_rsrc_t dwe = rows_from(p.w_exps, n0, p.N, L::kRowsN, kb);
    const __amdgpu_buffer_rsrc_t dxe = rows_from(p.x_scale, m0, p.M, L::kRowsM, kX == kX4 ? kb : 0);

    constexpr int kLoadW = L::kPiecesW / 256, kLoadX = L::kPiecesX / 256, kLoad = kLoadW + kLoadX;
    constexpr int kPer = L::kBytesX / 16, kLoadE = L::kScales / 256;
    // piece tid + 256 i: rows 64 (or 32) apart, whose turns are alike
    const int cw = ((tid & 3) ^ turn_w(tid >> 2)) * 16, ow = (tid >> 2) * row_w + cw;
    const int cx = ((tid % kPer) ^ turn_x<kX>(tid / kPer)) * 16, ox = tid / kPer * row_x + cx;
    u32x4 re[kLoadE];
    // sets of a stage's columns on their way; as many as the registers hold where a compute unit has but one
    // workgroup (5120 x 5120, 256 rows of x in 4 bits: 15.9 us with two, 13.0 with four, 13.4 with eight)
    constexpr int kSets = kM == 1 || (kM == 2 && kX == kX4) ? 4 : 2;
    struct Moved {
        u32x4 v[kLoad];
    } set[kSets];
    // piece i of a thread: weights' first; what lies behind the last column is 0
    auto fetch = [&](int s, int i, Moved& r) {
        if (i < kLoadW)
            r.v[i] = __builtin_amdgcn_raw_buffer_load_b128(
                dw, kEven || s * 64 + cw < row_w ? ow : kNowhere, s * 64 + i * 64 * row_w, 0);
        else
            r.v[i] = __builtin_amdgcn_raw_buffer_load_b128(
                dx, kEven || s * L::kBytesX + cx < row_x ? ox : kNowhere,
                s * L::kBytesX + (i - kLoadW) * (256 / kPer) * row_x, 0);
    };
    auto keep = [&](int to, int i, const Moved& r) {
        if (i < kLoadW) sh.w[to][tid + 256 * i] = r.v[i];
        else sh.x[to][tid + 256 * (i - kLoadW)] = r.v[i];
    };
    // a thread a row: the weights' first, then those of x, then none
    auto fetch_e = [&](int block) {
#pragma unroll
        for (int i = 0; i < kLoadE; ++i) {
            const int r0 = 256 * i + 64 * wave, r = tid + 256 * i;
            const bool w = r0 < L::kRowsN;
            re[i] = exponents<kEven>(w ? dwe : dxe, r0 < L::kUsed ? (w ? r : r - L::kRowsN) * kb : kNowhere,
                                     block, kb);
        }
    };
    auto keep_e = [&](int block) {      // 0 behind a row's end: the codes there are 0 as well
#pragma unroll
        for (int i = 0; i < kLoadE; ++i) {
            const u32x4 w = in_place<kEven>(re[i], block, kb);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sh.e[block & 1][c][tid + 256 * i] = 4 * (4 * block + c) < kb ? w[c] : 0;
        }
    };

    // Operands of a wave are the first + a constant: dealt() and 32 t leave the bits of the turns alone.
    const int rn = 64 * wn + dealt(0, row), rm = 32 * kM * wm + row;
    const int at_w = rn * 4, tw = turn_w(rn), at_x = rm * kPer, tx = turn_x<kX>(rm);
    f32x16 acc[2][kM] = {};
    const int stages = (K + 127) / 128;
    // Stage 4 block + j.  While a stage's products run, the next one's columns go into the other buffer and,
    // every second stage, those of two more are fetched, both halves of a line one after the other; in steps
    // of two products, whose order the compiler keeps.
    auto stage = [&](int block, auto j) {
        constexpr int kJ = decltype(j)::value, from = kJ & 1;
        const int s = 4 * block + kJ;
        const uint32_t* e = sh.e[block & 1][kJ];      // a row's four blocks
        i32x8 a[2][2] = {}, b[2] = {};        // weights: half of the stage, product
        int sa[2], sb[kM];       // from block g on
        auto read_w = [&](int h, int u) {
            const u32x4 v = sh.w[from][at_w + 16 * u + ((2 * h + g) ^ tw)];
#pragma unroll
            for (int c = 0; c < 4; ++c) a[h][u][c] = int(v[c]);
            if (h == 0) sa[u] = int(e[rn + 4 * u] >> (8 * g));
        };
        auto read_x = [&](int step) {
            const int o = step & 1, h = step / kM, t = step % kM;
            if constexpr (kX == kX4) {
                const u32x4 v = sh.x[from][at_x + 128 * t + ((2 * h + g) ^ tx)];
#pragma unroll
                for (int c = 0; c < 4; ++c) b[o][c] = int(v[c]);
                if (h == 0) sb[t] = int(e[L::kRowsN + rm + 32 * t] >> (8 * g));
            } else {
                const u32x4 v = sh.x[from][at_x + 256 * t + ((4 * h + g) ^ tx)];
                const u32x4 w = sh.x[from][at_x + 256 * t + ((4 * h + 2 + g) ^ tx)];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    b[o][c] = int(v[c]);
                    b[o][4 + c] = int(w[c]);
                }
            }
        };
        read_x(0);
        read_w(0, 0);
        read_w(0, 1);
#pragma unroll
        for (int step = 0; step < 2 * kM; ++step) {
            const int h = step / kM, t = step % kM, o = step & 1;
            if (step + 1 < 2 * kM) read_x(step + 1);
            if (step < 2) read_w(1, step);
#pragma unroll
            for (int i = step; i < kLoad; i += 2 * kM) {
                keep(from ^ 1, i, set[(kJ + 1) % kSets]);
                if constexpr (from == 0) {
                    fetch(s + kSets, i, set[kJ % kSets]);
                    fetch(s + kSets + 1, i, set[(kJ + 1) % kSets]);
                }
            }
            if constexpr (kX == kX8) {
                i32x8 large;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    large[c] = from_two(b[o][c]);
                    b[o][c] ^= large[c];
                }
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const i32x8& x = part ? b[o] : large;
                        acc[u][t] = h == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                                 a[h][u], x, acc[u][t], 4, 0, 0, sa[u], 0, 127)
                                           : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                                 a[h][u], x, acc[u][t], 4, 0, 2, sa[u], 0, 127);
                    }
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    acc[u][t] = h == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                             a[h][u], b[o], acc[u][t], 4, 4, 0, sa[u], 0, sb[t])
                                       : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                             a[h][u], b[o], acc[u][t], 4, 4, 2, sa[u], 2, sb[t]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // (pinned: the compiler would move products behind branches that follow)
#pragma unroll
        for (int t = 0; t < kM; ++t) asm volatile("" : "+v"(acc[0][t]), "+v"(acc[1][t]));
        if constexpr (kJ == 3) keep_e(block + 1);
        if constexpr (kJ == 0) fetch_e(block + 1);
        __syncthreads();
    };
#pragma unroll
    for (int i = 0; i < kLoad; ++i) {
        fetch(0, i, set[0]);
        fetch(1, i, set[1]);
    }
    fetch_e(0);
#pragma unroll
    for (int j = 2; j < kSets; j += 2)
#pragma unroll
        for (int i = 0; i < kLoad; ++i) {
            fetch(j, i, set[j]);
            fetch(j + 1, i, set[j + 1]);
        }
#pragma unroll
    for (int i = 0; i < kLoad; ++i) keep(0, i, set[0]);
    keep_e(0);
    __syncthreads();
    // four stages at a time without a branch, so that the waits inside are counted for what they wait
    const std::integral_constant<int, 0> j0;
    const std::integral_constant<int, 1> j1;
    const std::integral_constant<int, 2> j2;
    const std::integral_constant<int, 3> j3;
    int block = 0;
    for (; 4 * block + 4 <= stages; ++block) {
        stage(block, j0);
        stage(block, j1);
        stage(block, j2);
        stage(block, j3);
    }
    if (4 * block < stages) stage(block, j0);
    if (4 * block + 1 < stages) stage(block, j1);
    if (4 * block + 2 < stages) stage(block, j2);
    settle();      // (a product of 32 by 32 takes up to twice the wait)
    settle();
    // (no wave reads columns from LDS any more)
    static_assert(sizeof(L) >= 4 * 512 * sizeof(u32x4), "8 KB a wave");
    store_tile<kX, kM>(p, m0, n0, wn, wm, lane, acc, reinterpret_cast<u32x4*>(&sh) + 512 * wave);
}

template <int kX, int kM>
hipError_t launch_tiles(const Mx4Launch& p, hipStream_t s) {
    const int64_t m = (p.M + 64 * kM - 1) / (64 * kM), n = (p.N + 127) / 128;
    const dim3 grid(unsigned((m * n + 7) / 8 * 8));
    if (p.K % 128 == 0)
        hipLaunchKernelGGL((mx4_tile_kernel<kX, kM, true>), grid, dim3(256), 0, s, p, m, n);
    else
        hipLaunchKernelGGL((mx4_tile_kernel<kX, kM, false>), grid, dim3(256), 0, s, p, m, n);
    return hipGetLastError();
}

template <int kTiles, int kX, int kWaves>
hipError_t launch_rows(const Mx4Launch& p, hipStream_t s) {
    const dim3 grid(unsigned((p.N + 15) / 16), unsigned((p.M + 16 * kTiles - 1) / (16 * kTiles)));
    hipLaunchKernelGGL((mx4_rows_kernel<kTiles, kX, kWaves>), grid, dim3(64 * kWaves), 0, s, p);
    return hipGetLastError();
}

template <int kX>
hipError_t launch_mm(const Mx4Launch& p, hipStream_t s) {
    const Mx4Plan m = mx4_plan(p.M, p.N, p.K, kX != kX4);
    if (m.tiled) {
        if (m.high == 1) return launch_tiles<kX, 1>(p, s);
        if constexpr (kX == kX4)
            if (m.high == 4) return launch_tiles<kX, 4>(p, s);
        return launch_tiles<kX, 2>(p, s);
    }
    if (m.high == 4) return launch_rows<4, kX, 8>(p, s);
    if (m.high == 2) return m.waves == 16 ? launch_rows<2, kX, 16>(p, s) : launch_rows<2, kX, 8>(p, s);
    return m.waves == 16 ? launch_rows<1, kX, 16>(p, s) : launch_rows<1, kX, 8>(p, s);
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
    return p.fp8 ? launch_mm<kX8>(p, s) : launch_mm<kX4>(p, s);
}

}  // namespace ss
