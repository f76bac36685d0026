// Host bounds harness of the plans in ss_gr_plan.h (gated recurrence, layer norm, microscaled products),
// built with -fsanitize=address,undefined by tests/test_sanitize_gr.py.
//
// For every dims it tries (the benchmark's sizes, the largest of each kind, a seeded sweep, invalid and
// overflowing dims) it checks what the kernels assume: the workspace's regions lie inside it and apart,
// with their sizes recomputed in 128-bit arithmetic; a wave's rows and a tile's rows stay within a
// descriptor's 2^31 bytes; a norm's row fits its threads, in a shape that has a kernel; grids fit the
// runtime's 32 bits.  Prints "gr plan bounds ok: of <tried> taken <accepted>" and exits 0, or
// names the first failing case.
#include <algorithm>
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ss_gr_plan.h"

namespace {

using u128 = unsigned __int128;
using i128 = __int128;

constexpr i128 kDescriptor = i128(1) << 31;

int g_cases = 0, g_taken = 0;

struct Region {
    const char* name;
    u128 off, bytes, align;
};

[[noreturn]] void fail(const char* what, int64_t a, int64_t b, int64_t c, int64_t d) {
    std::printf("FAIL %s: %" PRId64 " %" PRId64 " %" PRId64 " %" PRId64 "\n", what, a, b, c, d);
    std::exit(1);
}

void check_regions(const std::vector<Region>& rs, u128 total, int64_t a, int64_t b, int64_t c, int64_t d) {
    for (size_t i = 0; i < rs.size(); ++i) {
        if (rs[i].off % rs[i].align != 0 || rs[i].off + rs[i].bytes > total) fail(rs[i].name, a, b, c, d);
        for (size_t j = 0; j < i; ++j)
            if (rs[i].bytes && rs[j].bytes && rs[i].off < rs[j].off + rs[j].bytes &&
                rs[j].off < rs[i].off + rs[i].bytes)
                fail("overlap", a, b, c, d);
    }
}

void check_gr(int64_t B, int64_t T, int64_t D, int64_t st, float c = 8.0f) {
    ss_gr_dims d{B, T, D, {st ? 1 : 0, st}, {0, 0}, {0, 0}, int32_t(D & 1), c};
    for (int form = 0; form < 3; ++form) {          // forward, gradient, gradient with checkpoints
        ss::GrPlan p;
        ++g_cases;
        if (ss::make_gr_plan(d, form > 0, form == 2, &p) != SS_OK) continue;
        ++g_taken;
        std::vector<Region> rs;
        u128 words = 0;
        auto chain = [&](const ss::GrChain& k, int64_t tokens, const char* name) {
            if (k.tiles == 0) return;
            if (i128(k.tiles) * tokens < T || i128(k.tiles - 1) * tokens >= T) fail("tiles", B, T, D, form);
            if (i128(k.groups) * k.group < k.tiles) fail("groups", B, T, D, form);
            if (k.tiles == 1) return;
            const u128 maps = u128(B) * k.tiles * D, ends = u128(B) * k.groups * D;
            words += maps + ends;
            rs.push_back({name, k.off_ticket, 4, 8});
            rs.push_back({name, k.off_maps, 8 * maps, 8});
            rs.push_back({name, k.off_ends, 8 * ends, 8});
            if (u128(k.off_ends) != k.off_maps + 8 * maps) fail("ends", B, T, D, form);
        };
        chain(p.fwd, ss::kGrFwdTile, "forward chain");
        chain(p.rev, SS_GR_CKPT, "gradient chain");
        if (words != u128(p.words)) fail("words", B, T, D, form);
        // one launch sets them, 16 bytes at a time, and both counters
        const u128 set = words ? p.off_words + (words + 1) / 2 * 16 : 0;
        if (set > p.total) fail("padding", B, T, D, form);
        if (form > 0) {
            const u128 row = u128(B) * p.rev.tiles * D * 4;
            if (form == 1) rs.push_back({"checkpoints", p.off_ckpt, row, 16});
            rs.push_back({"partial sums", p.off_part, row, 16});
            if (u128(form == 1 ? p.off_ckpt : p.off_part) < set) fail("set over others", B, T, D, form);
        }
        check_regions(rs, p.total, B, T, D, form);
        const i128 cols = i128(B) * ((D + 127) / 128);
        if (cols * p.fwd.tiles * 512 >> 32 || cols * p.rev.tiles * 512 >> 32) fail("grid", B, T, D, form);
        const int64_t step = T == 1 ? D : std::max(st, D);
        if ((i128(15) * step + D) * 4 >= kDescriptor) fail("a wave's rows", B, T, D, form);
        if (form == 0 && ss::gr_walks(T, int64_t(cols), step) &&
            ((i128(T) + 7) * step + D) * 4 >= kDescriptor)
            fail("a walk's rows", B, T, D, form);
    }
}

void check_ln(int64_t M, int64_t D, int q8) {
    const int shapes[] = {81, 321, 641, 642, 643, 644, 645, 646, 2561, 3201, 3841, 5121, 5122, 10242, 10244};
    for (int form = 0; form < 4; ++form) {           // forward, backward; float32, bfloat16
        const bool backward = form & 1;
        const int32_t t = form >> 1 ? SS_BF16 : SS_F32;
        ss_ln_dims d{M, D, t, t, backward ? int32_t(SS_Q8_NONE) : q8, 1e-5f};
        ss::RmsPlan p;
        ++g_cases;
        if (ss::make_ln_plan(d, backward, &p) != SS_OK) continue;
        ++g_taken;
        if (i128(p.threads) * p.pieces * 8 < D) fail("norm's row", M, D, p.threads, p.pieces);
        const int shape = p.threads * 10 + p.pieces;
        if (std::find(std::begin(shapes), std::end(shapes), shape) == std::end(shapes))
            fail("norm without a kernel", M, D, p.threads, p.pieces);
        if (backward && p.pieces > 2 && p.threads != 1024) fail("gradient without a kernel", M, D, p.threads, p.pieces);
        if (p.grid < 1 || i128(p.grid) * std::max(p.threads, 256) >> 32) fail("norm's grid", M, D, p.grid, form);
        if (backward && u128(p.total) < u128(p.grid) * 2 * D * 4) fail("norm's sums", M, D, p.grid, form);
        if (!backward && p.total != 0) fail("norm's workspace", M, D, p.grid, form);
    }
}

void check_mx4(int64_t M, int64_t N, int64_t K) {
    for (int fp8 = 0; fp8 < 2; ++fp8) {
        ss_mx4_dims d{M, N, K, SS_BF16, fp8 ? int32_t(SS_Q8_FP8) : int32_t(SS_Q4_MX), SS_F32};
        ++g_cases;
        if (ss::check_mx4(d, true) != SS_OK) continue;
        ++g_taken;
        const ss::Mx4Plan p = ss::mx4_plan(M, N, K, fp8);
        const i128 row_w = K / 2, row_x = fp8 ? K : K / 2;
        const i128 tall = (p.tiled ? 64 : 16) * p.high, wide = p.tiled ? 128 : 16;
        if (p.tiled ? !(p.high == 1 || p.high == 2 || (p.high == 4 && !fp8))
                    : !((p.high == 4 && p.waves == 8) || ((p.high == 1 || p.high == 2) && (p.waves == 8 || p.waves == 16))))
            fail("product without a kernel", M, N, K, fp8);
        if (p.tiled && p.high > 1 && M <= 32 * p.high) fail("a tile taller than its rows", M, N, K, fp8);
        // two stages beyond the last are asked for (and are behind the descriptor's end, or not issued)
        if (wide * row_w >= kDescriptor || tall * row_x >= kDescriptor) fail("a tile's operands", M, N, K, fp8);
        if (p.tiled && tall * N * 4 >= kDescriptor) fail("a tile's results", M, N, K, fp8);
        const i128 m = (M + tall - 1) / tall, n = (N + wide - 1) / wide;
        if (p.tiled ? (m * n + 7) / 8 * 8 * 256 >> 32 : (m > 65535 || m * n * 64 * p.waves >> 32))
            fail("a product's grid", M, N, K, fp8);
    }
}

uint64_t g_rng = 0x9E3779B97F4A7C15ull;
uint64_t rnd(uint64_t n) {   // xorshift64*, uniform enough for picking cases
    g_rng ^= g_rng >> 12; g_rng ^= g_rng << 25; g_rng ^= g_rng >> 27;
    return (g_rng * 0x2545F4914F6CDD1Dull) % n;
}
int64_t spread(int bits) { return 1 + int64_t(rnd(uint64_t(1) << (1 + rnd(bits)))); }

}  // namespace

int main(int argc, char**) {
    if (argc > 1) {      // the checks' own test: a region past the end, and two that overlap
        check_regions({{"inside", 0, 256, 8}, {"planted overlap", 128, 512, 8}}, 1024, 0, 0, 0, 0);
        return 0;
    }
    const int64_t gr[][3] = {{2, 37, 75}, {8, 2048, 5120}, {1, 262144, 256}, {4, 4096, 2048}, {3, 203, 100},
                             {256, 1, 5120}, {1, 1, 1}, {65535, 1, 1}, {65535, 128, 16}, {1, 128, 1 << 24},
                             {1, (1 << 23) - 1, 1}, {1, 1 << 29, 1}, {1, (int64_t(1) << 29) - 64, 128}};
    for (const auto& s : gr)
        for (int64_t st : {int64_t(0), int64_t(1), s[2], 3 * s[2] + 5, int64_t(1) << 25, (int64_t(1) << 25) + 1})
            check_gr(s[0], s[1], s[2], st);
    const int64_t bad[][3] = {{0, 1, 1}, {1, 0, 1}, {1, 1, 0}, {-1, 1, 1}, {65536, 1, 1}, {1, 1, (1 << 24) + 1},
                              {INT64_MAX, INT64_MAX, INT64_MAX}, {1, INT64_MAX, 1}, {2, INT64_MAX / 2, 1 << 24},
                              {1, 1, INT64_MAX}};
    for (const auto& s : bad) {
        ss::GrPlan p;
        ss_gr_dims d{s[0], s[1], s[2], {0, 0}, {0, 0}, {0, 0}, SS_BF16, 8.0f};
        for (int form = 0; form < 3; ++form)
            if (ss::make_gr_plan(d, form > 0, form == 2, &p) == SS_OK) fail("accepted", s[0], s[1], s[2], form);
        for (int64_t k : {s[0], s[1], s[2]}) check_mx4(s[0], s[1], k), check_ln(s[0], k, SS_Q8_NONE);
    }
    for (int64_t D = 1; D <= 32768; D += D < 9000 ? 1 : 37)
        for (int64_t M : {int64_t(1), int64_t(1023), int64_t(1024), int64_t(100000)}) check_ln(M, D, D % 32 ? int(rnd(3)) : int(rnd(4)));
    check_ln(int64_t(1) << 40, 32768, SS_Q8_NONE);
    for (int i = 0; i < 60000; ++i) {
        const int64_t B = std::min<int64_t>(spread(15), 65535), T = spread(i % 3 ? 12 : 28), D = spread(i % 5 ? 13 : 23);
        check_gr(B, T, D, i % 2 ? 0 : spread(25));
        check_mx4(spread(i % 4 ? 14 : 31), spread(i % 3 ? 15 : 27), 32 * spread(i % 7 ? 9 : 18));
    }
    for (int64_t N : {int64_t(1) << 20, (int64_t(1) << 20) - 1, (int64_t(1) << 27) - 16})
        for (int64_t M : {1, 16, 17, 32, 33, 64, 65, 257, 4096, 8192})
            for (int64_t K : {32, 2048, 2560, (1 << 23) - 32}) check_mx4(M, N, K);
    std::printf("gr plan bounds ok: of %d taken %d\n", g_cases, g_taken);
    return 0;
}
