// How the products behind la_linear_* are cut into tiles and parts of their sums: rules on sizes alone, on the
// host (no HIP in here).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace la {

// The workgroups of the few tokens' kernel read all tokens' codes for 16 channels, tiles of 64 x 64 for 64.
// us, that kernel and the tiles: 32 tokens, N = 8192, K = 2048 9.2 and 7.5, N = 2048 5.5 and 7.5, K = 8192
// 13 and 20; 64 tokens 12 and 7.7, 6.9 and 7.6, 21 and 20.
inline int few_tokens(int N, int K) { return N <= 4096 ? (K <= 4096 ? 64 : 32) : 16; }

// The tiles that a product is cut into (of 64 x 64 with two or four steps in LDS), their size, and the workgroups
// that a CU holds.
enum Tiling { kTiles256, kTiles128, kTiles64, kTiles64Deep };
constexpr int kTileSize[] = {256, 128, 64, 64}, kTilesPerCu[] = {1, 2, 3, 2};
inline int64_t gemm_units_of(Tiling t, int64_t I, int64_t J, int parts) {
    const int n = kTileSize[t];
    return (I + n - 1) / n * ((J + n - 1) / n) * parts;
}

inline int gemm_steps(int64_t kbytes, int shift) { return static_cast<int>((kbytes + 127) >> 7) << shift; }

// The tiles and parts of a product of I x J results with `steps` steps, by what they would take in
// microseconds: a launch's fixed time, and for every round of workgroups that the chip holds its steps,
// which are slower the fuller it is; parts write their sums, and a second kernel reads them (4 TB/s).
// Measured, us a step from a few workgroups to all: 256 x 256 1.1 to 1.75, 128 x 128 0.42 to 1.2 (two a CU),
// 64 x 64 0.27 to 0.65 (three a CU), with four steps in LDS 0.25 to 0.47 (two a CU).  256 tokens, 8192 channels,
// K = 2048 in 8 bits: 27, 13, 10 and 11 us; 2048 tokens: 36, 40, 65 and 65 us; 256 tokens, 2048 channels, K = 8192:
// 82, 39, 26 and 21 us; 1552 x 512 results over 4000 in FP16: one part 89, 50, 33 and 22 us, four 31, 18, 22 and 20.
// Short sums are not measured for all tilings, and stores are not in the model: 2000 x 1552 over 512 to FP32 takes
// 12 us where it says 7, 777 x 2305 over 1040 11 where it says 8.
struct Cut {
    Tiling tiling;
    int parts;
    float us;
};
inline float tiles_us(Tiling t, int64_t units, int steps) {
    constexpr struct { float fixed, few, full; } kinds[] = {{7.0f, 1.1f, 1.75f}, {5.0f, 0.42f, 1.2f}, {3.5f, 0.27f, 0.65f}, {3.5f, 0.25f, 0.47f}};
    const int64_t slots = 256 * kTilesPerCu[t];
    const float rest = static_cast<float>(units % slots) / slots;
    return kinds[t].fixed + steps * (static_cast<float>(units / slots) * kinds[t].full + (rest > 0.0f ? kinds[t].few + rest * (kinds[t].full - kinds[t].few) : 0.0f));
}
inline Cut cut_product(int64_t I, int64_t J, int steps, int most_parts) {
    Cut best{kTiles256, 1, tiles_us(kTiles256, gemm_units_of(kTiles256, I, J, 1), steps)};
    for (int k = 0; k < 4; k++) {
        const Tiling t = static_cast<Tiling>(k);
        for (int parts = 1; parts <= most_parts && (parts == 1 || steps / parts >= 4); parts *= 2) {
            float us = tiles_us(t, gemm_units_of(t, I, J, parts), (steps + parts - 1) / parts);
            if (parts > 1) us += 4.0f + static_cast<float>(parts) * I * J * 8e-6f / 4.0f;
            if (us < best.us) best = {t, parts, us};
        }
    }
    return best;
}
// Two products in whole sums whose workgroups the chip holds at once, if one launch of them beats the two cuts:
// both get its tiling (the gradients of 2000 tokens, 512 to 1552 in FP32: 58 us in two launches, 50 in one).
inline bool cut_pair(int64_t I0, int64_t J0, int steps0, Cut& c0, int64_t I1, int64_t J1, int steps1, Cut& c1) {
    bool pair = false;
    float least = c0.us + c1.us;
    for (const Tiling t : {kTiles128, kTiles64, kTiles64Deep}) {
        const int64_t units = gemm_units_of(t, I0, J0, 1) + gemm_units_of(t, I1, J1, 1);
        if (units > 256 * kTilesPerCu[t]) continue;
        const float us = tiles_us(t, units, steps0 > steps1 ? steps0 : steps1);
        if (us < least) least = us, c0 = c1 = {t, 1, us}, pair = true;
    }
    return pair;
}

// The tiles of la_linear_fwd beyond the few tokens' kernel.
inline Cut cut_forward(int M, int N, int K) { return cut_product(N, M, gemm_steps(K, 0), 1); }

// The products of la_linear_bwd: dx sums over N and dweight over M, in chunks of 64 elements with 1 << kShift
// parts of each.
constexpr int kShift = 1;
struct GradientCuts {
    Cut dx, dw;
    bool pair;  // in one launch where both are wanted (each is cut the same alone: the same bits)
};
inline GradientCuts cut_gradients(int M, int N, int K) {
    const auto most = [](int64_t n) { return n <= (int64_t{1} << 30) ? 16 : 1; };  // (the join's grid)
    const int64_t m = M, n = N, k = K, mc = (m + 63) / 64, nc = (n + 63) / 64;
    const int steps_x = gemm_steps(nc * 128, kShift), steps_w = gemm_steps(mc * 128, kShift);
    GradientCuts c{cut_product(k, m, steps_x, most(m * k)), cut_product(k, n, steps_w, most(n * k)), false};
    c.pair = cut_pair(k, m, steps_x, c.dx, k, n, steps_w, c.dw);
    return c;
}

}  // namespace la
