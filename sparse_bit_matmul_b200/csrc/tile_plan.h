// Choice of token tile and grid for the tensor-core launches (host).
#pragma once

#include <algorithm>
#include <cstdint>

namespace sherry {

// Token tile of the tensor-core kernel for M tokens (the dispatch of
// sherry_gemm_tc and sherry_w4a8_gemm_tc; the largest that splits tiles in
// the feed-forward entry points).
inline int tc_token_tile(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M < 1536 ? 128 : 192; }

// Token tile and grid of a tensor-core launch with M rows of int8 (tokens or
// digit rows), TN row tiles and Kc chunks, by the time each choice is
// estimated to take.  Per CTA: c(BN) us a chunk and e(BN) us for the epilogue
// of its last tile; whole tiles run in rounds of one per SM, and a round lasts
// no less than an epilogue; splitting the leftover tiles (or, with fewer tiles
// than SMs, every tile S ways) evens out the chunks but costs the sums through
// the workspace.  Constants fitted on one B200 to about 900 forced launches of 160
// shapes (forward and gradients, M 5 to 2048, 4 to 112 chunks): the choice is
// on average 0.8 % and at most 16 % above the best of them, the rule of
// sherry_gemm_tc 26 % (K = 1056, N = 2000, M = 1400: 21 us instead of 45;
// K = 4096, N = 4096, M = 700: 25.5 instead of 42.5).
struct TilePlan {
    int bn = 16;
    int64_t grid = 1;
    int whole = 1;
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline TilePlan plan_tiles(int64_t M, int64_t TN, int64_t Kc, int64_t sms)
{
    struct Tile {
        int bn;
        double chunk_us;
    };
    constexpr Tile kTiles[] = {{16, 0.155}, {32, 0.150}, {64, 0.177}, {128, 0.248}, {192, 0.300}};
    TilePlan best;
    double best_us = 1e300;
    for (const Tile& t : kTiles) {
        const int64_t T = ceil_div(M, t.bn) * TN;
        const double e = 0.6 + 0.004 * t.bn, sums = 3.4 + 0.08 * t.bn, tile = t.chunk_us * (double)Kc;
        const double whole = (double)(ceil_div(T, sms) - 1) * std::max(tile, e) + tile + e;
        if (whole < best_us) {
            best_us = whole;
            best = {t.bn, std::min(T, sms), 1};
        }
        // split launches stay within the workspace of sherry_reserve(M, ..)
        if (t.bn > tc_token_tile(M)) continue;
        double split;
        int64_t grid;
        if (T < sms) {
            const int64_t S = std::min(sms / T, Kc);
            if (S < 2) continue;
            grid = T * S;
            split = t.chunk_us * (double)ceil_div(Kc, S) + e + sums;
        } else {
            if (T % sms == 0) continue;
            grid = sms;
            // the sums hold up the epilogue warps; only a long tile behind
            // them hides that (all of it from about 60 us on)
            const double shown = std::min(1.0, std::max(0.0, 1.0 - (tile - 15.0) / 45.0));
            split = tile * (double)T / (double)sms + e + sums * shown;
        }
        if (split < best_us) {
            best_us = split;
            best = {t.bn, grid, 0};
        }
    }
    return best;
}

}  // namespace sherry
