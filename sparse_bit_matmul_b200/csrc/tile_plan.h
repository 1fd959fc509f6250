// Choice of token tile and grid for the tensor-core launches (host).
#pragma once

#include <algorithm>
#include <cstdint>

#include "sherry.h"
#include "sherry_internal.h"

namespace sherry {

// Token tile of the tensor-core kernel for M tokens (the dispatch of
// sherry_gemm_tc and sherry_w4a8_gemm_tc; the largest that splits tiles in
// the feed-forward entry points).
inline int tc_token_tile(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M < 1536 ? 128 : 192; }

// Token tile, epilogue groups and grid of a tensor-core launch with M rows of
// int8 (tokens or digit rows), TN row tiles and Kc chunks, by the time each
// choice is estimated to take.  Per CTA: c us a chunk and e us for the
// epilogue of a tile (w: the weight of the epilogue's arithmetic, 1 for a bare
// linear layer).  Whole tiles run in rounds of one per SM; but for the last, a
// round lasts as long as its chunks, or as its epilogue and the part of the
// chunks' issue that does not fit beside it.  A second epilogue group cuts the
// epilogue's share to a third and, one decoder group fewer, slows the chunks.
// Splitting the leftover tiles (or, with fewer tiles than SMs, every tile S
// ways) evens out the chunks but costs the sums through the workspace; small
// tiles are split within a cluster instead.
// Constants fitted on one B200 to about 1200 forced launches of 220 shapes
// (forward and gradients, M 5 to 2048, 1 to 112 chunks): the choice is on
// average 1.3 % and at most 16 % above the best of them; the rule of
// sherry_gemm_tc was 26 % above it (K = 1056, N = 2000, M = 1400: 21 us instead
// of 45; K = 4096, N = 4096, M = 700: 25.5 instead of 42.5), and one epilogue
// group 20 to 40 % on long batches of few chunks (M = 2048, N = 4096, gelu with
// residual, fp32: K = 768 68 -> 46 us, K = 4096 89 -> 72 us).  The clusters'
// constants come from 54 shapes of few rows (M 4 to 64): there the choice is
// 0.9 % above the best and at most 8 %, without clusters 7 % and up to 42 % (K = 14336,
// N = 4096, M = 16: 15.4 -> 13.3 us).  Clusters of eight never won and, at 128
// CTAs, lost 5 to 10 us: not all of them are resident.
struct TilePlan {
    int bn = 16;
    int eg = 1;
    int64_t grid = 1;
    int whole = 1;
    int cluster = 0;            // CTAs per tile
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// grad: the launch reads the transposed weight (kEpGrad).  split_bn: the
// largest tile that may be split through the workspace.
inline TilePlan plan_tiles(int64_t M, int64_t TN, int64_t Kc, int64_t sms, double w, bool grad, int split_bn)
{
    struct Tile {
        int bn, eg;
        double chunk_us;
    };
    // two epilogue groups: the tiles that measured best with them
    const Tile kTiles[] = {{16, 1, 0.159},  {32, 1, 0.154},  {64, 1, 0.172},
                           {128, 1, 0.221}, {192, 1, 0.260}, {grad ? 192 : 64, 2, grad ? 0.291 : 0.205},
                           {128, 2, grad ? 1e9 : 0.263}};
    TilePlan best;
    double best_us = 1e300;
    for (const Tile& t : kTiles) {
        const int64_t T = ceil_div(M, t.bn) * TN;
        const double e = (0.1 + 0.026 * t.bn) * w, chunks = t.chunk_us * (double)Kc;
        const double steady = std::max(chunks, (t.eg == 2 ? 0.34 * e : e) + 0.65 * chunks);
        // more than two thirds of the SMs at once slow the small tiles
        const bool crowded = t.bn <= 32 && T <= sms && 3 * T > 2 * sms;
        const double whole = (double)(ceil_div(T, sms) - 1) * steady + chunks + e + (crowded ? 0.5 : 0.0);
        if (whole < best_us) {
            best_us = whole;
            best = {t.bn, t.eg, std::min(T, sms), 1};
        }
        // a cluster of S CTAs per tile, while all clusters are resident (an SM
        // each CTA; a cluster of four may leave SMs of a GPC out)
        for (int S = 2; t.bn <= 32 && S <= 4 && S <= Kc && T * S <= sms * 7 / 8; S *= 2) {
            const double adds = (S == 2 ? 1.4 : 2.0) * (t.bn == 32 ? 1.6 : 1.0) + (3 * T * S > 2 * sms ? 1.5 : 0.0);
            const double us = t.chunk_us * (double)ceil_div(Kc, S) + e + adds;
            if (us < best_us) {
                best_us = us;
                best = {t.bn, 1, T * S, 0, S};
            }
        }
        if (t.eg == 2 || t.bn > split_bn) continue;
        const double sums = 3.6 + 0.075 * t.bn;
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
            const double shown = std::min(1.0, std::max(0.0, 1.0 - (chunks - 15.0) / 45.0));
            split = steady * (double)T / (double)sms + e + sums * shown;
        }
        if (split < best_us) {
            best_us = split;
            best = {t.bn, 1, grid, 0};
        }
    }
    return best;
}

// Tiles of a launch of T that are summed through the workspace, a slot of BN x
// 128 sums and a counter each.
inline int64_t split_tiles(const TilePlan& plan, int64_t T)
{
    return plan.whole || plan.cluster ? 0 : T - T / plan.grid * plan.grid;
}

// With split tiles within the workspace of sherry_reserve(M, ..).
inline TilePlan plan_tiles(int64_t M, int64_t TN, int64_t Kc, int64_t sms, double w, bool grad)
{
    return plan_tiles(M, TN, Kc, sms, w, grad, tc_token_tile(M));
}

// Weight of an epilogue for plan_tiles, beside a bare linear layer's: the
// activation's instructions, the residual, fp32 stores, kept sums.
inline double epilogue_weight(int dtype, int act, bool res, bool acc, bool gated)
{
    const double a = act == SHERRY_ACT_NONE                              ? 0.0
                     : act == SHERRY_ACT_RELU || act == SHERRY_ACT_RELU2 ? 0.1
                     : act == SHERRY_ACT_GELU                            ? 0.7
                                                                         : 0.55;
    const double w = 1.0 + a + (res ? 0.5 : 0.0) + (dtype == SHERRY_F32 ? 0.3 : 0.0) + (acc ? 0.4 : 0.0);
    return gated ? 0.75 * w : w;
}

inline TilePlan forward_plan(int dtype, int act, bool res, bool acc, bool gated, int64_t M, int64_t R, int64_t K, int sms)
{
    return plan_tiles(M, sherry_row_tiles(R), sherry_k_chunks(K), sms, epilogue_weight(dtype, act, res, acc, gated), false);
}

// Rows of int8 digits of M tokens' gradients: four a token, or 16 for five.
inline int64_t digit_rows(int dtype, int64_t M)
{
    return dtype == SHERRY_F32 ? 4 * M : (M + 4) / 5 * 16;
}

// sherry_grad_digits
inline int grad_digits(int dtype) { return dtype == SHERRY_BF16 ? 2 : dtype == SHERRY_F32 || dtype == SHERRY_F16 ? 4 : 0; }

// Split tiles stay within what sherry_reserve(sherry_grad_digits(dtype) M, ..) sets aside.
inline TilePlan grad_plan(int dtype, int64_t M, int64_t R, int64_t K, int sms)
{
    return plan_tiles(digit_rows(dtype, M), sherry_row_tiles(K), sherry_k_chunks(R), sms, 0.3, true,
                      tc_token_tile(grad_digits(dtype) * M));
}

}  // namespace sherry
