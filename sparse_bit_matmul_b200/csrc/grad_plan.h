// Launch shapes of the gradients' elementwise half (host; kernels in grad.cuh).
//
// A column sum is one fp32 chain per warp over every (warps * cluster)-th token,
// then the warps' sums and the cluster's in order.  Every choice below keeps it
// to at most M / 16 + 20 additions: 16 warps at least share the tokens from 64
// tokens on.
#pragma once

#include <algorithm>
#include <cstdint>

namespace sherry {
namespace grad {

constexpr int kSegMin = 1024;               // weight rows worth a block of their own
constexpr int kSegMax = 8192;               // above, a block's 32 KB keep its neighbours off the SM
constexpr int kClusterMax = 8;
constexpr int kColRows = 128;               // weight rows per block of the column sums
constexpr int kColWarps = 4;
constexpr int kColBlocks = 6;               // resident per SM (registers)
// So few rows that clusters of eight blocks leave SMs idle: blocks of 16 warps.
constexpr int kColWarpsWide = 16;
constexpr int kDigitThreads = 256;
// Digits and column sums in one launch up to here (see grad_both_kernel).
constexpr int64_t kBothMaxTokens = 1024;
constexpr int kBothBlocks = 4;

inline int64_t row_blocks(int64_t R) { return (R + kColRows - 1) / kColRows; }

// More than kBothMaxTokens tokens: blocks that share the columns, and their warps.
struct Columns {
    int warps, cluster;
};

// Of the cluster sizes from four on, the one whose last round of resident blocks
// is fullest; the smallest such.
inline Columns columns_shape(int64_t R, int sms)
{
    const int64_t bx = row_blocks(R), slots = (int64_t)kColBlocks * sms;
    if (bx * kClusterMax < sms) return {kColWarpsWide, kClusterMax};
    int cy = 4;
    double best = 0.0;
    for (int y = 4; y <= kClusterMax; ++y) {
        const int64_t blocks = bx * y, rounds = (blocks + slots - 1) / slots;
        const double full = (double)blocks / (double)(rounds * slots);
        if (full > best + 0.02) {
            best = full;
            cy = y;
        }
    }
    return {kColWarps, cy};
}

// Blocks per token of the digits: so many that a block holds at most kSegMax rows,
// and more while the grid leaves SMs without `per` blocks.
inline int token_blocks(int64_t M, int64_t R, int sms, int per)
{
    int cx = 1;
    while (cx < kClusterMax && (R > (int64_t)cx * kSegMax || (M * cx < per * (int64_t)sms && R >= (int64_t)cx * 2 * kSegMin)))
        cx *= 2;
    return cx;
}

// Up to kBothMaxTokens tokens: the cluster of a launch for both.  whole: a block,
// not a cluster, per token.
inline int both_cluster(int64_t M, int64_t R, int sms, bool* whole)
{
    int c = token_blocks(M, R, sms, 2);
    *whole = c == 1;
    // short rows: clusters for the column sums alone, four tokens a warp, while
    // they leave half the blocks of a round to the digits (M=300 K=512 N=203:
    // 15.7 -> 9.7 us); two blocks at least, for the length of the chains
    if (*whole)
        while (c < kClusterMax && M >= 2 * c * (kDigitThreads / 32) * 4 &&
               (c == 1 || 2 * c * row_blocks(R) <= kBothBlocks / 2 * (int64_t)sms))
            c *= 2;
    return c;
}

}  // namespace grad
}  // namespace sherry
