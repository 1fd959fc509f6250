// Host-side check of the feed-forward launches' tile choice (plan_tiles) with
// the kernel's work split (SegWalk), compiled from the library's headers: for
// many token, row-tile and chunk counts and SM counts, the grid has at most one
// CTA per SM, every (tile, chunk) unit is walked exactly once, a launch without
// splits cuts no tile, and a split one uses no larger token tile than
// sherry_reserve(M, ..) sets slots aside for, with its slots inside the grid,
// and a cluster launch gives every tile to one cluster, its first share to the
// first CTA.
// Prints "ok" and exits 0, or prints the first violation and exits 1.
#include <cstdio>
#include <cstdint>
#include <vector>

#include "tc_gemm.cuh"
#include "tile_plan.h"

using namespace sherry;

static int check(int64_t M, int64_t TN, int64_t Kc, int64_t sms, double w, bool grad)
{
    const TilePlan pl = plan_tiles(M, TN, Kc, sms, w, grad);
    tc::Params p{};
    p.TM = (M + pl.bn - 1) / pl.bn;
    p.TN = TN;
    p.Kc = Kc;
    p.U = p.TM * TN * Kc;
    p.whole = pl.whole;
    p.cluster = pl.cluster;
    const char* what = nullptr;
    if (pl.grid < 1 || pl.grid > sms || pl.grid > p.U) what = "grid";
    if (pl.cluster && (pl.bn > 32 || pl.eg != 1 || pl.cluster > 4 || pl.grid != p.TM * TN * pl.cluster || pl.cluster > Kc))
        what = "cluster";
    if (!pl.whole && !pl.cluster && pl.bn > tc_token_tile(M)) what = "split tile larger than the reserved slots";
    // the instantiated kernels
    if (pl.eg == 2 && !(grad ? pl.bn == 192 : pl.bn == 64 || pl.bn == 128)) what = "no such kernel";
    std::vector<uint8_t> seen(p.U, 0);
    for (int64_t b = 0; b < pl.grid && !what; ++b)
        for (tc::SegWalk w(p, b, pl.grid); !w.done() && !what; w.next()) {
            if (w.tile < 0 || w.tile >= p.TM * TN || w.cb < 0 || w.cb >= w.ce || w.ce > Kc) what = "segment";
            else if (pl.whole && !w.complete()) what = "cut tile";
            else
                for (int64_t c = w.cb; c < w.ce; ++c)
                    if (seen[w.tile * Kc + c]++) what = "unit walked twice";
            if (!what && pl.cluster && (w.tile != b / pl.cluster || (w.cb == 0) != (b % pl.cluster == 0))) what = "cluster share";
            if (!what && !w.complete() && !pl.cluster) {
                int64_t bf = 0, bl = 0;
                tc::split_owners(p, w.tile, pl.grid, &bf, &bl);
                if (bf < 0 || bl >= pl.grid || b < bf || b > bl) what = "owners";
            }
        }
    for (int64_t u = 0; u < p.U && !what; ++u)
        if (!seen[u]) what = "unit not walked";
    if (what)
        std::printf("%s: M=%lld TN=%lld Kc=%lld sms=%lld bn=%d grid=%lld whole=%d\n", what, (long long)M, (long long)TN,
                    (long long)Kc, (long long)sms, pl.bn, (long long)pl.grid, pl.whole);
    return what ? 1 : 0;
}

int main()
{
    const int64_t ms[] = {1, 2, 15, 16, 17, 33, 64, 65, 129, 333, 600, 1200, 1535, 1536, 2049, 4100};
    const int64_t tns[] = {1, 2, 7, 16, 32, 40, 112, 149, 224};
    const int64_t kcs[] = {1, 2, 4, 9, 17, 32, 79, 112};
    const int64_t smss[] = {148, 132, 5, 1};
    int n = 0, split = 0, two = 0, clusters = 0;
    for (int64_t M : ms)
        for (int64_t TN : tns)
            for (int64_t Kc : kcs)
                for (int64_t sms : smss) {
                    for (int k = 0; k < 3; ++k) {
                        const double w = k == 0 ? 1.0 : k == 1 ? 2.5 : 0.3;
                        const bool grad = k == 2;
                        if (check(M, TN, Kc, sms, w, grad)) return 1;
                        ++n;
                        split += !plan_tiles(M, TN, Kc, sms, w, grad).whole && !plan_tiles(M, TN, Kc, sms, w, grad).cluster;
                        clusters += plan_tiles(M, TN, Kc, sms, w, grad).cluster > 0;
                        two += plan_tiles(M, TN, Kc, sms, w, grad).eg == 2;
                    }
                }
    if (split == 0 || split == n || two == 0 || two == n || clusters == 0) {
        std::printf("only one kind of launch: %d split, %d with two epilogue groups of %d\n", split, two, n);
        return 1;
    }
    std::printf("ok %d shapes, %d split\n", n, split);
    return 0;
}
