// Host-side check of the gradients' launch shapes (grad_plan.h): for many token
// and row counts and SM counts, a column sum is a chain of at most M / 16 + 20
// additions (the tokens of one warp, then the warps of a block, then the blocks
// of a cluster), and clusters are of sizes the kernels are launched with.
// Prints "ok" and exits 0, or prints the first violation and exits 1.
#include <cstdio>
#include <cstdint>

#include "grad_plan.h"

using namespace sherry::grad;

int main()
{
    const int64_t rs[] = {1,    2,    100,   128,   129,   1000,  2048,  2400,   2501,   4096,   5001,    5632,
                          8192, 8193, 10002, 14336, 16385, 28672, 33000, 40000, 57344, 113664, 420003, (1 << 24) - 1};
    int n = 0, wide = 0;
    for (int sms : {148, 132, 16, 1})
        for (int64_t R : rs)
            for (int64_t M = 1; M <= 70000; M = M < 1100 ? M + 1 : M * 5 / 4) {
                int warps, cluster;
                bool whole = false;
                if (M <= kBothMaxTokens) {
                    warps = kDigitThreads / 32;
                    cluster = both_cluster(M, R, sms, &whole);
                } else {
                    warps = columns_shape(R, sms).warps;
                    cluster = columns_shape(R, sms).cluster;
                    wide += warps == kColWarpsWide;
                }
                const int64_t chain = (M + warps * cluster - 1) / (warps * cluster) + warps + (cluster - 1);
                if (cluster < 1 || cluster > kClusterMax || 16 * (chain - 20) > M) {
                    std::printf("M=%lld R=%lld sms=%d: %d warps, cluster %d, chain %lld\n", (long long)M, (long long)R, sms,
                                warps, cluster, (long long)chain);
                    return 1;
                }
                ++n;
            }
    if (!wide) return std::printf("no wide blocks\n"), 1;
    std::printf("ok %d\n", n);
    return 0;
}
