// Prints the path of feed-forward calls, one line each, from the library's own
// plans on a device of 148 SMs.  Arguments, per call:
//   kind (linear | gated | linear_grad | gated_grad) dtype act residual keep M N K
// Output: "decode/<rows per thread>", or "<token tile>/<epilogue groups>/<how
// tiles are cut>": c2, c4 (over a cluster), whole (at most one a CTA), whole+
// (several), splitS (fewer tiles than SMs, summed through the workspace),
// leftover (the last ones summed through it).
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "decode.cuh"
#include "tile_plan.h"

using namespace sherry;

int main(int argc, char** argv)
{
    const int sms = 148;
    for (int i = 1; i + 7 < argc; i += 8) {
        const bool gated = !std::strncmp(argv[i], "gated", 5), grad = std::strstr(argv[i], "grad") != nullptr;
        const int dt = std::atoi(argv[i + 1]), act = std::atoi(argv[i + 2]);
        const bool res = std::atoi(argv[i + 3]) != 0, keep = std::atoi(argv[i + 4]) != 0;
        const int64_t M = std::atoll(argv[i + 5]), N = std::atoll(argv[i + 6]), K = std::atoll(argv[i + 7]);
        const int64_t R = gated ? 2 * N : N;
        decode::Plan dp;
        if (!grad && M <= SHERRY_GEMM_DECODE_AUTO_MAX_M &&
            decode::plan(R, sherry_k_chunks(K), M, sms, &dp, decode::ep_rt_first(R, M, sms))) {
            std::printf("decode/%d\n", dp.RT);
            continue;
        }
        const TilePlan p = grad ? grad_plan(dt, M, R, K, sms) : forward_plan(dt, act, res, keep, gated, M, R, K, sms);
        const int64_t T = ceil_div(grad ? digit_rows(dt, M) : M, p.bn) * sherry_row_tiles(grad ? K : R);
        std::printf("%d/%d/%s\n", p.bn, p.eg,
                    p.cluster == 2          ? "c2"
                    : p.cluster == 4        ? "c4"
                    : split_tiles(p, T) > 0 ? (T < sms ? "splitS" : "leftover")
                    : T > sms               ? "whole+"
                                            : "whole");
    }
    return 0;
}
