// Launches of the elementwise half of the feed-forward gradients (grad.cuh),
// one kernel per activation and element type.
#include <algorithm>
#include <atomic>

#include "sherry.h"
#include "sherry_internal.h"
#include "host_common.h"
#include "grad.cuh"

namespace sherry {
namespace grad {
namespace {

constexpr int kCacheMax = 200 * 1024;       // bytes of e a block may hold
// The segments of cx blocks per token; returns the block's shared memory for e.
int64_t split_rows(Params& p, int cx)
{
    p.seg = (int)(((p.R + cx - 1) / cx + 15) & ~int64_t(15));
    const int64_t need = 4 * std::min<int64_t>(p.seg, (p.R + 3) & ~int64_t(3));
    p.cached = need <= kCacheMax;
    return p.cached ? need : 0;
}

template <class K>
int allow_cache(K kernel, std::atomic<uint64_t>& done)
{
    return once_per_device(done, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheMax);
    });
}

template <bool GATED, int ACT, int DT>
int digits(Params p, int sms, cudaStream_t stream)
{
    auto kernel = grad_digits_kernel<GATED, ACT, DT>;
    static std::atomic<uint64_t> done{0};
    const int st = allow_cache(kernel, done);
    if (st != SHERRY_OK) return st;
    const int cx = token_blocks(p.M, p.R, sms, 4);
    const int64_t smem = split_rows(p, cx);
    // tokens in grid.y: at most 65535 a launch (whole groups of 16 digit rows)
    Params q = p;
    for (int64_t m0 = 0; m0 < p.M; m0 += 65535) {
        const int64_t left = p.M - m0, n = left < 65535 ? left : 65535;
        q.dy = static_cast<const uint8_t*>(p.dy) + m0 * p.No * (DT == SHERRY_F32 ? 4 : 2);
        q.acc = p.acc ? p.acc + m0 * p.R : nullptr;
        q.x_scale = p.x_scale ? p.x_scale + m0 : nullptr;
        q.dig = p.dig + ep::first_row<kDigits<DT>>(m0) * p.ld;
        q.dscale = p.dscale + m0;
        const cudaError_t e = launch_pdl(kernel, dim3((unsigned)cx, (unsigned)n), dim3(kDigitThreads), (size_t)smem, stream,
                                         dim3((unsigned)cx), q);
        if (e != cudaSuccess) return cuda_status(e);
        q.zero_n = 0;                                        // cleared by the first
    }
    return SHERRY_OK;
}

// Few tokens: the column sums, and with dx the digits, in one launch.
template <bool GATED, int ACT, int DT>
int both(Params p, bool dx, int sms, cudaStream_t stream)
{
    auto kernel = grad_both_kernel<GATED, ACT, DT>;
    static std::atomic<uint64_t> done{0};
    const int st = allow_cache(kernel, done);
    if (st != SHERRY_OK) return st;
    bool whole = false;
    const int c = both_cluster(p.M, p.R, sms, &whole);
    const int64_t smem = split_rows(p, whole ? 1 : c), rb = row_blocks(p.R);
    const int64_t ahead = !dx ? 0 : whole ? (p.M + c - 1) / c : p.M;
    return cuda_status(launch_pdl(kernel, dim3((unsigned)(c * (ahead + rb))), dim3(kDigitThreads), (size_t)smem, stream,
                                  dim3((unsigned)c), p, (uint32_t)ahead, (uint32_t)c, (int)whole));
}

template <bool GATED, int ACT, int DT>
int columns(const Params& p, int sms, cudaStream_t stream)
{
    if (p.M <= kBothMaxTokens) return both<GATED, ACT, DT>(p, false, sms, stream);
    const Columns shape = columns_shape(p.R, sms);
    const unsigned bx = (unsigned)row_blocks(p.R), cy = (unsigned)shape.cluster;
    if (shape.warps == kColWarpsWide)
        return cuda_status(launch_pdl(grad_columns_kernel<GATED, ACT, DT, kColWarpsWide>, dim3(bx, cy),
                                      dim3(32 * kColWarpsWide), 0, stream, dim3(1, cy), p));
    return cuda_status(launch_pdl(grad_columns_kernel<GATED, ACT, DT, kColWarps>, dim3(bx, cy), dim3(32 * kColWarps), 0,
                                  stream, dim3(1, cy), p));
}

template <bool GATED, int ACT, int DT>
int ahead(const Params& p, int sms, cudaStream_t stream)
{
    const bool sums = p.dalpha || p.dbias;
    if (sums && p.M <= kBothMaxTokens) return both<GATED, ACT, DT>(p, true, sms, stream);
    // the digits first: the column sums then find their inputs in the second-level
    // cache (M=2048 K=14336 N=4096 bf16: 295 us for the call, 305 the other way
    // round; gated M=1386 K=1504 N=14319 f16: 333 and 352)
    const int st = digits<GATED, ACT, DT>(p, sms, stream);
    return st != SHERRY_OK || !sums ? st : columns<GATED, ACT, DT>(p, sms, stream);
}

template <bool GATED, int ACT>
int of_type(bool dx, const Params& p, int dtype, int sms, cudaStream_t s)
{
    if (dtype == SHERRY_F32) return dx ? ahead<GATED, ACT, SHERRY_F32>(p, sms, s) : columns<GATED, ACT, SHERRY_F32>(p, sms, s);
    if (dtype == SHERRY_BF16) return dx ? ahead<GATED, ACT, SHERRY_BF16>(p, sms, s) : columns<GATED, ACT, SHERRY_BF16>(p, sms, s);
    return dx ? ahead<GATED, ACT, SHERRY_F16>(p, sms, s) : columns<GATED, ACT, SHERRY_F16>(p, sms, s);
}

template <bool GATED>
int of_act(bool dx, const Params& p, int act, int dtype, int sms, cudaStream_t s)
{
    switch (act) {
    case SHERRY_ACT_NONE: return of_type<GATED, SHERRY_ACT_NONE>(dx, p, dtype, sms, s);
    case SHERRY_ACT_RELU: return of_type<GATED, SHERRY_ACT_RELU>(dx, p, dtype, sms, s);
    case SHERRY_ACT_RELU2: return of_type<GATED, SHERRY_ACT_RELU2>(dx, p, dtype, sms, s);
    case SHERRY_ACT_SILU: return of_type<GATED, SHERRY_ACT_SILU>(dx, p, dtype, sms, s);
    case SHERRY_ACT_GELU: return of_type<GATED, SHERRY_ACT_GELU>(dx, p, dtype, sms, s);
    default: return of_type<GATED, SHERRY_ACT_GELU_TANH>(dx, p, dtype, sms, s);
    }
}

}  // namespace

int launch_ahead(Params p, bool gated, int act, int dtype, int sms, cudaStream_t stream)
{
    return gated ? of_act<true>(true, p, act, dtype, sms, stream) : of_act<false>(true, p, act, dtype, sms, stream);
}

int launch_columns(const Params& p, bool gated, int act, int dtype, int sms, cudaStream_t stream)
{
    return gated ? of_act<true>(false, p, act, dtype, sms, stream) : of_act<false>(false, p, act, dtype, sms, stream);
}

}  // namespace grad
}  // namespace sherry
