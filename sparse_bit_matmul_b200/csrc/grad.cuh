// Elementwise halves of the feed-forward gradients (sherry_linear_grad,
// sherry_gated_grad): the gradient of every pre-activation from the kept
// int32 sums, its column sums, and its int8 digits for the tensor cores.
//
//   z = acc * alpha * s (+ bias), as the forward computes it
//   linear  dz = dy act'(z)
//   gated   dz[2n] = dh z[2n+1] act'(z[2n]),  dz[2n+1] = dh act(z[2n])
//   e = dz * alpha;  dx = e . T is sherry_gemm_tc_kernel<.., kEpGrad>
//   dalpha[n] = sum_m dz acc s,  dbias[n] = sum_m dz
//
// Fixed point.  e of a token is scaled to integers v below its largest |e|:
// D = 3 digits (bf16 and fp16 tensors) |v| <= 2^22 - 1, so e is off by at most
// 2^-23 of the token's largest;
// D = 4 (fp32) a power of two with |v| < 2^30, exact for every e within a
// factor 64 of the largest and off by at most 2^-30 of it below.
// The error is the token's, not the term's: beside one |e| r times the others,
// the columns of dx whose weight in that row is 0 (a quarter of them) hold the
// others alone, and are off by about 7e-8 r of themselves (D = 3; D = 4 5e-10 r
// to 3e-10 r).  A bf16 output rounds by 1.7e-3 in the same norm, an fp16 one by
// 2.1e-4: r = 20000 and r = 3000 reach that.  Two digits would reach it at r =
// 200 for bf16 (r = 1000: 0.9 %), and outliers of that size are ordinary behind
// a gate.  Four digits for fp16: M=1386 K=1504, gated to 14319 367 us, three 339.
// v = sum_d 256^d digit_d with digits in [-128, 127]: the integer sums over n
// below 2^24 rows stay inside int32.
#pragma once

#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "grad_plan.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "sherry_internal.h"

namespace sherry {
namespace grad {

struct Params {
    const void* dy;             // [M][No] of dtype
    const int32_t* acc;         // [M][R] or null (linear, act none: z is not needed)
    const float* x_scale;       // [M] (with acc)
    const float* alpha;         // [R]
    const float* bias;          // [R] or null
    int64_t M, R, No;           // R = No, or 2 No when gated
    int8_t* dig;                // [digit rows][ld]: a token's from ep::first_row<D>(m) on
    float* dscale;              // [M]
    int64_t ld;                 // a multiple of 16, >= R; what is past R is not read
    int seg;                    // rows of the weight per block of a cluster, a multiple of 4
    int cached;                 // a block's e fits in its shared memory
    int vec;                    // rows and bases allow 16-byte loads of four rows' values
    float* dalpha;              // [R] or null
    float* dbias;               // [R] or null
    uint4* zero;                // split-K workspace that the digits' launch clears
    int64_t zero_n;
};

// Block `block` of `blocks` clears its share of p.zero.
__device__ __forceinline__ void clear_split(const Params& p, int64_t block, int64_t blocks)
{
    for (int64_t i = block * blockDim.x + threadIdx.x; i < p.zero_n; i += blocks * blockDim.x)
        p.zero[i] = make_uint4(0u, 0u, 0u, 0u);
}

template <int DT>
struct Elem {
    using type = uint16_t;
};
template <>
struct Elem<SHERRY_F32> {
    using type = float;
};
template <int DT>
__device__ __forceinline__ float widen(typename Elem<DT>::type v)
{
    if constexpr (DT == SHERRY_F32) return v;
    else return ep::from16(v, DT);
}

template <int DT>
constexpr int kDigits = DT == SHERRY_F32 ? 4 : 3;

__device__ __forceinline__ float pre_act(int32_t acc, float al, float s, bool has_bias, float b)
{
    const float z = __fmul_rn(__fmul_rn((float)acc, al), s);
    return has_bias ? __fadd_rn(z, b) : z;
}

// A thread's unit is four weight rows.  Where rows and bases allow it (VEC) they
// are consecutive and read 16 bytes at a time.  Elsewhere the k-th is k * step
// rows on (gated: the two pairs are `step` pairs apart), step the number of
// threads side by side, so that every load of a warp is one contiguous piece:
// four consecutive rows a thread measured two to three times the L2 traffic.

// Four values, p[k * step] of the `left` there are from p on.
template <class T>
__device__ __forceinline__ void load4(const T* p, int left, bool vec, int step, T (&v)[4])
{
    if (vec) {
        const uint4 t = __ldcg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) memcpy(&v[k], &w[k], 4);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k * step < left ? __ldcg(p + k * step) : T(0);
    }
}

// The same for rows that come in pairs (8-byte aligned when they are sums).
template <bool GATED>
__device__ __forceinline__ void load_acc(const int32_t* p, int left, bool vec, int step, int32_t (&a)[4])
{
    if (!GATED || vec) {
        load4(p, left, vec, step, a);
    } else {
        const int2 t = 0 < left ? __ldcg(reinterpret_cast<const int2*>(p)) : make_int2(0, 0);
        const int2 u = 2 * step < left ? __ldcg(reinterpret_cast<const int2*>(p + 2 * step)) : make_int2(0, 0);
        a[0] = t.x; a[1] = t.y; a[2] = u.x; a[3] = u.y;
    }
}

// C values of dy (2 or 4), p[k * step] of the `left` there are.
template <int DT, int C>
__device__ __forceinline__ void load_dy(const typename Elem<DT>::type* p, int left, bool vec, int step, float (&g)[C])
{
    using E = typename Elem<DT>::type;
    if (vec) {
        if constexpr (DT == SHERRY_F32) {
#pragma unroll
            for (int k = 0; k < C; k += 2) {
                const float2 t = __ldcg(reinterpret_cast<const float2*>(p + k));
                g[k] = t.x;
                g[k + 1] = t.y;
            }
        } else {
            uint32_t t[C / 2];
            if constexpr (C == 4) {
                const uint2 w = __ldcg(reinterpret_cast<const uint2*>(p));
                t[0] = w.x;
                t[1] = w.y;
            } else {
                t[0] = __ldcg(reinterpret_cast<const uint32_t*>(p));
            }
#pragma unroll
            for (int k = 0; k < C / 2; ++k) {
                g[2 * k] = widen<DT>((E)(t[k] & 0xFFFFu));
                g[2 * k + 1] = widen<DT>((E)(t[k] >> 16));
            }
        }
    } else {
        E h[C];
#pragma unroll
        for (int k = 0; k < C; ++k) h[k] = k * step < left ? __ldcg(p + k * step) : E(0);
#pragma unroll
        for (int k = 0; k < C; ++k) g[k] = widen<DT>(h[k]);
    }
}

// What a unit's rows need of alpha and bias.
struct Rows4 {
    float al[4], b[4];
};
template <bool GATED, bool VEC>
__device__ __forceinline__ void load_row_values(const float* p, int left, int step, float (&v)[4])
{
    if constexpr (GATED && !VEC) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = 2 * (k >> 1) * step + (k & 1);
            v[k] = at < left ? __ldcg(p + at) : 0.0f;
        }
    } else {
        load4(p, left, VEC, step, v);
    }
}
template <bool GATED, bool VEC>
__device__ __forceinline__ Rows4 load_rows(const float* alpha, const float* bias, int left, int step)
{
    Rows4 w;
    load_row_values<GATED, VEC>(alpha, left, step, w.al);
    w.b[0] = w.b[1] = w.b[2] = w.b[3] = 0.0f;
    if (bias) load_row_values<GATED, VEC>(bias, left, step, w.b);
    return w;
}

// dz of a unit of one token, from its sums a and the
// token's dy (two columns when gated)
template <bool GATED, int ACT, int DT, int C>
__device__ __forceinline__ void dz4(const int32_t (&a)[4], const float (&g)[C], const Rows4& w, bool hb, float s,
                                    float (&dz)[4])
{
    if constexpr (GATED) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float f, d;
            ep::act_slope<DT == SHERRY_F32>(pre_act(a[2 * k], w.al[2 * k], s, hb, w.b[2 * k]), ACT, f, d);
            const float up = pre_act(a[2 * k + 1], w.al[2 * k + 1], s, hb, w.b[2 * k + 1]);
            dz[2 * k] = __fmul_rn(__fmul_rn(g[k], up), d);
            dz[2 * k + 1] = __fmul_rn(g[k], f);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f, d;
            ep::act_slope<DT == SHERRY_F32>(pre_act(a[k], w.al[k], s, hb, w.b[k]), ACT, f, d);
            dz[k] = __fmul_rn(g[k], d);
        }
    }
}

// e of units of one token's segment: from row `at` (gated: pair `at`) on.
template <bool GATED, int ACT, int DT, bool VEC>
struct Segment {
    static constexpr int C = GATED ? 2 : 4;
    using E = typename Elem<DT>::type;
    const E* dy;
    const int32_t* acc;
    const float *alpha, *bias;
    float s;
    int rows, cols;             // left in the segment's arrays

    __device__ __forceinline__ Segment(const Params& p, int64_t m, int64_t r0)
    {
        const int64_t c0 = GATED ? r0 >> 1 : r0;
        dy = static_cast<const E*>(p.dy) + m * p.No + c0;
        acc = p.acc ? p.acc + m * p.R + r0 : nullptr;
        alpha = p.alpha + r0;
        bias = p.bias ? p.bias + r0 : nullptr;
        s = p.acc ? p.x_scale[m] : 0.0f;
        rows = (int)(p.R - r0);
        cols = (int)(p.No - c0);
    }
    __device__ __forceinline__ void e4(int at, int step, float (&e)[4]) const
    {
        const int r = GATED ? 2 * at : at;
        float g[C], dz[4];
        int32_t a[4] = {0, 0, 0, 0};
        load_dy<DT, C>(dy + at, cols - at, VEC, step, g);
        if (acc) load_acc<GATED>(acc + r, rows - r, VEC, step, a);
        const Rows4 w = load_rows<GATED, VEC>(alpha + r, bias ? bias + r : nullptr, rows - r, step);
        dz4<GATED, ACT, DT, C>(a, g, w, bias != nullptr, s, dz);
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = __fmul_rn(dz[k], w.al[k]);
    }
};

// One cluster of blocks per token, `seg` weight rows per block: e into shared
// memory (recomputed when it does not fit), the token's largest |e| over the
// cluster, then the digit rows.
// Bound by instruction issue and DRAM in about equal parts: magnitudes are
// compared as integers (one mask and one maximum a value; Inf and NaN order
// above every number), and three digits come out of the low bits of
// e * inv + 1.5 * 2^23 without a conversion instruction.
constexpr uint32_t kInfBits = 0x7F800000u;

template <bool GATED, int ACT, int DT, bool VEC>
__device__ __forceinline__ void grad_digits(const Params& p, int64_t m, uint32_t rank, uint32_t CX, float* cache,
                                            uint32_t* warp_max, uint32_t* block_max)
{
    constexpr int D = kDigits<DT>;
    constexpr int kWarps = kDigitThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t r0 = (int64_t)rank * p.seg;
    const int U = (int)((min(r0 + p.seg, (p.R + 3) & ~int64_t(3)) - r0) >> 2);     // units of four rows, may be <= 0
    const Segment<GATED, ACT, DT, VEC> sg(p, m, r0);
    uint32_t mx = 0;
    // units: rows (gated: pairs) i * kUnit + .. of 4 U; strided ones only go to
    // the cache
    constexpr int kUnit = GATED ? 2 : 4;
    const bool strided = !VEC && p.cached;
    const int step = strided ? kDigitThreads : 1;
#pragma unroll 2
    for (int i = tid; i < U * (strided ? kUnit : 1); i += kDigitThreads * (strided ? kUnit : 1)) {
        const int at = strided ? i : kUnit * i;
        float e[4];
        sg.e4(at, step, e);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = max(mx, __float_as_uint(e[k]) & 0x7FFFFFFFu);
        if (strided) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int to = GATED ? 2 * (at + (k >> 1) * step) + (k & 1) : at + k * step;
                if (to < 4 * U) cache[to] = e[k];
            }
        } else if (p.cached) {
            *reinterpret_cast<float4*>(cache + 4 * i) = make_float4(e[0], e[1], e[2], e[3]);
        }
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) warp_max[tid >> 5] = mx;
    __syncthreads();
    mx = __reduce_max_sync(0xffffffffu, lane < kWarps ? warp_max[lane] : 0u);
    if (CX > 1) {
        if (tid == 0) *block_max = mx;
        ptx::cluster_arrive_release();
        ptx::cluster_wait_acquire();
        uint32_t other = 0;
        if (lane < (int)CX) other = ptx::ld_cluster_u32(ptx::smem_u32(block_max), (uint32_t)lane);
        mx = __reduce_max_sync(0xffffffffu, other);
        ptx::cluster_arrive_release();                       // waited for at the end: the maxima stay readable
    }

    // v = e * inv, dx = sum * sc
    const bool bad = mx >= kInfBits;
    const float big = __uint_as_float(mx);
    float inv = 0.0f, sc = 0.0f;
    if (mx != 0u && !bad) {
        if constexpr (D == 3) {
            if (big >= 7.8886091e-31f) {                     // 2^-100
                inv = __fdiv_rn(4194303.0f, big);
                sc = __fdiv_rn(big, 4194303.0f);
            } else {
                inv = 5.316912e36f;                          // 2^122
                sc = 1.8807910e-37f;
            }
        } else {
            const int ex = (int)(mx >> 23) - 127;            // big < 2^(ex + 1)
            const int k = min(29 - ex, 126);
            inv = __uint_as_float((uint32_t)(127 + k) << 23);
            sc = __uint_as_float((uint32_t)(127 - k) << 23);
        }
    }
    if (bad) sc = __uint_as_float(0x7FC00000u);              // the whole dx row becomes NaN
    if (tid == 0 && rank == 0) p.dscale[m] = sc;
    int8_t* dig = p.dig + ep::first_row<D>(m) * p.ld + r0;
#pragma unroll 2
    for (int u = tid; u < U; u += kDigitThreads) {
        float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (inv != 0.0f) {
            if (p.cached) {
                const float4 t = *reinterpret_cast<const float4*>(cache + 4 * u);
                e[0] = t.x; e[1] = t.y; e[2] = t.z; e[3] = t.w;
            } else {
                sg.e4(kUnit * u, 1, e);
            }
        }
        uint32_t v[4];
        // |v| < 2^22: rint(e inv) in the low bits of the sum, above its bits
        // for 0 (which reach the third byte)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = D < 4 ? __float_as_uint(__fmaf_rn(e[k], inv, quant::kRoundMagic))
                         : (uint32_t)__float2int_rn(__fmul_rn(e[k], inv));
            if constexpr (D < 4) v[k] -= __float_as_uint(quant::kRoundMagic);
        }
        // digit d is byte d of v once 128 was added to every byte below it:
        // (v - digit) / 256 is (v + 128) >> 8 for a digit in [-128, 127]
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const uint32_t sel = (uint32_t)d | (uint32_t)(4 + d) << 4;
            const uint32_t lo = __byte_perm(v[0], v[1], sel), hi = __byte_perm(v[2], v[3], sel);
            *reinterpret_cast<uint32_t*>(dig + d * p.ld + 4 * u) = __byte_perm(lo, hi, 0x5410u);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += 128u << (8 * d);
        }
    }
    if (CX > 1) ptx::cluster_wait_acquire();
}

template <bool GATED, int ACT, int DT>
__device__ __forceinline__ void digits_block(const Params& p, int64_t m, uint32_t rank, uint32_t CX)
{
    extern __shared__ __align__(16) float cache[];
    __shared__ uint32_t warp_max[kDigitThreads / 32];
    __shared__ uint32_t block_max;
    if (p.vec) grad_digits<GATED, ACT, DT, true>(p, m, rank, CX, cache, warp_max, &block_max);
    else grad_digits<GATED, ACT, DT, false>(p, m, rank, CX, cache, warp_max, &block_max);
}

// grid (blocks per token, tokens)
template <bool GATED, int ACT, int DT>
__global__ void __launch_bounds__(kDigitThreads) grad_digits_kernel(const Params p)
{
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    clear_split(p, (int64_t)blockIdx.y * gridDim.x + blockIdx.x, (int64_t)gridDim.x * gridDim.y);
    digits_block<GATED, ACT, DT>(p, blockIdx.y, blockIdx.x, gridDim.x);
}

// Column sums: a block owns the rows of 32 lanes x 4 weight rows, its warps
// (and the blocks of its cluster, which share the columns) take the tokens in
// turn, and the partial sums meet in a fixed order.

// One lane's sums over the tokens m0, m0 + step, ..: the loads of B tokens are
// issued before their arithmetic, without a branch between them; advances m
// and the pointers while B tokens are left.
template <bool GATED, int ACT, int DT, bool VEC, bool ACC>
struct Column {
    static constexpr int C = GATED ? 2 : 4;
    using E = typename Elem<DT>::type;
    const E* dy;
    const int32_t* acc;
    const float* s;
    int64_t dstep, astep, step;
    int64_t m;                  // next token
    int rows, cols;             // left in the arrays' rows
    Rows4 w;
    bool hb;
    static constexpr int kLanes = VEC ? 1 : 32;              // rows (pairs) between a unit's

    template <int B>
    __device__ __forceinline__ void run(int64_t M, float (&sa)[4], float (&sb)[4])
    {
        for (; m + (B - 1) * step < M; m += B * step) {
            float g[B][C], sc[B];
            int32_t a[B][4];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                load_dy<DT, C>(dy, cols, VEC, kLanes, g[i]);
                dy += dstep;
                sc[i] = 0.0f;
                a[i][0] = a[i][1] = a[i][2] = a[i][3] = 0;
                if constexpr (ACC) {
                    load_acc<GATED>(acc, rows, VEC, kLanes, a[i]);
                    acc += astep;
                    sc[i] = __ldcg(s);
                    s += step;
                }
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                float dz[4];
                dz4<GATED, ACT, DT, C>(a[i], g[i], w, hb, sc[i], dz);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sa[k] = __fmaf_rn(dz[k], __fmul_rn((float)a[i][k], sc[i]), sa[k]);
                    sb[k] = __fadd_rn(sb[k], dz[k]);
                }
            }
        }
    }
};

template <bool GATED, int ACT, int DT, bool VEC, bool ACC, int BATCH>
__device__ __forceinline__ void column_sums(const Params& p, int64_t r, int64_t m0, int64_t step, float (&sa)[4],
                                            float (&sb)[4])
{
    Column<GATED, ACT, DT, VEC, ACC> c;
    const int64_t col = GATED ? r >> 1 : r;
    c.dy = static_cast<const typename Elem<DT>::type*>(p.dy) + m0 * p.No + col;
    c.acc = ACC ? p.acc + m0 * p.R + r : nullptr;
    c.s = ACC ? p.x_scale + m0 : nullptr;
    c.step = step;
    c.dstep = step * p.No;
    c.astep = step * p.R;
    c.m = m0;
    c.rows = (int)min(p.R - r, int64_t(kColRows));
    c.cols = (int)min(p.No - col, int64_t(kColRows));
    c.hb = p.bias != nullptr;
    c.w = load_rows<GATED, VEC>(p.alpha + r, c.hb ? p.bias + r : nullptr, c.rows, c.kLanes);
    c.template run<BATCH>(p.M, sa, sb);
    c.template run<1>(p.M, sa, sb);
}

template <bool GATED, int ACT, int DT, int WARPS, int BATCH>
__device__ __forceinline__ void columns_block(const Params& p, int64_t bx, uint32_t rank, uint32_t CY)
{
    __shared__ float part[WARPS][2][kColRows];
    __shared__ float total[2][kColRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the lane's first row: four in a row, or every 32nd (gated: pair)
    const int64_t r = bx * kColRows + lane * (p.vec ? 4 : GATED ? 2 : 1);
    float sa[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r < p.R) {
        const int64_t m0 = (int64_t)rank * WARPS + warp, step = (int64_t)CY * WARPS;
        if constexpr (!GATED && ACT == SHERRY_ACT_NONE) {
            if (!p.acc) {                                    // dbias alone
                if (p.vec) column_sums<GATED, ACT, DT, true, false, BATCH>(p, r, m0, step, sa, sb);
                else column_sums<GATED, ACT, DT, false, false, BATCH>(p, r, m0, step, sa, sb);
            }
        }
        if (p.acc) {
            if (p.vec) column_sums<GATED, ACT, DT, true, true, BATCH>(p, r, m0, step, sa, sb);
            else column_sums<GATED, ACT, DT, false, true, BATCH>(p, r, m0, step, sa, sb);
        }
    }
    if (p.vec) {
        *reinterpret_cast<float4*>(&part[warp][0][4 * lane]) = make_float4(sa[0], sa[1], sa[2], sa[3]);
        *reinterpret_cast<float4*>(&part[warp][1][4 * lane]) = make_float4(sb[0], sb[1], sb[2], sb[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = GATED ? 2 * (lane + 32 * (k >> 1)) + (k & 1) : lane + 32 * k;
            part[warp][0][at] = sa[k];
            part[warp][1][at] = sb[k];
        }
    }
    __syncthreads();
    static_assert(32 * WARPS >= kColRows, "one thread per row");
    const int i = threadIdx.x;
    const bool mine = i < kColRows;
    float t[2] = {0.0f, 0.0f};
    if (mine) {
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
#pragma unroll
            for (int k = 0; k < 2; ++k) t[k] = __fadd_rn(t[k], part[w][k][i]);
    }
    if (CY > 1) {
        if (mine) {
            total[0][i] = t[0];
            total[1][i] = t[1];
        }
        ptx::cluster_arrive_release();
        ptx::cluster_wait_acquire();
        if (rank == 0 && mine)
            for (uint32_t y = 1; y < CY; ++y)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    t[k] = __fadd_rn(t[k], ptx::ld_cluster_f32(ptx::smem_u32(&total[k][i]), y));
        ptx::cluster_arrive_release();                       // the sums stay readable until read
        ptx::cluster_wait_acquire();
    }
    const int64_t n = bx * kColRows + i;
    if (rank == 0 && mine && n < p.R) {
        if (p.dalpha) p.dalpha[n] = t[0];
        if (p.dbias) p.dbias[n] = t[1];
    }
}

// grid (row blocks, blocks that share the columns)
template <bool GATED, int ACT, int DT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == kColWarps ? kColBlocks : 1)
    grad_columns_kernel(const Params p)
{
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    constexpr int kBatch = GATED ? 4 : 3;                    // what 80 registers hold
    columns_block<GATED, ACT, DT, WARPS, kBatch>(p, blockIdx.x, blockIdx.y, gridDim.y);
}

// Both in one launch, for few tokens, where a launch costs more than the work
// (M=5 K=1024, gated to 2816, bf16: 12.4 -> 9.6 us for the call): clusters of
// `cluster` blocks, the first `ahead` of them the tokens' digits (a cluster per
// token, or with `whole` a block), the others column sums, whose order does not
// depend on whether the digits are wanted.  In two launches and in one: M=750
// K=640, gated to 1197, bf16 30.9 and 23.1 us, M=1000, 4096 x 4096, bf16 64.5 and
// 61.7; M=2048 K=4096, gated to 14336, 754 and 795.  Four blocks an SM, so that
// the digits of other tokens hide a token's two passes; the column sums load
// fewer tokens at once for it (M=300 K=2080, gated to 5001, f16: 48.1 -> 44.0 us;
// M=380 K=1056 N=10001 f32 gelu 64 -> 56).
template <bool GATED, int ACT, int DT>
__global__ void __launch_bounds__(kDigitThreads, kBothBlocks)
    grad_both_kernel(const Params p, uint32_t ahead, uint32_t cluster, int whole)
{
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    clear_split(p, blockIdx.x, gridDim.x);
    const uint32_t id = blockIdx.x / cluster, rank = blockIdx.x - id * cluster;
    // what 64 registers hold
    constexpr int kBatch = ACT == SHERRY_ACT_GELU ? 1 : 2;
    const uint32_t token = whole ? blockIdx.x : id;
    if (id >= ahead) columns_block<GATED, ACT, DT, kDigitThreads / 32, kBatch>(p, id - ahead, rank, cluster);
    else if (token < p.M) digits_block<GATED, ACT, DT>(p, token, whole ? 0 : rank, whole ? 1 : cluster);
}

// Host (grad_cuda.cu): what a gradient call launches ahead of its product, and
// the column sums alone.
int launch_ahead(Params p, bool gated, int act, int dtype, int sms, cudaStream_t stream);
int launch_columns(const Params& p, bool gated, int act, int dtype, int sms, cudaStream_t stream);

}  // namespace grad
}  // namespace sherry
