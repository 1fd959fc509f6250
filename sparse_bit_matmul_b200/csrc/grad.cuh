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
// D = 2 digits (bf16 tensors) |v| <= 32639 = 127 (256 + 1), so e is off by at
// most 2^-16 of the token's largest (a bf16 output rounds by 2^-9 of itself);
// D = 4 (fp32, fp16) a power of two with |v| < 2^30, exact for every e within
// a factor 64 of the largest and off by at most 2^-30 of it below.
// v = sum_d 256^d digit_d with digits in [-128, 127]: the integer sums over n
// below 2^24 rows stay inside int32.
#pragma once

#include <cstdint>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "sherry_internal.h"

namespace sherry {
namespace grad {

struct Params {
    const void* dy;             // [M][No] of dtype
    const int32_t* acc;         // [M][R] or null (linear, act none: z is not needed)
    const float* x_scale;       // [M] (with acc)
    const float* alpha;         // [R]
    const float* bias;          // [R] or null
    int dtype, act;
    int64_t M, R, No;           // R = No, or 2 No when gated
    int8_t* dig;                // [M * D][ld] digit rows
    float* dscale;              // [M]
    int64_t ld;                 // a multiple of 16, >= R
    int cache;                  // floats of e that fit in the block's shared memory
    int vec;                    // rows and bases allow 16-byte loads of four rows' values
    float* dalpha;              // [R] or null
    float* dbias;               // [R] or null
};

// dz of one pre-activation (linear)
__device__ __forceinline__ float dz_linear(float dy, float z, int act)
{
    float f, d;
    ep::act_slope(z, act, f, d);
    return __fmul_rn(dy, d);
}

__device__ __forceinline__ float pre_act(int32_t acc, float al, float s, bool has_bias, float b)
{
    const float z = __fmul_rn(__fmul_rn((float)acc, al), s);
    return has_bias ? __fadd_rn(z, b) : z;
}

// four consecutive 16-byte aligned values, or element by element with a bound
__device__ __forceinline__ void load4(const float* p, int64_t i, int64_t end, bool vec, float (&v)[4])
{
    if (vec) {
        const float4 t = *reinterpret_cast<const float4*>(p + i);
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < end ? p[i + k] : 0.0f;
    }
}
__device__ __forceinline__ void load4(const int32_t* p, int64_t i, int64_t end, bool vec, int32_t (&v)[4])
{
    if (vec) {
        const int4 t = *reinterpret_cast<const int4*>(p + i);
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < end ? p[i + k] : 0;
    }
}

// dy of output columns c .. c + C - 1 of token m
template <int C>
__device__ __forceinline__ void load_dy(const Params& p, int64_t m, int64_t c, float (&g)[C])
{
    const int64_t at = m * p.No + c;
    if (p.vec) {
        if (p.dtype == SHERRY_F32) {
#pragma unroll
            for (int k = 0; k < C; k += 2) {
                const float2 t = *reinterpret_cast<const float2*>(static_cast<const float*>(p.dy) + at + k);
                g[k] = t.x;
                g[k + 1] = t.y;
            }
        } else {
#pragma unroll
            for (int k = 0; k < C; k += 2) {
                const uint32_t t = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.dy) + at + k);
                g[k] = ep::from16((uint16_t)(t & 0xFFFFu), p.dtype);
                g[k + 1] = ep::from16((uint16_t)(t >> 16), p.dtype);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < C; ++k) g[k] = c + k < p.No ? ep::load_elem(p.dy, at + k, p.dtype) : 0.0f;
    }
}

// e of rows 4u .. 4u + 3 of token m (0 past R)
template <bool GATED>
__device__ __forceinline__ void e4(const Params& p, int64_t m, int64_t u, float s, float (&e)[4])
{
    const int64_t r = 4 * u;
    if (r >= p.R) {
        e[0] = e[1] = e[2] = e[3] = 0.0f;
        return;
    }
    float al[4], b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int32_t a[4] = {0, 0, 0, 0};
    load4(p.alpha, r, p.R, p.vec, al);
    if (p.bias) load4(p.bias, r, p.R, p.vec, b);
    if (p.acc) load4(p.acc + m * p.R, r, p.R, p.vec, a);
    const bool hb = p.bias != nullptr;
    if constexpr (GATED) {
        float g[2];
        load_dy<2>(p, m, r >> 1, g);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float f, d;
            ep::act_slope(pre_act(a[2 * k], al[2 * k], s, hb, b[2 * k]), p.act, f, d);
            const float up = pre_act(a[2 * k + 1], al[2 * k + 1], s, hb, b[2 * k + 1]);
            e[2 * k] = __fmul_rn(__fmul_rn(__fmul_rn(g[k], up), d), al[2 * k]);
            e[2 * k + 1] = __fmul_rn(__fmul_rn(g[k], f), al[2 * k + 1]);
        }
    } else {
        float g[4];
        load_dy<4>(p, m, r, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = __fmul_rn(dz_linear(g[k], pre_act(a[k], al[k], s, hb, b[k]), p.act), al[k]);
    }
}

// One block per token: e into shared memory (recomputed when it does not
// fit), its largest magnitude, then the digit rows.
template <bool GATED, int D>
__global__ void __launch_bounds__(1024) grad_digits_kernel(const Params p)
{
    extern __shared__ __align__(16) float cache[];
    __shared__ float warp_max[32];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int64_t m = blockIdx.x;
    const int tid = threadIdx.x, nthr = blockDim.x;
    const int64_t U = (p.R + 3) >> 2;
    const bool cached = 4 * U <= p.cache;
    const float s = p.acc ? p.x_scale[m] : 0.0f;
    float mx = 0.0f;
    bool bad = false;
    for (int64_t u = tid; u < U; u += nthr) {
        float e[4];
        e4<GATED>(p, m, u, s, e);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float a = fabsf(e[k]);
            mx = fmaxf(mx, a);
            bad |= !(a <= 3.4028234e38f);
        }
        if (cached) *reinterpret_cast<float4*>(cache + 4 * u) = make_float4(e[0], e[1], e[2], e[3]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) warp_max[tid >> 5] = mx;
    bad = __syncthreads_or(bad);
    mx = (tid & 31) < (nthr >> 5) ? warp_max[tid & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));

    // v = e * inv, dx = sum * sc
    float inv = 0.0f, sc = 0.0f;
    if (mx > 0.0f && !bad) {
        if constexpr (D == 2) {
            if (mx >= 7.8886091e-31f) {                      // 2^-100
                inv = __fdiv_rn(32639.0f, mx);
                sc = __fdiv_rn(mx, 32639.0f);
            } else {
                inv = 2.0769187e34f;                         // 2^114
                sc = 4.8148249e-35f;
            }
        } else {
            const int ex = (int)(__float_as_uint(mx) >> 23) - 127;      // mx < 2^(ex + 1)
            const int k = min(29 - ex, 126);
            inv = __uint_as_float((uint32_t)(127 + k) << 23);
            sc = __uint_as_float((uint32_t)(127 - k) << 23);
        }
    }
    if (bad) sc = __uint_as_float(0x7FC00000u);              // the whole dx row becomes NaN
    if (tid == 0) p.dscale[m] = sc;
    for (int64_t u = tid; u < (p.ld >> 2); u += nthr) {
        float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (u < U && inv != 0.0f) {
            if (cached) {
                const float4 t = *reinterpret_cast<const float4*>(cache + 4 * u);
                e[0] = t.x; e[1] = t.y; e[2] = t.z; e[3] = t.w;
            } else {
                e4<GATED>(p, m, u, s, e);
            }
        }
        int32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __float2int_rn(__fmul_rn(e[k], inv));
#pragma unroll
        for (int d = 0; d < D; ++d) {
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w |= ((uint32_t)v[k] & 0xFFu) << (8 * k);
                v[k] = (v[k] - (int32_t)(int8_t)(v[k] & 0xFF)) >> 8;
            }
            *reinterpret_cast<uint32_t*>(p.dig + (m * D + d) * p.ld + 4 * u) = w;
        }
    }
}

// Column sums: a block owns 32 output columns, its warps take the tokens in
// turn, and the warps' sums meet in shared memory in a fixed order.
constexpr int kColWarps = 16;

template <bool GATED>
__global__ void __launch_bounds__(32 * kColWarps) grad_columns_kernel(const Params p)
{
    constexpr int S = GATED ? 4 : 2;                         // dalpha, dbias of each row of the column
    __shared__ float part[kColWarps][S][32];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const bool in = c < p.No;
    float sum[S];
#pragma unroll
    for (int i = 0; i < S; ++i) sum[i] = 0.0f;
    if (in) {
        const bool hb = p.bias != nullptr;
        float al[2] = {0.0f, 0.0f}, b[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < (GATED ? 2 : 1); ++k) {
            const int64_t r = GATED ? 2 * c + k : c;
            al[k] = p.alpha[r];
            if (hb) b[k] = p.bias[r];
        }
#pragma unroll 4
        for (int64_t m = warp; m < p.M; m += kColWarps) {
            const float g = ep::load_elem(p.dy, m * p.No + c, p.dtype);
            const float s = p.acc ? p.x_scale[m] : 0.0f;
            if constexpr (GATED) {
                const int2 a = *reinterpret_cast<const int2*>(p.acc + m * p.R + 2 * c);
                float f, d;
                ep::act_slope(pre_act(a.x, al[0], s, hb, b[0]), p.act, f, d);
                const float up = pre_act(a.y, al[1], s, hb, b[1]);
                const float z0 = __fmul_rn(__fmul_rn(g, up), d), z1 = __fmul_rn(g, f);
                sum[0] = __fmaf_rn(z0, __fmul_rn((float)a.x, s), sum[0]);
                sum[1] = __fmaf_rn(z1, __fmul_rn((float)a.y, s), sum[1]);
                sum[2] = __fadd_rn(sum[2], z0);
                sum[3] = __fadd_rn(sum[3], z1);
            } else {
                const int32_t a = p.acc ? p.acc[m * p.R + c] : 0;
                const float z = dz_linear(g, pre_act(a, al[0], s, hb, b[0]), p.act);
                sum[0] = __fmaf_rn(z, __fmul_rn((float)a, s), sum[0]);
                sum[1] = __fadd_rn(sum[1], z);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < S; ++i) part[warp][i][lane] = sum[i];
    __syncthreads();
    if (warp < S && in) {
        float t = 0.0f;
        for (int w = 0; w < kColWarps; ++w) t = __fadd_rn(t, part[w][warp][lane]);
        float* out = (GATED ? warp < 2 : warp < 1) ? p.dalpha : p.dbias;
        if (out) out[GATED ? 2 * c + (warp & 1) : c] = t;
    }
}

}  // namespace grad
}  // namespace sherry
