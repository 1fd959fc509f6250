// Element types, activations and their slopes, shared by the epilogues of the
// forward kernels (tc_gemm.cuh, decode.cuh) and the gradient kernels
// (grad.cuh).
//
// act(z):
//   none z | relu max(z, 0) | relu2 max(z, 0)^2 | gelu z Phi(z), Phi the
//   normal distribution function | silu z S(z) | gelu_tanh z S(t(z)) with
//   t(z) = 2 sqrt(2/pi) (z + 0.044715 z^3), S the logistic function
//   (z/2 (1 + tanh(t/2)) = z S(t)).
// silu and gelu_tanh share one body.
// S(t) = 1 / (1 + e^-t) with the hardware's approximate reciprocal (1 ulp).
// e^-t overflows to infinity for t < -88, where S is 0 to fp32 either way.  For
// 16-bit tensors it is the hardware's approximate power of two of -t log2 e (two
// special-function instructions a value: the epilogue has one warp per
// scheduler), whose relative error, 2 ulp and |t| half steps of the rounded
// argument, is far below the output's rounding; for fp32 tensors it is expf (2
// ulp at any t).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sherry.h"

namespace sherry {
namespace ep {

__host__ __device__ inline int elem_size(int dtype) { return dtype == SHERRY_F32 ? 4 : 2; }

__device__ __forceinline__ float from16(uint16_t u, int dtype)
{
    return dtype == SHERRY_BF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

__device__ __forceinline__ uint16_t to16(float v, int dtype)
{
    return dtype == SHERRY_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// Rows of digits, D per token.  16 of them (a slice of the tensor-core
// kernel's epilogue) hold 16 / D tokens whole: with D = 3 five tokens and a row
// that nobody writes and whose sums nobody reads.
template <int D>
__host__ __device__ constexpr int64_t first_row(int64_t token)
{
    return D == 3 ? token / 5 * 16 + token % 5 * 3 : token * D;
}

// of the rows from `row` on, for D = 3 a multiple of 16
template <int D>
__host__ __device__ constexpr int64_t first_token(int64_t row)
{
    return D == 3 ? row / 16 * 5 : row / D;
}

// element `i` of a tensor of `dtype`
__device__ __forceinline__ float load_elem(const void* p, int64_t i, int dtype)
{
    if (dtype == SHERRY_F32) return static_cast<const float*>(p)[i];
    return from16(static_cast<const uint16_t*>(p)[i], dtype);
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, float v, int dtype)
{
    if (dtype == SHERRY_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = to16(v, dtype);
}

constexpr float kGeluC1 = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kGeluC3 = 0.0713548162726009f;       // 2 sqrt(2 / pi) 0.044715
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

template <bool FULL>
__device__ __forceinline__ float logistic(float t)
{
    float e, r;
    if constexpr (FULL) e = expf(-t);
    else asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(t, -1.4426950408889634f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
    return r;
}

// t(z) of silu and gelu_tanh (silu apart: z^2 may overflow)
__device__ __forceinline__ float sigmoid_arg(float z, bool silu)
{
    return silu ? z : __fmul_rn(z, __fmaf_rn(__fmul_rn(z, z), kGeluC3, kGeluC1));
}

// max(z, 0); NaN stays NaN
__device__ __forceinline__ float relu(float z) { return z < 0.0f ? 0.0f : z; }

// act over an array held in registers: one switch for the whole array.  dtype:
// that of the tensors.
template <int N>
__device__ __forceinline__ void apply_act(float (&v)[N], int act, int dtype)
{
    if (act == SHERRY_ACT_NONE) return;
    if (act == SHERRY_ACT_SILU || act == SHERRY_ACT_GELU_TANH) {
        const bool silu = act == SHERRY_ACT_SILU;
        if (dtype == SHERRY_F32) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __fmul_rn(v[i], logistic<true>(sigmoid_arg(v[i], silu)));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __fmul_rn(v[i], logistic<false>(sigmoid_arg(v[i], silu)));
        }
    } else if (act == SHERRY_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = __fmul_rn(__fmul_rn(0.5f, v[i]), __fadd_rn(1.0f, erff(__fmul_rn(v[i], kSqrtHalf))));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float r = relu(v[i]);
            v[i] = act == SHERRY_ACT_RELU2 ? __fmul_rn(r, r) : r;
        }
    }
}

__device__ __forceinline__ float act_one(float z, int act, int dtype)
{
    float v[1] = {z};
    apply_act<1>(v, act, dtype);
    return v[0];
}

// act(z) and its derivative (0 at the corner of relu).  FULL: for fp32 tensors.
template <bool FULL>
__device__ __forceinline__ void act_slope(float z, int act, float& f, float& d)
{
    if (act == SHERRY_ACT_NONE) {
        f = z;
        d = 1.0f;
    } else if (act == SHERRY_ACT_SILU) {
        // d/dz [z S(z)] = S + z S (1 - S)
        const float s = logistic<FULL>(z);
        f = __fmul_rn(z, s);
        d = __fmaf_rn(f, __fsub_rn(1.0f, s), s);
    } else if (act == SHERRY_ACT_GELU_TANH) {
        // d/dz [z S(t)] = S + z S (1 - S) t',  t' = c1 + 3 c3 z^2; a far z:
        // z^2 may overflow where S (1 - S) is 0
        const float s = logistic<FULL>(sigmoid_arg(z, false));
        const float t1 = __fmaf_rn(__fmul_rn(z, z), 3.0f * kGeluC3, kGeluC1);
        f = __fmul_rn(z, s);
        const float w = __fmul_rn(f, __fsub_rn(1.0f, s));
        d = w == 0.0f ? s : __fmaf_rn(w, t1, s);
    } else if (act == SHERRY_ACT_GELU) {
        // d/dz [z Phi(z)] = Phi + z phi
        const float phi_cdf = __fmul_rn(0.5f, __fadd_rn(1.0f, erff(__fmul_rn(z, kSqrtHalf))));
        const float pdf = __fmul_rn(kInvSqrt2Pi, expf(__fmul_rn(-0.5f, __fmul_rn(z, z))));
        f = __fmul_rn(z, phi_cdf);
        d = pdf == 0.0f ? phi_cdf : __fmaf_rn(z, pdf, phi_cdf);
    } else {
        const float r = relu(z);
        f = act == SHERRY_ACT_RELU2 ? __fmul_rn(r, r) : r;
        d = z > 0.0f ? (act == SHERRY_ACT_RELU2 ? __fmul_rn(2.0f, z) : 1.0f) : 0.0f;
    }
}

}  // namespace ep
}  // namespace sherry
