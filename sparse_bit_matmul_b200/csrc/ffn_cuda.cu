// Feed-forward operators of the C ABI (include/sherry.h): the linear layer
// with bias, activation and residual, the gated pair of projections, their
// gradients, and the weight layouts they read.  The contractions are the
// decode and tensor-core kernels of decode.cuh and tc_gemm.cuh with other
// epilogues; grad.cuh holds the elementwise half of the gradients.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "sherry.h"
#include "sherry_internal.h"
#include "host_common.h"
#include "decode.cuh"
#include "grad.cuh"
#include "quant.cuh"
#include "tc_gemm.cuh"
#include "tile_plan.h"

namespace sherry {
namespace {

// ---------------------------------------------------------------------------
// Activation quantiser for any element type: the rule of quant_act_kernel, one
// block per token.  Rows of up to XV 16-byte loads a thread stay in registers
// between the absmax and the quantisation; longer ones are read twice.  When
// the tokens fill the SMs, blocks are as narrow as four loads a thread allow
// (little to synchronise, and other tokens hide a token's two passes: M=2048
// bf16, K=4096 11.9 us with 512 threads, 7.8 so, 9.2 with eight loads; K=1024
// 9.6, 4.4 and 4.4); when they do not, a thread has one load (M=333 K=1056 3.4
// and 2.7).  Bound by issue: 16-bit values tie at half integers often, and
// those take the exact division.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 512;
constexpr int kQuantLoads = 4;
constexpr int kQuantLoadsMax = 8;           // rows beyond kQuantLoads * kQuantThreads loads

int quant_threads(int64_t M, int64_t units, int sms)
{
    const int64_t t = M >= 4 * (int64_t)sms ? (units + kQuantLoads - 1) / kQuantLoads : units;
    return (int)std::min<int64_t>(kQuantThreads, (t + 31) & ~int64_t(31));
}

// Memory that a launch clears for the next one.
struct Zero {
    uint4* p;
    int64_t n;
};

// The largest magnitude of 16-byte pieces of a row (NaN if there is one), two
// values at a time where they are 16-bit.
template <class XT>
struct AbsMax {
    using Pair = std::conditional_t<std::is_same_v<XT, __half>, __half2, __nv_bfloat162>;
    static constexpr bool kWide = std::is_same_v<XT, float>;
    std::conditional_t<kWide, float, Pair> a;

    __device__ __forceinline__ AbsMax()
    {
        const uint32_t zero = 0u;
        memcpy(&a, &zero, 4);
    }
    __device__ __forceinline__ void add(const uint4& w)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kWide) {
                a = quant::larger<true>(a, fabsf(__uint_as_float(u[i])));
            } else {
                Pair p;
                memcpy(&p, &u[i], 4);
                a = __hmax2_nan(a, __habs2(p));
            }
        }
    }
    __device__ __forceinline__ float get() const
    {
        if constexpr (kWide) return a;
        else if constexpr (std::is_same_v<XT, __half>) return quant::larger<true>(__low2float(a), __high2float(a));
        else return quant::larger<true>(__bfloat162float(a.x), __bfloat162float(a.y));
    }
};

// The int8 codes of 16 bytes of activations.
template <class XT>
__device__ __forceinline__ void quantise16(int8_t* row, int unit, const uint4& w, const quant::Scale& sc)
{
    if constexpr (std::is_same_v<XT, float>) {
        reinterpret_cast<uint32_t*>(row)[unit] = quant::quantise4(decode::load_x4<XT>(reinterpret_cast<const XT*>(&w), 0), sc);
    } else {
        const uint2 lo = make_uint2(w.x, w.y), hi = make_uint2(w.z, w.w);
        reinterpret_cast<uint2*>(row)[unit] =
            make_uint2(quant::quantise4(decode::load_x4<XT>(reinterpret_cast<const XT*>(&lo), 0), sc),
                       quant::quantise4(decode::load_x4<XT>(reinterpret_cast<const XT*>(&hi), 0), sc));
    }
}

template <class XT, int XV>
__global__ void __launch_bounds__(kQuantThreads, XV == kQuantLoads ? 3 : 2)
    quant_rows_kernel(const XT* __restrict__ x, int64_t K, int8_t* __restrict__ q, float* __restrict__ scale,
                      uint4* __restrict__ zero, int64_t zero_n)
{
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int64_t m = blockIdx.x;
    const uint4* xr = reinterpret_cast<const uint4*>(x + m * K);
    int8_t* qr = q + m * K;
    const int U = (int)(K * sizeof(XT) / 16), nthr = blockDim.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool in_regs = U <= XV * nthr;

    uint4 v[XV];
    AbsMax<XT> mx;
    if (in_regs) {
#pragma unroll
        for (int u = 0; u < XV; ++u)
            v[u] = tid + u * nthr < U ? xr[tid + u * nthr] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < XV; ++u)
            if (u * nthr < U) mx.add(v[u]);
    } else {
#pragma unroll 4
        for (int i = tid; i < U; i += nthr) mx.add(xr[i]);
    }
    float a = mx.get();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = quant::larger<true>(a, __shfl_xor_sync(0xffffffffu, a, o));
    __shared__ float warp_max[kQuantThreads / 32];
    if (lane == 0) warp_max[warp] = a;
    __syncthreads();
    a = lane < nthr / 32 ? warp_max[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = quant::larger<true>(a, __shfl_xor_sync(0xffffffffu, a, o));

    const quant::Scale sc = quant::make_scale(a);
    if (tid == 0) scale[m] = sc.s;
    if (in_regs) {
#pragma unroll
        for (int u = 0; u < XV; ++u)
            if (tid + u * nthr < U) quantise16<XT>(qr, tid + u * nthr, v[u], sc);
    } else {
#pragma unroll 4
        for (int i = tid; i < U; i += nthr) quantise16<XT>(qr, i, xr[i], sc);
    }
    // the split-K workspace of the launch behind
    for (int64_t i = m * nthr + tid; i < zero_n; i += (int64_t)gridDim.x * nthr) zero[i] = make_uint4(0u, 0u, 0u, 0u);
}

template <class XT>
int launch_quant(const void* x, int64_t M, int64_t K, int8_t* q, float* scale, Zero zero, int sms, cudaStream_t s)
{
    const int64_t units = K * (int64_t)sizeof(XT) / 16;
    auto kernel = units <= kQuantLoads * kQuantThreads ? quant_rows_kernel<XT, kQuantLoads>
                                                       : quant_rows_kernel<XT, kQuantLoadsMax>;
    return cuda_status(launch_pdl(kernel, dim3((unsigned)M), dim3((unsigned)quant_threads(M, units, sms)), 0, s,
                                  static_cast<const XT*>(x), K, q, scale, zero.p, zero.n));
}

int launch_quant(const void* x, int dtype, int64_t M, int64_t K, int8_t* q, float* scale, Zero zero, int sms,
                 cudaStream_t s)
{
    if (dtype == SHERRY_F32) return launch_quant<float>(x, M, K, q, scale, zero, sms, s);
    if (dtype == SHERRY_BF16) return launch_quant<__nv_bfloat16>(x, M, K, q, scale, zero, sms, s);
    return launch_quant<__half>(x, M, K, q, scale, zero, sms, s);
}

// ---------------------------------------------------------------------------
// Weight layouts (one thread per output word, once per weight).
// ---------------------------------------------------------------------------
// Canonical row `r` of a weight, or of the gated pair (rows 2n, 2n + 1).
struct Codes {
    const uint8_t* a;
    const uint8_t* b;           // up projection, or null
    int64_t row_bytes;
    __device__ __forceinline__ const uint8_t* row(int64_t r) const
    {
        return b ? ((r & 1) ? b : a) + (r >> 1) * row_bytes : a + r * row_bytes;
    }
};

__global__ void repack_gated_kernel(Codes codes, int64_t R, int64_t K, uint32_t* __restrict__ out, int64_t words)
{
    const int64_t Kc = sherry_k_chunks(K);
    for (int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; idx < words;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int64_t j = (idx / SHERRY_TILE_ROWS) % SHERRY_CHUNK_WORDS;
        const int64_t r = (idx - 8 * j) & (SHERRY_TILE_ROWS - 1);
        const int64_t c = (idx / (SHERRY_TILE_ROWS * SHERRY_CHUNK_WORDS)) % Kc;
        const int64_t n = idx / (SHERRY_TILE_ROWS * SHERRY_CHUNK_WORDS * Kc) * SHERRY_TILE_ROWS + r;
        const int64_t b0 = c * (SHERRY_CHUNK_WORDS * 4) + 4 * j;
        uint32_t w = 0;
        if (n < R) {
            const uint8_t* src = codes.row(n);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b0 + b < codes.row_bytes) w |= (uint32_t)src[b0 + b] << (8 * b);
        }
        out[idx] = w;
    }
}

__global__ void repack_t_kernel(Codes codes, int64_t R, int64_t K, uint32_t* __restrict__ out, int64_t words)
{
    const int64_t RT = sherry_row_tiles(R);
    for (int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; idx < words;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int64_t i = idx & 3, kk = (idx >> 2) & 127, q = (idx >> 9) & 1, blk = idx >> 10;
        const int64_t rt = blk % RT, k = blk / RT * SHERRY_KCHUNK + kk;
        const int64_t n0 = rt * SHERRY_TILE_ROWS + 64 * q + 16 * i;
        const int64_t bit = 5 * (k >> 2);
        const int64_t byte = bit >> 3;
        const uint32_t pos = (uint32_t)(k & 3);
        uint32_t w = 0;
        for (int e = 0; e < 16; ++e) {
            const int64_t n = n0 + e;
            if (n >= R || k >= K) break;
            const uint8_t* src = codes.row(n);
            uint32_t two = src[byte];
            if (byte + 1 < codes.row_bytes) two |= (uint32_t)src[byte + 1] << 8;
            const uint32_t code = (two >> (bit & 7)) & 31u, z = code & 3u;
            if (pos == z) continue;
            const uint32_t t = ((code >> (2 + pos - (pos > z ? 1u : 0u))) & 1u) ? 2u : 1u;
            const int c = e >> 2;
            w |= t << (2 * (c & 1) + 16 * (c >> 1) + 4 * (e & 3));
        }
        out[idx] = w;
    }
}

// ---------------------------------------------------------------------------
// host helpers
// ---------------------------------------------------------------------------
bool dtype_ok(int dtype) { return dtype == SHERRY_F32 || dtype == SHERRY_BF16 || dtype == SHERRY_F16; }
bool act_ok(int act) { return act >= SHERRY_ACT_NONE && act <= SHERRY_ACT_GELU_TANH; }
bool aligned_elem(const void* p, int dtype)
{
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(ep::elem_size(dtype) - 1)) == 0;
}

// fp32 and int32 arrays (null counts as aligned)
template <class... P>
bool aligned4(const P*... p)
{
    return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) == 0;
}

struct Span {
    const void* p;              // or null: empty
    int64_t bytes;
};

bool overlap(const Span& a, const Span& b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Whether an output shares a byte with an input or with another output.
template <int O, int I>
bool overlaps(const Span (&out)[O], const Span (&in)[I])
{
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i)
            if (overlap(out[o], in[i])) return true;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out[q])) return true;
    }
    return false;
}

// out [Mo][No]: boxes of box_n columns x box_m rows, for complete tiles
int make_out_map(CUtensorMap* map, void* out, int dtype, int64_t Mo, int64_t No, int box_n, int box_m)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return SHERRY_ERR_CUDA;
    const CUtensorMapDataType t = dtype == SHERRY_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : dtype == SHERRY_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    cuuint64_t dims[2] = {(cuuint64_t)No, (cuuint64_t)Mo};
    cuuint64_t strides[1] = {(cuuint64_t)No * ep::elem_size(dtype)};
    cuuint32_t box[2] = {(cuuint32_t)box_n, (cuuint32_t)box_m};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, t, 2, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SHERRY_OK
               : SHERRY_ERR_CUDA;
}

// A call's split-K workspace: the caller's (any contents; cleared by the launch
// ahead of the product), or with a null p the reserved one (all zero between
// calls).
struct Split {
    void* p;
    size_t bytes;
};

// What launch_tc needs of it: the slots of the split tiles, and their counters.
size_t split_bytes(const TilePlan& plan, int64_t M, int64_t TN)
{
    const int64_t n = split_tiles(plan, ceil_div(M, plan.bn) * TN);
    return (size_t)(n * plan.bn * SHERRY_TILE_ROWS * 4 + ((4 * n + 15) & ~int64_t(15)));
}

// One tensor-core launch.  b: int8 rows [p.M][p.K], ld bytes apart.  p holds
// the problem; tiles, workspace and status are filled in here.  `ahead` launches
// what the product reads, once nothing but a launch can fail any more, and
// clears the workspace it is given.
template <int BN, int SC, int WF, int EK, int D, int EG = 1, class Ahead>
int launch_tc(const int8_t* b, int64_t ld, tc::EpParams p, const TilePlan& plan, Split split, cudaStream_t stream,
              const Ahead& ahead)
{
    using C = tc::Cfg<BN, SC, WF, EG>;
    DeviceInfo di;
    int st = device_info(&di);
    if (st != SHERRY_OK) return st;
    p.y = nullptr;
    p.TM = (p.M + BN - 1) / BN;
    p.TN = sherry_row_tiles(p.N);
    p.Kc = sherry_k_chunks(p.K);
    p.U = p.TM * p.TN * p.Kc;
    const int64_t grid = plan.grid;
    p.whole = plan.whole;
    p.cluster = plan.cluster;
    p.ws = nullptr;
    p.counters = nullptr;
    Zero zero = {nullptr, 0};
    if (const size_t need = split_bytes(plan, p.M, p.TN)) {
        if (split.p) {
            if (split.bytes < need) return SHERRY_ERR_WORKSPACE;
            zero = {static_cast<uint4*>(split.p), (int64_t)(need / 16)};
        } else {
            st = get_workspace(need, &split.p);
            if (st != SHERRY_OK) return st;
        }
        p.ws = static_cast<int32_t*>(split.p);
        p.counters = reinterpret_cast<uint32_t*>(p.ws + split_tiles(plan, p.TM * p.TN) * BN * SHERRY_TILE_ROWS);
    }
    p.status = device_status_ptr();
    if (!p.status) return SHERRY_ERR_CUDA;

    CUtensorMap map;
    tc::OutMaps maps;
    st = make_x_map(&map, b, p.M, p.K, ld, BN);
    if (st != SHERRY_OK) return st;
    std::memset(&maps, 0, sizeof(maps));
    p.y_tma = (p.No * ep::elem_size(p.dtype)) % 16 == 0 && aligned16(p.out);
    if (p.res) p.y_tma = p.y_tma && aligned16(p.res);
    if (p.y_tma) {
        st = make_out_map(&maps.out, p.out, p.dtype, p.Mo, p.No, EK == tc::kEpGated ? 16 : 32, (int)ep::first_token<D>(16));
        if (st == SHERRY_OK && p.res)
            st = make_out_map(&maps.res, const_cast<void*>(p.res), p.dtype, p.Mo, p.No, 32, 16);
        if (st != SHERRY_OK) return st;
    }

    const int smem = std::max(C::kSmemBytes, 120 * 1024);    // one CTA per SM
    if (smem > di.max_smem_optin) return SHERRY_ERR_DEVICE;
    auto kernel = tc::sherry_gemm_tc_kernel<BN, SC, WF, EK, D, EG>;
    static std::atomic<uint64_t> done{0};
    st = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (st != SHERRY_OK) return st;
    st = ahead(zero);
    if (st != SHERRY_OK) return st;
    return cuda_status(launch_pdl(kernel, dim3((unsigned)grid), dim3(C::kThreads), (size_t)smem, stream,
                                  dim3((unsigned)std::max(1, plan.cluster)), map, maps, p));
}

// Few tokens: the decode kernel, when it has a plan for the shape.
bool forward_few(int64_t M, int64_t R, int64_t K, int sms, decode::Plan* pl)
{
    return M <= SHERRY_GEMM_DECODE_AUTO_MAX_M &&
           decode::plan(R, sherry_k_chunks(K), M, sms, pl, decode::ep_rt_first(R, M, sms));
}

template <int EK, class Ahead>
int launch_forward_tc(const int8_t* b, const tc::EpParams& p, Split split, int sms, cudaStream_t s, const Ahead& ahead)
{
    constexpr int W = tc::kWeightSherry;
    const TilePlan plan = forward_plan(p.dtype, p.act, p.res, p.acc, EK == tc::kEpGated, p.M, p.N, p.K, sms);
    if (plan.eg == 2) return plan.bn == 64 ? launch_tc<64, 4, W, EK, 1, 2>(b, p.K, p, plan, split, s, ahead)
                                           : launch_tc<128, 2, W, EK, 1, 2>(b, p.K, p, plan, split, s, ahead);
    switch (plan.bn) {
    case 16: return launch_tc<16, 4, W, EK, 1>(b, p.K, p, plan, split, s, ahead);
    case 32: return launch_tc<32, 4, W, EK, 1>(b, p.K, p, plan, split, s, ahead);
    case 64: return launch_tc<64, 4, W, EK, 1>(b, p.K, p, plan, split, s, ahead);
    case 128: return launch_tc<128, 2, W, EK, 1>(b, p.K, p, plan, split, s, ahead);
    default: return launch_tc<192, 1, W, EK, 1>(b, p.K, p, plan, split, s, ahead);
    }
}

// kWeightT2 chunks are 4 KB: two-chunk stages from 64 rows on keep at least
// three stages in the ring.
template <int D, class Ahead>
int launch_grad_tc(const int8_t* b, int64_t ld, const tc::EpParams& p, const TilePlan& plan, Split split, cudaStream_t s,
                   const Ahead& ahead)
{
    constexpr int W = tc::kWeightT2, EK = tc::kEpGrad;
    if (plan.eg == 2) return launch_tc<192, 1, W, EK, D, 2>(b, ld, p, plan, split, s, ahead);
    switch (plan.bn) {
    case 16: return launch_tc<16, 4, W, EK, D>(b, ld, p, plan, split, s, ahead);
    case 32: return launch_tc<32, 4, W, EK, D>(b, ld, p, plan, split, s, ahead);
    case 64: return launch_tc<64, 2, W, EK, D>(b, ld, p, plan, split, s, ahead);
    case 128: return launch_tc<128, 2, W, EK, D>(b, ld, p, plan, split, s, ahead);
    default: return launch_tc<192, 1, W, EK, D>(b, ld, p, plan, split, s, ahead);
    }
}

template <int MT, bool FUSED, int RT, class XT, class Ahead>
int launch_decode_rt(const decode::EpParams& p, const decode::Plan& pl, cudaStream_t stream, const Ahead& ahead)
{
    auto kernel = decode::sherry_decode_kernel<MT, FUSED, RT, XT, true>;
    static std::atomic<uint64_t> done{0};
    int st = once_per_device(done, [&] {
        // one carveout for every shape, so that the next call's CTAs share the SM
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, decode::kSmemBudgetMax);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        return e;
    });
    if (st != SHERRY_OK) return st;
    st = ahead(Zero{nullptr, 0});
    if (st != SHERRY_OK) return st;
    return cuda_status(launch_pdl(kernel, dim3((unsigned)pl.G), dim3((unsigned)pl.threads), (size_t)pl.smem, stream, p));
}

template <int MT, bool FUSED, class XT, class Ahead>
int launch_decode(decode::EpParams p, const decode::Plan& pl, const DeviceInfo& di, cudaStream_t stream,
                  const Ahead& ahead)
{
    p.Kc = sherry_k_chunks(p.K);
    p.G = pl.G;
    p.R = pl.R;
    p.Q = pl.Q;
    p.P = pl.P;
    p.CPT = pl.CPT;
    p.NS = pl.NS;
    p.S = pl.S;
    if (pl.smem > di.max_smem_optin) return SHERRY_ERR_DEVICE;
    if (pl.RT == 4) return launch_decode_rt<MT, FUSED, 4, XT>(p, pl, stream, ahead);
    if (pl.RT == 2) return launch_decode_rt<MT, FUSED, 2, XT>(p, pl, stream, ahead);
    return launch_decode_rt<MT, FUSED, 1, XT>(p, pl, stream, ahead);
}

// Both forward operators: R weight rows, No output columns.
int forward(const void* x, int dtype, const void* wn, const float* alpha, const float* bias, int act,
            const void* res, void* out, int32_t* acc, int8_t* x_i8, float* x_scale, Split split, int64_t M, int64_t R,
            int64_t No, int64_t K, bool gated, cudaStream_t s)
{
    if (!dtype_ok(dtype) || !act_ok(act)) return SHERRY_ERR_INVALID_ARG;
    if (!x || !wn || !alpha || !out || (x_i8 && !x_scale)) return SHERRY_ERR_INVALID_ARG;
    if (M <= 0 || No <= 0 || K <= 0) return SHERRY_ERR_INVALID_ARG;
    if (!sherry_shape_ok(M, R, K)) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(x) || !aligned16(wn) || (x_i8 && !aligned16(x_i8)) || !aligned16(split.p)) return SHERRY_ERR_INVALID_ARG;
    if (!aligned_elem(out, dtype) || (res && !aligned_elem(res, dtype))) return SHERRY_ERR_INVALID_ARG;
    if (!aligned4(alpha, bias, acc, x_scale)) return SHERRY_ERR_INVALID_ARG;
    const int64_t es = ep::elem_size(dtype), rb = 4 * R;
    const Span outs[] = {{out, M * No * es}, {acc, M * rb}, {x_i8, M * K}, {x_scale, 4 * M},
                         {split.p, (int64_t)split.bytes}};
    const Span ins[] = {{x, M * K * es}, {wn, (int64_t)sherry_native_bytes(R, K)}, {alpha, rb}, {bias, rb},
                        {res == out ? nullptr : res, M * No * es}};
    if (overlaps(outs, ins)) return SHERRY_ERR_INVALID_ARG;
    DeviceInfo di;
    int st = device_info(&di);
    if (st != SHERRY_OK) return st;

    decode::Plan pl;
    const bool few = forward_few(M, R, K, di.sms, &pl);
    decode::EpParams d = {};
    if (few) {
        d.wnative = static_cast<const uint8_t*>(wn);
        d.alpha = alpha;
        d.acc = acc;
        d.M = M;
        d.N = R;
        d.K = K;
        d.bias = bias;
        d.res = res;
        d.out = out;
        d.dtype = dtype;
        d.act = act;
        d.gated = gated ? 1 : 0;
    }
    if (few && M <= SHERRY_LINEAR_FUSED_MAX_M) {
        static_assert(SHERRY_LINEAR_FUSED_MAX_M == 1, "fused launches instantiated for one token");
        d.x = static_cast<const float*>(x);
        d.xq_out = x_i8;
        d.xs_out = x_scale;
        const auto none = [](Zero) { return (int)SHERRY_OK; };
        if (dtype == SHERRY_F32) return launch_decode<1, true, float>(d, pl, di, s, none);
        if (dtype == SHERRY_BF16) return launch_decode<1, true, __nv_bfloat16>(d, pl, di, s, none);
        return launch_decode<1, true, __half>(d, pl, di, s, none);
    }
    if (!x_i8) {
        void* buf = nullptr;
        st = get_act_buffer(act_buffer_bytes(M, K), &buf);
        if (st != SHERRY_OK) return st;
        x_i8 = static_cast<int8_t*>(buf);
        if (!x_scale)
            x_scale = reinterpret_cast<float*>(static_cast<uint8_t*>(buf) + (((size_t)M * (size_t)K + 255) & ~size_t(255)));
    }
    const auto quantise = [&](Zero zero) { return launch_quant(x, dtype, M, K, x_i8, x_scale, zero, di.sms, s); };
    if (few) {
        d.xq = x_i8;
        d.x_scale = x_scale;
        return launch_decode<2, false, float>(d, pl, di, s, quantise);
    }
    tc::EpParams p = {};
    p.wnative = static_cast<const uint8_t*>(wn);
    p.alpha = alpha;
    p.x_scale = x_scale;
    p.acc = acc;
    p.M = M;
    p.N = R;
    p.K = K;
    p.bias = bias;
    p.res = res;
    p.out = out;
    p.Mo = M;
    p.No = No;
    p.dtype = dtype;
    p.act = act;
    return gated ? launch_forward_tc<tc::kEpGated>(x_i8, p, split, di.sms, s, quantise)
                 : launch_forward_tc<tc::kEpLinear>(x_i8, p, split, di.sms, s, quantise);
}

size_t forward_split_bytes(int dtype, int act, bool res, bool acc, bool gated, int64_t M, int64_t R, int64_t K)
{
    DeviceInfo di;
    decode::Plan pl;
    if (!dtype_ok(dtype) || !act_ok(act) || !sherry_shape_ok(M, R, K) || device_info(&di) != SHERRY_OK) return 0;
    if (forward_few(M, R, K, di.sms, &pl)) return 0;
    return split_bytes(forward_plan(dtype, act, res, acc, gated, M, R, K, di.sms), M, sherry_row_tiles(R));
}

// Row stride of the digit rows: whole 128-byte lines, so that a TMA box row is
// one of them and not parts of two.
int64_t digit_ld(int64_t R) { return (R + 127) & ~int64_t(127); }

int64_t digit_bytes(int dtype, int64_t M, int64_t R)
{
    return (digit_rows(dtype, M) * digit_ld(R) + 255) & ~int64_t(255);
}

constexpr int64_t kGradMaxRows = (int64_t(1) << 24) - 1;

bool grad_shape_ok(int64_t M, int64_t R, int64_t K)
{
    return sherry_shape_ok(M, R, K) && R <= kGradMaxRows && M <= SHERRY_MAX_DIM / 4;
}

int backward(const void* dy, int dtype, const int32_t* acc, const float* x_scale, const void* wt, const float* alpha,
             const float* bias, int act, void* dx, float* dalpha, float* dbias, void* work, Split split, int64_t M,
             int64_t R, int64_t No, int64_t K, bool gated, cudaStream_t s)
{
    if (!dtype_ok(dtype) || !act_ok(act)) return SHERRY_ERR_INVALID_ARG;
    if (!dy || !alpha || (!dx && !dalpha && !dbias)) return SHERRY_ERR_INVALID_ARG;
    if (dx && (!wt || !work)) return SHERRY_ERR_INVALID_ARG;
    if (!acc && (gated || act != SHERRY_ACT_NONE || dalpha)) return SHERRY_ERR_INVALID_ARG;
    if (acc && !x_scale) return SHERRY_ERR_INVALID_ARG;
    if (M <= 0 || No <= 0 || K <= 0) return SHERRY_ERR_INVALID_ARG;
    if (!grad_shape_ok(M, R, K)) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(split.p) || !aligned_elem(dy, dtype) || (reinterpret_cast<uintptr_t>(acc) & 7u)) return SHERRY_ERR_INVALID_ARG;
    if (!aligned4(x_scale, alpha, bias, dalpha, dbias)) return SHERRY_ERR_INVALID_ARG;
    if (dx && (!aligned16(wt) || !aligned16(work) || !aligned_elem(dx, dtype))) return SHERRY_ERR_INVALID_ARG;
    const int64_t es = ep::elem_size(dtype), rb = 4 * R;
    const Span outs[] = {{dx, M * K * es}, {dalpha, rb}, {dbias, rb}, {dx ? work : nullptr, digit_bytes(dtype, M, R) + 4 * M},
                         {dx ? split.p : nullptr, (int64_t)split.bytes}};
    const Span ins[] = {{dy, M * No * es}, {acc, M * rb}, {x_scale, 4 * M}, {alpha, rb}, {bias, rb},
                        {dx ? wt : nullptr, (int64_t)sherry_transposed_bytes(R, K)}};
    if (overlaps(outs, ins)) return SHERRY_ERR_INVALID_ARG;
    DeviceInfo di;
    int st = device_info(&di);
    if (st != SHERRY_OK) return st;

    grad::Params g = {};
    g.dy = dy;
    g.acc = acc;
    g.x_scale = x_scale;
    g.alpha = alpha;
    g.bias = bias;
    g.M = M;
    g.R = R;
    g.No = No;
    g.ld = digit_ld(R);
    g.dig = static_cast<int8_t*>(work);
    g.dscale = reinterpret_cast<float*>(static_cast<uint8_t*>(work) + digit_bytes(dtype, M, R));
    g.vec = R % 4 == 0 && aligned16(dy) && aligned16(acc) && aligned16(alpha) && aligned16(bias);
    g.dalpha = dalpha;
    g.dbias = dbias;
    if (!dx) return grad::launch_columns(g, gated, act, dtype, di.sms, s);
    const TilePlan plan = grad_plan(dtype, M, R, K, di.sms);
    const auto digits = [&](Zero zero) {
        g.zero = zero.p;
        g.zero_n = zero.n;
        return grad::launch_ahead(g, gated, act, dtype, di.sms, s);
    };
    tc::EpParams p = {};
    p.wnative = static_cast<const uint8_t*>(wt);
    p.x_scale = g.dscale;
    p.M = digit_rows(dtype, M);
    p.N = K;
    p.K = R;
    p.out = dx;
    p.Mo = M;
    p.No = K;
    p.dtype = dtype;
    if (dtype == SHERRY_F32) return launch_grad_tc<grad::kDigits<SHERRY_F32>>(g.dig, g.ld, p, plan, split, s, digits);
    static_assert(grad::kDigits<SHERRY_BF16> == grad::kDigits<SHERRY_F16>, "one kernel for the 16-bit types");
    return launch_grad_tc<grad::kDigits<SHERRY_F16>>(g.dig, g.ld, p, plan, split, s, digits);
}

int repack(bool transposed, const uint8_t* a, const uint8_t* b, int64_t N, int64_t R, int64_t K, void* out, void* stream)
{
    if (!a || !out) return SHERRY_ERR_INVALID_ARG;
    if (N <= 0 || K <= 0) return SHERRY_ERR_INVALID_ARG;
    if (!sherry_shape_ok(1, R, K)) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(out)) return SHERRY_ERR_INVALID_ARG;
    const int64_t words = (int64_t)((transposed ? sherry_transposed_bytes(R, K) : sherry_native_bytes(R, K)) / 4);
    const Span outs[] = {{out, 4 * words}}, ins[] = {{a, N * (K / 32 * 5)}, {b, N * (K / 32 * 5)}};
    if (overlaps(outs, ins)) return SHERRY_ERR_INVALID_ARG;
    const int threads = 256;
    const unsigned blocks = (unsigned)std::min<int64_t>((words + threads - 1) / threads, 148 * 32);
    const Codes codes = {a, b, K / 32 * 5};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (transposed) repack_t_kernel<<<blocks, threads, 0, s>>>(codes, R, K, static_cast<uint32_t*>(out), words);
    else repack_gated_kernel<<<blocks, threads, 0, s>>>(codes, R, K, static_cast<uint32_t*>(out), words);
    return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace sherry

using namespace sherry;

extern "C" {

int sherry_quant_act_dt(const void* x, int x_dtype, int64_t M, int64_t K, int8_t* x_i8, float* x_scale, void* stream)
{
    if (!dtype_ok(x_dtype)) return SHERRY_ERR_INVALID_ARG;
    if (!x || !x_i8 || !x_scale) return SHERRY_ERR_INVALID_ARG;
    if (M <= 0 || K <= 0) return SHERRY_ERR_INVALID_ARG;
    if (!sherry_shape_ok(M, 1, K)) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(x) || !aligned16(x_i8) || !aligned4(x_scale)) return SHERRY_ERR_INVALID_ARG;
    const Span outs[] = {{x_i8, M * K}, {x_scale, 4 * M}}, ins[] = {{x, M * K * ep::elem_size(x_dtype)}};
    if (overlaps(outs, ins)) return SHERRY_ERR_INVALID_ARG;
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != SHERRY_OK) return st;
    return launch_quant(x, x_dtype, M, K, x_i8, x_scale, Zero{nullptr, 0}, di.sms, static_cast<cudaStream_t>(stream));
}

int sherry_repack_gated(const uint8_t* gate_dev, const uint8_t* up_dev, int64_t N, int64_t K, void* native_dev,
                        void* stream)
{
    if (!up_dev) return SHERRY_ERR_INVALID_ARG;
    if (N > SHERRY_MAX_DIM / 2) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    return repack(false, gate_dev, up_dev, N, 2 * N, K, native_dev, stream);
}

int sherry_repack_t(const uint8_t* codes_dev, int64_t N, int64_t K, void* out_dev, void* stream)
{
    return repack(true, codes_dev, nullptr, N, N, K, out_dev, stream);
}

int sherry_repack_gated_t(const uint8_t* gate_dev, const uint8_t* up_dev, int64_t N, int64_t K, void* out_dev,
                          void* stream)
{
    if (!up_dev) return SHERRY_ERR_INVALID_ARG;
    if (N > SHERRY_MAX_DIM / 2) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    return repack(true, gate_dev, up_dev, N, 2 * N, K, out_dev, stream);
}

size_t sherry_linear_split_bytes(int x_dtype, int act, int residual, int acc, int64_t M, int64_t N, int64_t K)
{
    return forward_split_bytes(x_dtype, act, residual != 0, acc != 0, false, M, N, K);
}

size_t sherry_gated_split_bytes(int x_dtype, int act, int acc, int64_t M, int64_t N, int64_t K)
{
    return N < 1 || N > SHERRY_MAX_DIM / 2 ? 0 : forward_split_bytes(x_dtype, act, false, acc != 0, true, M, 2 * N, K);
}

int sherry_linear_epilogue_ws(const void* x, int x_dtype, const void* Wnative, const float* alpha, const float* bias,
                              int act, const void* residual, void* y, int32_t* acc, int8_t* x_i8, float* x_scale,
                              void* split, size_t split_size, int64_t M, int64_t N, int64_t K, void* stream)
{
    return forward(x, x_dtype, Wnative, alpha, bias, act, residual, y, acc, x_i8, x_scale, Split{split, split_size}, M, N,
                   N, K, false, static_cast<cudaStream_t>(stream));
}

int sherry_linear_epilogue(const void* x, int x_dtype, const void* Wnative, const float* alpha, const float* bias,
                           int act, const void* residual, void* y, int32_t* acc, int8_t* x_i8, float* x_scale,
                           int64_t M, int64_t N, int64_t K, void* stream)
{
    return sherry_linear_epilogue_ws(x, x_dtype, Wnative, alpha, bias, act, residual, y, acc, x_i8, x_scale, nullptr, 0, M,
                                     N, K, stream);
}

int sherry_gated_ws(const void* x, int x_dtype, const void* Wnative, const float* alpha, const float* bias, int act,
                    void* h, int32_t* acc, int8_t* x_i8, float* x_scale, void* split, size_t split_size, int64_t M,
                    int64_t N, int64_t K, void* stream)
{
    if (N > SHERRY_MAX_DIM / 2) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    return forward(x, x_dtype, Wnative, alpha, bias, act, nullptr, h, acc, x_i8, x_scale, Split{split, split_size}, M,
                   2 * N, N, K, true, static_cast<cudaStream_t>(stream));
}

int sherry_gated(const void* x, int x_dtype, const void* Wnative, const float* alpha, const float* bias, int act,
                 void* h, int32_t* acc, int8_t* x_i8, float* x_scale, int64_t M, int64_t N, int64_t K, void* stream)
{
    return sherry_gated_ws(x, x_dtype, Wnative, alpha, bias, act, h, acc, x_i8, x_scale, nullptr, 0, M, N, K, stream);
}

size_t sherry_transposed_bytes(int64_t R, int64_t K)
{
    if (!sherry_shape_ok(1, R, K)) return 0;
    return (size_t)sherry_row_tiles(R) * (size_t)sherry_k_chunks(K) * SHERRY_T2_CHUNK_BYTES;
}

int sherry_grad_digits(int dtype) { return grad_digits(dtype); }

size_t sherry_grad_work_bytes(int dtype, int64_t M, int64_t R)
{
    if (!dtype_ok(dtype) || M < 1 || M > SHERRY_MAX_DIM / 4 || R < 1 || R > kGradMaxRows) return 0;
    return (size_t)digit_bytes(dtype, M, R) + 4 * (size_t)M;
}

size_t sherry_grad_split_bytes(int dtype, int64_t M, int64_t R, int64_t K)
{
    DeviceInfo di;
    if (!dtype_ok(dtype) || !grad_shape_ok(M, R, K) || device_info(&di) != SHERRY_OK) return 0;
    return split_bytes(grad_plan(dtype, M, R, K, di.sms), digit_rows(dtype, M), sherry_row_tiles(K));
}

int sherry_linear_grad_ws(const void* dy, int dtype, const int32_t* acc, const float* x_scale, const void* Wt,
                          const float* alpha, const float* bias, int act, void* dx, float* dalpha, float* dbias,
                          void* work, void* split, size_t split_size, int64_t M, int64_t N, int64_t K, void* stream)
{
    return backward(dy, dtype, acc, x_scale, Wt, alpha, bias, act, dx, dalpha, dbias, work, Split{split, split_size}, M, N,
                    N, K, false, static_cast<cudaStream_t>(stream));
}

int sherry_linear_grad(const void* dy, int dtype, const int32_t* acc, const float* x_scale, const void* Wt,
                       const float* alpha, const float* bias, int act, void* dx, float* dalpha, float* dbias,
                       void* work, int64_t M, int64_t N, int64_t K, void* stream)
{
    return sherry_linear_grad_ws(dy, dtype, acc, x_scale, Wt, alpha, bias, act, dx, dalpha, dbias, work, nullptr, 0, M, N,
                                 K, stream);
}

int sherry_gated_grad_ws(const void* dh, int dtype, const int32_t* acc, const float* x_scale, const void* Wt,
                         const float* alpha, const float* bias, int act, void* dx, float* dalpha, float* dbias,
                         void* work, void* split, size_t split_size, int64_t M, int64_t N, int64_t K, void* stream)
{
    if (N > kGradMaxRows / 2) return SHERRY_ERR_UNSUPPORTED_SHAPE;
    return backward(dh, dtype, acc, x_scale, Wt, alpha, bias, act, dx, dalpha, dbias, work, Split{split, split_size}, M,
                    2 * N, N, K, true, static_cast<cudaStream_t>(stream));
}

int sherry_gated_grad(const void* dh, int dtype, const int32_t* acc, const float* x_scale, const void* Wt,
                      const float* alpha, const float* bias, int act, void* dx, float* dalpha, float* dbias,
                      void* work, int64_t M, int64_t N, int64_t K, void* stream)
{
    return sherry_gated_grad_ws(dh, dtype, acc, x_scale, Wt, alpha, bias, act, dx, dalpha, dbias, work, nullptr, 0, M, N,
                                K, stream);
}

}  // extern "C"
