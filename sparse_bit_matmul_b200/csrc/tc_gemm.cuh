// Sherry 3:4 ternary GEMM on the sm_100a tensor cores.
//
// What it computes (Sherry page, pnsm.cn/news/1195499, sec. 2.2 steps 2-4):
//   acc[m][n] = sum_k x_i8[m][k] * T[n][k]           (exact int32)
//   y[m][n]   = (float)((float)acc[m][n] * alpha[n]) * x_scale[m]
// with T decoded from the 5-bit group codes of sec. 2.1.
//
// How (the page's CPU/Jetson table-lookup kernels are prior art only): the
// problem is run "swap-AB" on tcgen05.mma.kind::i8 with M = 128 weight rows,
// N = BN tokens and K = 32 per instruction.
//   * A (weights) lives in tensor memory.  Decoder warps read the packed
//     codes of their row from shared memory, turn every 5-bit code into the
//     four int8 weights {-1,0,+1} of its group with one lookup in a 32-entry
//     table, and store them with tcgen05.st: one 32-bit TMEM cell is one
//     group, so a 128-wide K chunk of a row is 32 consecutive columns of that
//     row's lane.
//   * B (activations) is loaded by TMA into shared memory, K-major with the
//     128-byte swizzle, and described to the MMA by a shared-memory matrix
//     descriptor; rows past M and columns past K are zero-filled by TMA.
//   * D (int32 accumulators) lives in tensor memory; epilogue warps read it
//     with tcgen05.ld and apply the two fp32 products.
// Work is split so that every SM gets the same number of K chunks whatever
// the shape (one CTA per SM): each CTA first takes an even share of the
// units (token tile, row tile, K chunk) of the T mod G tiles left over, then
// T div G whole tiles of its own (SegWalk).  A tile whose K range spans
// several CTAs is summed exactly with int32 red.add into a workspace slot;
// the last contributor (an atomic counter) runs the epilogue and clears the
// slot and counter, so the workspace is all zero between calls.  The split
// tiles come first, so their reductions overlap the whole tiles after them.
//
// A pipeline stage carries SC consecutive K chunks of one tile (one bulk copy
// of SC * 2560 bytes of codes, SC 2D TMA boxes of activations, SC * 4 MMAs),
// so that the fixed cost of a stage's barriers is paid once per SC chunks.
//
// Warp roles (576 threads; 448 for 192-token tiles with two-chunk stages,
// which have two decoder groups; EG = 2 has eight epilogue warps from warp 10):
//   warp 0       producer: per stage one bulk copy of the codes (completing
//                the stage's code barrier, which the decoders wait for) and
//                one 2D TMA of the activation tile per chunk (completing its
//                full barrier, which the MMA warp waits for); the codes of
//                the first ring round go out before the dependency wait, so
//                the decoders work while the previous kernel finishes
//   warp 1       TMEM allocation and MMA issue (an elected lane)
//   warps 2-13   three decoder groups of four warps (each group covers the
//                four TMEM lane quadrants), taking stages in turn
//   warps 14-17  epilogue (one warp per lane quadrant)
// Loop indices (stage, phase, tile coordinates) advance incrementally: no
// integer division on the per-chunk path.
// Every wait is bounded in wall time; when a bound runs out the kernel
// records a status code, stops issuing work, waits (bounded) for what it has
// in flight, frees its tensor memory and returns.
//
// The same kernel runs the W4A8 FastGEMM of the OdysseyLLM review page
// (xllm-io.github.io/paper-review/blog/odysseyllm, sec. 3.1-3.2, 5.2) when
// WF = kWeightInt4: the weights are per-channel SINT4 (8 KB per 128 x 128
// chunk instead of 2560 bytes of codes), the decoders turn each 4-bit two's
// complement value into the int8 16 w by moving it into the high half of a
// byte (shift and mask, no table), the MMAs sum q * 16 w exactly in int32,
// and the epilogue divides those sums by 16 (an exact arithmetic shift)
// before the two fp32 products with the channel scale and the token scale.
//
// The feed-forward entry points (ffn_cuda.cu) run it with other epilogues
// (EK): kEpLinear adds bias, activation and residual; kEpGated has gate and
// up rows in adjacent TMEM lanes, exchanges them by one shuffle per two sums
// (the even lane finishes the even token of a pair, the odd lane the odd one,
// so no lane idles) and writes act(gate) * up; kEpGrad is the input gradient:
// the weights are T^T at two bits each (kWeightT2, four byte selectors per
// shift and mask, one byte permute per TMEM cell, no table), the "tokens" are
// the int8 base-256 digits of a fixed-point gradient, D per token (three: five
// tokens to 16 rows), and the epilogue joins a token's D sums.  Its sums are as exact as the forward's,
// so the split-K reductions stay free of order.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "sherry_internal.h"

namespace sherry {
namespace tc {

constexpr int kProducerWarp = 0;
constexpr int kMmaWarp = 1;
constexpr int kDecWarp0 = 2;
constexpr int kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;              // 2 s per wait

// weight formats
constexpr int kWeightSherry = 0;     // 5-bit 3:4 ternary group codes
constexpr int kWeightInt4 = 1;       // SINT4, two per byte
constexpr int kWeightT2 = 2;         // transposed ternary, 2 bits each (sherry_repack_t)

// epilogues
constexpr int kEpPlain = 0;          // y = acc * alpha * x_scale, fp32
constexpr int kEpLinear = 1;         // + bias, activation, residual; any element type
constexpr int kEpGated = 2;          // rows 2n, 2n + 1: act(z[2n]) * z[2n + 1]
constexpr int kEpGrad = 3;           // joins the digits of fixed-point gradients

// EG = 2: two epilogue groups take the segments in turn (each keeps to one of
// the two accumulators), in place of the third decoder group.  For tiles of
// few chunks, whose time is the epilogue's.
template <int BN, int SC, int WF = kWeightSherry, int EG = 1>
struct Cfg {
    static_assert(BN == 16 || BN == 32 || BN == 64 || BN == 128 || BN == 192, "BN");
    // 192-token tiles: two 192-column accumulators leave 128 TMEM columns:
    // four one-chunk A slots (SC = 1, three decoder groups, the form used)
    // or two two-chunk slots (SC = 2, then only two groups: the rings must be
    // at least as deep as the number of groups)
    static constexpr int kDecGroups = (BN == 192 && SC == 2) || EG == 2 ? 2 : 3;
    static constexpr int kEpiWarp0 = kDecWarp0 + 4 * kDecGroups;
    static constexpr int kThreads = 32 * (kEpiWarp0 + 4 * EG);
    static_assert(EG == 1 || EG == 2, "EG");
    static_assert(SC >= 1 && SC <= 4, "SC");
    static_assert(WF == kWeightSherry || WF == kWeightInt4 || WF == kWeightT2, "WF");
    // weight bytes of one (row tile, K chunk) block
    static constexpr int kChunkWBytes = WF == kWeightSherry ? SHERRY_CHUNK_BYTES_PER_TILE
                                        : WF == kWeightInt4 ? SHERRY_W4_CHUNK_BYTES
                                                            : SHERRY_T2_CHUNK_BYTES;
    // int32 sums of q * 16 w are divided by 16 before the epilogue uses them
    static constexpr int kAccShift = WF == kWeightInt4 ? 4 : 0;
    static constexpr int kBChunkBytes = BN * 128;
    static constexpr int kBStageBytes = SC * kBChunkBytes;
    static constexpr int kCodeStageBytes = SC * kChunkWBytes;
    static constexpr int kStageBytes = kBStageBytes + kCodeStageBytes;
    // output staging for TMA stores, per epilogue group: per warp two slices of
    // [kSlice tokens][32 rows] fp32
    static constexpr int kSlice = BN < 32 ? BN : 32;
    static constexpr int kStagingBytes = 4 * 2 * kSlice * 32 * 4;
    static constexpr int kStagesRaw = (192 * 1024 - (EG - 1) * (kStagingBytes + 4096)) / kStageBytes;
    static constexpr int kStagesCap = kStagesRaw > 12 ? 12 : kStagesRaw;
    // A whole number of rounds of decoder groups: stage s is then always
    // decoded by group s mod kDecGroups (see the ring rules below).
    static constexpr int kStages = kStagesCap - kStagesCap % kDecGroups;
    static constexpr int kACols = 32 * SC;                          // TMEM columns of one A stage
    static constexpr int kDBufs = (2 * BN + 2 * kACols <= kTmemCols) ? 2 : 1;
    static constexpr int kAStagesRaw = (kTmemCols - kDBufs * BN) / kACols;
    static constexpr int kAStages = kAStagesRaw > 8 ? 8 : kAStagesRaw;
    // A decoder group takes every kDecGroups-th stage.  A parity wait is exact
    // only while the waiter is not a whole phase ahead of the barrier: a wait
    // for phase k on a barrier still in phase k-1 sees the parity of phase
    // k-2, complete, and returns at once.
    //  - code(s) (the stage's codes; the decoders wait for it): the copies of
    //    different stages may land in any order, so the group waiting for the
    //    fill of iteration i must itself have seen the fill of iteration
    //    i - kStages: kStages a multiple of kDecGroups makes it the same
    //    group.  It cannot be two phases behind either: the next refill of
    //    stage s needs this group's arrival on empty(s).
    //  - full(s) (the stage's activation boxes): waited for by the MMA warp
    //    alone, in stage order; its refill needs the MMA's commit on empty(s).
    //  - aempty(a): completed by tcgen05.commit of the one MMA thread, in
    //    issue order; a group that saw its previous slot freed has seen every
    //    earlier MMA complete, which covers slot a's previous use once the
    //    ring is at least kDecGroups deep.
    static_assert(kStages >= kDecGroups && kStages % kDecGroups == 0, "stage ring not whole rounds of decoder groups");
    static_assert(kAStages >= kDecGroups, "A ring shallower than decoder groups");
    static constexpr int kACol0 = kDBufs * BN;
    // shared memory: [B stages][code stages][barriers + misc]
    static constexpr int kOffCodes = kStages * kBStageBytes;
    static constexpr int kOffBars = kOffCodes + kStages * kCodeStageBytes;
    static constexpr int kNumBars = 3 * kStages + 2 * kAStages + 2 * kDBufs + 1;
    static constexpr int kOffMisc = kOffBars + 8 * kNumBars;
    static constexpr int kMiscBytes = 64 + EG * 2 * BN * 4;   // tmem holder, flags, token scales [EG][2][BN]
    static constexpr int kOffStaging = (kOffMisc + kMiscBytes + 127) & ~127;
    static_assert(EG == 1 || kDBufs == 2, "one accumulator per epilogue group");
    // the other epilogues cut a warp's staging into slots of 16 sums x 32
    // rows: two at BN = 16 (one slice a tile), else four
    static constexpr int kEpSlots = kStagingBytes / (4 * 16 * 32 * 4);
    static_assert(kEpSlots == 2 || kEpSlots == 4, "rings of 1, 2 or 4 slots");
    static constexpr int kSmemBytes = kOffStaging + EG * kStagingBytes + 1024;   // + alignment slack
    // dynamic plus static (the table of the code path, 1 KB as compiled)
    // within the 227 KB per-block limit
    static_assert(kSmemBytes + (WF == kWeightSherry ? 1024 : 0) <= 232448, "shared memory");
    // instruction descriptor: s32 accumulate, signed int8 A and B, both
    // K-major, N = BN, M = 128
    static constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(BN >> 3) << 17) |
                                       (uint32_t(128 >> 4) << 24);
};

struct Params {
    const uint8_t* wnative;     // kernel-native codes
    const float* alpha;         // [N]
    const float* x_scale;       // [M]
    float* y;                   // [M][N] or null
    int32_t* acc;               // [M][N] or null
    int32_t* ws;                // split-K slots [grid][BN][128] (kEpPlain), else [split tiles][BN][128]
    uint32_t* counters;         // one per slot
    unsigned* status;           // device status word
    int64_t M, N, K;
    int64_t TM, TN, Kc;         // token tiles, row tiles, K chunks
    int64_t U;                  // total units TM*TN*Kc
    int y_tma;                  // y rows 16-byte multiples: complete tiles leave through TMA stores
    int whole;                  // leftover tiles are not split: one each to the first CTAs
    int cluster;                // CTAs per tile, a thread-block cluster (0: none); see kClusterSplit
};

// Parameters of the epilogues other than kEpPlain.  kEpGrad: M counts digit
// rows, N is the output's row length, x_scale one per token.
struct EpParams : Params {
    const float* bias;          // [N] or null
    const void* res;            // [Mo][No] or null (kEpLinear)
    void* out;                  // [Mo][No]
    int64_t Mo, No;             // output rows (tokens) and row length
    int dtype;                  // sherry_dtype of out and res
    int act;                    // sherry_act
};

// Tensor maps of the output, and of the residual in boxes of 32 columns x 16
// tokens (kEpLinear).  Apart from EpParams: taking a map's address makes the
// compiler read the struct it sits in through memory, field by field.
struct OutMaps {
    CUtensorMap out, res;
};

template <int EK>
struct ParamsOf {
    using type = EpParams;
    using maps = OutMaps;
};
template <>
struct ParamsOf<kEpPlain> {
    using type = Params;
    using maps = CUtensorMap;
};

// S sums of one weight row (32 lanes: 32 rows), of S consecutive tokens or
// digit rows with the scales sc, into output values: kEpLinear o[i] of token
// i, kEpGated o[i] of token 2 i + (lane & 1) and the lane's row pair, kEpGrad
// o[i] of token i (digit rows D i .. D i + D - 1, lowest first).
// All 32 lanes call it.
template <int EK, int D, int S, int O>
__device__ __forceinline__ void ep_values(const EpParams& p, const uint32_t (&v)[S], const float* sc, float al,
                                          float bi, int lane, float (&o)[O])
{
    if constexpr (EK == kEpGrad) {
        static_assert(O == S / D, "digits");
#pragma unroll
        for (int i = 0; i < O; ++i) {
            // every step rounds relative to the joined value
            float f = (float)(int32_t)v[i * D + D - 1];
#pragma unroll
            for (int d = D - 2; d >= 0; --d) f = __fmaf_rn(f, 256.0f, (float)(int32_t)v[i * D + d]);
            o[i] = __fmul_rn(f, sc[i]);
        }
    } else if constexpr (EK == kEpLinear) {
        static_assert(O == S, "one value per sum");
#pragma unroll
        for (int i = 0; i < O; ++i) o[i] = __fmul_rn(__fmul_rn((float)(int32_t)v[i], al), sc[i]);
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < O; ++i) o[i] = __fadd_rn(o[i], bi);
        }
        ep::apply_act<O>(o, p.act, p.dtype);
    } else {
        static_assert(2 * O == S, "one value per pair of sums");
        const bool odd = lane & 1;
        float up[O];
#pragma unroll
        for (int i = 0; i < O; ++i) {
            float z0 = __fmul_rn(__fmul_rn((float)(int32_t)v[2 * i], al), sc[2 * i]);
            float z1 = __fmul_rn(__fmul_rn((float)(int32_t)v[2 * i + 1], al), sc[2 * i + 1]);
            if (p.bias) {
                z0 = __fadd_rn(z0, bi);
                z1 = __fadd_rn(z1, bi);
            }
            const float got = __shfl_xor_sync(0xffffffffu, odd ? z0 : z1, 1);
            o[i] = odd ? got : z0;
            up[i] = odd ? z1 : got;
        }
        ep::apply_act<O>(o, p.act, p.dtype);
#pragma unroll
        for (int i = 0; i < O; ++i) o[i] = __fmul_rn(o[i], up[i]);
    }
}

// v[i] to base + i * stride bytes for i < cnt: one running address, no
// per-element products.
template <int O, class T>
__device__ __forceinline__ void store_strided(char* base, int64_t stride, int cnt, const T (&v)[O])
{
#pragma unroll
    for (int i = 0; i < O; ++i) {
        if (i < cnt) *reinterpret_cast<T*>(base) = v[i];
        base += stride;
    }
}

template <int O, class T>
__device__ __forceinline__ void load_strided(const char* base, int64_t stride, int cnt, uint32_t (&v)[O])
{
#pragma unroll
    for (int i = 0; i < O; ++i) {
        v[i] = i < cnt ? (uint32_t)*reinterpret_cast<const T*>(base) : 0u;
        base += stride;
    }
}

// Sums handled at once: kEpLinear has one value per sum where the others have
// one per two or more, and 16 of them beside a residual do not fit the 96
// registers that 18 warps leave a thread (with 16, spills made its slices 2.5
// times as long as kEpGated's).
template <int EK>
constexpr int kEpSums = EK == kEpLinear ? 8 : 16;

// The kept sums of S tokens from m0 on, row n.
template <int S>
__device__ __forceinline__ void ep_keep(const EpParams& p, const uint32_t (&v)[S], int64_t m0, int64_t n)
{
    if (!p.acc) return;
    const int64_t left = n < p.N ? p.M - m0 : 0;
    store_strided<S, uint32_t>(reinterpret_cast<char*>(p.acc + m0 * p.N + n), 4 * p.N, (int)(left < S ? left : S), v);
}

// ep_values of S sums, stored element by element: output rows from m0 on,
// column col (out of range: not stored).  The residual is loaded whole before
// the first store (it may be the output itself, so a load could not pass a
// store on its own).
template <int EK, int D, int S>
__device__ __forceinline__ void ep_store(const EpParams& p, const uint32_t (&v)[S], const float* sc, float al,
                                         float bi, int lane, int64_t m0, int64_t col)
{
    constexpr int O = EK == kEpGated ? S / 2 : S / D;
    constexpr int kStep = EK == kEpGated ? 2 : 1;            // output rows between values
    const int first = EK == kEpGated ? lane & 1 : 0;
    const int64_t left = (p.Mo - m0 - first + kStep - 1) / kStep;
    const int cnt = col >= p.No ? 0 : left < O ? (int)left : O;
    const int es = ep::elem_size(p.dtype);
    const int64_t at = ((m0 + first) * p.No + col) * es, stride = (int64_t)kStep * p.No * es;
    // as read, widened only when added: all loads are in flight at once
    [[maybe_unused]] uint32_t rs[EK == kEpLinear ? O : 1];
    if constexpr (EK == kEpLinear) {
        if (p.res) {
            const char* r = static_cast<const char*>(p.res) + at;
            if (p.dtype == SHERRY_F32) load_strided<O, uint32_t>(r, stride, cnt, rs);
            else load_strided<O, uint16_t>(r, stride, cnt, rs);
        }
    }
    float o[O];
    ep_values<EK, D, S, O>(p, v, sc, al, bi, lane, o);
    if constexpr (EK == kEpLinear) {
        if (p.res) {
#pragma unroll
            for (int i = 0; i < O; ++i)
                o[i] = __fadd_rn(o[i], p.dtype == SHERRY_F32 ? __uint_as_float(rs[i])
                                                             : ep::from16((uint16_t)rs[i], p.dtype));
        }
    }
    char* base = static_cast<char*>(p.out) + at;
    if (p.dtype == SHERRY_F32) {
        store_strided<O, float>(base, stride, cnt, o);
    } else {
        uint16_t h[O];
#pragma unroll
        for (int i = 0; i < O; ++i) h[i] = ep::to16(o[i], p.dtype);
        store_strided<O, uint16_t>(base, stride, cnt, h);
    }
}

// ep_values of S sums into a staging slot of 16 sums x 32 rows (sums part ..
// part + S - 1 of the slot): outputs [token][column], replacing the residual
// there in place when has_res.
template <int EK, int D, int S>
__device__ __forceinline__ void ep_stage(const EpParams& p, const uint32_t (&v)[S], const float* sc, float al,
                                         float bi, int lane, float* stg, int part, bool has_res)
{
    constexpr int O = EK == kEpGated ? S / 2 : S / D;
    constexpr int OW = EK == kEpGated ? 16 : 32;             // columns of the slot
    constexpr int kStep = EK == kEpGated ? 2 * OW : OW;
    float o[O];
    ep_values<EK, D, S, O>(p, v, sc, al, bi, lane, o);
    const int at0 = (int)ep::first_token<D>(part) * OW + (EK == kEpGated ? (lane & 1) * OW + (lane >> 1) : lane);
    if (p.dtype == SHERRY_F32) {
        if (has_res) {
#pragma unroll
            for (int i = 0; i < O; ++i) o[i] = __fadd_rn(o[i], stg[at0 + i * kStep]);
        }
#pragma unroll
        for (int i = 0; i < O; ++i) stg[at0 + i * kStep] = o[i];
    } else {
        uint16_t* st16 = reinterpret_cast<uint16_t*>(stg);
        if (has_res) {
            uint16_t h[O];
#pragma unroll
            for (int i = 0; i < O; ++i) h[i] = st16[at0 + i * kStep];
#pragma unroll
            for (int i = 0; i < O; ++i) o[i] = __fadd_rn(o[i], ep::from16(h[i], p.dtype));
        }
#pragma unroll
        for (int i = 0; i < O; ++i) st16[at0 + i * kStep] = ep::to16(o[i], p.dtype);
    }
}

// The work of one CTA as a sequence of tile segments (a segment = chunks
// [cb, ce) of one tile; units are numbered tile-major, unit = tile * Kc +
// chunk).  With T tiles and G CTAs, the last R = T mod G tiles are split
// stream-K: their RU = R * Kc units are cut into G contiguous shares (each
// under one tile; when RU < G, one unit to each of the first RU CTAs, so
// that no share is empty), walked first.  Then every CTA walks F = T div G whole tiles of
// its own.  So every CTA gets the same number of units within one, the
// tiles summed across CTAs come first (their reductions overlap the later
// tiles), and every CTA ends on whole tiles.  With `whole` the last R tiles
// are not cut: each of the first R CTAs walks one of them first, and no tile is
// summed across CTAs.  With `cluster` every tile is one cluster's, a share of
// its chunks each CTA's.  All roles walk this sequence.
struct SegWalk {
    int64_t Kc, tile, cb, ce, end_u, r1_tile, r1_end_tile;
    int range;                                  // 0 split share, 1 own tiles, 2 done
    SHERRY_HD SegWalk(const Params& p, int64_t b, int64_t G)
    {
        Kc = p.Kc;
        const int64_t T = p.TM * p.TN;
        const int64_t F = T / G, R = T - F * G;
        const int64_t L0 = (T - R) * Kc, RU = R * Kc;
        r1_tile = b * F;
        r1_end_tile = (b + 1) * F;
        int64_t a0, a1;
        if (p.cluster) {
            // one tile per cluster, its chunks cut evenly
            const int64_t S = p.cluster, t = b / S, q = b - t * S;
            a0 = t * Kc + Kc * q / S;
            a1 = t * Kc + Kc * (q + 1) / S;
            r1_tile = r1_end_tile = 0;
        } else if (p.whole) {
            a0 = L0 + Kc * b;
            a1 = b < R ? a0 + Kc : a0;
        } else if (RU >= G) {
            a0 = L0 + RU * b / G;
            a1 = L0 + RU * (b + 1) / G;
        } else {
            a0 = L0 + b;
            a1 = a0 + (b < RU ? 1 : 0);
        }
        if (a0 < a1) {
            range = 0;
            end_u = a1;
            tile = a0 / Kc;
            cb = a0 - tile * Kc;
            const int64_t te = (tile + 1) * Kc;
            ce = (te < a1 ? te : a1) - tile * Kc;
        } else {
            start_own();
        }
    }
    SHERRY_HD void start_own()
    {
        if (r1_tile < r1_end_tile) {
            range = 1;
            tile = r1_tile;
            cb = 0;
            ce = Kc;
        } else {
            range = 2;
        }
    }
    SHERRY_HD bool done() const { return range == 2; }
    SHERRY_HD bool complete() const { return cb == 0 && ce == Kc; }
    SHERRY_HD void next()
    {
        if (range == 0) {
            const int64_t u = tile * Kc + ce;
            if (u < end_u) {
                ++tile;
                cb = 0;
                ce = (end_u - u) < Kc ? (end_u - u) : Kc;
            } else {
                start_own();
            }
        } else if (++tile >= r1_end_tile) {
            range = 2;
        }
    }
};

// First and last CTA of a split tile t (one of the last R tiles): the owners
// of its first and last unit among the G shares of the split units.
SHERRY_HD inline void split_owners(const Params& p, int64_t t, int64_t G, int64_t* bf, int64_t* bl)
{
    const int64_t T = p.TM * p.TN;
    const int64_t R = T - (T / G) * G;
    const int64_t RU = R * p.Kc;
    const int64_t u = (t - (T - R)) * p.Kc;
    if (RU >= G) {
        *bf = ((u + 1) * G - 1) / RU;
        *bl = ((u + p.Kc) * G - 1) / RU;
    } else {
        *bf = u;
        *bl = u + p.Kc - 1;
    }
}

__device__ __forceinline__ uint64_t b_desc_sw128(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);          // start address
    d |= (uint64_t)1u << 16;                               // leading byte offset (unused, 16 B)
    d |= (uint64_t)(1024u >> 4) << 32;                     // stride byte offset: 8 rows x 128 B
    d |= (uint64_t)1u << 46;                               // descriptor version (sm_100)
    d |= (uint64_t)2u << 61;                               // 128-byte swizzle
    return d;
}

__device__ __forceinline__ void report(unsigned* status, volatile int* abort_flag, unsigned code)
{
    atomicCAS(status, 0u, code);
    *abort_flag = 1;
}

template <int BN, int SC, int WF = kWeightSherry, int EK = kEpPlain, int D = 1, int EG = 1>
__global__ void __launch_bounds__(Cfg<BN, SC, WF, EG>::kThreads, 1)
    sherry_gemm_tc_kernel(const __grid_constant__ CUtensorMap xmap,
                          const __grid_constant__ typename ParamsOf<EK>::maps ymap,
                          const typename ParamsOf<EK>::type p)
{
    using C = Cfg<BN, SC, WF, EG>;
    static_assert(EK != kEpPlain || EG == 1, "EG");
    static_assert(EK == kEpGrad ? D == 3 || D == 4 : D == 1, "digits per token");
    // Few tokens and fewer tiles than SMs: the CTAs of a cluster take a share of
    // a tile's chunks each and add their sums into the first one's staging
    // slots over distributed shared memory (M = 16 bf16: K = 4096, N = 4096
    // 10.2 us whole, 11.1 split through the workspace, 9.2 so; K = 14336 24.6,
    // 15.4, 13.3)
    constexpr bool kClusterSplit = EK != kEpPlain && EG == 1 && BN <= 32;
    const bool cluster = kClusterSplit && p.cluster > 0;
    // kEpLinear: a barrier per staging slot of each epilogue warp, for the
    // residual boxes loaded into it
    __shared__ __align__(8) uint64_t res_bars[EK == kEpLinear ? EG * 4 * C::kEpSlots : 1];
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(128) uint32_t table[32];
    // 1024-byte aligned start, computed by pointer arithmetic so that the
    // compiler keeps the shared address space (plain ld.shared/st.shared)
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t bar0 = sbase + C::kOffBars;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (C::kStages + s); };
    auto afull_bar = [&](int a) { return bar0 + 8u * (2 * C::kStages + a); };
    auto aempty_bar = [&](int a) { return bar0 + 8u * (2 * C::kStages + C::kAStages + a); };
    auto dfull_bar = [&](int d) { return bar0 + 8u * (2 * C::kStages + 2 * C::kAStages + d); };
    auto dempty_bar = [&](int d) { return bar0 + 8u * (2 * C::kStages + 2 * C::kAStages + C::kDBufs + d); };
    const uint32_t drain_bar = bar0 + 8u * (2 * C::kStages + 2 * C::kAStages + 2 * C::kDBufs);
    // a stage's codes land on code(s) (the decoders wait for it), its
    // activation boxes on full(s) (the MMA warp waits for it): the codes of
    // the first ring round are copied, and decoded, before the dependency wait
    auto code_bar = [&](int s) { return bar0 + 8u * (2 * C::kStages + 2 * C::kAStages + 2 * C::kDBufs + 1 + s); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    const int64_t G = gridDim.x;

    if (WF == kWeightSherry && threadIdx.x < 32) {
        // code -> four int8 weights of the group, byte i = position i
        const uint32_t c = threadIdx.x, z = c & 3u;
        uint32_t word = 0, slot = 2;
        for (uint32_t i = 0; i < 4; ++i) {
            uint32_t b = 0;
            if (i != z) {
                b = ((c >> slot) & 1u) ? 0xFFu : 0x01u;
                ++slot;
            }
            word |= b << (8 * i);
        }
        table[c] = word;
    }
    if (threadIdx.x == 32) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(code_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 4 + 1);
        }
        for (int a = 0; a < C::kAStages; ++a) {
            ptx::mbar_init(afull_bar(a), 4);
            ptx::mbar_init(aempty_bar(a), 1);
        }
        for (int d = 0; d < C::kDBufs; ++d) {
            ptx::mbar_init(dfull_bar(d), 1);
            ptx::mbar_init(dempty_bar(d), 4);
        }
        ptx::mbar_init(drain_bar, 1);
        if constexpr (EK == kEpLinear)
            for (int i = 0; i < EG * 4 * C::kEpSlots; ++i) ptx::mbar_init(ptx::smem_u32(&res_bars[i]), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    __syncwarp();
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_holder), kTmemCols);
        ptx::tmem_relinquish();
    }
    if (threadIdx.x == 0) ptx::prefetch_tensormap(&xmap);
    if constexpr (kClusterSplit) {
        // the sums start at zero; every CTA of the cluster has its slots ready
        // once the barrier that starts here completes
        if (cluster && warp >= C::kEpiWarp0) {
            uint32_t* z = reinterpret_cast<uint32_t*>(smem + C::kOffStaging) + (warp & 3) * (C::kEpSlots * 16 * 32);
            for (int i = lane; i < BN * 32; i += 32) z[i] = 0u;
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if constexpr (kClusterSplit)
        if (cluster) ptx::cluster_arrive_release();
    const uint32_t tmem = *tmem_holder;
    // Programmatic dependent launch: everything above (barriers, tensor
    // memory, table) overlaps the end of the previous kernel on the stream.
    // The roles that touch global memory the previous kernel may write or
    // read (the producer: activations; the epilogue: scales, y, acc and the
    // split-K workspace) wait for it to complete; the decoders and the MMA
    // warp only use this CTA's shared and tensor memory.
    ptx::pdl_launch_dependents();

    if (warp == kProducerWarp) {
        // Converged warp, elected-lane issue and a non-blocking test of the
        // next slot, for the same reason as the MMA loop below: a copy issued
        // late delays every role after it.
        //
        // The codes do not depend on the previous kernel: the first ring
        // round's code copies are issued before the dependency wait, so that
        // they (and their decoding) overlap the end of the previous kernel;
        // their activation boxes follow after the wait.
        int64_t npre = 0;
        {
            SegWalk w(p, blockIdx.x, G);
            while (!w.done() && npre < C::kStages) {
                const int64_t tn = w.tile % p.TN;
                int c = (int)w.cb;
                int left = (int)(w.ce - w.cb);
                while (left > 0 && npre < C::kStages) {
                    const int nch = left < SC ? left : SC;
                    const uint32_t st = (uint32_t)npre;          // first round: slot npre, no wait
                    ptx::mbar_arrive_expect_tx_elect(code_bar((int)st), (uint32_t)(nch * C::kChunkWBytes));
                    ptx::bulk_g2s_elect(sbase + C::kOffCodes + st * C::kCodeStageBytes,
                                        p.wnative + (tn * p.Kc + c) * (int64_t)C::kChunkWBytes,
                                        (uint32_t)(nch * C::kChunkWBytes), code_bar((int)st));
                    c += nch;
                    left -= nch;
                    ++npre;
                }
                w.next();
            }
        }
        ptx::pdl_wait();
        int s = 0;
        uint32_t ph = 0;
        bool ready = false;                      // empty(s) already seen complete
        bool ok = true;
        int64_t issued = 0;
        SegWalk w(p, blockIdx.x, G);
        while (!w.done()) {
            const int64_t tm = w.tile / p.TN, tn = w.tile - tm * p.TN;
            int c = (int)w.cb;                     // K chunk within the tile
            const uint8_t* src = p.wnative + (tn * p.Kc + c) * (int64_t)C::kChunkWBytes;
            const int32_t ty = (int32_t)(tm * BN);
            int left = (int)(w.ce - w.cb);
            while (left > 0) {
                const int nch = left < SC ? left : SC;
                const bool pre = issued < npre;      // codes already in flight, empty(s) fresh
                if (!ready && !pre) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(empty_bar(s), ph ^ 1u, kWaitLimitNs));
                    if (!ok) break;
                }
                const int s1 = (s + 1 == C::kStages) ? 0 : s + 1;
                const uint32_t ph1 = (s + 1 == C::kStages) ? ph ^ 1u : ph;
                const uint32_t t_e = ptx::mbar_test(empty_bar(s1), ph1 ^ 1u);
                if (!pre) {
                    ptx::mbar_arrive_expect_tx_elect(code_bar(s), (uint32_t)(nch * C::kChunkWBytes));
                    ptx::bulk_g2s_elect(sbase + C::kOffCodes + (uint32_t)s * C::kCodeStageBytes, src,
                                        (uint32_t)(nch * C::kChunkWBytes), code_bar(s));
                }
                ptx::mbar_arrive_expect_tx_elect(full_bar(s), (uint32_t)(nch * C::kBChunkBytes));
                if (nch == SC) {
#pragma unroll
                    for (int j = 0; j < SC; ++j)
                        ptx::tma_load_2d_elect(sbase + (uint32_t)(s * C::kBStageBytes + j * C::kBChunkBytes), &xmap,
                                               (c + j) * SHERRY_KCHUNK, ty, full_bar(s));
                } else {
                    for (int j = 0; j < nch; ++j)
                        ptx::tma_load_2d_elect(sbase + (uint32_t)(s * C::kBStageBytes + j * C::kBChunkBytes), &xmap,
                                               (c + j) * SHERRY_KCHUNK, ty, full_bar(s));
                }
                src += nch * C::kChunkWBytes;
                c += nch;
                left -= nch;
                ++issued;
                s = s1;
                ph = ph1;
                ready = __all_sync(0xffffffffu, t_e != 0u);
            }
            if (!ok) break;
            w.next();
        }
        if (!ok && lane == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_PRODUCER);
        // every copy issued has landed before the CTA may exit (in the
        // normal flow the consumers already waited for all of them)
        const int64_t from = issued > C::kStages ? issued - C::kStages : 0;
        int ds = (int)(from % C::kStages);
        uint32_t dph = (uint32_t)((from / C::kStages) & 1);
        for (int64_t i = from; i < issued; ++i) {
            const bool landed = ptx::mbar_wait_bounded(full_bar(ds), dph, kWaitLimitNs) &&
                                ptx::mbar_wait_bounded(code_bar(ds), dph, kWaitLimitNs);
            if (!__all_sync(0xffffffffu, landed)) {
                if (lane == 0) atomicCAS(p.status, 0u, (unsigned)SHERRY_DEV_TIMEOUT_DRAIN);
                break;
            }
            if (++ds == C::kStages) { ds = 0; dph ^= 1u; }
        }
    } else if (warp == kMmaWarp) {
        // The MMA issue blocks while the tensor pipe is busy and the pipe holds
        // almost no queued work, so every instruction between two MMAs is a
        // bubble.  Hence: the whole warp runs the loop converged, with every
        // loop value warp-uniform (votes make the wait results uniform), and
        // one elected lane issues inside the MMA's own instruction sequence;
        // and the next stage's barriers are tested (non-blocking) before the
        // current stage's MMAs, so a stage whose inputs are ready starts with
        // no wait.
        int s = 0, a = 0, d = 0;
        uint32_t sph = 0, aph = 0, dph = 0;
        bool issued_any = false, ok = true;
        bool ready = false;                      // this stage's full and afull already seen complete
        SegWalk w(p, blockIdx.x, G);
        while (!w.done()) {
            int left = (int)(w.ce - w.cb);         // chunks of this tile segment
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(dempty_bar(d), dph ^ 1u, kWaitLimitNs));
            if (!ok) break;
            const uint32_t d_tmem = tmem + (uint32_t)(d * BN);
            uint32_t acc0 = 0u;
            while (left > 0) {
                if (!ready) {
                    ok = ptx::mbar_wait_bounded(full_bar(s), sph, kWaitLimitNs) &&
                         ptx::mbar_wait_bounded(afull_bar(a), aph, kWaitLimitNs);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                ptx::tc_fence_after();
                const int s1 = (s + 1 == C::kStages) ? 0 : s + 1;
                const int a1 = (a + 1 == C::kAStages) ? 0 : a + 1;
                const uint32_t sph1 = (s + 1 == C::kStages) ? sph ^ 1u : sph;
                const uint32_t aph1 = (a + 1 == C::kAStages) ? aph ^ 1u : aph;
                // both tests issue before the MMAs; their results are read
                // only after the stage's last MMA
                const uint32_t t_full = ptx::mbar_test(full_bar(s1), sph1);
                const uint32_t t_a = ptx::mbar_test(afull_bar(a1), aph1);
                const uint32_t a_tmem = tmem + (uint32_t)(C::kACol0 + a * C::kACols);
                // descriptor of the stage's first K step; later steps only
                // add to the start-address field (16-byte units)
                const uint64_t desc0 = b_desc_sw128(sbase + (uint32_t)s * C::kBStageBytes);
                if (left >= SC) {
#pragma unroll
                    for (int j = 0; j < SC; ++j)
                        ptx::mma_i8_ts_chunk_elect(d_tmem, a_tmem + (uint32_t)(32 * j),
                                                   desc0 + (uint64_t)((j * C::kBChunkBytes) >> 4), C::kIdesc,
                                                   j == 0 ? acc0 : 1u);
                    left -= SC;
                } else {
                    for (int j = 0; j < left; ++j)
                        ptx::mma_i8_ts_chunk_elect(d_tmem, a_tmem + (uint32_t)(32 * j),
                                                   desc0 + (uint64_t)((j * C::kBChunkBytes) >> 4), C::kIdesc,
                                                   j == 0 ? acc0 : 1u);
                    left = 0;
                }
                ptx::tc_commit_elect(empty_bar(s));
                ptx::tc_commit_elect(aempty_bar(a));
                issued_any = true;
                acc0 = 1u;
                s = s1; a = a1; sph = sph1; aph = aph1;
                ready = __all_sync(0xffffffffu, (t_full & t_a) != 0u);
            }
            if (!ok) break;
            ptx::tc_commit_elect(dfull_bar(d));
            if (++d == C::kDBufs) { d = 0; dph ^= 1u; }
            w.next();
        }
        if (!ok && lane == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_MMA);
        if (issued_any) {
            // all MMAs of this warp complete before tensor memory is freed
            ptx::tc_commit_elect(drain_bar);
            const bool done = ptx::mbar_wait_bounded(drain_bar, 0, kWaitLimitNs);
            if (!__all_sync(0xffffffffu, done) && lane == 0)
                atomicCAS(p.status, 0u, (unsigned)SHERRY_DEV_TIMEOUT_DRAIN);
        }
    } else if (warp >= kDecWarp0 && warp < kDecWarp0 + 4 * C::kDecGroups) {
        const int grp = (warp - kDecWarp0) / 4;
        const int quad = warp & 3;                 // TMEM lane quadrant of this warp
        const int row = quad * 32 + lane;          // row within the 128-row tile
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        // 128-byte aligned: a code's entry address is (code * 4) | table_s
        const uint32_t table_s = ptx::smem_u32(table);
        // byte offsets of this row's five code words within a chunk
        uint32_t wpos[SHERRY_CHUNK_WORDS];
#pragma unroll
        for (int k = 0; k < SHERRY_CHUNK_WORDS; ++k) wpos[k] = 4u * (uint32_t)sherry_word_pos(k, row);
        int s = 0, a = 0;
        uint32_t sph = 0, aph = 0;
        int turn = 0;                               // iteration index modulo C::kDecGroups
        bool quit = false;
        SegWalk w(p, blockIdx.x, G);
        for (; !w.done() && !quit; w.next()) {
          for (int left = (int)(w.ce - w.cb); left > 0; left -= SC, turn = (turn + 1 == C::kDecGroups) ? 0 : turn + 1) {
            const int nch = left < SC ? left : SC;
            const bool mine = turn == grp;
            if (mine) {
                // no per-stage abort poll: after another role gave up, this
                // wait runs out by itself and the group leaves
                bool ok = ptx::mbar_wait_bounded(code_bar(s), sph, kWaitLimitNs);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_DECODER);
                    quit = true;
                    break;
                }
                const uint32_t codes_s = sbase + (uint32_t)(C::kOffCodes + s * C::kCodeStageBytes);
                if constexpr (WF == kWeightInt4) {
                    // SINT4 -> int8 16 w (shift into the high half of each
                    // byte); the stage's weights are read while its A slot is
                    // filled, then both are released
                    ok = ptx::mbar_wait_bounded(aempty_bar(a), aph ^ 1u, kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_DECODER);
                        quit = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t wrow = codes_s + (uint32_t)(16 * row);
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        if (j >= nch) break;
                        uint32_t a_vals[32];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];
                            ptx::lds_v4_u32(wrow + (uint32_t)(j * C::kChunkWBytes + q * SHERRY_TILE_ROWS * 16), v);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                a_vals[8 * q + 2 * i] = (v[i] << 4) & 0xF0F0F0F0u;
                                a_vals[8 * q + 2 * i + 1] = v[i] & 0xF0F0F0F0u;
                            }
                        }
                        ptx::tmem_st_32x32b_x32(lane_base + (uint32_t)(C::kACol0 + a * C::kACols + 32 * j), a_vals);
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(empty_bar(s));
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(afull_bar(a));
                } else if constexpr (WF == kWeightT2) {
                    // four 2-bit weights -> four int8 by one byte permute
                    ok = ptx::mbar_wait_bounded(aempty_bar(a), aph ^ 1u, kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_DECODER);
                        quit = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t wrow = codes_s + (uint32_t)(16 * row);
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        if (j >= nch) break;
                        uint32_t a_vals[32];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t v[4];
                            ptx::lds_v4_u32(wrow + (uint32_t)(j * C::kChunkWBytes + q * SHERRY_TILE_ROWS * 16), v);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    a_vals[16 * q + 4 * i + c] = __byte_perm(
                                        0x00FF0100u, 0u, (v[i] >> (2 * (c & 1) + 16 * (c >> 1))) & 0x3333u);
                        }
                        ptx::tmem_st_32x32b_x32(lane_base + (uint32_t)(C::kACol0 + a * C::kACols + 32 * j), a_vals);
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(empty_bar(s));
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(afull_bar(a));
                } else {
                uint32_t w[SC][SHERRY_CHUNK_WORDS];
#pragma unroll
                for (int j = 0; j < SC; ++j)
#pragma unroll
                    for (int k = 0; k < SHERRY_CHUNK_WORDS; ++k)
                        w[j][k] = (j < nch) ? ptx::lds_u32(codes_s + (uint32_t)(j * C::kChunkWBytes) + wpos[k]) : 0u;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty_bar(s));
                ok = ptx::mbar_wait_bounded(aempty_bar(a), aph ^ 1u, kWaitLimitNs);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_DECODER);
                    quit = true;
                    break;
                }
                ptx::tc_fence_after();
#pragma unroll
                for (int j = 0; j < SC; ++j) {
                    if (j >= nch) break;
                    uint32_t a_vals[32];
#pragma unroll
                    for (int g = 0; g < 32; ++g) {
                        // byte offset of the group's table entry: code * 4
                        const int bit = 5 * g, wi = bit >> 5, off = bit & 31;
                        uint32_t v;
                        if (off == 0) v = w[j][wi] << 2;
                        else if (off == 1) v = w[j][wi] << 1;
                        else if (off <= 27) v = w[j][wi] >> (off - 2);
                        else v = __funnelshift_r(w[j][wi], w[j][wi + 1], off - 2);
                        a_vals[g] = ptx::lds_u32_nv((v & 0x7Cu) | table_s);
                    }
                    ptx::tmem_st_32x32b_x32(lane_base + (uint32_t)(C::kACol0 + a * C::kACols + 32 * j), a_vals);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(afull_bar(a));
                }
            }
            if (++s == C::kStages) { s = 0; sph ^= 1u; }
            if (++a == C::kAStages) { a = 0; aph ^= 1u; }
          }
        }
    } else if (warp >= C::kEpiWarp0) {
        ptx::pdl_wait();
        const int quad = warp & 3;
        const int r = quad * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        const int grp = EG == 1 ? 0 : (warp - C::kEpiWarp0) / 4;
        const int etid = (threadIdx.x - C::kEpiWarp0 * 32) & 127;
        const uint32_t ebar = 1u + (uint32_t)grp;   // the group's named barrier
        int64_t seg = 0;                           // this group's segments so far
        int d = grp;
        uint32_t dph = 0;
        uint32_t stage_slice = 0;                  // output slices staged so far
        [[maybe_unused]] uint32_t res_phase = 0;   // parity of each slot's residual barrier
        [[maybe_unused]] bool res_ok = true;
        [[maybe_unused]] const uint32_t res_bar0 =
            ptx::smem_u32(&res_bars[EK == kEpLinear ? (4 * grp + quad) * C::kEpSlots : 0]);
        [[maybe_unused]] float* const stg_w =
            reinterpret_cast<float*>(smem + C::kOffStaging) + (4 * grp + quad) * (C::kEpSlots * 16 * 32);
        SegWalk w(p, blockIdx.x, G);
        [[maybe_unused]] int turn = 0;             // segment index modulo EG
        [[maybe_unused]] bool met = false;         // this thread passed the cluster's second barrier
        if constexpr (kClusterSplit)
            if (cluster) ptx::cluster_wait_acquire();
        for (; !w.done(); w.next()) {
            if constexpr (EG > 1) {
                const bool mine = turn == grp;
                turn = (turn + 1 == EG) ? 0 : turn + 1;
                if (!mine) continue;
            }
            const int64_t tile = w.tile;
            const int64_t tm = tile / p.TN, tn = tile - tm * p.TN;
            const int64_t n = tn * SHERRY_TILE_ROWS + r;
            const bool complete = w.complete();
            // the tile's token scales and this row's alpha do not depend on
            // the MMAs: fetch them into shared memory (double-buffered by
            // segment) before waiting for the accumulators
            float* sc_s = reinterpret_cast<float*>(smem + C::kOffMisc + 64) + (2 * grp + (int)(seg & 1)) * BN;
            int64_t Mo = p.M;                          // scales: one per token
            if constexpr (EK != kEpPlain) Mo = p.Mo;
            constexpr int kTileTokens = (int)ep::first_token<D>(BN);
            for (int i = etid; i < kTileTokens; i += 128) {
                const int64_t m = tm * kTileTokens + i;
                sc_s[i] = (m < Mo) ? __ldg(p.x_scale + m) : 0.0f;
            }
            float al = 0.0f, bi = 0.0f;
            if constexpr (EK != kEpGrad) al = (n < p.N) ? __ldg(p.alpha + n) : 0.0f;
            if constexpr (EK == kEpLinear || EK == kEpGated) bi = (p.bias && n < p.N) ? __ldg(p.bias + n) : 0.0f;
            // output column of this lane's row
            const int64_t col = EK == kEpGated ? n >> 1 : n;
            bool via_tma = complete && p.y_tma;
            if constexpr (EK == kEpPlain) via_tma = via_tma && p.y && !p.acc;
            // slices of 16 sums that hold tokens, and the residual's first boxes
            const int64_t rows_left = p.M - tm * BN;
            [[maybe_unused]] const int nslices = (int)((rows_left < BN ? rows_left : BN) + 15) >> 4;
            [[maybe_unused]] const int32_t out_x =
                (int32_t)((tn * SHERRY_TILE_ROWS + quad * 32) / (EK == kEpGated ? 2 : 1));
            [[maybe_unused]] auto load_res = [&](int q, uint32_t slot) {
                if constexpr (EK == kEpLinear) {
                    const uint32_t bar = res_bar0 + 8u * slot;
                    ptx::mbar_arrive_expect_tx(bar, (uint32_t)(16 * 32 * ep::elem_size(p.dtype)));
                    ptx::tma_load_2d(ptx::smem_u32(stg_w + slot * (16 * 32)), &ymap.res, out_x, (int32_t)(tm * BN + 16 * q),
                                     bar);
                }
            };
            [[maybe_unused]] bool has_res = false;
            [[maybe_unused]] int res_upto = 0;         // slices whose residual box was issued
            if constexpr (EK == kEpLinear) {
                has_res = via_tma && p.res && res_ok;
                if (has_res) {
                    res_upto = nslices < C::kEpSlots - 1 ? nslices : C::kEpSlots - 1;
                    if (lane == 0) {
                        ptx::bulk_wait_group_read<0>();
                        for (int q = 0; q < res_upto; ++q) load_res(q, (stage_slice + q) % C::kEpSlots);
                    }
                    __syncwarp();
                }
            }
            // every epilogue thread waits; the AND over the 128 of them makes
            // the leave-or-stay decision uniform
            bool ok = !*abort_flag && ptx::mbar_wait_bounded(dfull_bar(d), dph, kWaitLimitNs);
            ok = ptx::named_bar_and(ebar, 128, ok);
            if (!ok) {
                if (etid == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_EPILOGUE);
                if constexpr (EK == kEpLinear) {
                    // the residual boxes in flight land before the CTA may exit
                    if (has_res)
                        for (int q = 0; q < res_upto; ++q) {
                            const uint32_t slot = (stage_slice + q) % C::kEpSlots;
                            if (!ptx::mbar_wait_bounded(res_bar0 + 8u * slot, (res_phase >> slot) & 1u, kWaitLimitNs))
                                atomicCAS(p.status, 0u, (unsigned)SHERRY_DEV_TIMEOUT_DRAIN);
                        }
                }
                break;
            }
            ptx::tc_fence_after();
            int64_t slot = 0, nparts = 1;
            if (!complete && !cluster) {
                int64_t bf = 0, bl = 0;
                split_owners(p, tile, G, &bf, &bl);
                slot = bf;
                // the feed-forward launches' slots are as many as their split tiles
                if constexpr (EK != kEpPlain) slot = tile - p.TM * p.TN / G * G;
                nparts = bl - bf + 1;
            }
            int32_t* wsl = p.ws + slot * (int64_t)BN * SHERRY_TILE_ROWS;
            if constexpr (EK != kEpPlain) {
                if (via_tma) {
                    // As below, in slices of 16 sums x 32 rows with kEpSlots
                    // staging slots per warp.  A residual box is loaded by
                    // TMA into the slot its outputs will take, up to
                    // kEpSlots - 1 slices ahead (the first ones before the
                    // accumulators are complete), and replaced in place.
                    constexpr int S = kEpSums<EK>;
#pragma unroll 1
                    for (int q = 0; q < nslices; ++q) {
                        const int j0 = 16 * q;
                        const int64_t m0 = ep::first_token<D>(tm * BN + j0);
                        const uint32_t slot = stage_slice % C::kEpSlots;
                        float* stg = stg_w + slot * (16 * 32);
                        if (has_res) {
                            if constexpr (EK == kEpLinear) {
                                // every box issued is waited for; after a wait
                                // ran out no further one is issued
                                if (q < res_upto) {
                                    const bool in = ptx::mbar_wait_bounded(res_bar0 + 8u * slot,
                                                                           (res_phase >> slot) & 1u, kWaitLimitNs);
                                    if (!__all_sync(0xffffffffu, in)) {
                                        res_ok = false;
                                        if (lane == 0) report(p.status, abort_flag, SHERRY_DEV_TIMEOUT_EPILOGUE);
                                    }
                                    res_phase ^= 1u << slot;
                                }
                            }
                        } else {
                            // the slot's earlier store has read it
                            if (lane == 0) ptx::bulk_wait_group_read<C::kEpSlots - 1>();
                            __syncwarp();
                        }
#pragma unroll 1
                        for (int part = 0; part < 16; part += S) {
                            uint32_t v[S];
                            if constexpr (S == 16) ptx::tmem_ld_32x32b_x16(lane_base + (uint32_t)(d * BN + j0), v);
                            else ptx::tmem_ld_32x32b_x8(lane_base + (uint32_t)(d * BN + j0 + part), v);
                            ptx::tmem_wait_ld_of(v);
                            if constexpr (EK != kEpGrad) ep_keep<S>(p, v, m0 + part, n);
                            ep_stage<EK, D, S>(p, v, sc_s + ep::first_token<D>(j0 + part), al, bi, lane, stg, part, has_res);
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            ptx::tma_store_2d(&ymap.out, out_x, (int32_t)m0, ptx::smem_u32(stg));
                            ptx::bulk_commit_group();
                        }
                        if constexpr (EK == kEpLinear) {
                            if (has_res && res_ok && res_upto < nslices) {
                                if (lane == 0) {
                                    ptx::bulk_wait_group_read<1>();      // the store of slice q - 1, the slot's last
                                    load_res(res_upto, (stage_slice + C::kEpSlots - 1) % C::kEpSlots);
                                }
                                ++res_upto;
                            }
                        }
                        ++stage_slice;
                    }
                }
            } else if (via_tma) {
                // Each warp stores its own 32 rows x kSlice tokens through TMA
                // from its own double-buffered staging, with its own bulk
                // groups: no barrier across the epilogue warps per slice.
                constexpr int SL = C::kSlice;
                float* stg_w = reinterpret_cast<float*>(smem + C::kOffStaging) + quad * (2 * SL * 32);
#pragma unroll 1
                for (int j0 = 0; j0 < BN; j0 += SL) {
                    if (tm * BN + j0 >= p.M) break;     // tokens past M: nothing to store
                    uint32_t v[SL];
                    if constexpr (SL == 32) ptx::tmem_ld_32x32b_x32(lane_base + (uint32_t)(d * BN + j0), v);
                    else ptx::tmem_ld_32x32b_x16(lane_base + (uint32_t)(d * BN + j0), v);
                    // this slice's buffer is free once the store issued two
                    // slices ago has read it
                    if (lane == 0) ptx::bulk_wait_group_read<1>();
                    __syncwarp();
                    ptx::tmem_wait_ld();
                    float* stg = stg_w + (stage_slice & 1) * (SL * 32);
#pragma unroll
                    for (int jj = 0; jj < SL; ++jj)
                        stg[jj * 32 + lane] =
                            __fmul_rn(__fmul_rn((float)((int32_t)v[jj] >> C::kAccShift), al), sc_s[j0 + jj]);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_2d(&ymap, (int32_t)(tn * SHERRY_TILE_ROWS + quad * 32), (int32_t)(tm * BN + j0),
                                          ptx::smem_u32(stg));
                        ptx::bulk_commit_group();
                    }
                    ++stage_slice;
                }
            }
#pragma unroll 1
            for (int j0 = 0; j0 < (via_tma ? 0 : BN); j0 += 16) {
                if constexpr (EK != kEpPlain) {
                    if (complete) {
                        if (ep::first_token<D>(tm * BN + j0) >= p.Mo) break;
                        constexpr int S = kEpSums<EK>;
#pragma unroll 1
                        for (int j = j0; j < j0 + 16; j += S) {
                            uint32_t u[S];
                            if constexpr (S == 16) ptx::tmem_ld_32x32b_x16(lane_base + (uint32_t)(d * BN + j), u);
                            else ptx::tmem_ld_32x32b_x8(lane_base + (uint32_t)(d * BN + j), u);
                            ptx::tmem_wait_ld_of(u);
                            if constexpr (EK != kEpGrad) ep_keep<S>(p, u, tm * BN + j, n);
                            ep_store<EK, D, S>(p, u, sc_s + ep::first_token<D>(j), al, bi, lane, ep::first_token<D>(tm * BN + j),
                                               col);
                        }
                        continue;
                    }
                }
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(lane_base + (uint32_t)(d * BN + j0), v);
                ptx::tmem_wait_ld();
                if constexpr (kClusterSplit) {
                    if (cluster) {
                        // [token][32 rows] of the first CTA's warp of this quadrant
                        const uint32_t to = ptx::mapa(ptx::smem_u32(stg_w + j0 * 32 + lane), 0u);
#pragma unroll
                        for (int jj = 0; jj < 16; ++jj) ptx::red_shared_cluster_add_s32(to + 128u * (uint32_t)jj, (int32_t)v[jj]);
                        continue;
                    }
                }
#pragma unroll
                for (int jj = 0; jj < 16; ++jj) {
                    const int64_t m = tm * BN + j0 + jj;
                    if (m >= p.M) continue;
                    const int32_t a32 = (int32_t)v[jj];      // a partial sum goes to the slot as is
                    if (complete) {
                        const int32_t af = a32 >> C::kAccShift;
                        if (n < p.N) {
                            if (p.acc) p.acc[m * p.N + n] = af;
                            if (p.y) p.y[m * p.N + n] = __fmul_rn(__fmul_rn((float)af, al), sc_s[j0 + jj]);
                        }
                    } else {
                        ptx::red_add_s32(wsl + (j0 + jj) * SHERRY_TILE_ROWS + r, a32);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(dempty_bar(d));
            ++seg;
            if constexpr (EG > 1) {
                dph ^= 1u;                             // the group keeps its accumulator
            } else if (++d == C::kDBufs) {
                d = 0;
                dph ^= 1u;
            }
            const int64_t cur_tm = tm;
            if (!complete) {
                bool last;
                if (cluster) {
                    // every CTA's sums are in the first one's slots
                    if constexpr (kClusterSplit) {
                        __syncwarp();
                        ptx::cluster_arrive_release();
                        ptx::cluster_wait_acquire();
                        met = true;
                    }
                    last = w.cb == 0;
                } else {
                    __threadfence();
                    ptx::named_bar_sync(ebar, 128);
                    if (etid == 0) {
                        const uint32_t old = atomicAdd(p.counters + slot, 1u);
                        last_flag[grp] = (old == (uint32_t)(nparts - 1)) ? 1 : 0;
                    }
                    __syncwarp();
                    ptx::named_bar_sync(ebar, 128);
                    last = last_flag[grp];
                    if (last) __threadfence();
                }
                if (last) {
                    // 16 independent L2 loads in flight per batch: one round
                    // trip per 16 tokens, not one per token
                    const int64_t mleft = p.M - cur_tm * BN;
                    const int jn = mleft < BN ? (int)mleft : BN;
                    if constexpr (EK != kEpPlain) {
                        // The sums come back through the first half of the
                        // warp's staging slots, 16 tokens x its 32 rows each,
                        // one slice ahead, and with them an aligned residual
                        // into the second half, where the outputs then take
                        // its place and leave through TMA stores (unaligned
                        // ones element by element).  192 tokens with a
                        // residual: 64000 cycles beside the decoders when every
                        // slice waited for its sums and its residual, 44000
                        // so.
                        constexpr int S = kEpSums<EK>;
                        constexpr int kRing = C::kEpSlots / 2;
                        constexpr int kSlotFloats = 16 * 32;
                        const int nq = (jn + 15) >> 4;
                        const bool res_in = EK == kEpLinear && p.res && p.y_tma;
                        const uint32_t stg_a = ptx::smem_u32(stg_w);
                        const int es = ep::elem_size(p.dtype);
                        const int piece0 = (lane >> 3) * SHERRY_TILE_ROWS + 32 * quad + 4 * (lane & 7);
                        auto fetch = [&](int q) {
                            if (q < nq) {
                                // 16-byte piece `lane` of every group of four
                                // tokens; tokens past jn: zeros of the slot
                                const uint32_t to = stg_a + (uint32_t)(q % kRing) * (kSlotFloats * 4);
                                if (!cluster) {
                                    const int32_t* from = wsl + 16 * q * SHERRY_TILE_ROWS + piece0;
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        ptx::cp_async16(to + (uint32_t)(k * 4 * 32 * 4 + 16 * lane),
                                                        from + k * (4 * SHERRY_TILE_ROWS));
                                }
                                if constexpr (EK == kEpLinear) {
                                    if (res_in) {
                                        // rows of 32 es bytes: 2 es pieces each, whole inside the residual or outside
                                        const uint32_t rto = to + (uint32_t)kRing * (kSlotFloats * 4);
                                        const int64_t c0 = tn * SHERRY_TILE_ROWS + quad * 32;
                                        for (int i = lane; i < 16 * 2 * es; i += 32) {
                                            const int t = i / (2 * es), piece = i - t * (2 * es);
                                            const int64_t m = cur_tm * BN + 16 * q + t, c = c0 + piece * (16 / es);
                                            if (m < p.Mo && c < p.No)
                                                ptx::cp_async16(rto + 16u * (uint32_t)i,
                                                                static_cast<const char*>(p.res) + (m * p.No + c) * es);
                                        }
                                    }
                                }
                            }
                            ptx::cp_async_commit();
                        };
                        if (lane == 0) ptx::bulk_wait_group_read<0>();   // earlier output stores left the slots
                        __syncwarp();
                        fetch(0);
#pragma unroll 1
                        for (int q = 0; q < nq; ++q) {
                            if constexpr (kRing > 1) {
                                // into the slots of slice q - 1: its sums are
                                // read, its outputs gone once their store has read them
                                if (lane == 0) ptx::bulk_wait_group_read<0>();
                                __syncwarp();
                                fetch(q + 1);
                                ptx::cp_async_wait_group<1>();
                            } else {
                                ptx::cp_async_wait_group<0>();
                            }
                            __syncwarp();                    // every lane's pieces are in
                            const float* in = stg_w + (q % kRing) * kSlotFloats;
                            float* stg = stg_w + (kRing + q % kRing) * kSlotFloats;
                            const int64_t m0 = cur_tm * BN + 16 * q;
#pragma unroll 1
                            for (int part = 0; part < 16; part += S) {
                                uint32_t u[S];
#pragma unroll
                                for (int i = 0; i < S; ++i) u[i] = __float_as_uint(in[(part + i) * 32 + lane]);
                                if constexpr (EK != kEpGrad) ep_keep<S>(p, u, m0 + part, n);
                                const float* sc = sc_s + ep::first_token<D>(16 * q + part);
                                if (p.y_tma) ep_stage<EK, D, S>(p, u, sc, al, bi, lane, stg, part, res_in);
                                else ep_store<EK, D, S>(p, u, sc, al, bi, lane, ep::first_token<D>(m0 + part), col);
                            }
                            if (!cluster) {
                                // the slot's words are zero again for the next call
                                int4* z = reinterpret_cast<int4*>(wsl + 16 * q * SHERRY_TILE_ROWS + piece0);
#pragma unroll
                                for (int k = 0; k < 4; ++k) z[k * SHERRY_TILE_ROWS] = make_int4(0, 0, 0, 0);
                            }
                            if (p.y_tma) ptx::fence_proxy_async_smem();
                            __syncwarp();
                            if (p.y_tma && lane == 0) {
                                ptx::tma_store_2d(&ymap.out, out_x, (int32_t)ep::first_token<D>(m0), ptx::smem_u32(stg));
                                ptx::bulk_commit_group();
                            }
                            if constexpr (kRing == 1) fetch(q + 1);
                        }
                        // whole tiles take the slots in an order of their own
                        ptx::cp_async_wait_group<0>();
                        if (lane == 0) ptx::bulk_wait_group_read<0>();
                        __syncwarp();
                    } else {
                        for (int j0 = 0; j0 < jn; j0 += 16) {
                            int32_t v[16];
#pragma unroll
                            for (int jj = 0; jj < 16; ++jj)
                                v[jj] = (j0 + jj < jn) ? __ldcg(wsl + (j0 + jj) * SHERRY_TILE_ROWS + r) : 0;
#pragma unroll
                            for (int jj = 0; jj < 16; ++jj) {
                                const int j = j0 + jj;
                                if (j >= jn) break;
                                const int64_t m = cur_tm * BN + j;
                                wsl[j * SHERRY_TILE_ROWS + r] = 0;
                                const int32_t af = v[jj] >> C::kAccShift;
                                if (n < p.N) {
                                    if (p.acc) p.acc[m * p.N + n] = af;
                                    if (p.y) p.y[m * p.N + n] = __fmul_rn(__fmul_rn((float)af, al), sc_s[j]);
                                }
                            }
                        }
                    }
                    if (etid == 0 && !cluster) atomicExch(p.counters + slot, 0u);
                }
                __syncwarp();
                ptx::named_bar_sync(ebar, 128);
            }
        }
        if constexpr (kClusterSplit) {
            // a warp that gave up still meets the others
            __syncwarp();
            if (cluster && !met) {
                ptx::cluster_arrive_release();
                ptx::cluster_wait_acquire();
            }
        }
        // shared memory stays valid until every TMA store has read it
        if (lane == 0) ptx::bulk_wait_group<0>();
    }

    __syncwarp();
    if constexpr (kClusterSplit) {
        // the other warps' part in the cluster's two barriers
        if (cluster && warp < C::kEpiWarp0) {
            ptx::cluster_wait_acquire();
            ptx::cluster_arrive_release();
            ptx::cluster_wait_acquire();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

}  // namespace tc
}  // namespace sherry
