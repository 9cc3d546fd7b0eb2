// A mixture-of-experts layer for a few tokens on block-scaled FP8 weights,
// bf16 activations.
//
//   l[t, e] = sum_h X[t, h] Wr[e, h]                 (router logits, fp64 sums)
//   the top_k largest of a token, ties to the lowest expert; w[t, j] their
//   softmax weights (over all experts, or over the chosen ones)
//   h[t, j] = silu(X[t] Wg) * (X[t] Wu) of expert e = idx[t, j]
//   Y[t]    = sum_j w[t, j] (h[t, j] Wd), rounded once to bf16
//
// Launches: the router's logits; with more than kRouteInUp tokens one block
// that makes the choices and the lists of the reached experts; the gate and up
// projections, one block per reached expert and 16 intermediate columns; the
// down projection with the weighted sum, one block per 16 output columns. Each
// reached expert's weights are read once, so the layer is bound by HBM.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_common.h"
#include "fp8_common.h"
#include "internal.h"

namespace svdq {

namespace {

constexpr int kUpThreads = 512;
constexpr int kUpWaves = kUpThreads / 64;
constexpr int kDownThreads = 1024;
constexpr int kDownWaves = kDownThreads / 64;
constexpr int kRouteThreads = 1024;
constexpr int kRouteInUp = kUpWaves;  // tokens that the up kernel's blocks route themselves, one per wave
constexpr int kMaxPairs = SVDQ_FP8_MOE_MAX_TOKENS * SVDQ_FP8_MOE_MAX_TOP_K;
constexpr uint32_t kMoeOob = 0x80000000u;

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// ---- router logits -----------------------------------------------------------

constexpr int kLogitWaves = 4;
constexpr int kLogitExperts = 4;  // per block

// One block: 4 experts x TB tokens; its waves take steps of 512 features in
// turn, a lane 8 of them. bf16 values are widened to fp64 and multiplied and
// added there, so that the order of two logits is the exact one up to 2^-50.
// The lanes' sums are folded together so that each step halves the sums a lane
// holds (TB 4 - 1 exchanges instead of 6 TB 4), the waves' through LDS.
template <int TB>
__global__ __launch_bounds__(64 * kLogitWaves) void moe_logits_kernel(const uint16_t *__restrict__ X,
                                                                      const uint16_t *__restrict__ wr, int T, int H,
                                                                      int E, double *__restrict__ logits) {
    constexpr int kSums = kLogitExperts * TB;
    __shared__ double part[kLogitWaves][kSums];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = blockIdx.x * kLogitExperts, t0 = blockIdx.y * TB;
    double sum[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) sum[i] = 0.0;
    for (int h = wave * 512 + lane * 8; h < H; h += kLogitWaves * 512) {
        u32x4 w[kLogitExperts], x[TB];
#pragma unroll
        for (int i = 0; i < kLogitExperts; ++i)
            w[i] = *reinterpret_cast<const u32x4 *>(wr + (size_t)min(e0 + i, E - 1) * H + h);
#pragma unroll
        for (int i = 0; i < TB; ++i)
            x[i] = *reinterpret_cast<const u32x4 *>(X + (size_t)min(t0 + i, T - 1) * H + h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            auto value = [&](const u32x4 &v) {
                return (double)__uint_as_float(j & 1 ? v[j / 2] & 0xFFFF0000u : v[j / 2] << 16);
            };
            double wv[kLogitExperts];
#pragma unroll
            for (int i = 0; i < kLogitExperts; ++i) wv[i] = value(w[i]);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const double xv = value(x[t]);
#pragma unroll
                for (int i = 0; i < kLogitExperts; ++i)
                    sum[t * kLogitExperts + i] = __builtin_fma(xv, wv[i], sum[t * kLogitExperts + i]);
            }
        }
    }
    // after the steps with n sums left a lane holds those of its own low bits
    int n = kSums, d = 32;
#pragma unroll
    for (; n > 1 && d > 0; n >>= 1, d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const double give = up ? sum[i] : sum[i + n / 2], keep = up ? sum[i + n / 2] : sum[i];
            sum[i] = keep + __shfl_xor(give, d);
        }
    }
#pragma unroll
    for (; d > 0; d >>= 1) sum[0] += __shfl_xor(sum[0], d);
    // lane l holds sum number (its top log2 kSums bits)
    constexpr int kShift = 64 / kSums;
    if (lane % kShift == 0) part[wave][lane / kShift] = sum[0];
    __syncthreads();
    if (threadIdx.x < kSums) {
        double v = 0.0;
#pragma unroll
        for (int w = 0; w < kLogitWaves; ++w) v += part[w][threadIdx.x];
        const int t = t0 + threadIdx.x / kLogitExperts, e = e0 + threadIdx.x % kLogitExperts;
        if (t < T && e < E) logits[(size_t)t * E + e] = v;
    }
}

// ---- the choice ----------------------------------------------------------------

// One wave: the top_k largest of a token's logits and their softmax weights.
// Lane l holds experts l, l + 64, ...; top_k rounds of a wave-wide maximum over
// (logit, lowest expert), each expert chosen at most once whatever its logit;
// NaN orders below every number. idx and gate may be in LDS.
__device__ __forceinline__ void choose(const double *__restrict__ logit, int E, int top_k, bool renorm, int lane,
                                       int32_t *idx, float *gate) {
    constexpr int kPer = SVDQ_FP8_MOE_MAX_EXPERTS / 64;
    constexpr double kLowest = -1.7976931348623157e308;
    double raw[kPer], v[kPer];
    bool open[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        open[i] = lane + 64 * i < E;
        raw[i] = open[i] ? logit[lane + 64 * i] : kLowest;
        v[i] = raw[i] >= kLowest ? raw[i] : kLowest;  // NaN, -inf
    }
    double top = 0.0;
    float chosen = 0.0f, mine = 0.0f;
    int mine_e = 0;
    for (int j = 0; j < top_k; ++j) {
        double best = kLowest, best_raw = 0.0;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (open[i] && (at == 1 << 30 || v[i] > best)) {
                best = v[i];
                best_raw = raw[i];
                at = lane + 64 * i;
            }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const double ob = __shfl_xor(best, d);
            const int oa = __shfl_xor(at, d);
            if (oa != 1 << 30 && (at == 1 << 30 || ob > best || (ob == best && oa < at))) {
                best = ob;
                at = oa;
            }
        }
        best_raw = __shfl(best_raw, at & 63);  // the winner is its lane's own best
        if (j == 0) top = best_raw;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (at == lane + 64 * i) open[i] = false;
        const float e = expf((float)(best_raw - top));
        chosen += e;
        if (lane == j) {
            mine = e;
            mine_e = at;
        }
    }
    float total = chosen;
    if (!renorm) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 64 * i < E) total += expf((float)(raw[i] - top));
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) total += __shfl_xor(total, d);
    }
    if (lane < top_k) {
        idx[lane] = mine_e;
        gate[lane] = mine / total;
    }
}

// The reached experts of a batch, ascending, each with its pairs t top_k + j,
// ascending.
struct MoeLists {
    int32_t *reached;  // [1] how many
    int32_t *experts;  // [reached]
    int32_t *counts;   // [reached]
    int32_t *pairs;    // [reached][T]
};

// The a-th reached expert, or -1, and the number of reached ones, from a bit
// per expert.
__device__ __forceinline__ int reached_expert(const uint32_t *bits, int a, int &reached) {
    int e = -1;
    reached = 0;
#pragma unroll
    for (int i = 0; i < SVDQ_FP8_MOE_MAX_EXPERTS / 32; ++i) {
        uint32_t w = bits[i];
        const int c = __popc(w);
        if (e < 0 && a < reached + c) {
            for (int skip = a - reached; skip > 0; --skip) w &= w - 1;
            e = 32 * i + __ffs((int)w) - 1;
        }
        reached += c;
    }
    return e;
}

// One wave: the pairs of expert e, in order; their number.
__device__ __forceinline__ int collect_pairs(const int32_t *idx, int pairs, int e, int lane, int32_t *list) {
    int n = 0;
    for (int p0 = 0; p0 < pairs; p0 += 64) {
        const bool hit = p0 + lane < pairs && idx[p0 + lane] == e;
        const uint64_t mask = __ballot(hit);
        if (hit) list[n + __popcll(mask & ((1ull << lane) - 1))] = p0 + lane;
        n += __popcll(mask);
    }
    return n;
}

// One block for a batch of more than kRouteInUp tokens: the choices, one wave
// per token at a time, and the lists, one wave per reached expert.
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const double *__restrict__ logits, int T, int E,
                                                                  int top_k, int renorm, int32_t *__restrict__ idx,
                                                                  float *__restrict__ gate, MoeLists lists) {
    __shared__ int32_t idx_s[kMaxPairs];
    __shared__ uint32_t bits[SVDQ_FP8_MOE_MAX_EXPERTS / 32];
    constexpr int kWaves = kRouteThreads / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int pairs = T * top_k;
    if (threadIdx.x < SVDQ_FP8_MOE_MAX_EXPERTS / 32) bits[threadIdx.x] = 0u;
    for (int t = wave; t < T; t += kWaves)
        choose(logits + (size_t)t * E, E, top_k, renorm, lane, idx_s + t * top_k, gate + t * top_k);
    __syncthreads();
    if ((int)threadIdx.x < pairs) {
        const int e = idx_s[threadIdx.x];
        idx[threadIdx.x] = e;
        atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    static_assert(kMaxPairs <= kRouteThreads, "a thread per pair");
    int reached;
    reached_expert(bits, 0, reached);
    for (int a = wave; a < reached; a += kWaves) {
        int n;
        const int e = reached_expert(bits, a, n);
        n = collect_pairs(idx_s, pairs, e, lane, lists.pairs + (size_t)a * T);
        if (lane == 0) {
            lists.experts[a] = e;
            lists.counts[a] = n;
        }
    }
    if (threadIdx.x == 0) *lists.reached = reached;
}

// ---- gate and up projections ------------------------------------------------

constexpr int kUpAhead = 4;  // groups of weights in flight per wave

// One block: the a-th reached expert, 16 intermediate columns of gate and up.
// The waves take the groups of H in turn, their weights straight from global
// memory into the operands of the bf16 MFMA (an E4M3 value is exact in bf16),
// and add their sums in LDS. h is written as the sum of two bf16 numbers (hi +
// lo, 16 significant bits), so that its rounding stays far below that of Y.
// kRoute: few tokens; every block makes the choices itself (one wave per
// token), which saves a launch, and the blocks of column tile 0 write the
// choices and lists down.
template <bool kRoute>
__global__ __launch_bounds__(kUpThreads) void moe_up_kernel(
    const uint16_t *__restrict__ X, const uint8_t *__restrict__ w13, const float *__restrict__ s13,
    const double *__restrict__ logits, int32_t *__restrict__ idx, float *__restrict__ gate, int T, int H, int I, int E,
    int top_k, int renorm, uint16_t *__restrict__ h_hi, uint16_t *__restrict__ h_lo, MoeLists lists) {
    __shared__ int32_t list[SVDQ_FP8_MOE_MAX_TOKENS];
    __shared__ f32x4 red[kUpWaves][2][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int a = blockIdx.y;
    const int i0 = blockIdx.x * 16;
    int e, count;
    if constexpr (kRoute) {
        __shared__ int32_t idx_s[kRouteInUp * SVDQ_FP8_MOE_MAX_TOP_K];
        __shared__ float gate_s[kRouteInUp * SVDQ_FP8_MOE_MAX_TOP_K];
        __shared__ uint32_t bits[SVDQ_FP8_MOE_MAX_EXPERTS / 32];
        const int pairs = T * top_k;
        if (threadIdx.x < SVDQ_FP8_MOE_MAX_EXPERTS / 32) bits[threadIdx.x] = 0u;
        if (wave < T)
            choose(logits + (size_t)wave * E, E, top_k, renorm, lane, idx_s + wave * top_k, gate_s + wave * top_k);
        __syncthreads();
        static_assert(kRouteInUp * SVDQ_FP8_MOE_MAX_TOP_K <= kUpThreads, "a thread per pair");
        if ((int)threadIdx.x < pairs) {
            const int ei = idx_s[threadIdx.x];
            atomicOr(&bits[ei >> 5], 1u << (ei & 31));
            if (blockIdx.x == 0 && a == 0) {
                idx[threadIdx.x] = ei;
                gate[threadIdx.x] = gate_s[threadIdx.x];
            }
        }
        __syncthreads();
        int reached;
        e = __builtin_amdgcn_readfirstlane(reached_expert(bits, a, reached));
        if (blockIdx.x == 0 && a == 0 && threadIdx.x == 0) *lists.reached = reached;
        if (e < 0) return;  // the same for every thread of the block
        // every wave writes the same list
        count = __builtin_amdgcn_readfirstlane(collect_pairs(idx_s, pairs, e, lane, list));
        if (blockIdx.x == 0 && wave == 0) {
            if (lane < count) lists.pairs[(size_t)a * T + lane] = list[lane];
            if (lane == 0) {
                lists.experts[a] = e;
                lists.counts[a] = count;
            }
        }
    } else {
        if (a >= *lists.reached) return;
        e = __builtin_amdgcn_readfirstlane(lists.experts[a]);
        count = __builtin_amdgcn_readfirstlane(lists.counts[a]);
        if ((int)threadIdx.x < count) list[threadIdx.x] = lists.pairs[(size_t)a * T + threadIdx.x];
    }
    __syncthreads();
    const int r16 = lane & 15, q4 = lane >> 4;
    const int G = (H + kF8Block - 1) / kF8Block, gi = (I + kF8Block - 1) / kF8Block;
    const uint8_t *we = w13 + (size_t)e * 2 * I * H;
    const __amdgpu_buffer_rsrc_t rg = fp8_rsrc(we + (size_t)i0 * H, 16u * (uint32_t)H);
    const __amdgpu_buffer_rsrc_t ru = fp8_rsrc(we + (size_t)(I + i0) * H, 16u * (uint32_t)H);
    const float *sg = s13 + ((size_t)e * 2 * gi + i0 / kF8Block) * G;
    const float *su = sg + (size_t)gi * G;
    const uint32_t row = (uint32_t)r16 * (uint32_t)H;
    for (int m0 = 0; m0 < count; m0 += 16) {
        const uint16_t *x = X + (size_t)(list[min(m0 + r16, count - 1)] / top_k) * H;
        f32x4 accg = {0.f, 0.f, 0.f, 0.f}, accu = accg;
        for (int g0 = wave; g0 < G; g0 += kUpWaves * kUpAhead) {
            u32x4 cg[kUpAhead][2], cu[kUpAhead][2];
#pragma unroll
            for (int n = 0; n < kUpAhead; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = (g0 + n * kUpWaves) * kF8Block + 64 * i + 16 * q4;
                    const uint32_t off = k < H ? row + (uint32_t)k : kMoeOob;  // zeros past H
                    cg[n][i] = load16(rg, off);
                    cu[n][i] = load16(ru, off);
                }
#pragma unroll
            for (int n = 0; n < kUpAhead; ++n) {
                const int g = g0 + n * kUpWaves;
                if (g >= G) break;
                f32x4 pg = {0.f, 0.f, 0.f, 0.f}, pu = pg;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = g * kF8Block + 64 * i + 16 * q4;
                    u32x4 x0 = {0u, 0u, 0u, 0u}, x1 = x0;
                    if (k < H) {
                        x0 = *reinterpret_cast<const u32x4 *>(x + k);
                        x1 = *reinterpret_cast<const u32x4 *>(x + k + 8);
                    }
                    const bf16x8 b0 = __builtin_bit_cast(bf16x8, x0), b1 = __builtin_bit_cast(bf16x8, x1);
                    pg = mfma_bf16_16x16x32(fp8_widen8(cg[n][i][0], cg[n][i][1]), b0, pg);
                    pu = mfma_bf16_16x16x32(fp8_widen8(cu[n][i][0], cu[n][i][1]), b0, pu);
                    pg = mfma_bf16_16x16x32(fp8_widen8(cg[n][i][2], cg[n][i][3]), b1, pg);
                    pu = mfma_bf16_16x16x32(fp8_widen8(cu[n][i][2], cu[n][i][3]), b1, pu);
                }
                const float wg = sg[g], wu = su[g];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    accg[i] = __builtin_fmaf(wg, pg[i], accg[i]);
                    accu[i] = __builtin_fmaf(wu, pu[i], accu[i]);
                }
            }
        }
        if (m0) __syncthreads();  // the sums of the tokens before have been read
        red[wave][0][lane] = accg;
        red[wave][1][lane] = accu;
        __syncthreads();
        if (threadIdx.x < 256) {
            const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
            const int src = 16 * (c >> 2) + m;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kUpWaves; ++w) {
                g += red[w][0][src][c & 3];
                u += red[w][1][src][c & 3];
            }
            if (m0 + m < count) {
                const float h = g / (1.0f + expf(-g)) * u;
                const uint32_t hi = f32_to_bf16_bits(h);
                const size_t at = (size_t)list[m0 + m] * I + i0 + c;
                h_hi[at] = (uint16_t)hi;
                // no remainder of an infinity or NaN
                h_lo[at] = (hi & 0x7F80u) == 0x7F80u ? 0 : (uint16_t)f32_to_bf16_bits(h - bf16_bits_to_f32(hi));
            }
        }
    }
}

// ---- down projection and weighted sum ----------------------------------------

constexpr int kDownAhead = 4;  // groups of weights in flight per wave

// One block: 16 output columns of every token. A wave takes one reached expert
// and one of `splits` shares of I at a time, reads its 16 weight rows once and
// leaves each pair's 16 sums in LDS at its own place; then each output is the
// weighted sum over its token's pairs in order, so the result does not depend
// on which wave came first.
__global__ __launch_bounds__(kDownThreads) void moe_down_kernel(
    const uint8_t *__restrict__ w2, const float *__restrict__ s2, const uint16_t *__restrict__ h_hi,
    const uint16_t *__restrict__ h_lo, const float *__restrict__ gate, MoeLists lists, int T, int H, int I,
    int top_k, int splits, uint16_t *__restrict__ Y) {
    extern __shared__ __align__(16) float out[];  // [splits][T top_k][16]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q4 = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int pairs = T * top_k;
    const int G = (I + kF8Block - 1) / kF8Block, gh = (H + kF8Block - 1) / kF8Block;
    const uint32_t row = (uint32_t)r16 * (uint32_t)I;
    const int units = *lists.reached * splits;
    for (int unit = wave; unit < units; unit += kDownWaves) {
        const int a = unit / splits, s = unit % splits;
        const int e = __builtin_amdgcn_readfirstlane(lists.experts[a]);
        const int count = __builtin_amdgcn_readfirstlane(lists.counts[a]);
        const __amdgpu_buffer_rsrc_t rw = fp8_rsrc(w2 + ((size_t)e * H + n0) * I, 16u * (uint32_t)I);
        const float *sw = s2 + ((size_t)e * gh + n0 / kF8Block) * G;
        for (int m0 = 0; m0 < count; m0 += 16) {
            const int pair = lists.pairs[(size_t)a * T + min(m0 + r16, count - 1)];
            const uint16_t *hh = h_hi + (size_t)pair * I, *hl = h_lo + (size_t)pair * I;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            for (int g0 = s; g0 < G; g0 += splits * kDownAhead) {
                u32x4 c[kDownAhead][2];
#pragma unroll
                for (int n = 0; n < kDownAhead; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = (g0 + n * splits) * kF8Block + 64 * i + 16 * q4;
                        c[n][i] = load16(rw, k < I ? row + (uint32_t)k : kMoeOob);  // zeros past I
                    }
#pragma unroll
                for (int n = 0; n < kDownAhead; ++n) {
                    const int g = g0 + n * splits;
                    if (g >= G) break;
                    f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = g * kF8Block + 64 * i + 16 * q4;
                        u32x4 x0 = {0u, 0u, 0u, 0u}, x1 = x0, y0 = x0, y1 = x0;
                        if (k < I) {
                            x0 = *reinterpret_cast<const u32x4 *>(hh + k);
                            x1 = *reinterpret_cast<const u32x4 *>(hh + k + 8);
                            y0 = *reinterpret_cast<const u32x4 *>(hl + k);
                            y1 = *reinterpret_cast<const u32x4 *>(hl + k + 8);
                        }
                        const bf16x8 a0 = fp8_widen8(c[n][i][0], c[n][i][1]), a1 = fp8_widen8(c[n][i][2], c[n][i][3]);
                        p = mfma_bf16_16x16x32(a0, __builtin_bit_cast(bf16x8, y0), p);
                        p = mfma_bf16_16x16x32(a1, __builtin_bit_cast(bf16x8, y1), p);
                        p = mfma_bf16_16x16x32(a0, __builtin_bit_cast(bf16x8, x0), p);
                        p = mfma_bf16_16x16x32(a1, __builtin_bit_cast(bf16x8, x1), p);
                    }
                    const float w = sw[g];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(w, p[i], acc[i]);
                }
            }
            if (m0 + r16 < count)
                *reinterpret_cast<f32x4 *>(out + ((size_t)s * pairs + pair) * 16 + 4 * q4) = acc;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * 16; i += kDownThreads) {
        const int t = i >> 4, c = i & 15;
        float y = 0.0f;
        for (int j = 0; j < top_k; ++j) {
            float o = 0.0f;
            for (int s = 0; s < splits; ++s) o += out[((size_t)s * pairs + t * top_k + j) * 16 + c];
            y = __builtin_fmaf(gate[t * top_k + j], o, y);
        }
        Y[(size_t)t * H + n0 + c] = (uint16_t)f32_to_bf16_bits(y);
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: h (hi, lo planes of [pairs][I]), the logits, the reached experts'
// lists, and room for the choices and weights of a call that does not ask for
// them.
struct Layout {
    size_t h_lo, logits, lists, idx, gate, bytes;
    Layout(int T, int I, int E, int top_k) {
        const size_t pairs = (size_t)T * top_k, lists_n = std::min((size_t)E, pairs);
        h_lo = align256(pairs * I * 2);
        logits = 2 * h_lo;
        lists = logits + align256((size_t)T * E * 8);
        idx = lists + align256(4 * (lists_n * (2 + (size_t)T) + 1));
        gate = idx + align256(4 * pairs);
        bytes = gate + align256(4 * pairs);
    }
};

}  // namespace

size_t fp8_moe_workspace_size(int T, int I, int E, int top_k) { return Layout(T, I, E, top_k).bytes; }

hipError_t launch_fp8_moe(const uint16_t *X, const uint16_t *wr, const uint8_t *w13, const float *s13,
                          const uint8_t *w2, const float *s2, int T, int H, int I, int E, int top_k, bool renorm,
                          int32_t *idx, float *gate, void *workspace, uint16_t *Y, hipStream_t stream) {
    const Layout at(T, I, E, top_k);
    const int pairs = T * top_k, lists_n = std::min(E, pairs);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint16_t *h_hi = reinterpret_cast<uint16_t *>(ws), *h_lo = reinterpret_cast<uint16_t *>(ws + at.h_lo);
    double *logits = reinterpret_cast<double *>(ws + at.logits);
    int32_t *l = reinterpret_cast<int32_t *>(ws + at.lists);
    const MoeLists lists{l, l + 1, l + 1 + lists_n, l + 1 + 2 * lists_n};
    if (!idx) idx = reinterpret_cast<int32_t *>(ws + at.idx);
    if (!gate) gate = reinterpret_cast<float *>(ws + at.gate);

    const int eb = (E + kLogitExperts - 1) / kLogitExperts;
    if (T == 1)
        hipLaunchKernelGGL(moe_logits_kernel<1>, dim3(eb), dim3(64 * kLogitWaves), 0, stream, X, wr, T, H, E, logits);
    else
        hipLaunchKernelGGL(moe_logits_kernel<4>, dim3(eb, (T + 3) / 4), dim3(64 * kLogitWaves), 0, stream, X, wr, T, H,
                           E, logits);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 up(I / 16, lists_n);
    if (T <= kRouteInUp) {
        hipLaunchKernelGGL(moe_up_kernel<true>, up, dim3(kUpThreads), 0, stream, X, w13, s13, logits, idx, gate, T, H,
                           I, E, top_k, renorm ? 1 : 0, h_hi, h_lo, lists);
    } else {
        hipLaunchKernelGGL(moe_route_kernel, dim3(1), dim3(kRouteThreads), 0, stream, logits, T, E, top_k,
                           renorm ? 1 : 0, idx, gate, lists);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL(moe_up_kernel<false>, up, dim3(kUpThreads), 0, stream, X, w13, s13, logits, idx, gate, T,
                           H, I, E, top_k, renorm ? 1 : 0, h_hi, h_lo, lists);
    }
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    // as many shares of I as give every wave a unit, at most one per group and
    // what 32 KB of LDS hold
    const int G = fp8_blocks(I);
    int splits = std::min((kDownWaves + lists_n - 1) / lists_n, G);
    while (splits > 1 && splits * pairs * 64 > (32 << 10)) --splits;
    hipLaunchKernelGGL(moe_down_kernel, dim3(H / 16), dim3(kDownThreads), (size_t)splits * pairs * 64, stream, w2, s2,
                       h_hi, h_lo, gate, lists, T, H, I, top_k, splits, Y);
    return hipGetLastError();
}

}  // namespace svdq
