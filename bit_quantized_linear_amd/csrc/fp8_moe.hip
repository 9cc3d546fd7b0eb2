// A mixture-of-experts layer for a few tokens on block-scaled FP8 weights,
// bf16 activations.
//
//   l[t, e] = sum_h X[t, h] Wr[e, h]                 (router logits, fp64 sums)
//   the top_k largest of a token, ties to the lowest expert; w[t, j] their
//   softmax weights (over all experts, or over the chosen ones)
//   h[t, j] = silu(X[t] Wg) * (X[t] Wu) of expert e = idx[t, j]
//   Y[t]    = sum_j w[t, j] (h[t, j] Wd), rounded once to bf16
//
// Launches: the router's logits; the choices (where the up kernel's blocks do
// not make them themselves); the gate and up projections, at most 256 blocks that
// take items of a reached expert and 16 intermediate columns in turn; the down
// projection with the weighted sum, one block per 16 or 8 output columns. A reached
// expert's weights are read once for 4 to 16 of its tokens, so with few tokens each
// the layer is bound by HBM: 64 tokens of 128 experts (H 4096, I 1408, 8 choices)
// take 440 us, 5.0 TB/s over all launches; for few bytes by the chain of
// dependent loads: a token's logits, its choice, the experts' weights, then h and
// again weights, in three launches about 1.1 us apart (1 token, H 2048, I 768, 8 of
// 64 experts: 20.5 us, of which the weights alone would take 7.5).

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
constexpr int kMaxPairs = SVDQ_FP8_MOE_MAX_TOKENS * SVDQ_FP8_MOE_MAX_TOP_K;
constexpr uint32_t kMoeOob = 0x80000000u;

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// ---- router logits -----------------------------------------------------------

constexpr int kLogitWaves = 4;
constexpr int kLogitExperts = 2;  // per block

// One block: 2 experts x TB tokens; its waves take steps of 512 features in
// turn, 8 a lane. bf16 values are widened to fp64 and multiplied and added
// there, so that the order of two logits is the exact one up to 2^-50. The
// lanes' sums are folded so that each step halves the sums a lane holds, the
// waves' added in LDS in order. Bound by the fp64 arithmetic and its conversions
// for many tokens (64 x 4096 x 128: 8.4 us; 4 tokens share a weight's), by
// latency for one (1 x 2048 x 64: 2.8 us).
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
#pragma unroll 2
    for (int h = (wave * 64 + lane) * 8; h < H; h += 512 * kLogitWaves) {
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
    // fold: lanes with bit 32 / n of the number of sums left keep the upper half
#pragma unroll
    for (int step = 0; step < 6; ++step) {
        const int n = kSums >> step, d = 32 >> step;
        if (n > 1) {
            const bool up = lane & d;
#pragma unroll
            for (int i = 0; i < n / 2; ++i) {
                const double give = up ? sum[i] : sum[i + n / 2], keep = up ? sum[i + n / 2] : sum[i];
                sum[i] = keep + __shfl_xor(give, d);
            }
        } else {
            sum[0] += __shfl_xor(sum[0], d);
        }
    }
    constexpr int kLanes = 64 / kSums;  // lanes that hold the same sum
    if (lane % kLanes == 0) part[wave][lane / kLanes] = sum[0];
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

// NaN and -inf order below every number, alike.
__device__ __forceinline__ double order_key(double l) { return l > -__builtin_inf() ? l : -__builtin_inf(); }

// How many of the experts part, part + kParts, ... come before expert e: with a
// larger logit, or the same and a lower number. The sum over the parts is e's
// place, a permutation, so the first top_k places are the choice, in order,
// with no rounds that wait for each other.
constexpr int kParts = 4;
__device__ __forceinline__ int place(const double *key, int E, int e, int part) {
    const double mine = key[e];
    int before = 0;
#pragma unroll 4
    for (int o = part; o < E; o += kParts) {
        const double v = key[o];
        before += v > mine || (v == mine && o < e) ? 1 : 0;
    }
    return before;
}

// Weight numerators of a token's choices, in fp32: exp(l - largest l).
__device__ __forceinline__ float numerator(double l, double top) { return expf((float)(l - top)); }

// All experts' numerators (lane l takes experts l, l + 64, ...; then a fold).
__device__ __forceinline__ float all_numerators(const double *logit, double top, int E, int lane) {
    float sum = 0.0f;
    for (int o = lane; o < E; o += 64) sum += numerator(logit[o], top);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    return sum;
}

// The choices of `tokens` tokens by one block, kParts threads per token and
// expert at a time: first [tokens][top_k], in LDS like logit and key
// [tokens][E]. The block is in step afterwards.
__device__ __forceinline__ void choose(const double *__restrict__ logits, int tokens, int E, int top_k, int threads,
                                       double *logit, double *key, int32_t *first) {
    for (int i = threadIdx.x; i < tokens * E; i += threads) {
        logit[i] = logits[i];
        key[i] = order_key(logit[i]);
    }
    __syncthreads();
    const int items = tokens * E;
    for (int i0 = 0; i0 < items; i0 += threads / kParts) {
        const int i = i0 + (int)threadIdx.x / kParts;
        const int t = min(i, items - 1) / E, e = min(i, items - 1) % E;
        int j = place(key + t * E, E, e, threadIdx.x % kParts);
#pragma unroll
        for (int d = 1; d < kParts; d <<= 1) j += __shfl_xor(j, d);
        if (i < items && j < top_k && threadIdx.x % kParts == 0) first[t * top_k + j] = e;
    }
    __syncthreads();
}

// The choices and their weights to idx and gate, a wave per token. The weights'
// denominator is the sum of the chosen numerators in order, or of all.
__device__ __forceinline__ void write_choices(const double *logit, const int32_t *first, int tokens, int E, int top_k,
                                              bool renorm, int threads, int32_t *idx, float *gate) {
    const int lane = threadIdx.x & 63;
    for (int t = threadIdx.x >> 6; t < tokens; t += threads / 64) {
        const double *l = logit + t * E;
        const int32_t *f = first + t * top_k;
        const double top = l[f[0]];
        float total = 0.0f;
        if (renorm)
            for (int j = 0; j < top_k; ++j) total += numerator(l[f[j]], top);
        else
            total = all_numerators(l, top, E, lane);
        if (lane < top_k) {
            idx[t * top_k + lane] = f[lane];
            gate[t * top_k + lane] = numerator(l[f[lane]], top) / total;
        }
    }
}

constexpr int kRouteThreads = kParts * SVDQ_FP8_MOE_MAX_EXPERTS;

// One block per token. Latency: 4.7 us for 128 experts, 3.6 for 40.
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const double *__restrict__ logits, int E, int top_k,
                                                                  int renorm, int32_t *__restrict__ idx,
                                                                  float *__restrict__ gate) {
    __shared__ double logit[SVDQ_FP8_MOE_MAX_EXPERTS], key[SVDQ_FP8_MOE_MAX_EXPERTS];
    __shared__ int32_t first[SVDQ_FP8_MOE_MAX_TOP_K];
    const int t = blockIdx.x;
    choose(logits + (size_t)t * E, 1, E, top_k, kRouteThreads, logit, key, first);
    write_choices(logit, first, 1, E, top_k, renorm, kRouteThreads, idx + (size_t)t * top_k, gate + (size_t)t * top_k);
}

// Up to this many (token, expert) pairs the up kernel's blocks make the choices
// themselves. A layer, H 2048, I 768, with the choice in the up kernel / by
// itself: 1 token of 64 experts 20.9 / 22.8 us, 16 of 16 29.9 / 30.5, 4 of 64 46.2
// / 47.7; 4 of 128 52.1 / 50.7 and 64 of 8 39.3 / 37.9, as every block does all
// the comparisons.
constexpr int kRouteInUp = 256;

// ---- the reached experts ---------------------------------------------------------

// The reached experts (ascending; a single token's in the order of its choices)
// and the pairs t top_k + j sorted by expert, then token: reached expert number
// a has pairs pair[from[a]] .. pair[from[a + 1] - 1], each as token << 10 | pair
// (a division in place of it costs as much as a load). Written down for the
// down projection as it is.
struct MoeTable {
    int32_t reached;
    uint16_t expert[SVDQ_FP8_MOE_MAX_EXPERTS];
    uint16_t from[SVDQ_FP8_MOE_MAX_EXPERTS + 2];
    uint16_t pair[kMaxPairs];
};
static_assert(sizeof(MoeTable) % 4 == 0, "copied in dwords");
static_assert(kMaxPairs <= 1 << 10 && SVDQ_FP8_MOE_MAX_TOKENS <= 1 << 6, "both in 16 bits");
__device__ __forceinline__ uint32_t pair_of(uint16_t v) { return v & 1023u; }
__device__ __forceinline__ uint32_t token_of(uint16_t v) { return v >> 10; }

// Built by a whole block from the choices. tokens: [256] of LDS, the set of an
// expert's tokens as a bit each; an expert is at most once among a token's
// choices, so a pair's place is the number of its expert's earlier tokens.
__device__ __forceinline__ void build_table(const int32_t *idx, int T, int E, int top_k, int threads,
                                            unsigned long long *tokens, MoeTable &table) {
    static_assert(SVDQ_FP8_MOE_MAX_TOKENS <= 64, "a bit per token");
    const int lane = threadIdx.x & 63;
    if (T == 1) {  // each choice another expert: any order does
        for (int j = threadIdx.x; j <= top_k; j += threads) {
            if (j < top_k) table.expert[j] = (uint16_t)min((unsigned)idx[j], (unsigned)E - 1);
            table.from[j] = table.pair[j] = (uint16_t)j;
        }
        if (threadIdx.x == 0) table.reached = top_k;
        __syncthreads();
        return;
    }
    for (int e = threadIdx.x; e < SVDQ_FP8_MOE_MAX_EXPERTS; e += threads) tokens[e] = 0;
    __syncthreads();
    // the choices are in range; where a caller's other work writes the buffer
    // meanwhile, the clamp and the bounded search below keep every access and
    // loop inside the table
    auto choice = [&](int p) { return min((unsigned)idx[p], (unsigned)E - 1); };
    for (int p = threadIdx.x; p < T * top_k; p += threads) atomicOr(&tokens[choice(p)], 1ull << (p / top_k));
    __syncthreads();
    if (threadIdx.x < 64) {
        int reached = 0, start = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int n = __popcll(tokens[e0 + lane]);
            int sum = n;  // of the experts up to this one
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(sum, d);
                if (lane >= d) sum += o;
            }
            const uint64_t hit = __ballot(n > 0);
            if (n > 0) {
                const int a = reached + __popcll(hit & ((1ull << lane) - 1));
                table.expert[a] = (uint16_t)(e0 + lane);
                table.from[a] = (uint16_t)(start + sum - n);
            }
            reached += __popcll(hit);
            start += __shfl(sum, 63);
        }
        if (lane == 0) {
            table.from[reached] = (uint16_t)start;
            table.reached = reached;
        }
    }
    __syncthreads();
    // a thread per reached expert and token
    for (int i = threadIdx.x; i < table.reached * T; i += threads) {
        const int a = i / T, t = i % T, e = table.expert[a];
        const uint64_t set = tokens[e];
        if (set >> t & 1) {
            int j = 0;
            while (j < top_k - 1 && (int)choice(t * top_k + j) != e) ++j;
            table.pair[table.from[a] + __popcll(set & ((1ull << t) - 1))] = (uint16_t)(t << 10 | (t * top_k + j));
        }
    }
    __syncthreads();
}

// ---- rows of activations through LDS -----------------------------------------------

// The activations of a few tokens reach the MFMA through LDS: 4 tokens' 128
// features are one 1 KB load (a slot), where loads straight into the operand
// registers take four, mostly of lanes without a token. (Per load the address
// unit spends 16 cycles whatever its lanes hold: with 4 tokens per expert the
// straight loads cost both projections as much as the weights they meet.) Lane l
// brings the 16-byte chunk c of token l / 16 to chunk position c ^ 4 (l / 16),
// so that the four tokens' equal chunks are on different banks.
typedef __attribute__((address_space(3))) void moe_lds_void;
constexpr int kSlot = 1024;

__device__ __forceinline__ uint32_t slot_chunk(int lane) { return ((lane & 15) ^ (4 * (lane >> 4))) * 16; }

__device__ __forceinline__ void load_slot(__amdgpu_buffer_rsrc_t r, uint8_t *slot, uint32_t row, int k, int K,
                                          uint32_t chunk) {
    const int at = 2 * k + (int)chunk;  // bytes into the row; zeros past its end
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (moe_lds_void *)slot, 16, at < 2 * K ? row + (uint32_t)at : kMoeOob, 0,
                                             0, 0);
}

// Chunk c (of 16) of the lane's token (slots one after another, 4 tokens each).
__device__ __forceinline__ bf16x8 slot_read(const uint8_t *slots, int token, int c) {
    return *reinterpret_cast<const bf16x8 *>(slots + token * 256 + ((c ^ (4 * (token & 3))) * 16));
}

// Slots per group for at most 8 tokens.
__device__ __forceinline__ int slots_of(int tokens) { return tokens <= 4 ? 1 : 2; }

// ---- gate and up projections ------------------------------------------------

constexpr int kUpBlocks = 256;  // one per compute unit
constexpr int kUpRing = 3;      // steps under way per wave

// Blocks take items in turn: a reached expert and 16 intermediate columns of
// gate and up. The waves share H, a group each per step, and add their sums in
// LDS at an item's end. Weights and activations go straight from global memory
// into the operands of the bf16 MFMA (an E4M3 value is exact in bf16), kUpRing
// steps ahead of their use and across items, so that loads are under way all
// the time; the activations of few tokens come through kSlots slots of LDS,
// 4 kSlots tokens at a time (0: straight, 16 at a time). h is written as the sum of two bf16 numbers (hi + lo, 16
// significant bits), so that its rounding stays far below that of Y. kRoute:
// every block also makes the choices, which saves a launch. Block 0 writes the
// table down for the down projection. HBM-bound: 64 tokens, H 4096, I 1408, 128
// experts 265 us (1.48 GB, 5.6 TB/s). The address and data units are busy 73 and
// 90 % of that; 4 steps ahead gain 1 % there and lose 4 % for 23 tokens.
template <bool kRoute, int kSlots>
__global__ __launch_bounds__(kUpThreads) void moe_up_kernel(
    const uint16_t *__restrict__ X, const uint8_t *__restrict__ w13, const float *__restrict__ s13,
    const double *__restrict__ logits, int32_t *__restrict__ idx, float *__restrict__ gate, int T, int H, int I, int E,
    int top_k, int renorm, uint16_t *__restrict__ h_hi, uint16_t *__restrict__ h_lo, MoeTable *__restrict__ table_out) {
    constexpr int kTokens = kSlots ? 4 * kSlots : 16;  // of an expert at a time
    constexpr int kSlotBytes = kSlots ? kUpWaves * kSlots * kSlot : 16;
    // an array per place in the ring, so that a read waits for no other's loads
    __shared__ __align__(16) uint8_t slots0[kSlotBytes], slots1[kSlotBytes], slots2[kSlotBytes];
    static_assert(kUpRing == 3, "slots");
    __shared__ f32x4 red[2][kUpWaves][2][64];
    __shared__ unsigned long long tokens[SVDQ_FP8_MOE_MAX_EXPERTS];
    __shared__ MoeTable table;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q4 = lane >> 4;
    if constexpr (kRoute) {
        __shared__ double logit[kRouteInUp], key[kRouteInUp];
        __shared__ int32_t first[kRouteInUp];
        choose(logits, T, E, top_k, kUpThreads, logit, key, first);
        if (blockIdx.x == 0) write_choices(logit, first, T, E, top_k, renorm, kUpThreads, idx, gate);
        build_table(first, T, E, top_k, kUpThreads, tokens, table);
    } else {
        build_table(idx, T, E, top_k, kUpThreads, tokens, table);
    }
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < (int)sizeof(MoeTable) / 4; i += kUpThreads)
            reinterpret_cast<uint32_t *>(table_out)[i] = reinterpret_cast<const uint32_t *>(&table)[i];

    const int G = (H + kF8Block - 1) / kF8Block, gi = (I + kF8Block - 1) / kF8Block;
    const int tiles = I / 16, steps = (G + kUpWaves - 1) / kUpWaves;
    const int items = __builtin_amdgcn_readfirstlane(table.reached) * tiles;
    const __amdgpu_buffer_rsrc_t rx = fp8_rsrc(X, (uint32_t)T * (uint32_t)H * 2u);

    // A place in a wave's work: step `step` of the item for its tokens m0 ...
    // (all waves of a block take the same number of steps; past H they load
    // zeros).
    struct Place {
        int item, m0, step;
        int a, i0, e, from, count;  // a: the reached expert's number
    };
    const int next_a = (int)gridDim.x / tiles, next_i0 = (int)gridDim.x % tiles * 16;
    auto enter = [&](Place &p) __attribute__((always_inline)) {
        p.m0 = p.step = 0;
        const int a = min(p.a, table.reached - 1);
        p.e = __builtin_amdgcn_readfirstlane(table.expert[a]);
        p.from = __builtin_amdgcn_readfirstlane(table.from[a]);
        p.count = __builtin_amdgcn_readfirstlane(table.from[a + 1]) - p.from;
    };
    // Where rows are a multiple of 4 KB apart, the same group of all rows lies on a
    // few memory channels, so each tile starts at another group (G is then a multiple
    // of 32, and of a step). A layer for 64 tokens, H 4096, I 2048, 4 of 64 experts:
    // 314 us, 330 without.
    const int spread = H % 4096 ? 0 : (1 << (31 - __builtin_clz(G))) - 1;
    auto group_of = [&](const Place &p) __attribute__((always_inline)) {
        const int g = p.step * kUpWaves + wave, turned = g + ((p.i0 >> 4) & spread);
        return spread && turned >= G ? turned - G : turned;
    };
    auto advance = [&](Place &p) __attribute__((always_inline)) {
        if (++p.step < steps) return;
        p.step = 0;
        p.m0 += kTokens;
        if (p.m0 < p.count) return;
        p.item += (int)gridDim.x;
        p.a += next_a;
        p.i0 += next_i0;
        if (p.i0 >= I) {
            p.i0 -= I;
            ++p.a;
        }
        enter(p);
    };
    struct Step {
        u32x4 g[2], u[2], x[kSlots ? 1 : 2][2];
    };
    // the operands of place p's step, and on to the next place
    const uint32_t chunk = slot_chunk(lane);
    uint32_t xrow[kSlots ? kSlots : 1] = {};
    auto load = [&](Step &to, uint8_t *slots, Place &p) __attribute__((always_inline)) {
        const uint8_t *we = w13 + (size_t)p.e * 2 * I * H;
        const __amdgpu_buffer_rsrc_t rg = fp8_rsrc(we + (size_t)p.i0 * H, 16u * (uint32_t)H);
        const __amdgpu_buffer_rsrc_t ru = fp8_rsrc(we + (size_t)(I + p.i0) * H, 16u * (uint32_t)H);
        if (p.step == 0) {  // the lane's token, as a byte offset; lanes without one read zeros
            if constexpr (kSlots == 0)
                xrow[0] = p.m0 + r16 < p.count ? token_of(table.pair[p.from + p.m0 + r16]) * (uint32_t)H * 2u : kMoeOob;
            else
#pragma unroll
                for (int q = 0; q < kSlots; ++q)
                    xrow[q] = token_of(table.pair[p.from + min(p.m0 + 4 * q + q4, p.count - 1)]) * (uint32_t)H * 2u;
        }
        if constexpr (kSlots > 0) {
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): what the slots held has been read
            const int kx = p.item < items ? group_of(p) * kF8Block : H;
#pragma unroll
            for (int q = 0; q < kSlots; ++q) load_slot(rx, slots + (wave * kSlots + q) * kSlot, xrow[q], kx, H, chunk);
        }
        const int k0 = group_of(p) * kF8Block + 16 * q4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = k0 + 64 * i;
            const bool in = k < H && p.item < items;
            const uint32_t off = in ? (uint32_t)r16 * (uint32_t)H + (uint32_t)k : kMoeOob;
            const uint32_t xoff = kSlots == 0 && in ? xrow[0] + 2u * (uint32_t)k : kMoeOob;
            to.g[i] = load16(rg, off);
            to.u[i] = load16(ru, off);
            if constexpr (kSlots == 0) {
                to.x[i][0] = load16(rx, xoff);
                to.x[i][1] = load16(rx, xoff + 16);
            }
        }
        advance(p);
    };
    f32x4 accg = {0.f, 0.f, 0.f, 0.f}, accu = accg;
    int turn = 0;
    // one step: its products; the sums and the output behind an item's last one
    auto compute = [&](const Step &now, const uint8_t *slots, Place &p) __attribute__((always_inline)) {
        if constexpr (kSlots > 0) {
            __builtin_amdgcn_sched_barrier(0);
            // the slots are there; the loads of the later steps may stay under way
            constexpr int kLater = (kUpRing - 1) * (kSlots + 4);
            static_assert(kLater < 16, "what the wait below can count");
            __builtin_amdgcn_s_waitcnt(0x0F70 | kLater);  // vmcnt(kLater)
            __builtin_amdgcn_sched_barrier(0);
        }
        const int g = group_of(p);
        const size_t block = ((size_t)p.e * 2 * gi + p.i0 / kF8Block) * G + min(g, G - 1);
        const float wg = fp8_scale_within(s13[block], g, G), wu = fp8_scale_within(s13[block + (size_t)gi * G], g, G);
        f32x4 pg = {0.f, 0.f, 0.f, 0.f}, pu = pg;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bf16x8 b0, b1;
            if constexpr (kSlots == 0) {
                b0 = __builtin_bit_cast(bf16x8, now.x[i][0]), b1 = __builtin_bit_cast(bf16x8, now.x[i][1]);
            } else {
                const int c = 8 * i + 2 * q4, token = r16 & (kTokens - 1);
                b0 = slot_read(slots + wave * kSlots * kSlot, token, c);
                b1 = slot_read(slots + wave * kSlots * kSlot, token, c + 1);
            }
            pg = mfma_bf16_16x16x32(fp8_widen8(now.g[i][0], now.g[i][1]), b0, pg);
            pu = mfma_bf16_16x16x32(fp8_widen8(now.u[i][0], now.u[i][1]), b0, pu);
            pg = mfma_bf16_16x16x32(fp8_widen8(now.g[i][2], now.g[i][3]), b1, pg);
            pu = mfma_bf16_16x16x32(fp8_widen8(now.u[i][2], now.u[i][3]), b1, pu);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            accg[i] = __builtin_fmaf(wg, pg[i], accg[i]);
            accu[i] = __builtin_fmaf(wu, pu[i], accu[i]);
        }
    };
    auto finish = [&](const Place &p) __attribute__((always_inline)) {
        // two sets of sums take turns: one barrier per item
        red[turn][wave][0][lane] = accg;
        red[turn][wave][1][lane] = accu;
        accg = accu = f32x4{0.f, 0.f, 0.f, 0.f};
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0); the loads stay under way
        fp8_barrier();
        if (threadIdx.x < 256) {
            const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
            const int src = 16 * (c >> 2) + m;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kUpWaves; ++w) {
                g += red[turn][w][0][src][c & 3];
                u += red[turn][w][1][src][c & 3];
            }
            if (m < kTokens && p.m0 + m < p.count) {
                const float h = g / (1.0f + expf(-g)) * u;
                uint32_t hi = f32_to_bf16_bits(h);
                // a finite h past the largest bf16 number takes that one, and lo the rest
                if ((hi & 0x7FFFu) == 0x7F80u && __builtin_isfinite(h)) --hi;
                const size_t at = (size_t)pair_of(table.pair[p.from + p.m0 + m]) * I + p.i0 + c;
                h_hi[at] = (uint16_t)hi;
                // no remainder of an infinity or NaN
                h_lo[at] = (hi & 0x7F80u) == 0x7F80u ? 0 : (uint16_t)f32_to_bf16_bits(h - bf16_bits_to_f32(hi));
            }
        }
        turn ^= 1;
    };
    Place at, ahead;
    at.item = blockIdx.x;
    at.a = (int)blockIdx.x / tiles;
    at.i0 = (int)blockIdx.x % tiles * 16;
    enter(at);
    ahead = at;
    Step ring[kUpRing];
    auto slots_at = [&](int n) -> uint8_t * { return n == 0 ? slots0 : n == 1 ? slots1 : slots2; };
#pragma unroll
    for (int n = 0; n < kUpRing; ++n) load(ring[n], slots_at(n), ahead);
    while (at.item < items) {
#pragma unroll
        for (int n = 0; n < kUpRing; ++n) {
            if (at.item >= items) break;
            compute(ring[n], slots_at(n), at);
            load(ring[n], slots_at(n), ahead);
            if (at.step == steps - 1) finish(at);
            advance(at);
        }
    }
}

// ---- down projection and weighted sum ----------------------------------------

constexpr int kDownAhead = 4;  // groups of weights per set; two sets take turns

// One block: kCols output columns of every token. A wave takes one reached expert
// and one of 2^shift shares of I at a time (a unit; all of a wave's are the same
// share), reads its weight rows once, a batch of groups ahead of their use,
// and leaves each pair's sums in LDS at their own place; then each output is the
// weighted sum over its token's pairs in order, so the result does not depend on
// which wave came first. 16 waves of 4 groups' weights each are the loads under
// way; the rows of h come through LDS (above), filling kDownSlots slots at a time,
// each a wait for memory (a batch's first leaves the next batch's weights under
// way, the others wait for those too): 4 slots where the sums leave them room (a
// layer for 8 tokens of 64 experts 98.7 us, with 2 slots 99.4). HBM-bound: 64
// tokens, H 4096, I 1408, 128 experts 158 us (0.74 GB, 4.7 TB/s).
// kCols 8: the MFMA's rows 8 .. 15 are the same columns in the unit's next group,
// and its columns 8 .. 15 the tokens there, so that two quadrants of the result
// hold the sums of a group each.
template <int kDownSlots, int kCols>
__global__ __launch_bounds__(kDownThreads) void moe_down_kernel(
    const uint8_t *__restrict__ w2, const float *__restrict__ s2, const uint16_t *__restrict__ h_hi,
    const uint16_t *__restrict__ h_lo, const float *__restrict__ gate, const MoeTable *__restrict__ table_in, int T,
    int H, int I, int top_k, int shift, uint16_t *__restrict__ Y) {
    __shared__ MoeTable table;
    __shared__ float gate_s[kMaxPairs];
    extern __shared__ __align__(16) uint8_t smem[];  // slots [waves][2][kDownSlots], then sums [splits][T top_k][kCols]
    float *out = reinterpret_cast<float *>(smem + kDownWaves * 2 * kDownSlots * kSlot);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t *slots = smem + wave * 2 * kDownSlots * kSlot;
    const int r16 = lane & 15, q4 = lane >> 4;
    constexpr int kHalves = 16 / kCols;           // groups per step
    constexpr int kTokens = kHalves == 1 ? 8 : 4;  // of an expert at a time
    const int half = r16 / kCols, col = r16 % kCols;  // of the operands
    const int half_out = 4 * q4 / kCols;              // of the result's rows 4 q4 ...
    const int n0 = blockIdx.x * kCols;
    const int pairs = T * top_k;
    const int G = (I + kF8Block - 1) / kF8Block, gh = (H + kF8Block - 1) / kF8Block;
    const __amdgpu_buffer_rsrc_t rh = fp8_rsrc(h_hi, (uint32_t)pairs * (uint32_t)I * 2u);
    const __amdgpu_buffer_rsrc_t rl = fp8_rsrc(h_lo, (uint32_t)pairs * (uint32_t)I * 2u);
    const uint32_t chunk = slot_chunk(lane);
    // the table, and the choices' weights to wait in a register for their use
    constexpr int kTableWords = sizeof(MoeTable) / 4;
    static_assert(kTableWords <= kDownThreads && kMaxPairs == kDownThreads, "one of each for a thread");
    const uint32_t word = reinterpret_cast<const uint32_t *>(table_in)[min((int)threadIdx.x, kTableWords - 1)];
    const float weight = gate[min((int)threadIdx.x, pairs - 1)];
    if (threadIdx.x < kTableWords) reinterpret_cast<uint32_t *>(&table)[threadIdx.x] = word;
    gate_s[threadIdx.x] = weight;
    __syncthreads();
    const int splits = 1 << shift, s = wave & (splits - 1);
    const int reached = __builtin_amdgcn_readfirstlane(table.reached);
    const int groups = (G - s + splits - 1) >> shift, all = (groups + kHalves - 1) / kHalves;  // and steps of a unit

    // where a wave is (a: the reached expert's number): batch `first` (of the unit's groups) for tokens m0 ...
    struct Place {
        int a, e, from, count, m0, first;
    };
    auto enter = [&](Place &p) __attribute__((always_inline)) {
        if (p.a < reached) {
            p.e = __builtin_amdgcn_readfirstlane(table.expert[p.a]);
            p.from = __builtin_amdgcn_readfirstlane(table.from[p.a]);
            p.count = __builtin_amdgcn_readfirstlane(table.from[p.a + 1]) - p.from;
        }
        p.m0 = p.first = 0;
    };
    auto advance = [&](Place &p) __attribute__((always_inline)) {
        p.first += kDownAhead;
        if (p.first < all) return;
        p.first = 0;
        p.m0 += kTokens;
        if (p.m0 < p.count) return;
        p.a += kDownWaves >> shift;
        enter(p);
    };
    auto load_weights = [&](u32x4(&to)[kDownAhead][2], const Place &p) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t rw = fp8_rsrc(w2 + ((size_t)p.e * H + n0) * I, (uint32_t)kCols * (uint32_t)I);
#pragma unroll
        for (int n = 0; n < kDownAhead; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = (s + (((p.first + n) * kHalves + half) << shift)) * kF8Block + 64 * i + 16 * q4;
                to[n][i] = load16(rw, k < I ? (uint32_t)col * (uint32_t)I + (uint32_t)k : kMoeOob);  // zeros past I
            }
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    // one batch from `now`, the next one's weights to `next`
    auto batch = [&](Place &p, const u32x4(&now)[kDownAhead][2], u32x4(&next)[kDownAhead][2])
                     __attribute__((always_inline)) {
        const int here = min(kTokens, p.count - p.m0), per = kHalves == 1 ? slots_of(here) : 1;
        const Place at = p;
        uint32_t row[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
            row[q] = pair_of(table.pair[at.from + at.m0 + min(4 * q + q4, here - 1)]) * (uint32_t)I * 2u;
        const float *sw = s2 + ((size_t)at.e * gh + n0 / kF8Block) * G;
        if (at.first == 0) acc = f32x4{0.f, 0.f, 0.f, 0.f};
        advance(p);
#pragma unroll
        for (int n = 0; n < kDownAhead; ++n) {
            if (n * kHalves * per % kDownSlots == 0) {  // the slots are empty: fill them, lo behind hi
                __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): what they held has been read
#pragma unroll
                for (int q = 0; q < kDownSlots; ++q) {
                    const int k = (s + (((at.first + n) * kHalves + (per == 1 ? q : q / 2)) << shift)) * kF8Block;
                    load_slot(rh, slots + q * kSlot, (q & 1) && per > 1 ? row[1] : row[0], k, I, chunk);
                    load_slot(rl, slots + (kDownSlots + q) * kSlot, (q & 1) && per > 1 ? row[1] : row[0], k, I, chunk);
                }
                // the slots are there; the next batch's 2 kDownAhead loads may stay under way
                __builtin_amdgcn_sched_barrier(0);
                if (n == 0 && p.a < reached) {
                    load_weights(next, p);
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_waitcnt(0x0F70 | 2 * kDownAhead);  // vmcnt(2 kDownAhead)
                } else {
                    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (at.first + n >= all) break;
            const uint8_t *hi = slots + (n * kHalves * per % kDownSlots + half) * kSlot, *lo = hi + kDownSlots * kSlot;
            const int token = r16 & (4 * per - 1);
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bf16x8 a0 = fp8_widen8(now[n][i][0], now[n][i][1]), a1 = fp8_widen8(now[n][i][2], now[n][i][3]);
                const int c = 8 * i + 2 * q4;
                sum = mfma_bf16_16x16x32(a0, slot_read(lo, token, c), sum);
                sum = mfma_bf16_16x16x32(a1, slot_read(lo, token, c + 1), sum);
                sum = mfma_bf16_16x16x32(a0, slot_read(hi, token, c), sum);
                sum = mfma_bf16_16x16x32(a1, slot_read(hi, token, c + 1), sum);
            }
            const int group = (at.first + n) * kHalves;
            float w = sw[s + (group << shift)];
            if constexpr (kHalves == 2) {  // the second half may be past the last group
                const float w1 = fp8_scale_within(sw[s + (min(group + 1, groups - 1) << shift)], group, groups - 1);
                w = half_out ? w1 : w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(w, sum[i], acc[i]);
        }
        if (at.first + kDownAhead >= all) {
            if constexpr (kHalves == 2)  // rows 0 .. 7 of columns 0 .. 7, and rows 8 .. 15 of columns 8 .. 15
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor(acc[i], 40);
            if (r16 < here && half_out == 0) {
                const uint32_t pair = pair_of(table.pair[at.from + at.m0 + r16]);
                *reinterpret_cast<f32x4 *>(out + ((size_t)s * pairs + pair) * kCols + 4 * q4) = acc;
            }
        }
    };
    Place p;
    p.a = wave >> shift;
    enter(p);
    u32x4 c0[kDownAhead][2], c1[kDownAhead][2];
    if (p.a < reached) load_weights(c0, p);
    while (p.a < reached) {
        batch(p, c0, c1);
        if (p.a >= reached) break;
        batch(p, c1, c0);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * kCols; i += kDownThreads) {
        const int t = i / kCols, c = i % kCols;
        float y = 0.0f;
        for (int j = 0; j < top_k; ++j) {
            float o = 0.0f;
            for (int s = 0; s < splits; ++s) o += out[((size_t)s * pairs + t * top_k + j) * kCols + c];
            y = __builtin_fmaf(gate_s[t * top_k + j], o, y);
        }
        Y[(size_t)t * H + n0 + c] = (uint16_t)f32_to_bf16_bits(y);
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: h (hi, lo planes of [pairs][I]), the logits, the table of
// reached experts, and room for the choices and weights of a call that does not ask for
// them.
struct Layout {
    size_t h_lo, logits, table, idx, gate, bytes;
    Layout(int T, int I, int E, int top_k) {
        const size_t pairs = (size_t)T * top_k;
        h_lo = align256(pairs * I * 2);
        logits = 2 * h_lo;
        table = logits + align256((size_t)T * E * 8);
        idx = table + align256(sizeof(MoeTable));
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
    const int pairs = T * top_k, most = std::min(E, pairs);  // most: experts reached at the most
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint16_t *h_hi = reinterpret_cast<uint16_t *>(ws), *h_lo = reinterpret_cast<uint16_t *>(ws + at.h_lo);
    double *logits = reinterpret_cast<double *>(ws + at.logits);
    MoeTable *table = reinterpret_cast<MoeTable *>(ws + at.table);
    if (!idx) idx = reinterpret_cast<int32_t *>(ws + at.idx);
    if (!gate) gate = reinterpret_cast<float *>(ws + at.gate);

    const int eb = (E + kLogitExperts - 1) / kLogitExperts;
    if (T == 1)  // one token of 64 experts: 20.9 us, 21.6 with the other
        hipLaunchKernelGGL(moe_logits_kernel<1>, dim3(eb), dim3(64 * kLogitWaves), 0, stream, X, wr, T, H, E, logits);
    else
        hipLaunchKernelGGL(moe_logits_kernel<4>, dim3(eb, (T + 3) / 4), dim3(64 * kLogitWaves), 0, stream, X, wr, T, H,
                           E, logits);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 up((unsigned)std::min<int64_t>((int64_t)most * (I / 16), kUpBlocks));
    const auto launch_up = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, up, dim3(kUpThreads), 0, stream, X, w13, s13, logits, idx, gate, T, H, I, E, top_k,
                           renorm ? 1 : 0, h_hi, h_lo, table);
        return hipGetLastError();
    };
    if (T * E <= kRouteInUp) {
        err = T <= 4 ? launch_up(moe_up_kernel<true, 1>) : launch_up(moe_up_kernel<true, 0>);
    } else {
        hipLaunchKernelGGL(moe_route_kernel, dim3(T), dim3(kRouteThreads), 0, stream, logits, E, top_k,
                           renorm ? 1 : 0, idx, gate);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
        // slots for as many tokens as an expert mostly has, as with more than they
        // hold its weights are read again. Layer, H 4096, I 1408, slots / straight,
        // at tokens x choices per expert: 4 (64 x 8 of 128) 446 / 451 us, 6 (48 x 8
        // of 64) 265 / 261, 8 317 / 294.
        err = T <= 4             ? launch_up(moe_up_kernel<false, 1>)
              : pairs <= 4 * E ? launch_up(moe_up_kernel<false, 2>)
                                 : launch_up(moe_up_kernel<false, 0>);
    }
    if (err != hipSuccess) return err;
    // 8 columns per block where 16 would leave half the compute units without one:
    // twice the blocks, if an expert has few tokens (4 at a time instead of 8) and the
    // groups of I fill the steps of two. A layer with 16 / 8 columns: H 2048, I 768, 32
    // x 4 of 64 experts 80.8 / 73.0 us, 64 x 6 of 64 110.7 / 105.6, H 448, I 720, 37 x 6 of 60
    // 56.3 / 52.5; 17 x 6 of 6 31.8 / 32.7; I 336, H 768, 53 x 3 of 118 47.0 / 49.9; H 4096, I
    // 1408, 8 x 4 of 64 97 / 109. As many shares of I as give every wave a unit, at most
    // one per step and what 32 KB of LDS hold.
    const int G = fp8_blocks(I);
    const int cols = H / 16 <= kUpBlocks / 2 && G > 4 && pairs <= 8 * E ? 8 : 16;
    const int steps = (G * cols + 15) / 16;
    int shift = 0;
    while (most << shift < kDownWaves && 2 << shift <= steps && (2 << shift) * pairs * cols * 4 <= (32 << 10)) ++shift;
    const size_t sums = (size_t)pairs * cols * 4 << shift;
    const int slots = sums <= (24 << 10) ? 4 : 2;  // in 160 KB, 7 of them the table and weights
    const size_t lds = (size_t)kDownWaves * 2 * slots * kSlot + sums;
    const auto down = cols == 8 ? slots == 4 ? moe_down_kernel<4, 8> : moe_down_kernel<2, 8>
                                : slots == 4 ? moe_down_kernel<4, 16> : moe_down_kernel<2, 16>;
    hipLaunchKernelGGL(down, dim3(H / cols), dim3(kDownThreads), lds, stream, w2, s2, h_hi, h_lo, gate, table,
                       T, H, I, top_k, shift, Y);
    return hipGetLastError();
}

}  // namespace svdq
