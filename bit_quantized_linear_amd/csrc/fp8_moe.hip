// A mixture-of-experts layer for a few tokens on block-scaled FP8 weights,
// bf16 activations.
//
//   l[t, e] = sum_h X[t, h] Wr[e, h]                 (router logits, fp64 sums)
//   the top_k largest of a token, ties to the lowest expert; w[t, j] their
//   softmax weights (over all experts, or over the chosen ones)
//   h[t, j] = silu(X[t] Wg) * (X[t] Wu) of expert e = idx[t, j]
//   Y[t]    = sum_j w[t, j] (h[t, j] Wd), rounded once to bf16
//
// Three launches: the router, one block per token; the gate and up
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

constexpr int kMoeThreads = 512;
constexpr int kMoeWaves = kMoeThreads / 64;
constexpr uint32_t kMoeOob = 0x80000000u;

// ---- router ----------------------------------------------------------------

// One block per token. A wave takes four experts at a time; products of two
// bf16 values are exact in fp32 and summed in fp64, so that the order of two
// experts' logits is the exact one up to 2^-50. NaN logits order below every
// number. The choice: top_k rounds of a wave-wide maximum over (logit, lowest
// index), each expert chosen at most once whatever its logit.
__global__ __launch_bounds__(kMoeThreads) void moe_router_kernel(const uint16_t *__restrict__ X,
                                                                 const uint16_t *__restrict__ wr, int H, int E,
                                                                 int top_k, int renorm, int32_t *__restrict__ idx,
                                                                 float *__restrict__ gate) {
    __shared__ double logit[SVDQ_FP8_MOE_MAX_EXPERTS];
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint16_t *x = X + (size_t)t * H;
    for (int e0 = wave * 4; e0 < E; e0 += kMoeWaves * 4) {
        double sum[4] = {0.0, 0.0, 0.0, 0.0};
        for (int h = lane * 8; h < H; h += 512) {
            const u32x4 xv = *reinterpret_cast<const u32x4 *>(x + h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4 wv = *reinterpret_cast<const u32x4 *>(wr + (size_t)min(e0 + i, E - 1) * H + h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[i] += (double)(__uint_as_float(xv[j] << 16) * __uint_as_float(wv[j] << 16));
                    sum[i] += (double)(__uint_as_float(xv[j] & 0xFFFF0000u) * __uint_as_float(wv[j] & 0xFFFF0000u));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum[i] += __shfl_xor(sum[i], d);
            if (lane == 0 && e0 + i < E) logit[e0 + i] = sum[i];
        }
    }
    __syncthreads();
    if (wave != 0) return;
    // lane l holds experts l, l + 64, ...
    constexpr int kPer = SVDQ_FP8_MOE_MAX_EXPERTS / 64;
    constexpr double kLowest = -1.7976931348623157e308;
    double v[kPer];
    bool open[kPer];
    double top = kLowest;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        open[i] = lane + 64 * i < E;
        v[i] = open[i] ? logit[lane + 64 * i] : kLowest;
        if (!(v[i] >= kLowest)) v[i] = kLowest;  // NaN, -inf
    }
    float chosen_sum = 0.0f, mine = 0.0f, total = 0.0f;
    int mine_e = 0;
    for (int j = 0; j < top_k; ++j) {
        double best = kLowest;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (open[i] && (at == 1 << 30 || v[i] > best)) {
                best = v[i];
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
        if (j == 0) top = logit[at];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (at == lane + 64 * i) open[i] = false;
        const float e = expf((float)(logit[at] - top));
        chosen_sum += e;
        if (lane == j) {
            mine = e;
            mine_e = at;
        }
    }
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 64 * i < E) total += expf((float)(logit[lane + 64 * i] - top));
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) total += __shfl_xor(total, d);
    } else {
        total = chosen_sum;
    }
    if (lane < top_k) {
        idx[(size_t)t * top_k + lane] = mine_e;
        gate[(size_t)t * top_k + lane] = mine / total;
    }
}

// ---- gate and up projections ------------------------------------------------

struct MoeLists {
    int32_t *experts;  // [blocks of the reached list] expert of each
    int32_t *counts;   // tokens of each
    int32_t *pairs;    // [reached][tokens] the pairs t top_k + j of each, ascending
    int32_t *reached;  // [1]
};

// One block: the a-th reached expert (ascending), 16 intermediate columns.
// Every block finds its expert and its tokens from the router's choices
// itself (a bit set in LDS, then one wave collects the pairs in order); the
// blocks of column tile 0 write them down for the down projection. The waves
// take the groups of H in turn and add their sums in LDS; h is written as the
// sum of two bf16 numbers (hi + lo, 16 significant bits), so that its rounding
// stays far below that of Y.
__global__ __launch_bounds__(kMoeThreads) void moe_up_kernel(
    const uint16_t *__restrict__ X, const uint8_t *__restrict__ w13, const float *__restrict__ s13,
    const int32_t *__restrict__ idx, int T, int H, int I, int E, int top_k, uint16_t *__restrict__ h_hi,
    uint16_t *__restrict__ h_lo, MoeLists lists) {
    __shared__ uint32_t bits[SVDQ_FP8_MOE_MAX_EXPERTS / 32];
    __shared__ int32_t list[SVDQ_FP8_MOE_MAX_TOKENS];
    __shared__ int32_t count_s;
    __shared__ f32x4 red[kMoeWaves][2][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int pairs = T * top_k;
    const int a = blockIdx.y;
    const int i0 = blockIdx.x * 16;
    if (threadIdx.x < SVDQ_FP8_MOE_MAX_EXPERTS / 32) bits[threadIdx.x] = 0u;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kMoeThreads) atomicOr(&bits[idx[p] >> 5], 1u << (idx[p] & 31));
    __syncthreads();
    int e = -1, reached = 0;
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
    if (blockIdx.x == 0 && a == 0 && threadIdx.x == 0) *lists.reached = reached;
    e = __builtin_amdgcn_readfirstlane(e);
    if (e < 0) return;  // the same for every thread of the block
    if (wave == 0) {
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const bool hit = p0 + lane < pairs && idx[p0 + lane] == e;
            const uint64_t mask = __ballot(hit);
            if (hit) list[n + __popcll(mask & ((1ull << lane) - 1))] = p0 + lane;
            n += __popcll(mask);
        }
        if (lane == 0) count_s = n;
    }
    __syncthreads();
    const int count = count_s;
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < count; i += kMoeThreads) lists.pairs[(size_t)a * T + i] = list[i];
        if (threadIdx.x == 0) {
            lists.experts[a] = e;
            lists.counts[a] = count;
        }
    }
    const int r16 = lane & 15, q4 = lane >> 4;
    const int G = (H + kF8Block - 1) / kF8Block, gi = (I + kF8Block - 1) / kF8Block;
    const uint8_t *we = w13 + (size_t)e * 2 * I * H;
    const __amdgpu_buffer_rsrc_t rg = fp8_rsrc(we + (size_t)i0 * H, 16u * (uint32_t)H);
    const __amdgpu_buffer_rsrc_t ru = fp8_rsrc(we + (size_t)(I + i0) * H, 16u * (uint32_t)H);
    const float *sg = s13 + ((size_t)e * 2 * gi + i0 / kF8Block) * G;
    const float *su = sg + (size_t)gi * G;
    for (int m0 = 0; m0 < count; m0 += 16) {
        const int pair = list[min(m0 + r16, count - 1)];
        const uint16_t *x = X + (size_t)(pair / top_k) * H;
        f32x4 accg = {0.f, 0.f, 0.f, 0.f}, accu = accg;
        for (int g = wave; g < G; g += kMoeWaves) {
            f32x4 pg = {0.f, 0.f, 0.f, 0.f}, pu = pg;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = g * kF8Block + 64 * i + 16 * q4;
                const uint32_t off = k < H ? (uint32_t)r16 * (uint32_t)H + (uint32_t)k : kMoeOob;
                const u32x4 cg = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rg, off, 0, 0));
                const u32x4 cu = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ru, off, 0, 0));
                u32x4 x0 = {0u, 0u, 0u, 0u}, x1 = x0;
                if (k < H) {
                    x0 = *reinterpret_cast<const u32x4 *>(x + k);
                    x1 = *reinterpret_cast<const u32x4 *>(x + k + 8);
                }
                const bf16x8 b0 = __builtin_bit_cast(bf16x8, x0), b1 = __builtin_bit_cast(bf16x8, x1);
                pg = mfma_bf16_16x16x32(fp8_widen8(cg[0], cg[1]), b0, pg);
                pu = mfma_bf16_16x16x32(fp8_widen8(cu[0], cu[1]), b0, pu);
                pg = mfma_bf16_16x16x32(fp8_widen8(cg[2], cg[3]), b1, pg);
                pu = mfma_bf16_16x16x32(fp8_widen8(cu[2], cu[3]), b1, pu);
            }
            const float wg = sg[g], wu = su[g];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                accg[i] = __builtin_fmaf(wg, pg[i], accg[i]);
                accu[i] = __builtin_fmaf(wu, pu[i], accu[i]);
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
            for (int w = 0; w < kMoeWaves; ++w) {
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

// One block: 16 output columns of every token. A wave takes one reached expert
// and one of `splits` ranges of I at a time, reads its 16 weight rows once and
// leaves each pair's 16 sums in LDS at its own place; then each output is the
// weighted sum over its token's pairs in order, so the result does not depend
// on which wave came first.
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(
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
    const int units = *lists.reached * splits;
    for (int unit = wave; unit < units; unit += kMoeWaves) {
        const int a = unit / splits, s = unit % splits;
        const int e = __builtin_amdgcn_readfirstlane(lists.experts[a]);
        const int count = __builtin_amdgcn_readfirstlane(lists.counts[a]);
        const __amdgpu_buffer_rsrc_t rw = fp8_rsrc(w2 + ((size_t)e * H + n0) * I, 16u * (uint32_t)I);
        const float *sw = s2 + ((size_t)e * gh + n0 / kF8Block) * G;
        for (int m0 = 0; m0 < count; m0 += 16) {
            const int pair = lists.pairs[(size_t)a * T + min(m0 + r16, count - 1)];
            const uint16_t *hh = h_hi + (size_t)pair * I, *hl = h_lo + (size_t)pair * I;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            for (int g = s; g < G; g += splits) {
                f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = g * kF8Block + 64 * i + 16 * q4;
                    const uint32_t off = k < I ? (uint32_t)r16 * (uint32_t)I + (uint32_t)k : kMoeOob;
                    const u32x4 c = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, off, 0, 0));
                    u32x4 x0 = {0u, 0u, 0u, 0u}, x1 = x0, y0 = x0, y1 = x0;
                    if (k < I) {
                        x0 = *reinterpret_cast<const u32x4 *>(hh + k);
                        x1 = *reinterpret_cast<const u32x4 *>(hh + k + 8);
                        y0 = *reinterpret_cast<const u32x4 *>(hl + k);
                        y1 = *reinterpret_cast<const u32x4 *>(hl + k + 8);
                    }
                    const bf16x8 a0 = fp8_widen8(c[0], c[1]), a1 = fp8_widen8(c[2], c[3]);
                    p = mfma_bf16_16x16x32(a0, __builtin_bit_cast(bf16x8, y0), p);
                    p = mfma_bf16_16x16x32(a1, __builtin_bit_cast(bf16x8, y1), p);
                    p = mfma_bf16_16x16x32(a0, __builtin_bit_cast(bf16x8, x0), p);
                    p = mfma_bf16_16x16x32(a1, __builtin_bit_cast(bf16x8, x1), p);
                }
                const float w = sw[g];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(w, p[i], acc[i]);
            }
            if (m0 + r16 < count)
                *reinterpret_cast<f32x4 *>(out + ((size_t)s * pairs + pair) * 16 + 4 * q4) = acc;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * 16; i += kMoeThreads) {
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

}  // namespace

// Workspace: h (hi, lo planes of [pairs][I]), then the reached experts' lists,
// then room for the choices and weights of a call that does not ask for them.
size_t fp8_moe_workspace_size(int T, int I, int E, int top_k) {
    const size_t pairs = (size_t)T * top_k, lists = std::min((size_t)E, pairs);
    return 2 * align256(pairs * I * 2) + align256(4 * (lists * (2 + (size_t)T) + 1)) + 2 * align256(4 * pairs);
}

hipError_t launch_fp8_moe(const uint16_t *X, const uint16_t *wr, const uint8_t *w13, const float *s13,
                          const uint8_t *w2, const float *s2, int T, int H, int I, int E, int top_k, bool renorm,
                          int32_t *idx, float *gate, void *workspace, uint16_t *Y, hipStream_t stream) {
    const size_t pairs = (size_t)T * top_k;
    const int lists_n = (int)std::min((size_t)E, pairs);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint16_t *h_hi = reinterpret_cast<uint16_t *>(ws);
    ws += align256(pairs * I * 2);
    uint16_t *h_lo = reinterpret_cast<uint16_t *>(ws);
    ws += align256(pairs * I * 2);
    int32_t *l = reinterpret_cast<int32_t *>(ws);
    ws += align256(4 * (lists_n * (2 + (size_t)T) + 1));
    if (!idx) idx = reinterpret_cast<int32_t *>(ws);
    ws += align256(4 * pairs);
    if (!gate) gate = reinterpret_cast<float *>(ws);
    const MoeLists lists{l + 1, l + 1 + lists_n, l + 1 + 2 * lists_n, l};
    hipLaunchKernelGGL(moe_router_kernel, dim3(T), dim3(kMoeThreads), 0, stream, X, wr, H, E, top_k, renorm ? 1 : 0,
                       idx, gate);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(moe_up_kernel, dim3(I / 16, lists_n), dim3(kMoeThreads), 0, stream, X, w13, s13, idx, T, H, I,
                       E, top_k, h_hi, h_lo, lists);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    // as many ranges of I as give every wave a unit, at most one per group and
    // what 32 KB of LDS hold
    const int G = fp8_blocks(I);
    int splits = (int)std::min<size_t>((kMoeWaves + lists_n - 1) / lists_n, G);
    while (splits > 1 && splits * pairs * 64 > (32u << 10)) --splits;
    hipLaunchKernelGGL(moe_down_kernel, dim3(H / 16), dim3(kMoeThreads), splits * pairs * 64, stream, w2, s2, h_hi,
                       h_lo, gate, lists, T, H, I, top_k, splits, Y);
    return hipGetLastError();
}

}  // namespace svdq
