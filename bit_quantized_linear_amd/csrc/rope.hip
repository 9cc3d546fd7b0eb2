// Rotary positions of one or several axes on heads of bf16 rows.
//
//   angle[t, j] = positions[t, axis of pair j] * freqs[j]      (fp64)
//   (a, b) -> (a cos - b sin, a sin + b cos)                   (fp32, rounded once)
//
// The product and its reduction to a part of a turn are fp64: at position 2^20
// an angle kept in fp32 would be off by a twentieth of a radian. Sine and cosine
// of a token's pairs are worked out once for all its heads.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace svdq {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 1024;  // of a block's tokens, in LDS

struct RopeArgs {
    const uint16_t *X;
    int64_t x_stride;
    const int32_t *positions;
    const double *freqs;
    int ends[SVDQ_ROPE_MAX_AXES];  // pairs up to and with each axis
    int axes, R, T, H, D, tokens;
    uint16_t *Y;
    int64_t y_stride;
};

__device__ __forceinline__ void rope_turn(float c, float s, float &a, float &b) {
    const float x = a;
    a = __builtin_fmaf(a, c, -(b * s));
    b = __builtin_fmaf(x, s, b * c);
}

// A block takes `tokens` tokens: their angles' sines and cosines to LDS, then the
// heads in pieces of 8 features (two of them, R / 2 apart, where pairs are).
// HBM-bound: 2 bytes in and 2 out per feature; 32760 tokens of 80 heads of 128 take
// 245 us, 5.5 TB/s (a large copy: 5.15); 16 tokens of 40 heads 3.3 us, an empty launch 2 to 3.
template <bool kInterleaved>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    __shared__ __align__(16) float cs[kRopeAngles], sn[kRopeAngles];
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int tokens = min(a.tokens, (int)(a.T - t0)), pairs = a.R / 2;
    for (int i = threadIdx.x; i < tokens * pairs; i += kRopeThreads) {
        const int t = tokens == 1 ? 0 : i / pairs, j = i - t * pairs;
        int axis = 0;
        while (axis + 1 < a.axes && j >= a.ends[axis]) ++axis;
        const double turns = (double)a.positions[(t0 + t) * a.axes + axis] * a.freqs[j] * 0.15915494309189533577;
        const float f = (float)(2.0 * (turns - rint(turns)));
        sincospif(f, &sn[i], &cs[i]);
    }
    __syncthreads();
    const int turned = a.R / (kInterleaved ? 8 : 16), per = turned + (a.D - a.R) / 8, all = a.H * per;
    for (int i = threadIdx.x; i < tokens * all; i += kRopeThreads) {
        const int t = tokens == 1 ? 0 : i / all, head = (i - t * all) / per, c = i - t * all - head * per;
        const uint16_t *x = a.X + (t0 + t) * a.x_stride + (int64_t)head * a.D;
        uint16_t *y = a.Y + (t0 + t) * a.y_stride + (int64_t)head * a.D;
        if (c >= turned) {
            const int k = a.R + (c - turned) * 8;
            *reinterpret_cast<u32x4 *>(y + k) = *reinterpret_cast<const u32x4 *>(x + k);
            continue;
        }
        const int k = c * 8;
        const float *ct = cs + t * pairs, *st = sn + t * pairs;
        u32x4 u = *reinterpret_cast<const u32x4 *>(x + k);
        if (kInterleaved) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                float v = __uint_as_float(u[p] << 16), w = __uint_as_float(u[p] & 0xFFFF0000u);
                rope_turn(ct[4 * c + p], st[4 * c + p], v, w);
                u[p] = bf16x2_bits(v, w);
            }
            *reinterpret_cast<u32x4 *>(y + k) = u;
        } else {
            u32x4 v = *reinterpret_cast<const u32x4 *>(x + k + pairs);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                float a0 = __uint_as_float(u[p] << 16), a1 = __uint_as_float(u[p] & 0xFFFF0000u);
                float b0 = __uint_as_float(v[p] << 16), b1 = __uint_as_float(v[p] & 0xFFFF0000u);
                rope_turn(ct[8 * c + 2 * p], st[8 * c + 2 * p], a0, b0);
                rope_turn(ct[8 * c + 2 * p + 1], st[8 * c + 2 * p + 1], a1, b1);
                u[p] = bf16x2_bits(a0, a1);
                v[p] = bf16x2_bits(b0, b1);
            }
            *reinterpret_cast<u32x4 *>(y + k) = u;
            *reinterpret_cast<u32x4 *>(y + k + pairs) = v;
        }
    }
}

}  // namespace

// Tokens of a block: as many as give each of its threads two pieces, while there are
// 2048 blocks (32760 tokens of 8 heads of 128: 27.7 us with 512 pieces a block, 30.3 with
// 1024, 36.5 with one token, 256; of 1 head of 64: 5.4 and 13.9 with one token).
constexpr int kRopePieces = 512, kRopeBlocks = 2048;

hipError_t launch_rope(const uint16_t *X, int64_t x_stride, const int32_t *positions, const double *freqs,
                       const int *sections, int axes, int interleaved, int T, int H, int D, uint16_t *Y,
                       int64_t y_stride, hipStream_t stream) {
    RopeArgs a{X, x_stride, positions, freqs, {}, axes, 0, T, H, D, 1, Y, y_stride};
    int pairs = 0;
    for (int i = 0; i < axes; ++i) a.ends[i] = pairs += sections[i];
    a.R = 2 * pairs;
    const int pieces = H * (a.R / (interleaved ? 8 : 16) + (D - a.R) / 8);
    a.tokens = std::max(1, std::min({kRopePieces / pieces, kRopeAngles / pairs, T / kRopeBlocks}));
    return launch_kernel(interleaved ? rope_kernel<true> : rope_kernel<false>, dim3((unsigned)((T + a.tokens - 1) / a.tokens)),
                         kRopeThreads, stream, a);
}

}  // namespace svdq
