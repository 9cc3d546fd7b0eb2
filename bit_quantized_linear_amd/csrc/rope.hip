// Rotary positions of one or several axes on heads of bf16 rows.
//
//   angle[t, j] = positions[t, axis of pair j] * freqs[j]      (fp64)
//   (a, b) -> (a cos - b sin, a sin + b cos)                   (fp32, rounded once)
//
// The product and its reduction to a part of a turn are fp64: at position 2^20
// an angle kept in fp32 would be off by a twentieth of a radian. Sine and cosine
// of a token's pairs are worked out once for all its heads.

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "internal.h"

namespace svdq {

namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    const uint16_t *X;
    int64_t x_stride;
    const int32_t *positions;
    const double *freqs;
    int ends[SVDQ_ROPE_MAX_AXES];  // pairs up to and with each axis
    int axes, R, H, D;
    uint16_t *Y;
    int64_t y_stride;
};

__device__ __forceinline__ void rope_turn(float c, float s, float &a, float &b) {
    const float x = a;
    a = __builtin_fmaf(a, c, -(b * s));
    b = __builtin_fmaf(x, s, b * c);
}

template <bool kInterleaved>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    __shared__ __align__(16) float cs[SVDQ_ROPE_MAX_PAIRS], sn[SVDQ_ROPE_MAX_PAIRS];
    const int64_t t = blockIdx.x;
    const int pairs = a.R / 2;
    for (int j = threadIdx.x; j < pairs; j += kRopeThreads) {
        int axis = 0;
        while (axis + 1 < a.axes && j >= a.ends[axis]) ++axis;
        const double turns = (double)a.positions[t * a.axes + axis] * a.freqs[j] * 0.15915494309189533577;
        const float f = (float)(2.0 * (turns - rint(turns)));
        sincospif(f, &sn[j], &cs[j]);
    }
    __syncthreads();
    const uint16_t *x = a.X + t * a.x_stride;
    uint16_t *y = a.Y + t * a.y_stride;
    // pieces of 8 features (two of them, R / 2 apart, where pairs are)
    const int turned = a.R / (kInterleaved ? 8 : 16), per = turned + (a.D - a.R) / 8;
    for (int i = threadIdx.x; i < a.H * per; i += kRopeThreads) {
        const int head = i / per, c = i - head * per;
        const int64_t at = (int64_t)head * a.D;
        if (c >= turned) {
            const int64_t k = at + a.R + (c - turned) * 8;
            *reinterpret_cast<u32x4 *>(y + k) = *reinterpret_cast<const u32x4 *>(x + k);
            continue;
        }
        const int64_t k = at + c * 8;
        u32x4 u = *reinterpret_cast<const u32x4 *>(x + k);
        if (kInterleaved) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                float v = __uint_as_float(u[p] << 16), w = __uint_as_float(u[p] & 0xFFFF0000u);
                rope_turn(cs[4 * c + p], sn[4 * c + p], v, w);
                u[p] = bf16x2_bits(v, w);
            }
            *reinterpret_cast<u32x4 *>(y + k) = u;
        } else {
            u32x4 v = *reinterpret_cast<const u32x4 *>(x + k + pairs);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                float a0 = __uint_as_float(u[p] << 16), a1 = __uint_as_float(u[p] & 0xFFFF0000u);
                float b0 = __uint_as_float(v[p] << 16), b1 = __uint_as_float(v[p] & 0xFFFF0000u);
                rope_turn(cs[8 * c + 2 * p], sn[8 * c + 2 * p], a0, b0);
                rope_turn(cs[8 * c + 2 * p + 1], sn[8 * c + 2 * p + 1], a1, b1);
                u[p] = bf16x2_bits(a0, a1);
                v[p] = bf16x2_bits(b0, b1);
            }
            *reinterpret_cast<u32x4 *>(y + k) = u;
            *reinterpret_cast<u32x4 *>(y + k + pairs) = v;
        }
    }
}

}  // namespace

hipError_t launch_rope(const uint16_t *X, int64_t x_stride, const int32_t *positions, const double *freqs,
                       const int *sections, int axes, int interleaved, int T, int H, int D, uint16_t *Y,
                       int64_t y_stride, hipStream_t stream) {
    RopeArgs a{X, x_stride, positions, freqs, {}, axes, 0, H, D, Y, y_stride};
    int pairs = 0;
    for (int i = 0; i < axes; ++i) a.ends[i] = pairs += sections[i];
    a.R = 2 * pairs;
    hipLaunchKernelGGL(interleaved ? rope_kernel<true> : rope_kernel<false>, dim3((unsigned)T), dim3(kRopeThreads), 0,
                       stream, a);
    return hipGetLastError();
}

}  // namespace svdq
