// The residual's addition and root-mean-square norm before a block-scaled FP8
// linear, with the linear's E4M3 codes and scales as its output.
//
//   h[m, k]  = X + residual                                      (fp32)
//   y[m, k]  = h / sqrt(mean_k h^2 + eps) * w[k]                 (fp32)
//   A[m, g]  = max(max_{k in g} |y|, 2^-100)
//   sx[g, m] = fp32(A / 448),  qx = E4M3(fp32(y fp32(448 / A)))
//
// y is not rounded to bf16 on its way to the codes. The sum of squares is kept in
// fp64: it neither overflows nor underflows for any bf16 input, and what its order
// changes is far below fp32's rounding.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_common.h"
#include "fp8_common.h"
#include "internal.h"

namespace svdq {

namespace {

constexpr int kCus = 256;  // compute units

// The largest of 16 lanes' values (lanes 16 n .. 16 n + 15), in all of them.
__device__ __forceinline__ uint32_t max_of_16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // lane ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // lane ^ 2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // 7 - lane, of 8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // 15 - lane, of 16
    return v;
}

__device__ __forceinline__ void widen8(u32x4 v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ u32x4 narrow8(const float (&x)[8]) {
    return u32x4{bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]), bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7])};
}

struct NormArgs {
    const uint16_t *X, *residual, *w;
    float eps;
    int M, K;
    uint16_t *sum, *Y;
    uint8_t *qx;
    float *sx;
};

// h of 8 features.
__device__ __forceinline__ void norm_input(const NormArgs &a, size_t at, float (&h)[8]) {
    widen8(*reinterpret_cast<const u32x4 *>(a.X + at), h);
    if (a.residual) {
        float r[8];
        widen8(*reinterpret_cast<const u32x4 *>(a.residual + at), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
}

// What a token's h is multiplied with, 1 / sqrt(mean + eps), as the product of a power
// of two and an ordinary number: for tokens near the smallest or the largest bf16
// numbers (2^-133, subnormal; 2^128) it is itself past the largest fp32 number, or
// subnormal with fewer bits. h times the first factor is exact, as far as the norm shows
// it: it is 1 for all other tokens.
struct NormFactor {
    float power, rest;
};

__device__ __forceinline__ NormFactor norm_factor(double mean, float eps) {
    const double r = 1.0 / sqrt(mean + (double)eps);
    if (__builtin_expect(r > 0x1p100 || r < 0x1p-100, 0)) {
        const float power = r > 1.0 ? 0x1p64f : 0x1p-64f;
        return {power, (float)(r * (r > 1.0 ? 0x1p-64 : 0x1p64))};
    }
    return {1.0f, (float)r};
}

// Outputs of 8 features of token m from feature k on; the 16 lanes of a group of
// 128 features call it together, h is 0 past K.
__device__ __forceinline__ void norm_output(const NormArgs &a, int m, int k, float (&h)[8], NormFactor f) {
    const size_t at = (size_t)m * a.K + k;
    const bool in = k < a.K;
    if (in && a.sum) *reinterpret_cast<u32x4 *>(a.sum + at) = narrow8(h);
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
        float w[8];
        widen8(*reinterpret_cast<const u32x4 *>(a.w + k), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[i] * f.power * f.rest * w[i];
        if (a.Y) *reinterpret_cast<u32x4 *>(a.Y + at) = narrow8(y);
    }
    if (!a.qx) return;
    uint32_t top = __float_as_uint(0x1p-100f);  // on the bit patterns NaN is above all
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    const float A = __uint_as_float(max_of_16(top));
    const float r = kF8Max / A;
    if (!in) return;
    u32x2 q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i] * r, y[4 * i + 1] * r, 0, false);
        q[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2] * r, y[4 * i + 3] * r, lo, true);
    }
    *reinterpret_cast<u32x2 *>(a.qx + at) = q;
    if (k % kF8Block == 0) a.sx[(size_t)(k / kF8Block) * a.M + m] = A / kF8Max;
}

// HBM-bound: 2 bytes in, 2 of the residual, 2 of the sum out and 1 of a code per
// feature, each once; 32760 x 5120 takes 214 us, 5.5 TB/s (a large copy: 5.15), 8 x
// 4096 3.6 us (3.4 among others in a graph), of which an empty launch is 2 to 3.
// TR threads a token, C pieces of 8 features per thread in registers; the rest of a
// longer row is read again for the second pass (each thread reads what it has read
// before and writes there afterwards, so that the sum may replace the residual).
template <int TR, int C>
__global__ __launch_bounds__(TR < 256 ? 256 : TR) void fp8_norm_kernel(NormArgs a) {
    constexpr int NT = TR < 256 ? 256 : TR;
    __shared__ double part[NT / 64];
    const int m = blockIdx.x * (NT / TR) + threadIdx.x / TR, t = threadIdx.x % TR;
    if (TR < 256 && m >= a.M) return;
    const size_t row = (size_t)m * a.K;
    float h[C][8];
    double ss = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * TR + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = 0.0f;
        if (k < a.K) norm_input(a, row + k, h[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)h[c][i], (double)h[c][i], ss);
    for (int k = (C * TR + t) * 8; k < a.K; k += TR * 8) {
        float g[8];
        norm_input(a, row + k, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)g[i], (double)g[i], ss);
    }
#pragma unroll
    for (int d = 1; d < 64 && d < TR; d <<= 1) ss += __shfl_xor(ss, d);
    if constexpr (TR > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
        __syncthreads();
        ss = 0.0;
#pragma unroll
        for (int w = 0; w < TR / 64; ++w) ss += part[w];
    }
    const NormFactor f = norm_factor(ss / a.K, a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * TR + t) * 8;
        if (k - (t & 15) * 8 < a.K) norm_output(a, m, k, h[c], f);
    }
    for (int k = (C * TR + t) * 8; k - (t & 15) * 8 < a.K; k += TR * 8) {
        float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (k < a.K) norm_input(a, row + k, g);
        norm_output(a, m, k, g, f);
    }
}

}  // namespace

hipError_t launch_fp8_norm(const uint16_t *X, const uint16_t *residual, const uint16_t *w, float eps, int M, int K,
                           uint16_t *sum, uint16_t *Y, uint8_t *qx, float *sx, hipStream_t stream) {
    const NormArgs a{X, residual, w, eps, M, K, sum, Y, qx, sx};
    const auto launch = [&](auto kernel, int per_token) {
        const int threads = std::max(per_token, 256), tokens = threads / per_token;
        return launch_kernel(kernel, dim3((unsigned)((M + tokens - 1) / tokens)), (unsigned)threads, stream, a);
    };
    // Short rows: several tokens a block, so that its threads have work (32760 x 256: 12.6
    // us against 49.7 with a block per token, x 1024: 47.9 against 66.5, x 2048: 95 and 85.5)
    if (K <= 128) return launch(fp8_norm_kernel<16, 1>, 16);
    if (K <= 256) return launch(fp8_norm_kernel<32, 1>, 32);
    if (K <= 512) return launch(fp8_norm_kernel<64, 1>, 64);
    const bool few = M <= kCus;
    if (!few && K <= 1024) return launch(fp8_norm_kernel<64, 2>, 64);
    if (K <= 2048) return launch(fp8_norm_kernel<256, 1>, 256);
    // Long rows: 512 threads where a compute unit has one token (16 x 8192: 3.8 us against
    // 5.1 with 256) or they spare registers (4096 x 8192: 49.6 against 55.1; 32760 x
    // 5120: 231 against 213)
    if (few || K > 6144) return launch(fp8_norm_kernel<512, 2>, 512);
    return launch(fp8_norm_kernel<256, 3>, 256);
}

}  // namespace svdq
