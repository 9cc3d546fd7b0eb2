// New keys and values into the 8-bit cache.
//
//   page of 64 tokens and head:  A = max(max |x| over its new tokens, 2^-100)
//   need = the least power of two with A <= 448 need
//   s    = max(need, the page's scale if it holds earlier tokens)
//   codes E4M3(x / s); earlier codes become E4M3(code * (old scale / s))
//
// Scales are powers of two: an E4M3 code has the same three bits of mantissa at
// any scale, so nothing is lost against A / 448, and rounding earlier codes to a
// larger scale is exact but below 2^-6 s (the codes' subnormal range), where any
// scale that holds the page's largest value would round them too.
// Values that are not finite become the NaN code and leave the scale alone, so
// that they reach the attention of the queries that see them and nothing else.

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "fp8_common.h"
#include "internal.h"
#include "kv8_common.h"

namespace svdq {

namespace {

constexpr int kAppThreads = 256;

struct AppendArgs {
    KvBatch kv;
    const uint16_t *K, *V;
    int64_t k_stride, v_stride;
    int Hk, D;
    uint8_t *kc, *vc;
    float *ks, *vs;
};

// The least power of two s with a <= 448 s = 1.75 * 2^8 s; a is a bf16 number
// from 2^-100 up.
__device__ __forceinline__ float kv_scale(float a) {
    const uint32_t u = __float_as_uint(a);
    const uint32_t e = (u >> 23) - 8u + ((u & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
    return __uint_as_float(e << 23);
}

// A bf16 number as fp32; infinities become NaN.
__device__ __forceinline__ float kv_value(uint32_t bits16) {
    return __uint_as_float((bits16 & 0x7FFFu) == 0x7F80u ? 0x7FC00000u : bits16 << 16);
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Four codes times a power of two.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    return codes4(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * ratio, __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * ratio,
                  __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * ratio, __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * ratio);
}

// The largest finite magnitude of 8 bf16 values, on their bit patterns.
__device__ __forceinline__ uint32_t top_finite(u32x4 v) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = v[i] & 0x7FFFu, hi = (v[i] >> 16) & 0x7FFFu;
        top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
    return top;
}

// One page and head, keys or values (blockIdx.y % 2). A thread has 8 features of 4
// tokens. Of keys, neighbouring threads have neighbouring features, so that rows are
// read and written whole; of values, neighbouring tokens, whose codes are 8 pieces
// of 4 tokens as a page holds them. The tokens are under way while the page's
// number, then its scale and the codes that share a piece with new ones are.
// HBM-bound: 4 bytes in and 2 out per token, head and feature. 4680 tokens of 40 heads of
// 128: 35 us, 4.1 TB/s from memory (a large copy: 5.15; 27 to 30 us where the 96 MB of keys
// and values are in the last-level cache), as a block is three memory latencies in turn;
// one token each of 16 sequences 6.4 us, four of them (sequence, page, scale and shared
// codes, codes).
__global__ __launch_bounds__(kAppThreads) void kv8_append_kernel(AppendArgs a) {
    __shared__ uint32_t tops[kAppThreads / 64];
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    int b, nth;
    KvSeq seq;
    if (!kv_find(a.kv, blockIdx.x, b, seq, nth, [](const KvSeq &s) {
            const int first = max(0, s.length - s.rows);
            return s.rows > 0 && s.length > 0 ? (s.length - 1) / kKvPage - first / kKvPage + 1 : 0;
        }))
        return;
    const int first = max(0, seq.length - seq.rows);
    const int p = first / kKvPage + nth;
    // new tokens low .. high - 1 of the page; token t is row row0 + t
    const int low = max(first - p * kKvPage, 0), high = min(seq.length - p * kKvPage, kKvPage);
    const int64_t row0 = seq.row0 + seq.rows - seq.length + (int64_t)p * kKvPage;
    const int64_t stride = values ? a.v_stride : a.k_stride;
    const uint16_t *x = (values ? a.V : a.K) + (int64_t)head * a.D;

    const int per = a.D / 8;  // threads of a row of keys
    const int token = values ? 4 * (threadIdx.x & 15) : threadIdx.x / per, step = values ? 1 : kAppThreads / per;
    const int f = values ? (threadIdx.x >> 4) * 8 : threadIdx.x % per * 8;
    const bool mine = f < a.D;
    u32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = token + i * step;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (mine && t >= low && t < high) v[i] = *reinterpret_cast<const u32x4 *>(x + (row0 + t) * stride + f);
    }
    const int page = kv_page(a.kv, b, p);
    if (page < 0) return;
    const int64_t unit = (int64_t)page * a.Hk + head;
    uint8_t *codes = (values ? a.vc : a.kc) + unit * kKvPage * a.D;
    float *scale = (values ? a.vs : a.ks) + unit;
    const float old = *scale;
    // of values: bytes of the new tokens among the thread's 4, and the codes there if others share their pieces
    uint32_t fresh = 0, was[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) fresh |= token + i >= low && token + i < high ? 0xFFu << (8 * i) : 0u;
    const bool shared = values && mine && fresh != 0u && fresh != 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        was[j] = shared ? *reinterpret_cast<const uint32_t *>(codes + (f + j) * kKvPage + token) : 0u;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, top_finite(v[i]));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppThreads / 64; ++w) top = max(top, tops[w]);
    float s = kv_scale(bf16_bits_to_f32(max(top, kF8TinyBits)));
    if (low > 0) s = fmaxf(s, old);
    const float r = 1.0f / s, ratio = old / s;
    const bool shrink = low > 0 && s != old;
    if (threadIdx.x == 0) *scale = s;
    if (!mine) return;

    if (!values) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = token + i * step;
            u32x2 *at = reinterpret_cast<u32x2 *>(codes + t * a.D + f);
            if (t >= low && t < high) {
                u32x2 w;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t lo = v[i][2 * j], hi = v[i][2 * j + 1];
                    w[j] = codes4(kv_value(lo & 0xFFFFu) * r, kv_value(lo >> 16) * r, kv_value(hi & 0xFFFFu) * r,
                                  kv_value(hi >> 16) * r);
                }
                *at = w;
            } else if (shrink && t < low) {
                const u32x2 w = *at;
                *at = u32x2{rescale4(w[0], ratio), rescale4(w[1], ratio)};
            }
        }
        return;
    }
    uint32_t before = 0;  // bytes of earlier tokens, to be rounded to a larger scale
#pragma unroll
    for (int i = 0; i < 4; ++i) before |= shrink && token + i < low ? 0xFFu << (8 * i) : 0u;
    if (!(fresh | before)) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t *at = reinterpret_cast<uint32_t *>(codes + (f + j) * kKvPage + token);
        if (!fresh) {
            *at = rescale4(*at, ratio);
            continue;
        }
        const int sh = 16 * (j & 1);
        uint32_t w = codes4(kv_value(v[0][j / 2] >> sh & 0xFFFFu) * r, kv_value(v[1][j / 2] >> sh & 0xFFFFu) * r,
                            kv_value(v[2][j / 2] >> sh & 0xFFFFu) * r, kv_value(v[3][j / 2] >> sh & 0xFFFFu) * r);
        if (shared) {
            w = (w & fresh) | (was[j] & ~(fresh | before));
            if (before) w |= rescale4(was[j], ratio) & before;
        }
        *at = w;
    }
}

}  // namespace

// Pages that the new tokens of B sequences reach at the most, T tokens in all: n
// tokens reach (n + 62) / 64 + 1.
static int64_t append_pages(int T, int B) { return ((int64_t)T + 62LL * B) / kKvPage + B; }

hipError_t launch_kv8_append(const KvBatch &kv, const uint16_t *K, int64_t k_stride, const uint16_t *V, int64_t v_stride,
                             int Hk, int D, uint8_t *kc, float *ks, uint8_t *vc, float *vs, hipStream_t stream) {
    const AppendArgs a{kv, K, V, k_stride, v_stride, Hk, D, kc, vc, ks, vs};
    return launch_kernel(kv8_append_kernel, dim3((unsigned)append_pages(kv.T, kv.B), 2u * (unsigned)Hk), kAppThreads, stream, a);
}

}  // namespace svdq
