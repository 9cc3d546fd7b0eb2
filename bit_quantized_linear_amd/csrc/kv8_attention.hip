// Attention of a batch's newest tokens over the 8-bit key and value cache.
//
//   o[q] = sum_t softmax_t(scale q . k_t) v_t   over the tokens t that q sees
//
// in one pass over the pages with a running maximum and sum: for a page with
// scores s_t (base-2 logarithms, the page's key scale among their factors)
//   m' = max(m, max s_t),  p_t = 2^(s_t - m'),  l' = l 2^(m - m') + sum p_t,
//   O' = O 2^(m - m') + sum (p_t vs) v_t
// with vs the page's value scale. Products run on the bf16 matrix core: E4M3
// codes are exact in bf16, p vs is rounded to bf16 (2^-9 of each weight; vs is a
// power of two), sums and statistics are fp32.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T, so that a lane holds one
// query: its statistics need no broadcast, and the weights of S^T are the next
// product's operand where they are. A matrix-core tile's rows 4 apart belong to
// different lanes, so the key rows are dealt to them in an order that leaves each
// lane with the weights of consecutive tokens, as it reads them of V^T.
//
// The queries of a sequence that share a key head (`group` per token) are the
// rows of one problem, token by token.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_common.h"
#include "fp8_common.h"
#include "internal.h"
#include "kv8_common.h"

namespace svdq {

namespace {

constexpr float kLn2 = 0.69314718055994530942f;

struct AttnArgs {
    KvBatch kv;
    const uint16_t *Q;
    int64_t q_stride;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    int Hq, Hk, group;
    float scale;  // with log2 e
    int causal, window;
    uint16_t *O;
    float *lse;
    float *part;  // splits' sums [T][Hq][splits][D], then maxima and sums of weights [T][Hq][splits][2]
    int splits;
};

// Tokens low .. high - 1 are what the query of new token i sees.
__device__ __forceinline__ void kv_seen(const AttnArgs &a, const KvSeq &s, int i, int &low, int &high) {
    const int pos = s.length - s.rows + i;
    high = a.causal ? max(pos + 1, 0) : s.length;
    low = a.window ? max(0, pos + 1 - a.window) : 0;
}

// Bytes of a dword of 4 tokens from t on that lie in low .. high - 1.
__device__ __forceinline__ uint32_t byte_mask(int t, int low, int high) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m |= t + i >= low && t + i < high ? 0xFFu << (8 * i) : 0u;
    return m;
}

// Whether one of 4 codes is NaN (0x7F or 0xFF): the top bits of the result.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// 8 bf16 values, NaN replaced by 0 in v and 1.0 in their place in nan.
__device__ __forceinline__ void split_nan(bf16x8 &v, bf16x8 &nan) {
    u32x4 u = __builtin_bit_cast(u32x4, v), n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (u[i] & 0x7FFFu) > 0x7F80u ? 0xFFFFu : 0u;
        const uint32_t hi = (u[i] & 0x7FFF0000u) > 0x7F800000u ? 0xFFFF0000u : 0u;
        n[i] = (lo | hi) & 0x3F803F80u;
        u[i] &= ~(lo | hi);
    }
    v = __builtin_bit_cast(bf16x8, u);
    nan = __builtin_bit_cast(bf16x8, n);
}

__device__ __forceinline__ bf16x8 pack8(const float *p, float f) {
    return __builtin_bit_cast(bf16x8, u32x4{bf16x2_bits(p[0] * f, p[1] * f), bf16x2_bits(p[2] * f, p[3] * f),
                                            bf16x2_bits(p[4] * f, p[5] * f), bf16x2_bits(p[6] * f, p[7] * f)});
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- few queries -----------------------------------------------------------

constexpr int kDecWaves = 4;
constexpr int kDecRows = 16;

// A block takes up to 16 queries at a time and a run of the sequence's pages, its
// waves every fourth of them, straight into registers, the next page while this
// one is computed; the waves' sums are joined in LDS and, where a sequence's pages
// are split over blocks, by a second kernel.
template <int D>
__global__ __launch_bounds__(64 * kDecWaves) void kv8_decode_kernel(AttnArgs a) {
    constexpr int KC = D / 64;  // 64-byte pieces of a key
    constexpr int DT = D / 16;  // 16-row tiles of V^T
    __shared__ __align__(16) float o_s[kDecWaves][kDecRows][D + 4];
    __shared__ float m_s[kDecWaves][kDecRows], l_s[kDecWaves][kDecRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q16 = lane & 15, g4 = lane >> 4;
    const int split = blockIdx.x, head = blockIdx.y, b = blockIdx.z;
    const KvSeq seq = kv_seq(a.kv, b);
    const int rows = seq.rows * a.group;
    for (int r0 = 0; r0 < rows; r0 += kDecRows) {
        const int last = min(r0 + kDecRows, rows) - 1;
        const int r = min(r0 + q16, last);
        int low, high, low0, high0, low1, high1;
        kv_seen(a, seq, r / a.group, low, high);
        kv_seen(a, seq, r0 / a.group, low0, high0);
        kv_seen(a, seq, last / a.group, low1, high1);
        // low0 <= low <= low1 and high0 <= high <= high1
        const int first_page = low0 / kKvPage, pages = max(0, (high1 + kKvPage - 1) / kKvPage - first_page);
        const int per = (pages + a.splits - 1) / a.splits;
        const int p0 = first_page + split * per, p1 = min(p0 + per, first_page + pages);

        bf16x8 q[2 * KC];
        {
            const uint16_t *src = a.Q + (int64_t)(seq.row0 + r / a.group) * a.q_stride +
                                  (int64_t)(head * a.group + r % a.group) * D + 16 * g4;
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                q[2 * i] = bitcast<bf16x8>(src + 64 * i);
                q[2 * i + 1] = bitcast<bf16x8>(src + 64 * i + 8);
            }
        }
        float m = -INFINITY, l = 0.0f;
        f32x4 o[DT];
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

        u32x4 k[4][KC], v[DT];
        float ks = 0.0f, vs = 0.0f;
        int page = -1;
        auto fetch = [&](int p) __attribute__((always_inline)) {
            page = p < p1 ? kv_page(a.kv, b, p) : -1;
            if (page < 0) return;
            const int64_t unit = (int64_t)page * a.Hk + head;
            const uint8_t *kp = a.kc + unit * kKvPage * D, *vp = a.vc + unit * kKvPage * D;
            ks = a.ks[unit];
            vs = a.vs[unit];
            // tile j's row i is token 16 (i / 4) + 4 j + i % 4
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < KC; ++i)
                    k[j][i] = bitcast<u32x4>(kp + (16 * (q16 >> 2) + 4 * j + (q16 & 3)) * D + 64 * i + 16 * g4);
#pragma unroll
            for (int i = 0; i < DT; ++i) v[i] = bitcast<u32x4>(vp + (16 * i + q16) * kKvPage + 16 * g4);
        };
        fetch(p0 + wave);
        for (int p = p0 + wave; p < p1; p += kDecWaves) {
            if (page < 0) {
                fetch(p + kDecWaves);
                continue;
            }
            const float c = ks * a.scale, vscale = vs;
            f32x4 s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < KC; ++i) {
                    s[j] = mfma_bf16_16x16x32(fp8_widen8(k[j][i][0], k[j][i][1]), q[2 * i], s[j]);
                    s[j] = mfma_bf16_16x16x32(fp8_widen8(k[j][i][2], k[j][i][3]), q[2 * i + 1], s[j]);
                }
            }
            u32x4 vc[DT];
#pragma unroll
            for (int i = 0; i < DT; ++i) vc[i] = v[i];
            const int t0 = p * kKvPage;
            fetch(p + kDecWaves);
            // a page that some query does not see whole: hidden tokens' weights are
            // 0, and their values are not multiplied, as they may be NaN
            uint32_t nan = 0;
            bf16x8 seen[2];
            if (t0 < low1 || t0 + kKvPage > high0) {
                uint32_t see[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t mask = byte_mask(t0 + 16 * g4 + 4 * j, low0, high1);
#pragma unroll
                    for (int i = 0; i < DT; ++i) {
                        vc[i][j] &= mask;
                        nan |= nan_codes(vc[i][j]);
                    }
                    see[j] = byte_mask(t0 + 16 * g4 + 4 * j, low, high);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[j][e] = see[j] >> (8 * e) & 1 ? s[j][e] : -INFINITY;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    u32x4 w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t two = see[2 * u + i / 2] >> (16 * (i & 1));
                        w[i] = (two & 1 ? 0x3F80u : 0u) | (two & 0x100u ? 0x3F800000u : 0u);
                    }
                    seen[u] = __builtin_bit_cast(bf16x8, w);
                }
            }
            float top = s[0][0];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, s[j][e]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m_new = fmaxf(m, top * c);
            const float base = m_new == -INFINITY ? 0.0f : m_new;
            const float alpha = exp2_of(m - base);
            m = m_new;
            l *= alpha;
            float w[16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[4 * j + e] = exp2_of(__builtin_fmaf(s[j][e], c, -base));
                    l += w[4 * j + e];
                }
            const bf16x8 w0 = pack8(w, vscale), w1 = pack8(w + 8, vscale);
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= alpha;
            if (!__any(nan != 0)) {
#pragma unroll
                for (int i = 0; i < DT; ++i) {
                    o[i] = mfma_bf16_16x16x32(fp8_widen8(vc[i][0], vc[i][1]), w0, o[i]);
                    o[i] = mfma_bf16_16x16x32(fp8_widen8(vc[i][2], vc[i][3]), w1, o[i]);
                }
            } else {  // NaN reaches the queries that see its token, and no other
#pragma unroll
                for (int i = 0; i < DT; ++i) {
                    bf16x8 v0 = fp8_widen8(vc[i][0], vc[i][1]), v1 = fp8_widen8(vc[i][2], vc[i][3]), n0, n1;
                    split_nan(v0, n0);
                    split_nan(v1, n1);
                    f32x4 count = mfma_bf16_16x16x32(n0, seen[0], f32x4{0.f, 0.f, 0.f, 0.f});
                    count = mfma_bf16_16x16x32(n1, seen[1], count);
                    o[i] = mfma_bf16_16x16x32(v0, w0, o[i]);
                    o[i] = mfma_bf16_16x16x32(v1, w1, o[i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] = count[e] > 0.0f ? NAN : o[i][e];
                }
            }
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g4 == 0) {
            m_s[wave][q16] = m;
            l_s[wave][q16] = l;
        }
#pragma unroll
        for (int i = 0; i < DT; ++i) *reinterpret_cast<f32x4 *>(&o_s[wave][q16][16 * i + 4 * g4]) = o[i];
        __syncthreads();
        for (int i = tid; i < kDecRows * D / 4; i += 64 * kDecWaves) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            if (r0 + row > last) continue;
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kDecWaves; ++w) top = fmaxf(top, m_s[w][row]);
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kDecWaves; ++w) {
                const float f = top == -INFINITY ? 1.0f : exp2_of(m_s[w][row] - top);
                sum += l_s[w][row] * f;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += o_s[w][row][d + e] * f;
            }
            const int64_t at = (int64_t)(seq.row0 + (r0 + row) / a.group) * a.Hq + head * a.group + (r0 + row) % a.group;
            if (a.splits == 1) {
                const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
                *reinterpret_cast<u32x2 *>(a.O + at * D + d) =
                    u32x2{bf16x2_bits(acc[0] * f, acc[1] * f), bf16x2_bits(acc[2] * f, acc[3] * f)};
                if (a.lse && d == 0) a.lse[at] = (top + log2f(sum)) * kLn2;
            } else {
                *reinterpret_cast<f32x4 *>(a.part + (at * a.splits + split) * D + d) = acc;
                if (d == 0) {
                    float *ml = a.part + (int64_t)a.kv.T * a.Hq * a.splits * D + (at * a.splits + split) * 2;
                    ml[0] = top;
                    ml[1] = sum;
                }
            }
        }
        __syncthreads();
    }
}

// The splits' sums of one query joined, by the waves of a block each a part.
template <int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    __shared__ float o_s[4][D], f_s[SVDQ_KV8_MAX_SPLITS];
    __shared__ float red[2][4];
    const int64_t at = (int64_t)blockIdx.x * a.Hq + blockIdx.y;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int first = min(max(a.kv.starts[0], 0), a.kv.T);
    if (row < first || row >= min(max(a.kv.starts[a.kv.B], first), a.kv.T)) return;
    const float *ml = a.part + (int64_t)a.kv.T * a.Hq * a.splits * D + at * a.splits * 2;
    float top = -INFINITY;
    for (int s = tid; s < a.splits; s += 256) top = fmaxf(top, ml[2 * s]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) red[0][wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float sum = 0.0f;
    for (int s = tid; s < a.splits; s += 256) {
        const float l = ml[2 * s + 1];
        const float f = top == -INFINITY ? 1.0f : exp2_of(ml[2 * s] - top);
        f_s[s] = l == 0.0f ? 0.0f : f;
        sum += l * f;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) red[1][wave] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    const float *src = a.part + at * a.splits * D + lane * E;
#pragma unroll 8
    for (int s = wave; s < a.splits; s += 4) {
        const float f = f_s[s];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(f, src[(int64_t)s * D + e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o_s[wave][lane * E + e] = acc[e];
    __syncthreads();
    if (tid < D / 2) {
        float v[2];
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int d = 2 * tid + e;
            v[e] = ((o_s[0][d] + o_s[1][d]) + (o_s[2][d] + o_s[3][d])) * f;
        }
        reinterpret_cast<uint32_t *>(a.O + at * D)[tid] = bf16x2_bits(v[0], v[1]);
        if (a.lse && tid == 0) a.lse[at] = (top + log2f(sum)) * kLn2;
    }
}

// ---- many queries ----------------------------------------------------------

constexpr int kPreRows = 128;

// A block takes 128 queries, 32 a wave, and walks the pages that they see: a page
// goes to LDS as bf16, by all threads, into one of two buffers while the other is
// read; its loads are under way a page earlier.
template <int D>
__global__ __launch_bounds__(256, 2) void kv8_prompt_kernel(AttnArgs a) {
    constexpr int KS = D / 16, DT = D / 32, KCH = D / 8, BPT = D / 4;  // BPT: bytes of a page per thread
    struct Stage {
        u32x4 k[kKvPage * KCH];
        u32x4 v[D * 8];
    };
    __shared__ Stage stage[2];
    __shared__ uint32_t nan_s[2][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q32 = lane & 31, h = lane >> 5;
    const int head = blockIdx.y;
    int b, tile;
    const int group = a.group;
    if (!kv_find(a.kv, blockIdx.x, b, tile, [=](const KvSeq &s) { return (s.rows * group + kPreRows - 1) / kPreRows; }))
        return;
    b = __builtin_amdgcn_readfirstlane(b);
    const KvSeq seq = kv_seq(a.kv, b);
    const int rows = seq.rows * group;
    tile = (rows + kPreRows - 1) / kPreRows - 1 - __builtin_amdgcn_readfirstlane(tile);  // the longest first
    const int r0 = tile * kPreRows, last = min(r0 + kPreRows, rows) - 1;
    const int wr0 = min(r0 + 32 * wave, last), wlast = min(wr0 + 31, last);
    const int r = min(wr0 + q32, last);
    int low, high, low0, high0, low1, high1, wlow0, whigh0, wlow1, whigh1;
    kv_seen(a, seq, r / group, low, high);
    kv_seen(a, seq, r0 / group, low0, high0);
    kv_seen(a, seq, last / group, low1, high1);
    kv_seen(a, seq, wr0 / group, wlow0, whigh0);
    kv_seen(a, seq, wlast / group, wlow1, whigh1);
    const int p0 = low0 / kKvPage, p1 = (high1 + kKvPage - 1) / kKvPage;

    bf16x8 q[KS];
    {
        const uint16_t *src = a.Q + (int64_t)(seq.row0 + r / group) * a.q_stride +
                              (int64_t)(head * group + r % group) * D + 8 * h;
#pragma unroll
        for (int i = 0; i < KS; ++i) q[i] = bitcast<bf16x8>(src + 16 * i);
    }
    float m = -INFINITY, l = 0.0f;
    f32x16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;

    // this thread's part of a page: BPT bytes of key tid / 4 and of a row of V^T
    u32x4 kr[BPT / 16], vr[BPT / 16];
    float ks = 0.0f, vs = 0.0f;
    int page = -1;
    auto fetch = [&](int p) __attribute__((always_inline)) {
        page = p < p1 ? kv_page(a.kv, b, p) : -1;
        if (page < 0) return;
        const int64_t unit = (int64_t)page * a.Hk + head;
        ks = a.ks[unit];
        vs = a.vs[unit];
        const uint8_t *kp = a.kc + unit * kKvPage * D + tid * BPT, *vp = a.vc + unit * kKvPage * D + tid * BPT;
#pragma unroll
        for (int i = 0; i < BPT / 16; ++i) {
            kr[i] = bitcast<u32x4>(kp + 16 * i);
            vr[i] = bitcast<u32x4>(vp + 16 * i);
        }
    };
    const int krow = tid / 4, kch = tid % 4 * (BPT / 8), vrow = tid * BPT / 64, vch = tid * BPT % 64 / 8;
    // matrix-core row i of a tile of 32 keys is token 16 (i / 16) + 8 (i / 4 % 2) + 4 (i / 8 % 2) + i % 4
    const int key = 16 * (q32 >> 4) + 8 * (q32 >> 2 & 1) + 4 * (q32 >> 3 & 1) + (q32 & 3);

    fetch(p0);
    int buf = 0;
    for (int p = p0; p < p1; ++p) {
        if (page < 0) {
            fetch(p + 1);
            continue;
        }
        const int t0 = p * kKvPage;
        Stage &st = stage[buf];
        // a page that some query does not see whole (see the kernel above)
        const bool cut = t0 < low1 || t0 + kKvPage > high0;
        if (cut) {
            uint32_t nan = 0;
#pragma unroll
            for (int i = 0; i < BPT / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    vr[i][j] &= byte_mask(t0 + 8 * vch + 16 * i + 4 * j, low0, high1);
                    nan |= nan_codes(vr[i][j]);
                }
            const bool any = __any(nan != 0);
            if (lane == 0) nan_s[buf][wave] = any;
        }
#pragma unroll
        for (int i = 0; i < BPT / 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                st.k[krow * KCH + ((kch + 2 * i + j) ^ (krow & 7))] =
                    __builtin_bit_cast(u32x4, fp8_widen8(kr[i][2 * j], kr[i][2 * j + 1]));
                st.v[vrow * 8 + ((vch + 2 * i + j) ^ (vrow & 7))] =
                    __builtin_bit_cast(u32x4, fp8_widen8(vr[i][2 * j], vr[i][2 * j + 1]));
            }
        const float c = ks * a.scale, vscale = vs;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's part is in LDS
        fp8_barrier();
        fetch(p + 1);
        const bool slow = cut && (nan_s[buf][0] | nan_s[buf][1] | nan_s[buf][2] | nan_s[buf][3]);
        buf ^= 1;
        if (t0 >= whigh1 || t0 + kKvPage <= wlow0) continue;  // none of this wave's queries sees it

        f32x16 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
                s[t] = mfma_bf16_32x32x16(
                    __builtin_bit_cast(bf16x8, st.k[(32 * t + key) * KCH + ((2 * i + h) ^ (key & 7))]), q[i], s[t]);
        }
        if (t0 < wlow1 || t0 + kKvPage > whigh0) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int at = t0 + 32 * t + 16 * (e >> 3) + 8 * h + (e & 7);
                    s[t][e] = at >= low && at < high ? s[t][e] : -INFINITY;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][e]);
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top * c);
        const float base = m_new == -INFINITY ? 0.0f : m_new;
        const float alpha = exp2_of(m - base);
        m = m_new;
        l *= alpha;
        bf16x8 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = exp2_of(__builtin_fmaf(s[u >> 1][8 * (u & 1) + e], c, -base));
                l += x[e];
            }
            w[u] = pack8(x, vscale);
        }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] *= alpha;
        auto value = [&](int i, int u) __attribute__((always_inline)) {
            const int d = 32 * i + q32;
            return __builtin_bit_cast(bf16x8, st.v[d * 8 + ((2 * u + h) ^ (d & 7))]);
        };
        if (!slow) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < DT; ++i) o[i] = mfma_bf16_32x32x16(value(i, u), w[u], o[i]);
        } else {
#pragma unroll
            for (int i = 0; i < DT; ++i) {
                f32x16 count;
#pragma unroll
                for (int e = 0; e < 16; ++e) count[e] = 0.0f;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int at = t0 + 16 * u + 8 * h;
                    u32x4 see;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        see[e] = (at + 2 * e >= low && at + 2 * e < high ? 0x3F80u : 0u) |
                                 (at + 2 * e + 1 >= low && at + 2 * e + 1 < high ? 0x3F800000u : 0u);
                    bf16x8 v = value(i, u), nan;
                    split_nan(v, nan);
                    count = mfma_bf16_32x32x16(nan, __builtin_bit_cast(bf16x8, see), count);
                    o[i] = mfma_bf16_32x32x16(v, w[u], o[i]);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] = count[e] > 0.0f ? NAN : o[i][e];
            }
        }
    }
    l += __shfl_xor(l, 32);
    if (wr0 + q32 > wlast || r0 + 32 * wave > last) return;
    const int64_t at = (int64_t)(seq.row0 + r / group) * a.Hq + head * group + r % group;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<u32x2 *>(a.O + at * D + 32 * i + 8 * e + 4 * h) =
                u32x2{bf16x2_bits(o[i][4 * e] * f, o[i][4 * e + 1] * f),
                      bf16x2_bits(o[i][4 * e + 2] * f, o[i][4 * e + 3] * f)};
    if (a.lse && h == 0) a.lse[at] = (m + log2f(l)) * kLn2;
}

// Few queries per sequence and key head on average: the kernel that splits pages.
bool few_queries(int T, int B, int group) { return (int64_t)T * group <= (int64_t)kDecRows * B; }

// Blocks that share a sequence's pages: as many as give the chip four blocks per
// compute unit, a page for each wave at the least.
int split_count(int B, int Hk, int max_pages) {
    const int64_t want = (1024 + (int64_t)B * Hk - 1) / ((int64_t)B * Hk);
    const int64_t most = (max_pages + kDecWaves - 1) / kDecWaves;
    return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, SVDQ_KV8_MAX_SPLITS}));
}

}  // namespace

size_t kv8_attention_workspace(int T, int B, int max_pages, int Hq, int Hk, int D) {
    if (T == 0 || B == 0 || !few_queries(T, B, Hq / Hk)) return 0;
    const int splits = split_count(B, Hk, max_pages);
    return splits == 1 ? 0 : (size_t)T * Hq * splits * (D + 2) * sizeof(float);
}

hipError_t launch_kv8_attention(const KvBatch &kv, const uint16_t *Q, int64_t q_stride, const uint8_t *kc,
                                const float *ks, const uint8_t *vc, const float *vs, int Hq, int Hk, int D, float scale,
                                bool causal, int window, uint16_t *O, float *lse, void *workspace, hipStream_t stream) {
    AttnArgs a{kv, Q,  q_stride, kc,  vc, ks, vs, Hq, Hk, Hq / Hk, scale * 1.44269504088896340736f, causal, window,
               O,  lse, static_cast<float *>(workspace), 1};
    if (few_queries(kv.T, kv.B, a.group)) {
        a.splits = split_count(kv.B, Hk, kv.max_pages);
        hipLaunchKernelGGL(D == 64 ? kv8_decode_kernel<64> : kv8_decode_kernel<128>,
                           dim3((unsigned)a.splits, (unsigned)Hk, (unsigned)kv.B), dim3(64 * kDecWaves), 0, stream, a);
        if (a.splits == 1) return hipGetLastError();
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(D == 64 ? kv8_join_kernel<64> : kv8_join_kernel<128>, dim3((unsigned)kv.T, (unsigned)Hq),
                           dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    const int64_t tiles = ((int64_t)kv.T * a.group + (int64_t)(kPreRows - 1) * kv.B) / kPreRows;
    hipLaunchKernelGGL(D == 64 ? kv8_prompt_kernel<64> : kv8_prompt_kernel<128>, dim3((unsigned)tiles, (unsigned)Hk),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace svdq
