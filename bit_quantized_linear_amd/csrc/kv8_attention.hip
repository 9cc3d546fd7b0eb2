// Attention of a batch's newest tokens over the 8-bit key and value cache.
//
//   o[q] = sum_t softmax_t(scale q . k_t) v_t   over the tokens t that q sees
//
// in one pass over the pages with a running maximum and sum: for a page with
// scores s_t (base-2 logarithms, the page's key scale among their factors)
//   m' = max(m, max s_t),  p_t = 2^(s_t - m'),  l' = l 2^(m - m') + sum p_t,
//   O' = O 2^(m - m') + sum (p_t vs) v_t
// with vs the page's value scale. Products run on the bf16 matrix core: E4M3
// codes are exact in bf16, p vs is rounded to bf16 (2^-8 of each weight at most; vs
// is a power of two), sums and statistics are fp32.
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
#include <type_traits>

#include "device_common.h"
#include "fp8_common.h"
#include "internal.h"
#include "kv8_common.h"

namespace svdq {

namespace {

constexpr float kLn2 = 0.69314718055994530942f;
// Of scores: a page's key scale may be 0, a hidden score -infinity. The least number there
// is: large queries and a small scale have factors below the smallest normal one
constexpr float kLeastFactor = 0x1p-149f;

constexpr uint32_t kNanCodes = 0x7F7F7F7Fu;  // those of a page whose scale is no number
constexpr int kInfinityBits = 0x7F800000;    // all set in infinities and NaN

// The factor of a page's scores, or -1 where its key scale is no number (or the product
// overflows): the scores of its tokens are NaN then, for those who see them, and 1 serves.
// NaN as a factor would reach the others through the scores that a mask has made -infinity.
__device__ __forceinline__ float score_factor(float ks, float scale) {
    const float f = ks * scale;
    return fabsf(f) < INFINITY ? fmaxf(f, kLeastFactor) : -1.0f;
}

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
    bool sorted;  // prompts: tiles in the order of all sequences' pages
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
constexpr int kDecRows = 16;  // of a matrix-core tile
constexpr int kMostSequences = 65535;  // of a call, and of a grid's last dimension

// A block takes up to 16, 32 or 64 queries of a sequence and a run of its
// pages, its waves every fourth of them (or every second, half of the queries each),
// straight into registers: the next page's keys as soon as this one's scores are
// there, its values as soon as this one's are multiplied. A wave takes QT tiles of 16
// queries, one after the other up to their weights, then each value to all of them.
// The numbers and scales of a wave's next 64 pages are in its lanes, the queries in
// LDS. The waves' sums are joined in LDS and, where a sequence's pages are split over
// blocks, by a second kernel.
// HBM-bound: 2 D bytes a token and key head, read once. 32 sequences of up to 8191
// tokens, 8 heads of 128: 61 us, 5.2 TB/s (a large copy: 5.15); one token after
// 32759 in 32 parts: 14.7 us, 4.6 TB/s, of which a block's start (its sequence, page
// numbers, first keys, each waiting for the last) is 3 to 4. With 64 queries a head
// 130 us: 2 waves a SIMD work out weights as long as they wait for keys.
template <int D, int QT, int WR>
__global__ __launch_bounds__(64 * kDecWaves, 2) void kv8_decode_kernel(AttnArgs a) {
    constexpr int KC = D / 64;  // 64-byte pieces of a key
    constexpr int DT = D / 16;  // 16-row tiles of V^T
    constexpr int kRows = kDecRows * QT * WR, kStride = kDecWaves / WR;
    static_assert(QT <= kStride, "one wave for each tile of queries");
    __shared__ __align__(16) float o_s[kDecWaves][kDecRows][D + 4];
    __shared__ u32x4 q_s[WR * QT][2 * KC][64];
    __shared__ float m_s[kDecWaves][kDecRows], l_s[kDecWaves][kDecRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q16 = lane & 15, g4 = lane >> 4;
    const int split = blockIdx.x;
    const int wp = wave / WR, wr = wave % WR * QT;  // which pages are the wave's, and the first of its tiles
    // The first queries of each sequence, then the others of those that have more (256
    // tokens among 31 of one each, after 4000, 32 / 8 heads: 111 us, 946 where a
    // sequence's queries are one block's)
    int head = blockIdx.y, b = blockIdx.z, r0 = 0;
    if (head >= a.Hk) {
        head -= a.Hk;
        b += kMostSequences;
    }
    KvSeq seq;
    if (b < a.kv.B) {
        seq = kv_seq(a.kv, b);
    } else {
        int nth;
        if (!kv_find(a.kv, b - a.kv.B, b, seq, nth, [&](const KvSeq &s) { return max(s.rows * a.group - 1, 0) / kRows; })) return;
        r0 = (nth + 1) * kRows;
    }
    const int rows = seq.rows * a.group;
    if (r0 >= rows) return;
    const int last = min(r0 + kRows, rows) - 1;
    int low[QT], high[QT], low0, high0, low1, high1;
#pragma unroll
    for (int t = 0; t < QT; ++t) kv_seen(a, seq, min(r0 + kDecRows * (wr + t) + q16, last) / a.group, low[t], high[t]);
    kv_seen(a, seq, r0 / a.group, low0, high0);
    kv_seen(a, seq, last / a.group, low1, high1);
    // low0 <= low[t] <= low1 and high0 <= high[t] <= high1
    const int first_page = low0 / kKvPage, pages = max(0, (high1 + kKvPage - 1) / kKvPage - first_page);
    const int per = (pages + a.splits - 1) / a.splits;
    const int p0 = first_page + split * per, p1 = min(p0 + per, first_page + pages);

    if (wp < QT) {  // a tile's queries to LDS
        const int r = min(r0 + kDecRows * (wr + wp) + q16, last);
        const uint16_t *src = a.Q + (int64_t)(seq.row0 + r / a.group) * a.q_stride +
                              (int64_t)(head * a.group + r % a.group) * D + 16 * g4;
#pragma unroll
        for (int i = 0; i < 2 * KC; ++i) q_s[wr + wp][i][lane] = bitcast<u32x4>(src + 64 * (i / 2) + 8 * (i & 1));
    }
    __syncthreads();
    float m[QT], l[QT];
    f32x4 o[QT][DT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // lane i: page p0 + wp + kStride (first + i) of the sequence
    int number = -1, first = 0;
    float factor = 0.0f, vs = 0.0f;
    auto look_up = [&](int from) __attribute__((always_inline)) {
        first = from;
        const int p = p0 + wp + kStride * (from + lane);
        number = p < p1 ? kv_page(a.kv, b, p) : -1;
        const int64_t unit = (int64_t)max(number, 0) * a.Hk + head;
        factor = score_factor(a.ks[unit], a.scale);
        vs = number >= 0 ? a.vs[unit] : 0.0f;
    };
    u32x4 k[4][KC], v[DT];
    auto unit_of = [&](int i) {
        return (int64_t)max(__builtin_amdgcn_readlane(number, i - first), 0) * a.Hk + head;
    };
    auto load_keys = [&](int i) __attribute__((always_inline)) {
        const uint8_t *kp = a.kc + unit_of(i) * kKvPage * D;
        // tile j's row i is token 16 (i / 4) + 4 j + i % 4
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < KC; ++n)
                k[j][n] = bitcast<u32x4>(kp + (16 * (q16 >> 2) + 4 * j + (q16 & 3)) * D + 64 * n + 16 * g4);
    };
    auto load_values = [&](int i) __attribute__((always_inline)) {
        const uint8_t *vp = a.vc + unit_of(i) * kKvPage * D;
#pragma unroll
        for (int n = 0; n < DT; ++n) v[n] = bitcast<u32x4>(vp + (16 * n + q16) * kKvPage + 16 * g4);
    };
    const int count = p1 > p0 + wp ? (p1 - p0 - wp + kStride - 1) / kStride : 0;
    if (count > 0) {
        look_up(0);
        load_keys(0);
        // the loop's order: its waits for keys then leave values under way (67 us against 72, 32 sequences)
        __builtin_amdgcn_sched_barrier(0);
        load_values(0);
    }
    for (int i = 0; i < count; ++i) {
        const int p = p0 + wp + kStride * i;
        const bool there = __builtin_amdgcn_readlane(number, i - first) >= 0, more = i + 1 < count;
        const int c_bits = __builtin_amdgcn_readlane(__float_as_int(factor), i - first);
        const bool lost = c_bits < 0;
        const float c = __int_as_float(c_bits & 0x7FFFFFFF);
        const int v_bits = __builtin_amdgcn_readlane(__float_as_int(vs), i - first);
        const bool lost_values = (v_bits & kInfinityBits) == kInfinityBits;
        const float vscale = lost_values ? 1.0f : __int_as_float(v_bits);
        const int t0 = p * kKvPage;
        // a page that some query does not see whole: hidden tokens' weights are
        // 0, and their values are not multiplied, as they may be NaN. Of a page
        // that is not there, all are hidden. Scores or values that are NaN take this path as well
        const bool cut = !there || lost || lost_values || t0 < low1 || t0 + kKvPage > high0;
        uint32_t nan = 0;
        bf16x8 w[QT][2];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            f32x4 s[4];
            bf16x8 q[2 * KC];
#pragma unroll
            for (int n = 0; n < 2 * KC; ++n) q[n] = __builtin_bit_cast(bf16x8, q_s[wr + t][n][lane]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                __builtin_amdgcn_sched_barrier(0);  // few converted operands at a time: registers
                s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int n = 0; n < KC; ++n) {
                    s[j] = mfma_bf16_16x16x32(fp8_widen8(k[j][n][0], k[j][n][1]), q[2 * n], s[j]);
                    s[j] = mfma_bf16_16x16x32(fp8_widen8(k[j][n][2], k[j][n][3]), q[2 * n + 1], s[j]);
                }
            }
            if (QT > 1) __builtin_amdgcn_sched_barrier(0);
            if (t < QT - 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int n = 0; n < KC; ++n) asm volatile("" : "+v"(k[j][n]));  // widened again for each tile: registers
            } else if (more) {
                if (i + 1 - first == 64) look_up(i + 1);
                load_keys(i + 1);
            }
            if (cut) {
                if (t == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t mask = byte_mask(t0 + 16 * g4 + 4 * j, low0, there ? high1 : 0);
#pragma unroll
                        for (int n = 0; n < DT; ++n) {
                            if (lost_values) v[n][j] = kNanCodes;
                            v[n][j] &= mask;
                            nan |= nan_codes(v[n][j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t see = byte_mask(t0 + 16 * g4 + 4 * j, low[t], there ? high[t] : 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[j][e] = see >> (8 * e) & 1 ? (lost ? NAN : s[j][e]) : -INFINITY;
                }
            }
            float top = s[0][0];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, s[j][e]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m_new = fmaxf(m[t], top * c);
            const float base = m_new == -INFINITY ? 0.0f : m_new;
            const float alpha = exp2_of(m[t] - base);
            m[t] = m_new;
            l[t] *= alpha;
#pragma unroll
            for (int n = 0; n < DT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][n][e] *= alpha;
            float x[16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[4 * j + e] = exp2_of(__builtin_fmaf(s[j][e], c, -base));
                    l[t] += x[4 * j + e];
                }
            w[t][0] = pack8(x, vscale);
            w[t][1] = pack8(x + 8, vscale);
        }
        if (__any(nan != 0)) {  // NaN reaches the queries that see its token, and no other
#pragma unroll
            for (int n = 0; n < DT; ++n) {
                u32x4 one;  // the code of 1 for each NaN, which becomes 0 itself
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = (nan_codes(v[n][j]) >> 7) * 0xFFu;
                    one[j] = at & 0x38383838u;
                    v[n][j] &= ~at;
                }
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    __builtin_amdgcn_sched_barrier(0);
                    f32x4 count = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        u32x4 seen;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t two = byte_mask(t0 + 16 * g4 + 8 * u + 2 * e, low[t], high[t]);
                            seen[e] = (two & 1 ? 0x3F80u : 0u) | (two & 0x100u ? 0x3F800000u : 0u);
                        }
                        count = mfma_bf16_16x16x32(fp8_widen8(one[2 * u], one[2 * u + 1]),
                                                   __builtin_bit_cast(bf16x8, seen), count);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][n][e] = count[e] > 0.0f ? NAN : o[t][n][e];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < DT; ++n) {
            if (QT > 1 || n % 2 == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 value = fp8_widen8(v[n][2 * u], v[n][2 * u + 1]);
#pragma unroll
                for (int t = 0; t < QT; ++t) o[t][n] = mfma_bf16_16x16x32(value, w[t][u], o[t][n]);
            }
        }
        if (more) load_values(i + 1);
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {  // the waves' sums of a tile
        const int first_row = r0 + kDecRows * t;
        if (first_row > last) break;
        l[t] += __shfl_xor(l[t], 16);
        l[t] += __shfl_xor(l[t], 32);
        if (g4 == 0) {
            m_s[wave][q16] = m[t];
            l_s[wave][q16] = l[t];
        }
#pragma unroll
        for (int i = 0; i < DT; ++i) *reinterpret_cast<f32x4 *>(&o_s[wave][q16][16 * i + 4 * g4]) = o[t][i];
        __syncthreads();
        for (int i = tid; i < WR * kDecRows * D / 4; i += 64 * kDecWaves) {
            const int part = i / (kDecRows * D / 4), row = i / (D / 4) % kDecRows, d = i % (D / 4) * 4;
            const int r = first_row + kDecRows * QT * part + row;
            if (r > last) continue;
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = part; w < kDecWaves; w += WR) top = fmaxf(top, m_s[w][row]);
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = part; w < kDecWaves; w += WR) {
                const float f = top == -INFINITY ? 1.0f : exp2_of(m_s[w][row] - top);
                sum += l_s[w][row] * f;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += o_s[w][row][d + e] * f;
            }
            const int64_t at = (int64_t)(seq.row0 + r / a.group) * a.Hq + head * a.group + r % a.group;
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

// The parts' sums of a query joined: by a wave, where it has at most 8 parts, or by
// the W waves of a block. What is read does not depend on what is read before, so
// that one wait covers all: 3 to 4 us for 32 queries, an empty launch 2 to 3.
constexpr int kJoinAlone = 8;

template <int D, int W>
__global__ __launch_bounds__(256) void kv8_join_kernel(AttnArgs a) {
    constexpr int E = D / 64, kEach = W == 1 ? kJoinAlone : SVDQ_KV8_MAX_SPLITS / W;
    __shared__ float o_s[W == 1 ? 1 : W][D];
    const int lane = threadIdx.x & 63, wave = W == 1 ? 0 : threadIdx.x >> 6;
    const int64_t at = W == 1 ? 4 * (int64_t)blockIdx.x + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
    if (at >= (int64_t)a.kv.T * a.Hq) return;
    const int row = (int)(at / a.Hq);
    const float *src = a.part + at * a.splits * D + lane * E;
    float x[kEach][E];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = W * i + wave < a.splits ? src[(int64_t)(W * i + wave) * D + e] : 0.0f;
    const float *ml = a.part + (int64_t)a.kv.T * a.Hq * a.splits * D + at * a.splits * 2;
    const float m = lane < a.splits ? ml[2 * lane] : -INFINITY, l = lane < a.splits ? ml[2 * lane + 1] : 0.0f;
    const int first = min(max(a.kv.starts[0], 0), a.kv.T);
    const int last = min(max(a.kv.starts[a.kv.B], first), a.kv.T);
    float top = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float f = top == -INFINITY ? 1.0f : exp2_of(m - top);
    const float weight = l == 0.0f ? 0.0f : f;  // a part of nothing
    float sum = l * weight;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const float w = __shfl(weight, (W * i + wave) & 63);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(w, x[i][e], acc[e]);
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) o_s[wave][lane * E + e] = acc[e];
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[e] = o_s[0][lane * E + e];
#pragma unroll
            for (int w = 1; w < W; ++w) acc[e] += o_s[w][lane * E + e];
        }
    }
    // A row from the first start up to the last one is some sequence's. Others mostly are
    // none's; but starts may fall, behind the last sequence for instance, and then all say
    if (row < first || row >= last) {
        bool found = false;
        for (int b = lane; b < a.kv.B; b += 64) {
            const KvSeq s = kv_seq(a.kv, b);
            found |= row >= s.row0 && row < s.row0 + s.rows;
        }
        if (!__any(found)) return;
    }
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *out = a.O + at * D + lane * E;
    if constexpr (E == 2)
        *reinterpret_cast<uint32_t *>(out) = bf16x2_bits(acc[0] * r, acc[1] * r);
    else
        *out = (uint16_t)bf16x2_bits(acc[0] * r, 0.0f);
    if (a.lse && lane == 0) a.lse[at] = (top + log2f(sum)) * kLn2;
}

// ---- many queries ----------------------------------------------------------

// 8 codes as bf16 values times a page's scale, a power of two, which goes into the
// conversion; and times another scale (of a cache filled elsewhere), for a rounding.
__device__ __forceinline__ u32x4 widen_scaled(u32x2 v, float scale) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], scale, false));
        w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], scale, true));
    }
    return w;
}

__device__ __forceinline__ u32x4 widen_rounded(u32x2 v, float scale) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = (int)v[i];
        w[2 * i] = bf16x2_bits(__builtin_amdgcn_cvt_f32_fp8(x, 0) * scale, __builtin_amdgcn_cvt_f32_fp8(x, 1) * scale);
        w[2 * i + 1] = bf16x2_bits(__builtin_amdgcn_cvt_f32_fp8(x, 2) * scale, __builtin_amdgcn_cvt_f32_fp8(x, 3) * scale);
    }
    return w;
}

__device__ __forceinline__ bool power_of_two(float x) { return !(__float_as_uint(x) & 0x807FFFFFu) && x > 0.0f && x < INFINITY; }

// The larger of a lane's and the other half wave's value.
__device__ __forceinline__ float max_of_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

constexpr float kRise = 6.0f;  // how far, in powers of two, a score may pass the base that weights are taken to

// The sum of a wave's values: of 16 lanes each by rotations, of the four rows by hand.
__device__ __forceinline__ int wave_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);   // lane ^ 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);   // lane ^ 2
    v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);  // 7 - lane, of 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);  // 15 - lane, of 16
    return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
           __builtin_amdgcn_readlane(v, 48);
}

// kv_find for the tiles of up to 64 sequences in the order of the pages that they see
// (windows apart), the longest first: the last blocks of a launch are then short
// ones. Tile k of a sequence sees at least P pages from a k on that is easily worked
// out; a search over P finds the item's.
__device__ __forceinline__ bool find_longest(const AttnArgs &a, int item, int tile_rows, int &b, KvSeq &seq, int &tile) {
    const int lane = threadIdx.x & 63;
    const KvSeq mine = kv_seq(a.kv, min(lane, a.kv.B - 1));
    const int rows = lane < a.kv.B ? mine.rows * a.group : 0, tiles = (rows + tile_rows - 1) / tile_rows;
    // the first tile that sees at least `pages` pages
    auto first_with = [&](int pages) {
        if (!a.causal) return mine.length > (pages - 1) * kKvPage ? 0 : tiles;
        const int token = max(0, (pages - 1) * kKvPage - (mine.length - mine.rows));  // the first that does
        return token < mine.rows ? min(tiles, max(0, (a.group * token + tile_rows) / tile_rows - 1)) : tiles;
    };
    if (item >= wave_sum(tiles)) return false;
    // low: at least item + 1 tiles see so many pages, high: they do not
    int low = 0, high = a.kv.max_pages + 1;
    while (high - low > 1) {
        const int mid = low + (high - low) / 2;
        if (wave_sum(tiles - first_with(mid)) > item)
            low = mid;
        else
            high = mid;
    }
    const int from = low > 0 ? first_with(low) : 0, n = first_with(low + 1) - from;
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int other = __shfl_up(upto, d);
        upto += lane >= d ? other : 0;
    }
    item -= wave_sum(tiles - first_with(low + 1));
    b = __ffsll((unsigned long long)__ballot(item < upto)) - 1;
    seq.row0 = __builtin_amdgcn_readlane(mine.row0, b);
    seq.rows = __builtin_amdgcn_readlane(mine.rows, b);
    seq.length = __builtin_amdgcn_readlane(mine.length, b);
    tile = __builtin_amdgcn_readlane(from, b) + item - __builtin_amdgcn_readlane(upto - n, b);
    return true;
}

constexpr int kPreInfo = 512;  // pages whose numbers and scales are in LDS at a time

// A block takes 32 queries a wave and walks the pages that they see, or its part of
// them, in steps of 32 tokens. A page goes to LDS as bf16, by all threads, a page
// before it is read, its loads a page earlier; its number and scales are read for
// 512 pages at once, so that no load waits for another in the loop.
// Pages that every query of the block sees whole are pipelined: a step multiplies
// the next step's scores and the last one's weights while it works out its own
// weights, three things that do not wait for each other. The base of the weights
// (m above) is a whole number and rises only where a score passes it by more than
// kRise: weights are then below 2^kRise, and what is multiplied when it does rise
// (O, l and the weights not yet multiplied) is multiplied exactly.
// Bound by the matrix cores, at a clock set by power: 4680 queries over 32760 tokens,
// 40 heads of 128: 2.74 ms, 1145 TFLOP/s (the library's bf16 product of 8192^3: 1210
// to 1230). 8 waves of 32 queries, two a SIMD, as one wave's weights then overlap the
// other's products: one wave of 64 a SIMD took 3.2 ms. Prompts of three sequences, up
// to 2777 tokens after up to 1500: 236 to 240 us, 940 TFLOP/s; a block's start takes 6 to
// 7 us, its outputs 2, and pages with masks are not pipelined. 8192 tokens over themselves,
// 32 / 8 heads: 507 us, 1084 TFLOP/s, with a window of 1024 171 us, 753; heads of 64, whose
// products have half the work for the same weights: 341 us, 807 TFLOP/s.
// Waves a SIMD: two, where D = 64 in two blocks if they have 4 waves (100 queries after 1000
// of 16 sequences of 16 heads: 32.4 us, 36.5 with one); with D = 128 4 waves need the
// registers of one (with two, spilled: 49 against 39 us), and two blocks' LDS is not there.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 64 ? 2 : NW / 4) void kv8_prompt_kernel(AttnArgs a, int tiles) {
    constexpr int KS = D / 16, DT = D / 32, KCH = D / 8;
    constexpr int PC = D / 8 / NW;  // pieces of 8 codes of a page's keys, and of its values, per thread
    constexpr int kRows = 32 * NW;
    constexpr int KP = KCH + 1, VP = 9;  // pieces of 16 bytes from row to row in LDS: 8 rows at a piece fall on distinct banks
    __shared__ u32x4 k_s[2][kKvPage * KP];
    __shared__ u32x4 v_s[3][D * VP];
    __shared__ u32x4 info_s[kPreInfo];
    __shared__ uint32_t nan_s[3][NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q32 = lane & 31, h = lane >> 5;
    const int group = a.group;
    // Blocks are dealt to the 8 XCDs in turn: a head's tiles go to one of them, so
    // that its pages are read once per L2; the heads left over go to all
    int head, item;
    const int split = blockIdx.y;
    {
        const int whole = a.Hk / 8 * 8, id = blockIdx.x;
        if (id < whole * tiles) {
            head = id / (8 * tiles) * 8 + id % 8;
            item = id / 8 % tiles;
        } else {
            const int rest = a.Hk - whole, j = id - whole * tiles;
            head = whole + j % rest;
            item = j / rest;
        }
    }
    int b, tile;
    KvSeq seq;
    if (a.sorted) {
        if (!find_longest(a, item, kRows, b, seq, tile)) return;
    } else {
        if (!kv_find(a.kv, item, b, seq, tile, [=](const KvSeq &s) { return (s.rows * group + kRows - 1) / kRows; })) return;
        tile = (seq.rows * group + kRows - 1) / kRows - 1 - tile;  // a sequence's longest first
    }
    const int rows = seq.rows * group;
    const int r0 = tile * kRows, last = min(r0 + kRows, rows) - 1;
    const int row = min(r0 + 32 * wave + q32, last);
    int low, high, low0, high0, low1, high1;
    kv_seen(a, seq, row / group, low, high);
    kv_seen(a, seq, r0 / group, low0, high0);
    kv_seen(a, seq, last / group, low1, high1);
    // pages p0 .. p1 - 1 are this block's, of them f0 .. f1 - 1 seen whole by every query
    int p0 = low0 / kKvPage, p1 = (high1 + kKvPage - 1) / kKvPage;
    {
        const int per = (max(p1 - p0, 0) + a.splits - 1) / a.splits;
        p0 += split * per;
        p1 = min(p1, p0 + per);
    }
    const int f0 = (low1 + kKvPage - 1) / kKvPage, f1 = high0 / kKvPage;

    bf16x8 q[KS];
    {
        const uint16_t *src = a.Q + (int64_t)(seq.row0 + row / group) * a.q_stride +
                              (int64_t)(head * group + row % group) * D + 8 * h;
#pragma unroll
        for (int i = 0; i < KS; ++i) q[i] = bitcast<bf16x8>(src + 16 * i);
    }
    float base = -3.4028235e38f, l = 0.0f;
    f32x16 o[DT];
    auto zero = [](f32x16 &x) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.0f;
    };
#pragma unroll
    for (int i = 0; i < DT; ++i) zero(o[i]);

    // ---- pages to LDS ----
    // info_s: page number (-1: not there), the factor of its scores (-1: they are NaN), its
    // value scale, and whether it is plain: there, seen whole by every query, its scores
    // numbers, its value scale a power of two. Plain pages are what the pipelined steps take
    int info0 = 0;  // the page of info_s[0]
    auto load_info = [&](int from, int to) __attribute__((always_inline)) {
        info0 = from;
        for (int i = tid; i < to - from; i += 64 * NW) {
            const int p = from + i, page = kv_page(a.kv, b, p);
            u32x4 x = {(uint32_t)page, 0u, 0u, 0u};
            if (page >= 0) {
                const int64_t unit = (int64_t)page * a.Hk + head;
                const float ks = a.ks[unit], vs = a.vs[unit];
                const float factor = score_factor(ks, a.scale);
                x[1] = __float_as_uint(factor);
                x[2] = __float_as_uint(vs);
                x[3] = p >= f0 && p < f1 && factor > 0.0f && power_of_two(vs);
            }
            info_s[i] = x;
        }
    };
    // this thread's part of a page: PC pieces of a key and of a row of V^T
    u32x2 kr[PC], vr[PC];
    u32x4 held = {0u, 0u, 0u, 0u};  // info of the page in kr, vr
    auto fetch = [&](u32x4 info) __attribute__((always_inline)) {
        held = info;
        const int page = max(__builtin_amdgcn_readfirstlane((int)info[0]), 0);
        const int64_t unit = (int64_t)page * a.Hk + head;
        const uint8_t *kp = a.kc + unit * kKvPage * D + tid * PC * 8, *vp = a.vc + unit * kKvPage * D + tid * PC * 8;
        if constexpr (PC == 1) {
            kr[0] = bitcast<u32x2>(kp);
            vr[0] = bitcast<u32x2>(vp);
        } else {
#pragma unroll
            for (int i = 0; i < PC; i += 2) {
                const u32x4 k = bitcast<u32x4>(kp + 8 * i), v = bitcast<u32x4>(vp + 8 * i);
                kr[i] = u32x2{k[0], k[1]};
                kr[i + 1] = u32x2{k[2], k[3]};
                vr[i] = u32x2{v[0], v[1]};
                vr[i + 1] = u32x2{v[2], v[3]};
            }
        }
    };
    auto held_factor = [&]() __attribute__((always_inline)) { return fabsf(__uint_as_float(held[1])); };
    auto held_plain = [&]() __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane((int)held[3]) != 0; };
    // matrix-core row i of a tile of 32 keys is token 16 (i / 16) + 8 (i / 4 % 2) + 4 (i / 8 % 2) + i % 4, so that
    // element e of a lane's scores is token 16 (e / 8) + 8 h + e % 8: keys lie in LDS in that order
    const int token = tid * PC / KCH, krow = (token & 0x33) | (token & 8) >> 1 | (token & 4) << 1;
    const int k_at = krow * KP + tid * PC % KCH, v_at = tid * PC / 8 * VP + tid * PC % 8;
    // The page held to LDS, as page p.
    // Of a page that some query does not see whole, values that none sees become 0 (a
    // hidden token's weight is 0, but its value may be NaN), and it is noted whether
    // one of the others is NaN
    auto store = [&](int p, int ki, int vi) __attribute__((always_inline)) {
        const bool there = (int)held[0] >= 0;
        float vs = __uint_as_float(held[2]);
        if (!there) {
#pragma unroll
            for (int i = 0; i < PC; ++i) kr[i] = vr[i] = u32x2{0u, 0u};
        }
        if ((int)held[1] < 0) {
#pragma unroll
            for (int i = 0; i < PC; ++i) kr[i] = u32x2{kNanCodes, kNanCodes};
        }
        if (!(fabsf(vs) < INFINITY)) {  // codes, as a mask clears those
            vs = 1.0f;
#pragma unroll
            for (int i = 0; i < PC; ++i) vr[i] = u32x2{kNanCodes, kNanCodes};
        }
        if (p < f0 || p >= f1) {
            uint32_t nan = 0;
#pragma unroll
            for (int i = 0; i < PC; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    vr[i][j] &= byte_mask(p * kKvPage + tid * PC % 8 * 8 + 8 * i + 4 * j, low0, high1);
                    nan |= nan_codes(vr[i][j]);
                }
            const bool any = __any(nan != 0);
            if (lane == 0) nan_s[vi][wave] = any;
        } else if (lane == 0) {
            nan_s[vi][wave] = 0;
        }
        const bool two = power_of_two(vs);
#pragma unroll
        for (int i = 0; i < PC; ++i) {
            k_s[ki][k_at + i] = widen_scaled(kr[i], 1.0f);
            v_s[vi][v_at + i] = two ? widen_scaled(vr[i], vs) : widen_rounded(vr[i], there ? vs : 1.0f);
        }
    };
    // One of the 2 PC pieces of a plain page
    auto store_piece = [&](int n, int ki, int vi) __attribute__((always_inline)) {
        if (n < PC)
            k_s[ki][k_at + n] = widen_scaled(kr[n], 1.0f);
        else
            v_s[vi][v_at + n - PC] = widen_scaled(vr[n - PC], __uint_as_float(held[2]));
    };
    auto meet = [&]() __attribute__((always_inline)) {  // what this wave wrote is in LDS, and everyone is here
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        fp8_barrier();
    };

    // ---- a step of 32 tokens: half a page ----
    auto key = [&](int ki, int half, int i) __attribute__((always_inline)) {  // 8 features from 16 i on of 32 tokens
        return __builtin_bit_cast(bf16x8, k_s[ki][(32 * half + q32) * KP + 2 * i + h]);
    };
    auto value = [&](int vi, int half, int u, int i) __attribute__((always_inline)) {  // 8 tokens of 32 features
        return __builtin_bit_cast(bf16x8, v_s[vi][(32 * i + q32) * VP + 4 * half + 2 * u + h]);
    };
    auto top_of = [&](const f32x16 &s) __attribute__((always_inline)) {
        float m = fmaxf(s[0], s[1]);
#pragma unroll
        for (int e = 2; e < 16; e += 2) m = fmaxf(fmaxf(m, s[e]), s[e + 1]);
        return max_of_halves(m);
    };
    // The base raised to a step's largest score, what was taken to the old one
    // multiplied with the factor that is returned
    auto raise_to = [&](float top) __attribute__((always_inline)) {
        const float to = top > base ? ceilf(top) : base;
        const float f = exp2_of(base - to);
        base = to;
        l *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] *= f;
        return f;
    };
    auto raise = [&](float top, bf16x8 (&pending)[2]) __attribute__((always_inline)) {
        if (!__any(top > base + kRise)) return;
        const float f = raise_to(top);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            u32x4 w = __builtin_bit_cast(u32x4, pending[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = bf16x2_bits(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
            pending[u] = __builtin_bit_cast(bf16x8, w);
        }
    };
    // The pipelined step. It has KS + 2 DT parts, pinned in this order: each issues the
    // matrix-core instruction of one operand from LDS, fetches the operand kAhead
    // parts on, and does a share of everything else.
    //   s: this step's scores, whose weights go to w; c their factor
    //   sn, top: the next step's scores (keys kn, half hn) and their largest
    //   wp: the last step's weights (values vp, half hp)
    //   (ka, ha): the keys of the step after the next
    // kStage: store the page held to (ki, vi), meet the other waves, fetch the page of info_s[next]
    constexpr int kParts = KS + 2 * DT;
    constexpr int kAhead = D == 64 ? 3 : 5, kRing = 8;
    static_assert(kAhead <= 2 * DT && kParts % kRing == 0, "the page is stored before the waves meet");
    bf16x8 operand[kRing];
    auto step = [&](auto kStage, int ki, int vi, int next, const float (&s)[16], float c, bf16x8 (&w)[2], int kn, int hn,
                    float (&sn)[16], float &top, int vp, int hp, const bf16x8 (&wp)[2], int ka,
                    int ha) __attribute__((always_inline)) {
        float x[16], sum[2] = {0.0f, 0.0f}, most = -INFINITY;
        uint32_t packed[2][4];
        f32x16 acc;
        zero(acc);
        u32x4 info = held;
#pragma unroll
        for (int n = 0; n < kParts; ++n) {
            __builtin_amdgcn_sched_barrier(0);
            if (kStage && n == kParts - kAhead) meet();
            const int v = n - KS;
            if (n < KS)
                acc = mfma_bf16_32x32x16(operand[n % kRing], q[n], acc);
            else
                o[v % DT] = mfma_bf16_32x32x16(operand[n % kRing], wp[v / DT], o[v % DT]);
            const int r = n + kAhead, rv = r - KS;
            operand[r % kRing] = r < KS       ? key(kn, hn, r)
                                 : r < kParts ? value(vp, hp, rv / DT, rv % DT)
                                              : key(ka, ha, r - kParts);
            if (kStage && n == 0) info = info_s[next];
            if (kStage && n < KS) {
#pragma unroll
                for (int i = n * 2 * PC / KS; i < (n + 1) * 2 * PC / KS; ++i) store_piece(i, ki, vi);
            }
            if (kStage && n == KS) fetch(info);
            // this part's share of the 16 weights
#pragma unroll
            for (int e = n * 16 / kParts; e < (n + 1) * 16 / kParts; ++e) {
                x[e] = exp2_of(__builtin_fmaf(s[e], c, -base));
                sum[e & 1] += x[e];
                asm volatile("" : "+v"(x[e]), "+v"(sum[e & 1]));  // here, not later
                if (e & 1) {
                    packed[e / 8][e % 8 / 2] = bf16x2_bits(x[e - 1], x[e]);
                    asm volatile("" : "+v"(packed[e / 8][e % 8 / 2]));
                }
            }
            // and, from the second part behind the scores on, of the largest scores
            if (n > KS) {
                constexpr int kTopParts = kParts - KS - 1;
                const int at = n - KS - 1;
#pragma unroll
                for (int j = at * 8 / kTopParts; j < (at + 1) * 8 / kTopParts; ++j) {
                    sn[2 * j] = acc[2 * j];
                    sn[2 * j + 1] = acc[2 * j + 1];
                    most = fmaxf(fmaxf(most, sn[2 * j]), sn[2 * j + 1]);
                    asm volatile("" : "+v"(most));
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        l += sum[0] + sum[1];
        top = max_of_halves(most);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            w[u] = __builtin_bit_cast(bf16x8, u32x4{packed[u][0], packed[u][1], packed[u][2], packed[u][3]});
    };
    // A page, one thing after the other, with its masks
    auto cut_page = [&](int p, int ki, int vi, float c) __attribute__((always_inline)) {
        uint32_t slow = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) slow |= nan_s[vi][i];
        if (!(c > 0.0f)) return;
        // the tokens that the lane's query sees, counted as its elements are: count of them, from `from` on
        const int from = low - p * kKvPage - 8 * h;
        const uint32_t count = (uint32_t)max(high - low, 0);
        auto sees = [&](int half, int e) { return (uint32_t)(32 * half + 16 * (e >> 3) + (e & 7) - from) < count; };
        f32x16 s[2];
        zero(s[0]);
        zero(s[1]);
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) s[half] = mfma_bf16_32x32x16(key(ki, half, i), q[i], s[half]);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[half][e] = sees(half, e) ? s[half][e] : -INFINITY;
        const float top = fmaxf(top_of(s[0]), top_of(s[1])) * c;
        if (__any(top > base + kRise)) raise_to(top);
        bf16x8 w[2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = exp2_of(__builtin_fmaf(s[half][8 * u + e], c, -base));
                    l += x[e];
                }
                w[half][u] = pack8(x, 1.0f);
            }
        if (!slow) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < DT; ++i) o[i] = mfma_bf16_32x32x16(value(vi, half, u, i), w[half][u], o[i]);
            return;
        }
        // NaN reaches the queries that see its token, and no other
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            bf16x8 seen[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                u32x4 see;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    see[e] = (sees(half, 8 * u + 2 * e) ? 0x3F80u : 0u) | (sees(half, 8 * u + 2 * e + 1) ? 0x3F800000u : 0u);
                seen[u] = __builtin_bit_cast(bf16x8, see);
            }
#pragma unroll
            for (int i = 0; i < DT; ++i) {
                __builtin_amdgcn_sched_barrier(0);  // one tile at a time: registers
                f32x16 nans;
                zero(nans);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    bf16x8 v = value(vi, half, u, i), nan;
                    split_nan(v, nan);
                    nans = mfma_bf16_32x32x16(nan, seen[u], nans);
                    o[i] = mfma_bf16_32x32x16(v, w[half][u], o[i]);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] = nans[e] > 0.0f ? NAN : o[i][e];
            }
        }
    };

    for (int s0 = p0; s0 < p1; s0 += kPreInfo) {
        const int s1 = min(p1, s0 + kPreInfo);
        if (s0 > p0) meet();  // the last run's pages have been read
        load_info(s0, s1);
        meet();
        // Page p is in k_s[kc], v_s[vc], its factor is c and `plain` says what it is; page p + 1 is held
        int kc = 0, vc = 0;
        const auto after = [&](int v) { return v == 2 ? 0 : v + 1; };
        const auto info_at = [&](int p) { return min(p, s1 - 1) - info0; };
        fetch(info_s[0]);
        float c = held_factor();
        bool plain = held_plain();
        store(s0, kc, vc);
        fetch(info_s[info_at(s0 + 1)]);
        meet();
        for (int p = s0; p < s1; ++p) {
            if (plain && p + 1 < s1 && held_plain()) {
                float t0[16], t1[16], top0, top1;
                bf16x8 w0[2], w1[2] = {};
                {
                    f32x16 x;
                    zero(x);
#pragma unroll
                    for (int i = 0; i < KS; ++i) x = mfma_bf16_32x32x16(key(kc, 0, i), q[i], x);
                    top0 = top_of(x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) t0[e] = x[e];
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) operand[i] = key(kc, 1, i);
                int vw = vc;  // the values of w1 (at first zeros: any page that all see)
                do {
                    const float cn = held_factor();
                    const int vn = after(vc);
                    raise(top0 * c, w1);
                    step(std::true_type(), kc ^ 1, vn, info_at(p + 2), t0, c, w0, kc, 1, t1, top1, vw, 1, w1, kc ^ 1, 0);
                    raise(top1 * c, w0);
                    step(std::false_type(), 0, 0, 0, t1, c, w1, kc ^ 1, 0, t0, top0, vc, 0, w0, kc ^ 1, 1);
                    vw = vc;
                    vc = vn;
                    kc ^= 1;
                    c = cn;
                    ++p;
                } while (p + 1 < s1 && held_plain());
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < DT; ++i) o[i] = mfma_bf16_32x32x16(value(vw, 1, u, i), w1[u], o[i]);
            }
            const float cn = held_factor();
            const int vn = after(vc);
            plain = held_plain();
            if (p + 1 < s1) {
                store(p + 1, kc ^ 1, vn);
                fetch(info_s[info_at(p + 2)]);
            }
            cut_page(p, kc, vc, c);
            meet();
            kc ^= 1;
            vc = vn;
            c = cn;
        }
    }

    l += __shfl_xor(l, 32);
    if (r0 + 32 * wave + q32 > last) return;
    const int64_t at = (int64_t)(seq.row0 + row / group) * a.Hq + head * group + row % group;
    if (a.splits > 1) {
        float *dst = a.part + (at * a.splits + split) * D;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<f32x4 *>(dst + 32 * i + 8 * e + 4 * h) =
                    f32x4{o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
        if (h == 0) {
            float *ml = a.part + (int64_t)a.kv.T * a.Hq * a.splits * D + (at * a.splits + split) * 2;
            ml[0] = base;
            ml[1] = l;
        }
        return;
    }
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    // A lane has 4 of each 8 features and its half wave's other lane the rest: one takes
    // the first 8, one the next (2048 queries of 32 heads over themselves: 73.5 us
    // against 77.6 with 8-byte stores)
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
            const auto two = [&](int j) { return bf16x2_bits(o[i][e + j] * f, o[i][e + j + 1] * f); };
            const auto x = __builtin_amdgcn_permlane32_swap(two(0), two(4), false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(two(2), two(6), false, false);
            *reinterpret_cast<u32x4 *>(a.O + at * D + 32 * i + 2 * e + 8 * h) = u32x4{x[0], y[0], x[1], y[1]};
        }
    if (a.lse && h == 0) a.lse[at] = (base + log2f(l)) * kLn2;
}

// Parts of a sequence's pages. Few queries: as many as give each compute unit a
// block (8 heads, one token after 32759: 17.6 us in 32 parts, 20.6 in 16, 17.9 in 64;
// 32 sequences of up to 8192, 8 heads: 67 in one, 69 in two, 68 in four); tables of
// more than 128 pages in parts of 64 pages at the most, while that makes no more than
// 16 blocks a unit, so that a long sequence among short ones is not one block's alone
// (one of 18000 tokens, 35 of 100: 98 us in one part, 41 in 3, 29 in 5, 25 in 9; one of
// 32000, 31 of 500: 168, 51 in 4, 31 in 8, 45 in 16; 40 of 16000: 277, 244 in two, 227
// in four; 32 of 8000, where the second launch is not worth it: 93 and 98); and one
// up to 16 pages (500 tokens: 7.0 in one, 8.9 in two; 1000: 9.5 and 8.8, but a launch
// less, 3.4 on the host).
// Pages are the table's width, which the host knows, not the lengths, which it does not:
// 32 sequences of 1000 tokens 15.4 us up to 128 pages wide, 39.7 with 1024, in 16 parts.
// Prompts: what takes least by the time of a page in a block, of the second launch
// and of a query's part on its way through memory (32 / 8 heads: 64 tokens after 32000
// 57 us in 32 parts, 583 in one; after 8000 30, in all parts that there is room for 33,
// in one 156; 1000 tokens alone 30 in one, 38 in two; 16 / 2 heads: 300 tokens after
// 3000 29, 48 in all, 71 in one).
constexpr int kCus = 256;
constexpr int kAlonePages = 16, kDeepPages = 128, kDeepPart = 64;
constexpr int kIdle = kCus * 3 / 4;
constexpr float kPageTime = 1.3f, kJoinTime = 6.0f, kPartTime = 0.00026f;

// How a call is cut: which kernel, its queries per block (`rows`), the blocks of a
// head (`tiles`, prompts) and the parts of a sequence's pages.
// Queries per block: the least of 16, 32, 64, 128 and 256 that the average sequence
// fits, up to 64 in the kernel for few (32 sequences of up to 8192, 8 heads: 32
// queries 76 us, 64 queries 130, 164 both with 128 to a block; 128 queries 170 with
// 128, 193 twice 64, 229 with 256; 100 queries after 8000 alone 22, 26 and 24; 64
// sequences of 128 queries after 500 51, 47 and 59; of 256 queries 98 with 128, 72
// with 256). But 128, not 256, where blocks of 256 would leave a quarter of the compute
// units idle (32 / 8 heads: 256 tokens alone 17 us against 20, 1000 30.6 and 33.7,
// 1400, 176 blocks of 256, 38 and 43, 2000, 256 blocks, 62 and 59; 64 after 8000 29 and
// 33, after 32000, in 32 parts, 62 and 56). Sequences far from the average pay for it: 31
// decoded tokens after 4000 and a prompt of 2048 290 us, 218 in two calls, of 256 105 and
// 83, of 64 59 and 69.
struct AttnPlan {
    bool few, sorted;
    int rows, tiles, splits;
};

// A plan with blocks of `rows` queries.
AttnPlan attn_plan_of(int rows, int64_t queries, int B, int pages, int Hk) {
    AttnPlan p;
    p.rows = rows;
    p.few = rows <= 64;
    p.tiles = p.few ? B : (int)((queries + (int64_t)(rows - 1) * B) / rows);
    // more blocks than units: in order, where the sequences fit a wave
    p.sorted = !p.few && B > 1 && B <= 64 && (int64_t)p.tiles * Hk > kCus;
    p.splits = 1;
    const int fill = (int)std::min<int64_t>(SVDQ_KV8_MAX_SPLITS, kCus / ((int64_t)p.tiles * Hk));
    if (p.few) {
        if (pages > kAlonePages) {
            const int parts = pages > kDeepPages ? (pages + kDeepPart - 1) / kDeepPart : 1;
            const int deep = (int)std::min<int64_t>(parts, 16 * kCus / ((int64_t)B * Hk));
            p.splits = std::min({std::max({fill, deep, 1}), (pages + kDecWaves - 1) / kDecWaves, SVDQ_KV8_MAX_SPLITS});
        }
    } else {
        float best = kPageTime * pages;
        for (int s = 2; s <= fill && s <= pages; ++s) {
            const float time = kPageTime * ((pages + s - 1) / s) + kJoinTime + kPartTime * (float)queries * Hk * s;
            if (time < best) {
                best = time;
                p.splits = s;
            }
        }
    }
    return p;
}

AttnPlan attn_plan(int T, int B, int pages, int Hk, int group) {
    const int64_t queries = (int64_t)T * group;
    int rows = kDecRows;
    while (rows < 256 && queries > (int64_t)rows * B) rows *= 2;
    const AttnPlan p = attn_plan_of(rows, queries, B, pages, Hk);
    return rows == 256 && (int64_t)p.tiles * Hk * p.splits <= kIdle ? attn_plan_of(128, queries, B, pages, Hk) : p;
}

template <int D>
auto decode_kernel(int rows) {
    return rows == 16 ? kv8_decode_kernel<D, 1, 1> : rows == 32 ? kv8_decode_kernel<D, 2, 1> : kv8_decode_kernel<D, 2, 2>;
}

}  // namespace

size_t kv8_attention_workspace(int T, int B, int max_pages, int Hq, int Hk, int D) {
    if (T == 0 || B == 0) return 0;
    const int splits = attn_plan(T, B, max_pages, Hk, Hq / Hk).splits;
    return splits == 1 ? 0 : (size_t)T * Hq * splits * (D + 2) * sizeof(float);
}

hipError_t launch_kv8_attention(const KvBatch &kv, const uint16_t *Q, int64_t q_stride, const uint8_t *kc,
                                const float *ks, const uint8_t *vc, const float *vs, int Hq, int Hk, int D, float scale,
                                bool causal, int window, uint16_t *O, float *lse, void *workspace, hipStream_t stream) {
    AttnPlan plan = attn_plan(kv.T, kv.B, kv.max_pages, Hk, Hq / Hk);
    // With a window, parts of what it shows (a sequence has at most T new tokens), and
    // no more than the workspace was made for (8 heads, one token after 32000, a window
    // of 128: 5.2 us, in parts of the context 8.1; 64 tokens after 8000, 512: 16.6, 19.7)
    if (window > 0) {
        const int64_t pages = ((int64_t)window + kv.T + kKvPage - 3) / kKvPage + 1;
        const int most = plan.splits;
        if (pages < kv.max_pages) plan = attn_plan(kv.T, kv.B, (int)pages, Hk, Hq / Hk);
        plan.splits = std::min(plan.splits, most);
    }
    window = std::min(window, 1 << 30);  // no position is further
    const AttnArgs a{kv, Q, q_stride, kc, vc, ks, vs, Hq, Hk, Hq / Hk, scale * 1.44269504088896340736f, causal, window,
                     O, lse, plan.sorted, static_cast<float *>(workspace), plan.splits};
    hipError_t e;
    if (plan.few) {
        const int blocks = kv.B + (int)((int64_t)kv.T * (Hq / Hk) / plan.rows);  // of a head and part: at most 2 B
        const bool more = blocks > kMostSequences;
        e = launch_kernel(D == 64 ? decode_kernel<64>(plan.rows) : decode_kernel<128>(plan.rows),
                          dim3((unsigned)plan.splits, (unsigned)(more ? 2 * Hk : Hk), (unsigned)(more ? kMostSequences : blocks)),
                          64 * kDecWaves, stream, a);
    } else {
        const dim3 grid((unsigned)(plan.tiles * Hk), (unsigned)plan.splits);
        e = plan.rows == 128
                ? launch_kernel(D == 64 ? kv8_prompt_kernel<64, 4> : kv8_prompt_kernel<128, 4>, grid, 256, stream, a, plan.tiles)
                : launch_kernel(D == 64 ? kv8_prompt_kernel<64, 8> : kv8_prompt_kernel<128, 8>, grid, 512, stream, a, plan.tiles);
    }
    if (e != hipSuccess || plan.splits == 1) return e;
    const int64_t queries = (int64_t)kv.T * Hq;
    if (plan.splits <= kJoinAlone)
        return launch_kernel(D == 64 ? kv8_join_kernel<64, 1> : kv8_join_kernel<128, 1>, dim3((unsigned)((queries + 3) / 4)), 256,
                             stream, a);
    return launch_kernel(D == 64 ? kv8_join_kernel<64, 4> : kv8_join_kernel<128, 4>, dim3((unsigned)queries), 256, stream, a);
}

}  // namespace svdq
