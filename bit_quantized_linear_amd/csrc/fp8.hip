// The block-scaled FP8 linear: E4M3 codes with one fp32 scale per block of
// 128 -- weights in 128 x 128 blocks, activations per token and 128 features.
//
//   A[m, g]  = max(max_{k in g} |X[m, k]|, 2^-100)
//   sx[g, m] = fp32(A / 448),  qx = E4M3(fp32(X fp32(448 / A)))
//   acc[m,n] = sum_g (sx[g, m] sw[n / 128, g]) sum_{k in g} qx[m, k] qw[n, k]
//   Y        = acc + bias, rounded once to bf16 (nearest even) or kept fp32
//
// A group of 128 codes is summed by the matrix core (products of two E4M3
// numbers are exact, fp32 accumulation); the scale of a group's partial sum
// is one fp32 product per token and 128 output columns, and is applied with
// one fp32 FMA per output element and group.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "fp8_common.h"
#include "internal.h"

namespace svdq {

namespace {

// ---- activation pass -------------------------------------------------------

constexpr int kF8QThreads = 256;
constexpr int kF8QRows = 16;    // tokens per block
constexpr int kF8QGroups = 4;   // groups of 128 features per block

// One block quantizes 16 tokens x 4 groups. 16 lanes hold one token's group,
// 8 consecutive features (one 16-byte load) each; their largest magnitude is
// found on the bf16 bit patterns (an integer maximum orders magnitudes, and
// puts NaN above all, so a NaN reaches the scale). All four loads of a thread
// are in flight together. The scales of the block go through LDS so that 16
// tokens' scales of a group are stored as one 64-byte segment.
// HBM-bound: 3 bytes and a group's scale per feature, each once; 32760 x 5120
// takes 102 us, 5.0 TB/s, the rate of a large copy (16 x 5120: 3.5 us, of which
// an empty launch is 2 to 3).
__global__ __launch_bounds__(kF8QThreads) void fp8_quantize_kernel(const uint16_t *__restrict__ X, int M, int K,
                                                                   int G, uint8_t *__restrict__ qx,
                                                                   float *__restrict__ sx) {
    __shared__ float sxs[kF8QGroups][kF8QRows];
    const int row = threadIdx.x >> 4, part = threadIdx.x & 15;
    const int m = blockIdx.x * kF8QRows + row;
    const int g0 = blockIdx.y * kF8QGroups;
    const size_t base = (size_t)m * K;
    u32x4 v[kF8QGroups];
#pragma unroll
    for (int i = 0; i < kF8QGroups; ++i) {
        const int k = (g0 + i) * kF8Block + part * 8;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (m < M && k < K) v[i] = *reinterpret_cast<const u32x4 *>(X + base + k);
    }
#pragma unroll
    for (int i = 0; i < kF8QGroups; ++i) {
        const float a = fp8_block_top(v[i]);
        const float r = kF8Max / a;
        if (part == 0) sxs[i][row] = a / kF8Max;
        const int k = (g0 + i) * kF8Block + part * 8;
        if (m < M && k < K) *reinterpret_cast<u32x2 *>(qx + base + k) = fp8_codes8(v[i], r);
    }
    __syncthreads();
    const int g = threadIdx.x >> 4;
    if (g < kF8QGroups && g0 + g < G) {
        const int mm = blockIdx.x * kF8QRows + part;
        if (mm < M) sx[(size_t)(g0 + g) * M + mm] = sxs[g][part];
    }
}

// ---- the product, many tokens ----------------------------------------------

constexpr uint32_t kF8Oob = 0x80000000u;
constexpr int kF8Cus = 256;  // compute units
// one MFMA tile: with two, 20 x 5120 x 5120 took 14.6 us, in tiles of 32 x 32 it takes 8.5
constexpr int kF8SkinnyTokens = 16;

typedef __attribute__((address_space(3))) void f8_lds_void;

// One stage: KW groups of 128 bytes of K, the rows of both operands, and each
// wave's token scales.
template <int BN, int BM, int NW, int KW>
struct F8Stage {
    struct Group {
        uint8_t a[BN * kF8Block];
        uint8_t b[BM * kF8Block];
        float scale[NW][64];
    } group[KW];
};

// Operands of one 16-row tile and group: the codes, or their bf16 values.
struct F8Codes {
    i32x8 v;
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
        v = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    }
    __device__ __forceinline__ static f32x4 product(const F8Codes &a, const F8Codes &b) {
        return mfma_fp8_16x16x128(a.v, b.v, f32x4{0.f, 0.f, 0.f, 0.f});
    }
};

struct F8Wide {
    bf16x8 v[4];
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
        v[0] = fp8_widen8(lo[0], lo[1]);
        v[1] = fp8_widen8(lo[2], lo[3]);
        v[2] = fp8_widen8(hi[0], hi[1]);
        v[3] = fp8_widen8(hi[2], hi[3]);
    }
    __device__ __forceinline__ static f32x4 product(const F8Wide &a, const F8Wide &b) {
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) c = mfma_bf16_16x16x32(a.v[i], b.v[i], c);
        return c;
    }
};

// Block tile BN = 16 WN TN (output columns) x BM = 16 WM TM (tokens), WN x WM
// waves of TN x TM MFMA tiles of 16 x 16. One LDS stage is one group of 128
// bytes of K for the block's rows of both operands, double buffered; operands
// go straight from global memory to LDS (1 KB per load: 8 rows x 128 bytes).
// The 16-byte chunk c of row r sits at chunk position c ^ ((r >> 1) & 7), so
// that the operand reads of 16 consecutive rows fall on distinct banks; a
// lane fetches the global chunk that belongs at the position it writes. Rows
// past N or M and chunks past K read zeros (their offset is past the buffer).
// One 16x16x128 MFMA is a whole group of a tile, so its result is scaled and
// added (4 FMAs a lane) while the next row tile's MFMAs run: the 16 x 16 x 128
// MFMA and not the 32 x 32 x 64 one, whose results take two per group and four
// times the registers (1.19 times the time at 32768 x 5120 x 5120).
// NS stages take turns, loads NS - 1 ahead. KW parts of the block share K and add
// their sums at the end, for grids too small to fill the chip.
// kWide: sums to fp32 precision on bf16 MFMAs, for fp32 outputs; otherwise bf16.
template <int WN, int WM, int TN, int TM, int NS, int KW, bool kWide, class Stage>
__device__ __forceinline__ void fp8_tile(Stage &st0, Stage &st1, Stage &st2, float *bias_s,
                                         const uint8_t *__restrict__ qx, const float *__restrict__ sx,
                                         const uint8_t *__restrict__ qw, const float *__restrict__ sw,
                                         const uint16_t *__restrict__ bias, int M, int N, int K, void *__restrict__ Y,
                                         int n0, int m0) {
    constexpr int BN = 16 * WN * TN, BM = 16 * WM * TM, NW = WN * WM, kThreads = 64 * NW * KW;
    using Frag = std::conditional_t<kWide, F8Wide, F8Codes>;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int kw = KW == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6) / NW;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % NW;
    const int wn = wave % WN;
    const int wm = wave / WN;
    const int r16 = lane & 15;
    const int q4 = lane >> 4;
    const int G = (K + kF8Block - 1) / kF8Block, S = (G + KW - 1) / KW;

    const __amdgpu_buffer_rsrc_t ra = fp8_rsrc(qw + (size_t)n0 * K, (uint32_t)min(BN, N - n0) * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rb = fp8_rsrc(qx + (size_t)m0 * K, (uint32_t)min(BM, M - m0) * (uint32_t)K);

    // Each wave loads kA KB of the weights' rows and kB of the activations':
    // a load fills 8 staged rows r, r + 1, ... (lane l row r + l / 8 at chunk
    // position l % 8), rows 16 apart share their chunk order
    constexpr int kA = BN / 8 / NW, kB = BM / 8 / NW, kLoads = kA + kB;
    static_assert(kA % 2 == 0 && kB % 2 == 0, "a wave loads pairs of 8 rows");
    int gchunk[2];
    uint32_t ga[2], gb[2], oa[2], ob[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + lane / 8;
        gchunk[i] = ((lane % 8) ^ ((r >> 1) & 7)) * 16;
        ga[i] = (uint32_t)(wave * kA * 8 + r) * (uint32_t)K + (uint32_t)gchunk[i];
        gb[i] = (uint32_t)(wave * kB * 8 + r) * (uint32_t)K + (uint32_t)gchunk[i];
    }
    // offsets of stage s, and its load i into st
    auto aim = [&](int s) __attribute__((always_inline)) {
        const int k0 = (s * KW + kw) * kF8Block;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = k0 + gchunk[i] < K;
            oa[i] = in ? ga[i] + (uint32_t)k0 : kF8Oob;
            ob[i] = in ? gb[i] + (uint32_t)k0 : kF8Oob;
        }
    };
    auto issue = [&](Stage &st, int i) __attribute__((always_inline)) {
        const bool a = i < kA;
        const int n = a ? i : i - kA;
        uint8_t *dst = a ? st.group[kw].a + (wave * kA + n) * 1024 : st.group[kw].b + (wave * kB + n) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(a ? ra : rb, (f8_lds_void *)dst, 16,
                                                 (a ? oa : ob)[n & 1] + (uint32_t)(n / 2) * 16u * (uint32_t)K, 0, 0, 0);
    };
    // a lane's operand of row tile i: chunks q4 and 4 + q4 of row 16 i + l % 16
    const int x = (r16 >> 1) & 7;
    const int c_lo = r16 * kF8Block + (q4 ^ x) * 16, c_hi = r16 * kF8Block + ((4 + q4) ^ x) * 16;
    auto read = [&](Frag &f, const uint8_t *base, int i) __attribute__((always_inline)) {
        f.set(*reinterpret_cast<const u32x4 *>(base + i * 16 * kF8Block + c_lo),
              *reinterpret_cast<const u32x4 *>(base + i * 16 * kF8Block + c_hi));
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // this wave's columns lie in one block of 128: one weight scale a group
    static_assert(kF8Block % (16 * TN) == 0, "a wave's columns lie in one block");
    const int wblock = (n0 + wn * 16 * TN) / kF8Block;
    const float *swr = sw + (size_t)(wblock < (N + kF8Block - 1) / kF8Block ? wblock : 0) * G;
    // The scales of the wave's 16 TM tokens go to LDS with the stage, one load
    // of 4 bytes a lane (zeros past M, and for a group past K: an infinite scale
    // would make NaN of its zeros); a wave's loads per stage are kLoads and this
    // one, all of them to LDS, so that a wait can count them.
    static_assert(TM <= 4, "a lane per token");
    float raw[TM], sc[TM];
    const int first_m = m0 + wm * TM * 16;
    auto load_scales = [&](int s, Stage &st) __attribute__((always_inline)) {
        const int g = s * KW + kw;
        const __amdgpu_buffer_rsrc_t r = fp8_rsrc(sx + (size_t)min(g, G - 1) * M + min(first_m, M - 1),
                                                  g < G ? 4u * (uint32_t)max(0, min(16 * TM, M - first_m)) : 0u);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (f8_lds_void *)st.group[kw].scale[wave], 4, 4u * (uint32_t)lane, 0,
                                                 0, 0);
    };

    for (int i = tid; i < BN; i += kThreads)
        bias_s[i] = bias && n0 + i < N ? bf16_bits_to_f32(bias[n0 + i]) : 0.0f;
    static_assert(NS == 2 || NS == 3, "stages");
    auto stage = [&](int i) -> Stage & { return i == 0 ? st0 : i == 1 ? st1 : st2; };
#pragma unroll
    for (int f = 0; f < NS - 1; ++f) {
        aim(f);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) issue(stage(f), i);
        load_scales(f, stage(f));
    }

    // kRing row tiles' operands in registers, tile i in slot i % kRing; the
    // products of MFMA t of a stage (t = row tile * TM + token tile) in slot
    // t % 4 of p, scaled and added kDelay MFMAs later
    constexpr int kRing = TN % 4 == 0 && !kWide ? 4 : 2, kLate = kRing - 1, kDelay = TM >= 4 ? 3 : 2;
    static_assert(TN % kRing == 0 && TN * TM % 4 == 0, "slots are the same in every stage");
    Frag fa[kRing], fb[TM];
    f32x4 p[4];
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        sc[j] = 0.0f;
        fb[j].set(zero, zero);
    }
#pragma unroll
    for (int i = 0; i < kRing; ++i) fa[i].set(zero, zero);
#pragma unroll
    for (int t = 0; t < 4; ++t) p[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](int t) __attribute__((always_inline)) {
        const int i = t / TM, j = t % TM;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(sc[j], p[t % 4][e], acc[i][j][e]);
    };
    auto multiply = [&](int i, int j) __attribute__((always_inline)) {
        const int t = i * TM + j;
        __builtin_amdgcn_sched_barrier(0);
        add((t + TN * TM - kDelay) % (TN * TM));
        __builtin_amdgcn_s_setprio(1);
        p[t % 4] = Frag::product(fa[i % kRing], fb[j]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // stage s has landed (the NS - 2 behind it may be under way; loads return
    // in order) and everyone has read stage s - 1
    constexpr int kPending = (NS - 2) * (kLoads + 1);
    static_assert(kPending < 16, "what the wait below can count");
    auto next_stage = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (NS == 2)
            __builtin_amdgcn_s_waitcnt(0);
        else  // vmcnt(kPending) lgkmcnt(0)
            __builtin_amdgcn_s_waitcnt(kPending | (7 << 4) | (0 << 8));
        fp8_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    // The last kLate row tiles of stage s - 1 are multiplied after the barrier
    // that opens stage s, from operands read before it, so that stage s's
    // first operands are read under their MFMAs: a token tile's as soon as
    // its last MFMA has issued. The loads of stage s + NS - 1 are spread over
    // the MFMAs, TM / 2 apart (issued together they block the wave until the
    // load unit has taken them all: 5 % slower at 32760 x 5120 x 5120). Two
    // stages run in pairs without a branch (a stage past K loads zeros and adds
    // none): with one the compiler spills.
    constexpr int kTogether = (kLoads + 2 * TN - 1) / (2 * TN);  // loads at a time
    auto load_before = [&](Stage &nxt, int u) __attribute__((always_inline)) {
        if (u % (TM / 2) == 0)
#pragma unroll
            for (int i = u / (TM / 2) * kTogether; i < min((u / (TM / 2) + 1) * kTogether, kLoads); ++i) issue(nxt, i);
    };
    auto run_stage = [&](int s, const Stage &cur, Stage &nxt) __attribute__((always_inline)) {
        next_stage();
        const int g = s * KW + kw;
        const float weight_scale = fp8_scale_within(swr[min(g, G - 1)], g, G);
        aim(s + NS - 1);
        load_scales(s + NS - 1, nxt);
#pragma unroll
        for (int k = 0; k < TM; ++k) raw[k] = cur.group[kw].scale[wave][k * 16 + r16];
        read(fa[0], cur.group[kw].a, wn * TN);
#pragma unroll
        for (int r = 0; r < kLate; ++r) {
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                load_before(nxt, r * TM + j);
                multiply(TN - kLate + r, j);
                if (r == kLate - 1) read(fb[j], cur.group[kw].b, wm * TM + j);
            }
            read(fa[r + 1], cur.group[kw].a, wn * TN + r + 1);
        }
#pragma unroll
        for (int i = 0; i < TN - kLate; ++i) {
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                load_before(nxt, (kLate + i) * TM + j);
                multiply(i, j);
                if (i * TM + j == kDelay - 1) {  // stage s - 1 is all added
#pragma unroll
                    for (int k = 0; k < TM; ++k) sc[k] = raw[k] * weight_scale;
                }
            }
            if (i + kRing < TN) read(fa[i % kRing], cur.group[kw].a, wn * TN + i + kRing);
        }
    };
    if constexpr (NS == 2) {
        for (int s = 0; s < S; s += 2) {
            run_stage(s, st0, st1);
            run_stage(s + 1, st1, st0);
        }
    } else {
        for (int s = 0; s < S;) {  // stage s in slot s % NS
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                run_stage(s, stage(i), stage((i + NS - 1) % NS));
                if (++s >= S) break;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kLate; ++r)
#pragma unroll
        for (int j = 0; j < TM; ++j) multiply(TN - kLate + r, j);
#pragma unroll
    for (int t = TN * TM - kDelay; t < TN * TM; ++t) add(t);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    // the waves of the upper parts of K give their sums to those of the lower, in halves
    if constexpr (KW > 1) {
        static_assert(sizeof(Stage) >= sizeof(f32x4) * TN * TM * 64 * NW * (KW / 2),
                      "half the parts, through one stage");
#pragma unroll
        for (int half = KW / 2; half > 0; half /= 2) {
            f32x4 *sums = reinterpret_cast<f32x4 *>(&st0) + ((kw % half) * NW + wave) * TN * TM * 64 + lane;
            if (kw >= half && kw < 2 * half)
#pragma unroll
                for (int t = 0; t < TN * TM; ++t) sums[t * 64] = acc[t / TM][t % TM];
            __syncthreads();
            if (kw < half)
#pragma unroll
                for (int t = 0; t < TN * TM; ++t) acc[t / TM][t % TM] += sums[t * 64];
            __syncthreads();
        }
    }

    // Output: 32 tokens x BN columns at a time through LDS (the waves of one
    // wm write, everyone stores whole row segments), alternating between the
    // two stages.
    constexpr int wide = kWide ? 4 : 2;
    constexpr int pitch = BN * wide + 16;
    static_assert(sizeof(Stage) >= 32 * pitch && TM % 2 == 0, "LDS too small for the output tile");
    constexpr int pieces = BN * wide / 16;  // 16-byte pieces of a row
#pragma unroll
    for (int pass = 0; pass < WM * TM / 2; ++pass) {
        uint8_t *buf = reinterpret_cast<uint8_t *>((pass & 1) ? &st1 : &st0);
        if (kw == 0 && wm == pass / (TM / 2)) {
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const int nl = (wn * TN + i) * 16 + 4 * q4;
                const f32x4 bv = *reinterpret_cast<const f32x4 *>(bias_s + nl);
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const f32x4 v = acc[i][pass % (TM / 2) * 2 + jj] + bv;
                    uint8_t *to = buf + (jj * 16 + r16) * pitch + nl * wide;
                    if constexpr (kWide)
                        *reinterpret_cast<f32x4 *>(to) = v;
                    else
                        *reinterpret_cast<u32x2 *>(to) = u32x2{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
                }
            }
        }
        __syncthreads();
        for (int c = tid; c < 32 * pieces; c += kThreads) {
            const int row = c / pieces, piece = c % pieces;
            const int m = m0 + 32 * pass + row;
            const int64_t n = n0 + piece * (16 / wide);
            if (m < M && n < N) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(buf + row * pitch + piece * 16);
                u32x4 *to = reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(Y) + ((int64_t)m * N + n) * wide);
                // an output of many 256-wide tiles is larger than the L2 and
                // would push the operands out of it (2 to 6 % slower)
                if constexpr (BN == 256)
                    __builtin_nontemporal_store(v, to);
                else
                    *to = v;
            }
        }
    }
}

template <int WN, int WM, int TN, int TM, int NS, int KW, bool kWide>
__global__ __launch_bounds__(64 * WN * WM * KW, 1) void fp8_gemm_kernel(
    const uint8_t *__restrict__ qx, const float *__restrict__ sx, const uint8_t *__restrict__ qw,
    const float *__restrict__ sw, const uint16_t *__restrict__ bias, int M, int N, int K, void *__restrict__ Y,
    int tiles_n) {
    constexpr int BN = 16 * WN * TN, BM = 16 * WM * TM;
    using Stage = F8Stage<BN, BM, WN * WM, KW>;
    __shared__ __attribute__((aligned(16))) Stage st0;
    __shared__ __attribute__((aligned(16))) Stage st1;
    __shared__ __attribute__((aligned(16))) float bias_s[BN];
    int tile_n, tile_m;
    fp8_tile_of_block(blockIdx.x, gridDim.x, gridDim.x, tiles_n, tile_n, tile_m);
    if constexpr (NS == 2) {
        fp8_tile<WN, WM, TN, TM, NS, KW, kWide>(st0, st1, st0, bias_s, qx, sx, qw, sw, bias, M, N, K, Y, tile_n * BN,
                                            tile_m * BM);
    } else {
        __shared__ __attribute__((aligned(16))) Stage st2;
        fp8_tile<WN, WM, TN, TM, NS, KW, kWide>(st0, st1, st2, bias_s, qx, sx, qw, sw, bias, M, N, K, Y, tile_n * BN,
                                            tile_m * BM);
    }
}

// 256 x 256 tiles, of which the grid's first `whole` blocks take one each; two
// blocks share each of the others (128 of its tokens each). 8 waves, one block
// per compute unit: 133 KB of LDS hold two stages, and a stage's operands feed
// 4 times the MFMAs that they take LDS reads for. Bound by the matrix cores: they
// are busy 63 % of the time, at the clock that their power leaves (32760 x 5120 x
// 5120: 690 to 720 us, 2.4 to 2.5 PFLOP/s; 4608 x 5120 x 12288: 250, 2.3; the
// library's product of the same codes with one scale for all, 650 and 214). The rest is the epilogue, which nothing
// overlaps (one tile's output is 128 KB), and the fill of each tile's first stage.
__global__ __launch_bounds__(512, 1) void fp8_gemm256_kernel(
    const uint8_t *__restrict__ qx, const float *__restrict__ sx, const uint8_t *__restrict__ qw,
    const float *__restrict__ sw, const uint16_t *__restrict__ bias, int M, int N, int K, void *__restrict__ Y,
    int tiles_n, int tiles, int whole) {
    __shared__ __attribute__((aligned(16))) F8Stage<256, 256, 8, 1> st0;
    __shared__ __attribute__((aligned(16))) F8Stage<256, 256, 8, 1> st1;
    __shared__ __attribute__((aligned(16))) float bias_s[256];
    int tile_n, tile_m;
    const int b = blockIdx.x;
    if (b < whole) {
        fp8_tile_of_block(b, whole, tiles, tiles_n, tile_n, tile_m);
        fp8_tile<2, 4, 8, 4, 2, 1, false>(st0, st1, st0, bias_s, qx, sx, qw, sw, bias, M, N, K, Y, tile_n * 256,
                                          tile_m * 256);
    } else {
        const int id = whole + (b - whole) / 2, m0_half = (b - whole) % 2 * 128;
        fp8_tile_at(id, tiles, tiles_n, tile_n, tile_m);
        if (tile_m * 256 + m0_half < M)
            fp8_tile<4, 2, 4, 4, 2, 1, false>(st0, st1, st0, bias_s, qx, sx, qw, sw, bias, M, N, K, Y, tile_n * 256,
                                              tile_m * 256 + m0_half);
    }
}

// ---- the product, few tokens -----------------------------------------------

// One block computes 16 NT output columns of at most 16 tokens; its W waves take
// the groups of K in turn (part p of 16 has groups p, p + 16, ...; wave w of 8 the
// parts w and w + 8, so that the order of a sum is the same with 16 waves and
// with 8; of 64 columns, where there are always 8 waves, 8 parts), straight from
// global memory into the operands of the 16x16x128 MFMA (weights as A: row =
// output column; tokens as B, for all NT tiles of columns), and add the parts in
// LDS in order. The weight is read once: bound by HBM, and at these sizes by the
// way to the first of it (a launch, a load's latency, the sums): 8 x 2048 x 12288
// (M x K x N) takes 7.7 us (25 MB, 3.3 TB/s), 1 x 5120 x 5120 in one launch 8.6 (26
// MB, 3.0 TB/s). Waves hide a load's latency better than loads ahead, whose
// registers keep waves out: 1, 2, 3 and 4 groups in flight per wave take 8.5, 9.6,
// 9.3 and 10.5 us for 1 x 5120 x 5120, 13.4, 14.6, 14.5 and 16.2 for 8 x 5120 x 12288.
// kFused: from bf16 activations. While its first weights are on their way, each
// block quantizes all tokens' features into LDS, exactly as the activation pass
// does, which saves that launch; dynamic LDS: the codes [M][K rounded up to
// groups], then the scales [G][M].
template <int W, int NT, bool kWide, bool kFused>
__global__ __launch_bounds__(64 * W) void fp8_skinny_kernel(
    const uint8_t *__restrict__ qx, const float *__restrict__ sx, const uint16_t *__restrict__ X,
    const uint8_t *__restrict__ qw, const float *__restrict__ sw, const uint16_t *__restrict__ bias, int M, int N,
    int K, void *__restrict__ Y) {
    constexpr int kSums = NT == 4 ? 8 : 16, kParts = kSums / W;  // parts of K, and how many a wave has
    __shared__ f32x4 red[kSums][NT][64];
    extern __shared__ __align__(16) uint8_t codes_s[];
    const int n0 = blockIdx.x * 16 * NT;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q4 = lane >> 4;
    const int G = (K + kF8Block - 1) / kF8Block;
    const __amdgpu_buffer_rsrc_t rw = fp8_rsrc(qw + (size_t)n0 * K, (uint32_t)min(16 * NT, N - n0) * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rx = fp8_rsrc(qx, kFused ? 0u : (uint32_t)M * (uint32_t)K);
    const float *swr = sw + (size_t)(n0 / kF8Block) * G;
    float *scales_s = reinterpret_cast<float *>(codes_s + (size_t)M * G * kF8Block);

    auto join = [](u32x4 lo, u32x4 hi) __attribute__((always_inline)) {
        return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    };
    // a lane's 32 codes of a group: chunks of 16 at k = 16 q4 and 64 + 16 q4
    auto operand = [&](__amdgpu_buffer_rsrc_t r, int row, int g) __attribute__((always_inline)) {
        const int k = g * kF8Block + 16 * q4;
        const uint32_t off = (uint32_t)row * (uint32_t)K + (uint32_t)k;
        return join(
            __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, k < K ? off : kF8Oob, 0, 0)),
            __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, k + 64 < K ? off + 64 : kF8Oob, 0, 0)));
    };

    f32x4 acc[kParts][NT];
#pragma unroll
    for (int x = 0; x < kParts; ++x)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[x][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int mrow = min(r16, M - 1);

    // Where rows are a multiple of 4 KB apart, the same group of all rows lies on a
    // few memory channels, so each block starts at another group. Weights that the
    // last-level cache holds gain by it, those from HBM little (us, with / without: 8 x
    // 8192 x 8192 14.1 / 17.8, from HBM 18.0 / 18.0; 8 x 4096 x 16384 13.3 / 13.7 and
    // 15.1 / 16.6; fp32 16 x 8192 x 8192 15.7 / 18.4 and 19.4 / 18.5); rows at other
    // distances lose (1 x 2048 x 151936 57 / 49).
    const int first = K % 4096 ? 0 : (int)blockIdx.x & ((1 << (31 - __builtin_clz(G))) - 1);
    auto turned = [&](int i) __attribute__((always_inline)) { return i + first < G ? i + first : i + first - G; };
    i32x8 a[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) a[t] = operand(rw, 16 * t + r16, turned(wave));
    if constexpr (kFused) {
        // 16 threads per token and group, 8 features each
        const int part = threadIdx.x & 15;
        for (int i = threadIdx.x >> 4; i < M * G; i += 4 * W) {
            const int m = i / G, g = i % G, k = g * kF8Block + part * 8;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (k < K) v = *reinterpret_cast<const u32x4 *>(X + (size_t)m * K + k);
            const float top = fp8_block_top(v);
            *reinterpret_cast<u32x2 *>(codes_s + (size_t)i * kF8Block + part * 8) = fp8_codes8(v, kF8Max / top);
            if (part == 0) scales_s[g * M + m] = top / kF8Max;
        }
        __syncthreads();
    }
    auto group = [&](int i, f32x4(&to)[NT]) __attribute__((always_inline)) {
        const int g = turned(i);
        if (i != wave) {
#pragma unroll
            for (int t = 0; t < NT; ++t) a[t] = operand(rw, 16 * t + r16, g);
        }
        i32x8 b;
        float s;
        if constexpr (kFused) {
            const uint8_t *at = codes_s + ((size_t)mrow * G + g) * kF8Block + 16 * q4;
            b = join(*reinterpret_cast<const u32x4 *>(at), *reinterpret_cast<const u32x4 *>(at + 64));
            s = scales_s[g * M + mrow] * swr[g];
        } else {
            b = operand(rx, mrow, g);
            s = sx[(size_t)g * M + mrow] * swr[g];
        }
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 p = kWide ? mfma_wide_16x16x128(a[t], b, zero) : mfma_fp8_16x16x128(a[t], b, zero);
#pragma unroll
            for (int e = 0; e < 4; ++e) to[t][e] = __builtin_fmaf(s, p[e], to[t][e]);
        }
    };
    for (int i = wave; i < G; i += kSums) {
        group(i, acc[0]);
        if constexpr (kParts == 2)
            if (i + W < G) group(i + W, acc[1]);
    }
#pragma unroll
    for (int x = 0; x < kParts; ++x)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[x * W + wave][t][lane] = acc[x][t];
    __syncthreads();
    for (int i = threadIdx.x; i < 256 * NT; i += 64 * W) {
        const int m = i / (16 * NT), c = i % (16 * NT);  // consecutive threads: consecutive columns of a token
        const int src = 16 * ((c >> 2) & 3) + m;
        const int n = n0 + c;
        if (m < M && n < N) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kSums; ++w) v += red[w][c >> 4][src][c & 3];
            if (bias) v += bf16_bits_to_f32(bias[n]);
            if constexpr (kWide)
                static_cast<float *>(Y)[(size_t)m * N + n] = v;
            else
                static_cast<uint16_t *>(Y)[(size_t)m * N + n] = (uint16_t)f32_to_bf16_bits(v);
        }
    }
}

}  // namespace

hipError_t launch_fp8_quantize_act(const uint16_t *X, int M, int K, uint8_t *qx, float *sx, hipStream_t stream) {
    const int G = fp8_blocks(K);
    hipLaunchKernelGGL(fp8_quantize_kernel,
                       dim3((M + kF8QRows - 1) / kF8QRows, (G + kF8QGroups - 1) / kF8QGroups), dim3(kF8QThreads), 0,
                       stream, X, M, K, G, qx, sx);
    return hipGetLastError();
}

template <int WN, int WM, int TN, int TM, int NS, int KW, bool kWide>
static hipError_t launch_tile(const uint8_t *qx, const float *sx, const uint8_t *qw, const float *sw,
                              const uint16_t *bias, int M, int N, int K, void *Y, hipStream_t stream) {
    constexpr int BN = 16 * WN * TN, BM = 16 * WM * TM;
    const int tiles_n = (N + BN - 1) / BN, tiles_m = (M + BM - 1) / BM;
    hipLaunchKernelGGL((fp8_gemm_kernel<WN, WM, TN, TM, NS, KW, kWide>), dim3(tiles_n * tiles_m),
                       dim3(64 * WN * WM * KW), 0, stream, qx, sx, qw, sw, bias, M, N, K, Y, tiles_n);
    return hipGetLastError();
}

// As many columns per block as leave one block for each compute unit, up to 64:
// the tokens are read, and with kFused quantized, once per block. Beyond that,
// 32. Times in us of codes, 1 token / 16 tokens: N = 2560, K = 5120, 16 columns 5.3 /
// 7.5, 32 columns 7.5 / 9.6; 5120 x 5120 16 columns 8.4 / 12.0, 32 7.6 / 9.6, 64 11.8 /
// 14.4; N = 16384, K = 4096 32 columns 13.8 / 15.0, 64 11.7 / 12.8; N = 20480, K = 2048
// 32 9.1 / 11.4, 64 11.2 / 12.6. 16 waves for 16 columns, and for 32 where they
// share the quantization and have a group of K each (8 tokens, 5120 x 5120: 11.8,
// with 8 waves 14.3; of codes 9.2 and 8.6).
template <bool kWide, bool kFused>
static hipError_t launch_skinny(const uint8_t *qx, const float *sx, const uint16_t *X, const uint8_t *qw,
                                const float *sw, const uint16_t *bias, int M, int N, int K, void *Y, size_t lds,
                                hipStream_t stream) {
    const int tiles = (N + 15) / 16;
    const auto launch = [&](auto kernel, int columns, int waves) {
        hipLaunchKernelGGL(kernel, dim3((N + columns - 1) / columns), dim3(64 * waves), lds, stream, qx, sx, X, qw, sw,
                           bias, M, N, K, Y);
        return hipGetLastError();
    };
    if (tiles <= kF8Cus) return launch(fp8_skinny_kernel<16, 1, kWide, kFused>, 16, 16);
    if (tiles > 2 * kF8Cus && tiles <= 4 * kF8Cus) return launch(fp8_skinny_kernel<8, 4, kWide, kFused>, 64, 8);
    if constexpr (kFused)
        if (fp8_blocks(K) > 8) return launch(fp8_skinny_kernel<16, 2, kWide, true>, 32, 16);
    return launch(fp8_skinny_kernel<8, 2, kWide, kFused>, 32, 8);
}

template <bool kWide>
static hipError_t launch_gemm(const uint8_t *qx, const float *sx, const uint8_t *qw, const float *sw,
                              const uint16_t *bias, int M, int N, int K, void *Y, hipStream_t stream) {
    const auto tiles = [&](int64_t tn, int64_t tm) { return ((N + tn - 1) / tn) * ((M + tm - 1) / tm); };
    // Up to 16 tokens: where the linear is one launch by the kernel for few tokens,
    // its product alone gives the same bits. Elsewhere bf16 of more than 8 tokens is
    // faster in tiles, which read them once for 32 or 64 columns: 8 tokens, 5120 x
    // 5120 (K x N) 8.5 / 7.6 us, 4096 x 8192 7.8 / 8.2, 12288 x 1024 11.6 / 12.2; 16 tokens
    // 9.7 / 7.8, 8.8 / 8.4, 13.7 / 12.2; fp32 9.8 / 10.0, 8.9 / 9.2, 13.7 / 18.0.
    const bool few = M <= (kWide ? kF8SkinnyTokens : 8) ||
                     (M <= kF8SkinnyTokens && (fp8_linear_in_one(M, N, K) || tiles(64, 32) > kF8Cus));
    if (few) return launch_skinny<kWide, false>(qx, sx, nullptr, qw, sw, bias, M, N, K, Y, 0, stream);
    // The smallest tile of which no compute unit has more than one: the larger, the
    // less each operand is read; the smaller, the more compute units have one, and
    // the more parts of K fit into LDS (4, 4, 2, 2 and, of 128 x 128, 1 for bf16 and 2
    // for fp32, whose sums are slower). Times in us of M x 5120 x 5120, bf16 / fp32:
    // M = 32 in tiles of 32 x 32 8.0 / 9.9, of 64 columns x 32 tokens 10.1 / 11.4, of
    // 64 x 64 11.0 / 17.4; M = 96 13.5 / 18.1, 10.0 / 11.8, 11.6 / 17.9; M = 160 26 / 34, 20
    // / 22, 11.7 / 18.1; M = 256 in 64 x 64 22.4 / 34.3, 64 columns x 128 tokens 16.9 /
    // 28.6, 128 x 128 22.7 / 40.8; M = 512 33.3 / 51.3, 31.8 / 51.8, 22.9 / 41.2.
    const int64_t small = tiles(64, 64), medium = tiles(128, 128);
    if (tiles(32, 32) <= kF8Cus) return launch_tile<1, 1, 2, 2, 3, 4, kWide>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
    if (tiles(64, 32) <= kF8Cus) return launch_tile<2, 1, 2, 2, 3, 4, kWide>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
    if (small <= kF8Cus) return launch_tile<2, 2, 2, 2, 3, 2, kWide>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
    if (tiles(64, 128) <= kF8Cus) return launch_tile<2, 2, 2, 4, 3, 2, kWide>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
    if constexpr (kWide) {
        // beyond, several small blocks on a compute unit, or two of 128 x 128: M = 1024
        // 65.8 / 74.4, 1280 89.7 / 75.1, 4608 292 / 232
        if (medium <= kF8Cus) return launch_tile<2, 2, 4, 4, 2, 2, true>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
        if (small <= 6 * kF8Cus) return launch_tile<2, 2, 2, 2, 3, 1, true>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
        return launch_tile<2, 2, 4, 4, 2, 1, true>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
    } else {
        // 8 waves and three stages of a 128 x 128 tile, 4 waves and two where two
        // blocks share a compute unit (M = 768 25.4, 1024 45.1 / 35.0, 37.9); 256 x 256
        // from half a round of them on (M = 1536 46.6, with 128 42.2; 2048 57, with 128 73)
        const int64_t big = tiles(256, 256);
        if (medium <= kF8Cus) return launch_tile<2, 4, 4, 2, 3, 1, false>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
        if (big < kF8Cus / 2) return launch_tile<2, 2, 4, 4, 2, 1, false>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
        // the tiles of a last round that would leave half the compute units
        // idle are shared by two blocks each
        const int rest = (int)(big % kF8Cus), split = rest <= kF8Cus / 2 ? rest : 0;
        hipLaunchKernelGGL(fp8_gemm256_kernel, dim3((unsigned)(big + split)), dim3(512), 0, stream, qx, sx, qw, sw,
                           bias, M, N, K, Y, (N + 255) / 256, (int)big, (int)big - split);
        return hipGetLastError();
    }
}

template <bool kWide>
static hipError_t launch_few(const uint16_t *X, const uint8_t *qw, const float *sw, const uint16_t *bias, int M, int N,
                             int K, void *Y, hipStream_t stream) {
    const size_t lds = (size_t)M * fp8_blocks(K) * (kF8Block + sizeof(float));
    return launch_skinny<kWide, true>(nullptr, nullptr, X, qw, sw, bias, M, N, K, Y, lds, stream);
}

// Every block quantizes all tokens anew: one launch pays where a block does not do
// it for too many groups (a token's 128 features; its threads do 32 or 64 at a
// time), nor a compute unit in all its blocks. Times of a call in us, in one / two
// launches: 1 x 5120 x 5120 (M x K x N) 8.2 / 11.0, 6 x 5120 x 5120 10.5 / 11.8, 16
// x 2048 x 2048 6.8 / 8.5, 8 x 4096 x 4096 8.8 / 9.2, 2 x 8192 x 8192 14.9 / 16.8, 8 x
// 2048 x 12288 9.9 / 10.2, 1 x 5120 x 30720 29.3 / 32.4, 4 x 2048 x 151936 54 / 58; 8 x
// 5120 x 5120 11.9 / 11.8, 12 x 4096 x 4096 11.8 / 10.5, 13 x 2048 x 12288 11.4 / 10.7.
// At most 256 groups: 34 KB of LDS.
bool fp8_linear_in_one(int M, int N, int K) {
    const int64_t groups = (int64_t)M * fp8_blocks(K), rounds = ((int64_t)N + 32 * kF8Cus - 1) / (32 * kF8Cus);
    return M <= kF8SkinnyTokens && (groups <= 64 || groups * rounds <= 256);
}

hipError_t launch_fp8_linear_in_one(const uint16_t *X, const uint8_t *qw, const float *sw, const uint16_t *bias,
                                    int M, int N, int K, void *Y, bool y_f32, hipStream_t stream) {
    return y_f32 ? launch_few<true>(X, qw, sw, bias, M, N, K, Y, stream)
                 : launch_few<false>(X, qw, sw, bias, M, N, K, Y, stream);
}

hipError_t launch_fp8_gemm(const uint8_t *qx, const float *sx, const uint8_t *qw, const float *sw,
                           const uint16_t *bias, int M, int N, int K, void *Y, bool y_f32, hipStream_t stream) {
    return y_f32 ? launch_gemm<true>(qx, sx, qw, sw, bias, M, N, K, Y, stream)
                 : launch_gemm<false>(qx, sx, qw, sw, bias, M, N, K, Y, stream);
}

}  // namespace svdq
