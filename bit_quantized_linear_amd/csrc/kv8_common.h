// Shared by the kernels on the 8-bit key and value cache (kv8_append.hip,
// kv8_attention.hip): what a batch's device arrays say of one sequence, held
// within the buffers whatever they contain.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"

namespace svdq {

constexpr int kKvPage = SVDQ_KV8_PAGE;

// The batch of a call: rows starts[b] .. starts[b + 1] - 1 of T are the newest
// tokens of sequence b, which has lengths[b] tokens in the pages table[b].
struct KvSeq {
    int row0, rows;  // the new tokens' rows
    int length;      // tokens in the cache, the new ones among them
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatch &kv, int b) {
    KvSeq s;
    s.row0 = min(max(kv.starts[b], 0), kv.T);
    s.rows = min(max(kv.starts[b + 1], s.row0), kv.T) - s.row0;
    s.length = min(max(kv.lengths[b], 0), kv.max_pages * kKvPage);
    return s;
}

// Page number of a sequence's page p, or -1 where the table has none there.
__device__ __forceinline__ int kv_page(const KvBatch &kv, int b, int p) {
    const int page = kv.table[(int64_t)b * kv.max_pages + p];
    return page >= 0 && page < kv.num_pages ? page : -1;
}

// Work item `item` of a batch whose sequence b has count(sequence) of them: the
// sequence, in b and seq, and the number within it, or false past the last. A wave
// looks at 64 sequences at a time; every lane takes part and has the same answer.
template <class Count>
__device__ __forceinline__ bool kv_find(const KvBatch &kv, int item, int &b, KvSeq &seq, int &within, Count count) {
    const int lane = threadIdx.x & 63;
    for (int b0 = 0; b0 < kv.B; b0 += 64) {
        const KvSeq mine = kv_seq(kv, min(b0 + lane, kv.B - 1));
        const int n = b0 + lane < kv.B ? count(mine) : 0;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int other = __shfl_up(upto, d);
            upto += lane >= d ? other : 0;
        }
        const uint64_t past = __ballot(item < upto);
        if (past) {
            const int at = __ffsll((unsigned long long)past) - 1;
            b = b0 + at;
            seq.row0 = __builtin_amdgcn_readlane(mine.row0, at);
            seq.rows = __builtin_amdgcn_readlane(mine.rows, at);
            seq.length = __builtin_amdgcn_readlane(mine.length, at);
            within = item - __builtin_amdgcn_readlane(upto - n, at);
            return true;
        }
        item -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

}  // namespace svdq
