// Ragged batches of new tokens, shared by the kernels that take several tokens
// of several sequences in one call (rope_chunk.cu, attention_chunk.cu).
//
// Rows q_start[b] .. q_start[b + 1] - 1 of the call's tensors are the new tokens
// of sequence b, and ctx_len[b] counts that sequence's tokens including them, so
// new token i of n stands at position ctx_len[b] - n + i.
#pragma once

#include "common.cuh"

namespace i4 {

// The "pdl" option: the kernels of these calls start while the one before ends, and wait (grid_dep_wait) before they read or
// write any memory.
extern bool g_pdl;

// The rows of sequence b, clamped to the T rows that exist: (first row, number of rows).
__device__ __forceinline__ int2 chunk_rows(const int32_t *q_start, int b, int T) {
    const int a = min(max(q_start[b], 0), T), e = min(max(q_start[b + 1], 0), T);
    return make_int2(a, max(e - a, 0));
}

// The sequence that row t belongs to: the number of ends q_start[1..B] that are <= t (B for a row behind the
// last sequence). A 32-way search by one warp: B <= 32 takes one load, B <= 1024 two.
__device__ __forceinline__ int chunk_find(const int32_t *q_start, int B, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = B;
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int i = (lane + 1) * step - 1;
        const bool below = i < len && q_start[1 + lo + i] <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, below));
        lo += c * step;
        len = min(step - 1, len - c * step);
    }
    return lo;
}

}  // namespace i4
