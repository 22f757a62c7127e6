// What the kernels on the paged KV cache share: where a query row stands in a
// batch of sequences.
//
// Query rows of all sequences lie behind each other; q_start[0 .. B] are their
// borders.  Row t belongs to the last sequence whose start is <= t, if t lies
// before that sequence's end.  Every index that these functions read with is
// bounded by B alone, so that borders that do not rise give wrong places, and
// never a read outside the arrays.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace spin {

// What a sequence's new tokens count their places back from: its length, which may pass its table (tokens there have no
// page, and the others keep their places), held to numbers that positions behind a prefix fit 32 bits with.
__device__ __forceinline__ int placed(int kv_len) { return min(max(kv_len, 0), 1 << 30); }

// The sequence of row t, or -1, found by the 16 lanes of a DPP row together (l
// = 0 .. 15 its lane, all 16 with the same t): a 16-way search, one load deep
// per factor of 16 in B.
__device__ __forceinline__ int find_sequence16(const int32_t* __restrict__ q_start, int B, int t, int l) {
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 15) >> 4;
        const int at = l * step;
        const bool before = at < n && q_start[lo + at] <= t;
        const int seen = __popcll((__ballot(before) >> (threadIdx.x & 48)) & 0xFFFFull);
        const int skip = max(seen - 1, 0) * step;
        lo += skip;
        n = min(step, n - skip);
    }
    return q_start[lo] <= t && t < q_start[lo + 1] ? lo : -1;
}

// The last of 0 .. B - 1 that `before` holds for (it holds up to there, and not behind), or 0: by the 64 lanes of a wave
// together, one load deep per factor of 64 in B.
template <typename F>
__device__ __forceinline__ int find_last64(int B, int lane, F before) {
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int at = lane * step;
        const bool yes = at < n && before(lo + at);
        const int seen = __popcll(__ballot(yes));
        const int skip = max(seen - 1, 0) * step;
        lo += skip;
        n = min(step, n - skip);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The sequence of row t, or -1, by one lane alone: a binary search.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ q_start, int B, int t) {
    int lo = 0, n = B;
    while (n > 1) {
        const int half = n >> 1;
        const bool before = q_start[lo + half] <= t;
        lo += before ? half : 0;
        n = before ? n - half : half;
    }
    return q_start[lo] <= t && t < q_start[lo + 1] ? lo : -1;
}

}  // namespace spin
