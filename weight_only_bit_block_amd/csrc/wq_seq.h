// wq_seq.h -- packed sequences on the device: which sequence a token or a tile
// belongs to. cu holds B + 1 nondecreasing token offsets; whatever it holds,
// every range returned here lies inside [0, T].
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wq {

struct SeqRange {
    int begin, end;      // tokens; empty when begin >= end
};

__device__ __forceinline__ int clamp_token(int x, int T) { return x < 0 ? 0 : x > T ? T : x; }

__device__ __forceinline__ SeqRange seq_range(const int32_t *cu, int T, int b)
{
    if (!cu) return {0, T};
    return {clamp_token(cu[b], T), clamp_token(cu[b + 1], T)};
}

// The sequence that holds token t: the last b with cu[b] <= t, which is the
// nonempty one where several start there. The caller checks t < end (tokens
// before cu[0] and after cu[B] have no sequence).
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int B, int t)
{
    if (!cu) return 0;
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace wq
