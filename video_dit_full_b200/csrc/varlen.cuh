// Device helpers of the packed attention kernels: where a sequence lies on the token axes.
#pragma once

#include "wan_attn_internal.h"

namespace wan {
namespace varlen {

// Rows [begin, begin + len) of sequence n on an axis of T tokens, offsets clipped to [0, T].
struct Span {
    int begin, len;
};
__device__ __forceinline__ Span span_of(const int* cu, int n, int T) {
    const int a = min(max(cu[n], 0), T), b = min(max(cu[n + 1], 0), T);
    return {a, max(b - a, 0)};
}

// The sequence that owns token t: the last n with cu[n] <= t, if t < cu[n + 1]; else -1.
__device__ __forceinline__ int sequence_of(const int* cu, int N, int t) {
    int lo = 0, hi = N + 1;                     // cu[lo - 1] <= t < cu[hi] (with cu[-1] = -inf, cu[N + 1] = inf)
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return (lo >= 1 && lo <= N) ? lo - 1 : -1;
}

}  // namespace varlen
}  // namespace wan
