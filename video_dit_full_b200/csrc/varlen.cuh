// Device helpers of the packed attention kernels: where a sequence lies on the token axes.
#pragma once

#include <climits>

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

// Item `target` of all sequences' items: the sequence and the item within it, or seq = -1 past the last.  A
// sequence has an item for every `rows` of its queries (the last may have fewer) and every `keys` of its keys
// (keys = 0: for all of its keys; one for a sequence without keys).  The whole warp calls it; 32 sequences a
// step, a sequence to a lane, so no table has to be built (and no extra launch made) before the attention
// kernel.  Up to 32 sequences are taken by their number of items, most first, so that the work handed out last
// is short; more are taken as they come.  `scan` keeps the step where the last target was found: targets that
// grow are found from there on, without reading the offsets again.
struct ItemAt {
    int seq, item, items;          // items: of that sequence
    Span q, k;
};
struct ItemScan {
    int n0 = -1, before = 0;       // first sequence of the step (-1: none read yet), items before it
    int total = INT_MAX;           // of all sequences, once known
    Span q, k;                     // this lane's sequence
    int mine, upto;                // its items; the step's up to and including it
};
// The join kernel's number of parts of a token's sequence, as the forward stored it.  A forward that timed out
// may have left the workspace as it was: never more than the plan's most, and 1 (nothing to join) for no count.
__host__ __device__ inline int parts_to_join(int stored, int most) { return stored < 1 ? 1 : stored < most ? stored : most; }
__device__ __forceinline__ int parts_of(int len, int size) { return (len + size - 1) / size; }
__device__ __forceinline__ void scan_step(const int* cu_q, const int* cu_k, int N, int Tq, int Tk, int rows, int keys,
                                          int n0, ItemScan& scan) {
    const int lane = threadIdx.x & 31;
    const bool here = n0 + lane < N;
    scan.n0 = n0;
    scan.q = here ? span_of(cu_q, n0 + lane, Tq) : Span{0, 0};
    scan.k = here ? span_of(cu_k, n0 + lane, Tk) : Span{0, 0};
    const int mine = parts_of(scan.q.len, rows) * (keys ? max(parts_of(scan.k.len, keys), 1) : 1);
    int upto;
    if (N <= 32) {
        upto = 0;
#pragma unroll 4
        for (int l = 0; l < N; ++l) {
            const int o = __shfl_sync(0xffffffffu, mine, l);
            if (o > mine || (o == mine && l <= lane)) upto += o;
        }
    } else {
        upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += o;
        }
    }
    scan.mine = mine;
    scan.upto = upto;
}
__device__ __forceinline__ ItemAt item_at(const int* cu_q, const int* cu_k, int N, int Tq, int Tk, int rows, int keys,
                                          int target, ItemScan& scan) {
    if (target >= scan.total) return {-1, 0, 0, {0, 0}, {0, 0}};
    if (scan.n0 < 0 || target < scan.before) {
        scan.before = 0;
        scan_step(cu_q, cu_k, N, Tq, Tk, rows, keys, 0, scan);
    }
    while (true) {
        const unsigned here = __ballot_sync(0xffffffffu, scan.before + scan.upto > target &&
                                                             scan.before + scan.upto - scan.mine <= target);
        if (here) {
            const int l = __ffs(here) - 1;
            auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, l); };
            const int items = of(scan.mine);
            return {scan.n0 + l, target - scan.before - of(scan.upto) + items, items,
                    {of(scan.q.begin), of(scan.q.len)}, {of(scan.k.begin), of(scan.k.len)}};
        }
        const int upto = scan.before + static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(scan.mine)));
        if (scan.n0 + 32 >= N) {
            scan.total = upto;
            return {-1, 0, 0, {0, 0}, {0, 0}};
        }
        scan.before = upto;
        scan_step(cu_q, cu_k, N, Tq, Tk, rows, keys, scan.n0 + 32, scan);
    }
}

}  // namespace varlen
}  // namespace wan
