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

// Tile `target` of the tiles that all sequences' rows (on the axis of `cu`) split into, `rows` to a
// tile and each sequence starting a tile of its own: the sequence and the tile within it, or seq = -1
// past the last.  The whole warp calls it; 32 sequences a step, so no table has to be built (and no
// extra launch made) before the attention kernel.  Up to 32 sequences are taken longest first, so that
// the work handed out last is short; more are taken as they come.  `from`
// keeps the step where the last target was found: targets that grow are found from there on.
struct TileAt {
    int seq, tile, tiles;          // tiles: of that sequence
};
struct ScanFrom {
    int n0 = 0, before = 0;        // first sequence of the step, tiles before it
};
__device__ __forceinline__ TileAt tile_at(const int* cu, int N, int T, int rows, int target, ScanFrom& from) {
    const int lane = threadIdx.x & 31;
    if (target < from.before) from = ScanFrom{};
    int before = from.before;
    for (int n0 = from.n0; n0 < N; n0 += 32) {
        const int mine = n0 + lane < N ? (span_of(cu, n0 + lane, T).len + rows - 1) / rows : 0;
        int upto;                                  // tiles up to and including this lane's sequence
        if (N <= 32) {
            upto = 0;
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
        const unsigned here = __ballot_sync(0xffffffffu, before + upto > target && before + upto - mine <= target);
        if (here) {
            const int l = __ffs(here) - 1;
            from.n0 = n0;
            from.before = before;
            const int tiles = __shfl_sync(0xffffffffu, mine, l);
            return {n0 + l, target - before - __shfl_sync(0xffffffffu, upto, l) + tiles, tiles};
        }
        before += __reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine));
    }
    return {-1, 0, 0};
}

}  // namespace varlen
}  // namespace wan
