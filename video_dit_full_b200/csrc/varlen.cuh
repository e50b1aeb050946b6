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

// Tile `target` of the tiles that all sequences' query rows split into, `rows` to a tile and each sequence
// starting a tile of its own: the sequence and the tile within it, or seq = -1 past the last.  The whole
// warp calls it; 32 sequences a step, a sequence to a lane, so no table has to be built (and no extra launch
// made) before the attention kernel.  Up to 32 sequences are taken longest first, so that the work handed
// out last is short; more are taken as they come.  `scan` keeps the step where the last target was found:
// targets that grow are found from there on, without reading the offsets again.
struct TileAt {
    int seq, tile, tiles;          // tiles: of that sequence
    Span q, k;
};
struct TileScan {
    int n0 = -1, before = 0;       // first sequence of the step (-1: none read yet), tiles before it
    Span q, k;                     // this lane's sequence
    int mine, upto;                // its tiles; the step's up to and including it
};
__device__ __forceinline__ void scan_step(const int* cu_q, const int* cu_k, int N, int Tq, int Tk, int rows, int n0,
                                          TileScan& scan) {
    const int lane = threadIdx.x & 31;
    const bool here = n0 + lane < N;
    scan.n0 = n0;
    scan.q = here ? span_of(cu_q, n0 + lane, Tq) : Span{0, 0};
    scan.k = here ? span_of(cu_k, n0 + lane, Tk) : Span{0, 0};
    const int mine = (scan.q.len + rows - 1) / rows;
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
__device__ __forceinline__ TileAt tile_at(const int* cu_q, const int* cu_k, int N, int Tq, int Tk, int rows, int target,
                                          TileScan& scan) {
    if (scan.n0 < 0 || target < scan.before) {
        scan.before = 0;
        scan_step(cu_q, cu_k, N, Tq, Tk, rows, 0, scan);
    }
    while (true) {
        const unsigned here = __ballot_sync(0xffffffffu, scan.before + scan.upto > target &&
                                                             scan.before + scan.upto - scan.mine <= target);
        if (here) {
            const int l = __ffs(here) - 1;
            auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, l); };
            const int tiles = of(scan.mine);
            return {scan.n0 + l, target - scan.before - of(scan.upto) + tiles, tiles,
                    {of(scan.q.begin), of(scan.q.len)}, {of(scan.k.begin), of(scan.k.len)}};
        }
        if (scan.n0 + 32 >= N) return {-1, 0, 0, {0, 0}, {0, 0}};
        scan.before += static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(scan.mine)));
        scan_step(cu_q, cu_k, N, Tq, Tk, rows, scan.n0 + 32, scan);
    }
}

}  // namespace varlen
}  // namespace wan
