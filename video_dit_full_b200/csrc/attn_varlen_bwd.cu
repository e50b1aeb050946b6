// Packed attention backward on sm_100a: gradients for sequences of different lengths on one token
// axis, full or causal, grouped heads.
//
// With P_ij = 2^(s_ij - lse_i log2 e) for the pairs that row i sees (0 elsewhere), D_i = dO_i . O_i and
// dS = P (dP - D), dP = dO V^T:
//     dV = P^T dO,  dK = dS^T Q / sqrt(D),  dQ = dS K / sqrt(D);  dK, dV summed over a group's query heads.
//
// Three kernels:
//   varlen_prep  D_i (fp32), zeroing of the fp32 dQ accumulator, and (one block) the key tiles of all
//                sequences in the order of their work, most first
//   varlen_main  one CTA per 128-key tile of a sequence and kv head.  K_j and V_j stay in shared memory
//                while the CTA walks the 128-row Q tiles that see any of its keys, of all query heads of the
//                group: dK and dV gather the group's sum in TMEM, with no atomics.  A Q tile's rows are
//                (token, query head) pairs, as many heads to a token as the largest power of two in the
//                group: a short sequence then fills its tiles better (700 sequences of 1 to 30 tokens, 8
//                heads over 2: 136 us against 254 with a head to a tile).  Per Q tile
//                the five products of the dense backward, with the same roles (8 gradient warps, two
//                threads per key row; TMA producer; tcgen05 issuer; dQ reducer):
//                  S^T = K Q^T, dP^T = V dO^T;  dV += P^T dO;  dK += dS^T Q;  dQ^T = K^T dS^T -> TMA reduce-add
//   varlen_cast  dQ (and split dK, dV) = bf16(accumulator x scale), rows of the sequences only
// What packing adds:
//   - causal: Q tiles before the diagonal are never loaded; key tiles then differ by the length of a
//     sequence in Q tiles, so the ones with most start first, of the kv heads of a group in turn (HeadOrder;
//     head by head the last head's longest tile starts late: 571 us against 443 for packed documents of 5 to
//     2049 tokens; all heads in turn, a wave reads every head's Q and dO and adds to every head's dQ, past L2:
//     16384 tokens of 40 heads 8.6 ms against 7.9)
//   - pairs that do not see each other get P = 0 and dS = 0 by selection, never by arithmetic, so that an
//     infinite or NaN score, lse or dP there leaves no trace (diagonal and edge tiles only)
//   - rows behind the sequence in an edge tile belong to another one: K, Q and dO rows there are zeroed in
//     shared memory before the tensor core reads them (0 x NaN is NaN), and what is added into their
//     dQ, dK, dV accumulators is exactly zero
//   - rows that see no key (causal, more queries than keys) are zeroed there too: their dO, a gradient at
//     o = 0, is often not finite
//   - few key tiles: gridDim.z CTAs split a tile's Q tiles and add dK, dV into fp32 accumulators
#include <cuda.h>

#include "sm100_ptx.cuh"
#include "varlen.cuh"

namespace wan {
namespace varlen_bwd {

using varlen::Span;
using varlen::span_of;

constexpr int BM = 128;                  // keys per CTA and queries per Q tile
constexpr int HD = 128;
constexpr int TILE_BYTES = BM * HD * 2;  // 32 KB bf16 tile
constexpr int HALF_BYTES = TILE_BYTES / 2;

constexpr int OFF_K = 0;
constexpr int OFF_V = OFF_K + TILE_BYTES;
// Two stages of [Q_i | dO_i] (64 KB each).  Within a tile, dS^T overwrites dO_i once dV is done;
// after the dK and dQ MMAs the whole stage holds the fp32 dQ^T tile [query][d] for the TMA reduce.
constexpr int OFF_STAGE = OFF_V + TILE_BYTES;
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int OFF_VEC = OFF_STAGE + 2 * STAGE_BYTES;   // per warp: 64 fp32 lse*log2(e), 64 fp32 D_i
constexpr int VEC_BYTES = 2 * 64 * 4;
constexpr int OFF_BAR = OFF_VEC + 8 * VEC_BYTES;
enum Bar { KV_FULL = 0, QDO_FULL = 1, QDO_EMPTY = 3, S_FULL = 5, DP_FULL = 6, P_READY = 7, DV_DONE = 8,
           DS_READY = 9, DQ_FULL = 10, DQ_DRAINED = 11, FINAL = 12, DRAIN = 13, STAGED = 14, DS_SMEM = 15,
           RED_DONE = 16, EPI_STAGED = 17, EDGE = 18, NBARS = 19 };
// split epilogue: dV (stage 0) and dK (stage 1) as four [128 key][32 d] fp32 sub-tiles each,
// 128-byte swizzled, one TMA reduce-add per sub-tile
constexpr int SUB_BYTES = BM * 32 * 4;
constexpr int OFF_TMEM_SLOT = OFF_BAR + NBARS * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
constexpr int SMEM_BYTES = OFF_ABORT + 8 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");
// warps 0-7 gradients (two threads per key row: warps 0-3 take queries 0-63 of a tile,
// warps 4-7 queries 64-127), 8 TMA, 9 MMA, 10 dQ reducer
constexpr int NTHREADS = 352;
constexpr int WARP_TMA = 8, WARP_MMA = 9, WARP_RED = 10;
constexpr int G_WARPS = 8;
constexpr uint32_t TMEM_COLS = 512;      // S^T | dP^T | dV | dK
constexpr uint32_t T_S = 0, T_DP = 128, T_DV = 256, T_DK = 384;
constexpr float LOG2E = 1.4426950408889634f;

// A gradient warp's arrival, after every lane's writes and fences: one per warp.
__device__ __forceinline__ void g_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// The 8 MMAs of K = 16 of a 128 x 128 x 128 product: both operands K-major in shared memory; A in TMEM
// (columns of K = 64-127 64 past those of 0-63) and B MN-major; both MN-major.
__device__ __forceinline__ void mma_kmajor(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc) {
    mma8_f16_ss<HALF_BYTES / 16, 2>(d, sdesc_lo(a, 16), sdesc_lo(b, 16), hi, idesc, 0u);
}
__device__ __forceinline__ void mma_ts_bmn(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t hi, uint32_t idesc,
                                           bool accumulate) {
    mma8_f16_ts<64, 512, 128>(d, a_tmem, sdesc_lo(b, HALF_BYTES), hi, idesc, accumulate ? 1u : 0u);
}
__device__ __forceinline__ void mma_ss_mn(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc) {
    mma8_f16_ss<512, 128>(d, sdesc_lo(a, HALF_BYTES), sdesc_lo(b, HALF_BYTES), hi, idesc, 0u);
}

// The first Q tile that sees any key of key tile `tile` of a sequence, and how many do.
__device__ __forceinline__ int first_q_tile(const VarlenBwdParams& p, Span sq, Span sk, int tile) {
    return p.causal ? max(tile * BM - (sk.len - sq.len), 0) / (BM >> p.pack_log2) : 0;
}
__device__ __forceinline__ int q_tiles(const VarlenBwdParams& p, Span sq, Span sk, int tile) {
    const int tokens = BM >> p.pack_log2;
    return max((sq.len + tokens - 1) / tokens - first_q_tile(p, sq, sk, tile), 0);
}

// A CTA's walk over its Q tiles: the tile, counted from the first, of the packed head, counted from the group's.
struct Walk {
    int tile, head, per_head;
    __device__ __forceinline__ Walk(int it0, int per_head_) : tile(0), head(0), per_head(per_head_) {
        if (per_head > 0) {
            head = it0 / per_head;
            tile = it0 - head * per_head;
        }
    }
    __device__ __forceinline__ void next() {
        if (++tile == per_head) {
            tile = 0;
            ++head;
        }
    }
};

// One warp: zero rows [first, end) of a tile (two halves of d, a row 128 bytes of each).
__device__ __forceinline__ void zero_rows(uint32_t tile, int first, int end, int lane) {
    for (int half = 0; half < 2; ++half)
        for (int c = lane; c < (end - first) * 8; c += 32)
            st_shared_v4(tile + half * HALF_BYTES + first * 128 + c * 16, 0u, 0u, 0u, 0u);
}

__global__ void __launch_bounds__(NTHREADS, 1)
varlen_main_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmdo,
                   const __grid_constant__ CUtensorMap tmdq, const __grid_constant__ CUtensorMap tmdk,
                   const __grid_constant__ CUtensorMap tmdv, const VarlenBwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_addr);

    const int warp = warp_id();
    const int lane = lane_id();
    int unit, hk;
    p.heads.at(blockIdx.x, unit, hk);
    const int group = p.H / p.Hkv;
    grid_dependency_wait();
    const int2 at = p.order[unit];          // sequence, key tile
    if (at.x < 0) return;                                 // the grid is an upper bound
    const Span sq = span_of(p.cu_q, at.x, p.Tq), sk = span_of(p.cu_k, at.x, p.Tk);
    const int kv0 = at.y * BM;
    const int shift = sk.len - sq.len;                    // causal: query i sees keys 0 .. i + shift
    // Q tiles [i_first, i_first + per_head) of every packed head; this split's run [it0, it0 + n)
    const int pack_log2 = p.pack_log2, tokens = BM >> pack_log2;
    const int i_first = first_q_tile(p, sq, sk, at.y), per_head = q_tiles(p, sq, sk, at.y);
    const int all = per_head * (group >> pack_log2);
    const int it0 = static_cast<int>(static_cast<long long>(blockIdx.z) * all / p.splits);
    const int n = static_cast<int>(static_cast<long long>(blockIdx.z + 1) * all / p.splits) - it0;

    const uint32_t sK = base + OFF_K, sV = base + OFF_V;
    auto sQ = [&](int s) { return base + OFF_STAGE + s * STAGE_BYTES; };
    auto sDO = [&](int s) { return base + OFF_STAGE + s * STAGE_BYTES + TILE_BYTES; };
    const uint32_t bar0 = base + OFF_BAR;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const WaitCtl wc{abort_flag, p.wait_budget_ns, p.status};

    if (threadIdx.x == 0) {
        mbar_init(bar(KV_FULL), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(QDO_FULL + s), 1);
            mbar_init(bar(QDO_EMPTY + s), 2);    // the MMAs' commit + the dQ reducer's read-out
        }
        mbar_init(bar(S_FULL), 1);
        mbar_init(bar(DP_FULL), 1);
        mbar_init(bar(P_READY), G_WARPS);
        mbar_init(bar(DV_DONE), 1);
        mbar_init(bar(DS_READY), G_WARPS);        // dS^T in TMEM (dK may start)
        mbar_init(bar(DS_SMEM), G_WARPS);         // dS^T in shared memory (dQ may start)
        mbar_init(bar(DQ_FULL), 1);
        mbar_init(bar(DQ_DRAINED), G_WARPS);
        mbar_init(bar(FINAL), 1);
        mbar_init(bar(DRAIN), 1);
        mbar_init(bar(STAGED), G_WARPS);
        mbar_init(bar(RED_DONE), 1);
        mbar_init(bar(EPI_STAGED), G_WARPS);
        mbar_init(bar(EDGE), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(base + OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

    if (warp == WARP_TMA) {
        // ------------------------------ TMA producer ------------------------------
        // The whole warp walks the tiles, lane 0 issues.  A tile with rows behind the sequence, or rows that
        // see no key, lands on EDGE; the warp zeroes those rows and only then hands the tile over.
        if (n > 0) {
            const int kv_rows = min(sk.len - kv0, BM);
            const uint32_t kv_bar = bar(kv_rows < BM ? EDGE : KV_FULL);
            int edge = 0;                                  // EDGE phases used so far
            if (lane == 0) {
                tma_prefetch_desc(&tmq);
                tma_prefetch_desc(&tmdo);
                mbar_arrive_expect_tx(kv_bar, 2 * TILE_BYTES);
                tma_load_3d(sK, &tmk, kv_bar, 0, hk, sk.begin + kv0);
                tma_load_3d(sK + HALF_BYTES, &tmk, kv_bar, 64, hk, sk.begin + kv0);
                tma_load_3d(sV, &tmv, kv_bar, 0, hk, sk.begin + kv0);
                tma_load_3d(sV + HALF_BYTES, &tmv, kv_bar, 64, hk, sk.begin + kv0);
            }
            __syncwarp();
            bool ok = true;
            bool pending = kv_rows < BM;                   // copies in flight on EDGE
            if (pending) {
                ok = wait_warp(bar(EDGE), 0, wc);
                if (ok) {
                    pending = false;
                    edge = 1;
                    zero_rows(sK, kv_rows, BM, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(KV_FULL));
                }
            }
            const uint64_t keep = l2_policy_evict_last();
            int par[2] = {-1, -1};
            Walk at_tile(it0, per_head);
            for (int i = 0; i < n && ok; ++i, at_tile.next()) {
                const int s = i & 1;
                const int use = (i >> 1) & 1;
                const int h = hk * group + (at_tile.head << pack_log2), tok0 = (i_first + at_tile.tile) * tokens;
                const int rows = min(sq.len - tok0, tokens) << pack_log2;
                // rows before `seen` see no key (causal, more queries than keys)
                const int seen = p.causal ? min(max(-shift - tok0, 0), tokens) << pack_log2 : 0;
                const bool edge_tile = rows < BM || seen > 0;
                bool got = true;
                if (lane == 0) got = wait_thread(bar(QDO_EMPTY + s), use ^ 1, wc);
                ok = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
                if (!ok) break;
                const uint32_t fb = bar(edge_tile ? EDGE : QDO_FULL + s);
                if (lane == 0) {
                    mbar_arrive_expect_tx(fb, 2 * TILE_BYTES);
                    const int tok = sq.begin + tok0;
                    tma_load_3d_hint(sQ(s), &tmq, fb, 0, h, tok, keep);
                    tma_load_3d_hint(sQ(s) + HALF_BYTES, &tmq, fb, 64, h, tok, keep);
                    tma_load_3d_hint(sDO(s), &tmdo, fb, 0, h, tok, keep);
                    tma_load_3d_hint(sDO(s) + HALF_BYTES, &tmdo, fb, 64, h, tok, keep);
                }
                __syncwarp();
                if (edge_tile) {
                    pending = true;
                    ok = wait_warp(bar(EDGE), edge & 1, wc);
                    if (!ok) break;
                    pending = false;
                    ++edge;
                    zero_rows(sQ(s), 0, seen, lane);
                    zero_rows(sQ(s), rows, BM, lane);
                    zero_rows(sDO(s), 0, seen, lane);
                    zero_rows(sDO(s), rows, BM, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(QDO_FULL + s));
                } else {
                    par[s] = use;
                }
            }
            if (!ok && lane == 0) {
                // let the copies already issued land before the CTA's shared memory goes away
                if (pending) drain_wait(bar(EDGE), edge & 1);
                if (kv_rows == BM) drain_wait(bar(KV_FULL), 0);
                for (int s = 0; s < 2; ++s)
                    if (par[s] >= 0) drain_wait(bar(QDO_FULL + s), par[s]);
            }
        }
    } else if (warp == WARP_MMA) {
        // ------------------------------ MMA issuer --------------------------------
        if (lane == 0 && n > 0) {
            const uint32_t id_kk = make_idesc(1, 1, 1, 0, 0, BM, BM);   // both K-major
            const uint32_t id_tb = make_idesc(1, 1, 1, 0, 1, BM, HD);   // A in TMEM, B MN-major
            const uint32_t id_mm = make_idesc(1, 1, 1, 1, 1, HD, BM);   // both MN-major
            const uint32_t hi = sdesc_hi();
            bool ok = wait_thread(bar(KV_FULL), 0, wc);
            if (ok) ok = wait_thread(bar(QDO_FULL + 0), 0, wc);
            if (ok) {
                tc_fence_after();
                mma_kmajor(tmem + T_S, sK, sQ(0), hi, id_kk);           // S^T = K Q^T of the first tile
                mma_commit(bar(S_FULL));
                mma_kmajor(tmem + T_DP, sV, sDO(0), hi, id_kk);         // dP^T = V dO^T
                mma_commit(bar(DP_FULL));
            }
            for (int i = 0; i < n && ok; ++i) {
                const int s = i & 1;
                const uint32_t q_s = sQ(s), do_s = sDO(s);
                ok = wait_thread(bar(P_READY), i & 1, wc);
                if (!ok) break;
                tc_fence_after();
                mma_ts_bmn(tmem + T_DV, tmem + T_S, do_s, hi, id_tb, i > 0);   // dV += P^T dO
                mma_commit(bar(DV_DONE));
                ok = wait_thread(bar(DS_READY), i & 1, wc);
                if (!ok) break;
                tc_fence_after();
                mma_ts_bmn(tmem + T_DK, tmem + T_DP, q_s, hi, id_tb, i > 0);   // dK += dS^T Q
                ok = wait_thread(bar(DS_SMEM), i & 1, wc);
                if (!ok) break;
                // dQ^T = K^T dS^T (dS^T in dO's buffer) into dP^T's columns, which the dK MMA just
                // read: S^T's columns are free for the next tile at once
                mma_ss_mn(tmem + T_DP, sK, do_s, hi, id_mm);
                mma_commit(bar(DQ_FULL));
                mma_commit(bar(QDO_EMPTY + s));
                if (i + 1 < n) {
                    // the next tile's S^T runs while the gradient warps copy dQ^T out; its dP^T
                    // (needed only after its P) once that copy has freed the columns
                    const int s1 = (i + 1) & 1;
                    ok = wait_thread(bar(QDO_FULL + s1), ((i + 1) >> 1) & 1, wc);
                    if (!ok) break;
                    tc_fence_after();
                    mma_kmajor(tmem + T_S, sK, sQ(s1), hi, id_kk);
                    mma_commit(bar(S_FULL));
                    ok = wait_thread(bar(DQ_DRAINED), i & 1, wc);
                    if (!ok) break;
                    tc_fence_after();
                    mma_kmajor(tmem + T_DP, sV, sDO(s1), hi, id_kk);
                    mma_commit(bar(DP_FULL));
                }
            }
            if (ok) mma_commit(bar(FINAL));
            mma_commit(bar(DRAIN));
            drain_wait(bar(DRAIN), 0);
        }
    } else if (warp == WARP_RED) {
        // ------------------ dQ reducer: TMA reduce-add of each dQ tile ------------
        if (lane == 0 && n > 0) {
            bool ok = true;
            Walk at_tile(it0, per_head);
            for (int i = 0; i < n && ok; ++i, at_tile.next()) {
                ok = wait_thread(bar(STAGED), i & 1, wc);
                if (!ok) break;
                tma_reduce_add_3d(&tmdq, base + OFF_STAGE + (i & 1) * STAGE_BYTES, 0, hk * group + (at_tile.head << pack_log2),
                                  sq.begin + (i_first + at_tile.tile) * tokens);
                bulk_commit_group();
                bulk_wait_read_all();                         // the stage may be refilled now
                mbar_arrive(bar(QDO_EMPTY + (i & 1)));
            }
            bulk_wait_all();
            if (p.splits > 1 && ok) {
                // split Q range: add this CTA's dV and dK tiles into the fp32 accumulators
                mbar_arrive(bar(RED_DONE));                   // the stages are free for them
                ok = wait_thread(bar(EPI_STAGED), 0, wc);
                if (ok) {
                    for (int which = 0; which < 2; ++which)
                        for (int st = 0; st < 4; ++st)
                            tma_reduce_add_3d(which ? &tmdk : &tmdv,
                                              base + OFF_STAGE + which * STAGE_BYTES + st * SUB_BYTES, st * 32, hk,
                                              sk.begin + kv0);
                    bulk_commit_group();
                    bulk_wait_all();
                }
            }
        }
    } else {
        // -------- gradient warps: two threads per key row (or per d for dQ^T) -------
        // Thread (j, hq): key row / TMEM lane j = 32*(warp%4) + lane; query half hq = warp/4
        // covers queries 64hq..64hq+63 of each Q tile.  It writes P^T and dS^T (bf16) into the
        // first 32 of the 64 TMEM columns it has just read, so the halves never race.
        const int hq = warp >> 2;
        const int cb = hq * 64;                            // first query column of this half
        const int j = (warp & 3) * 32 + lane;              // 0..127
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + T_S + lane_off + cb, tDP = tmem + T_DP + lane_off + cb;
        const int key = kv0 + j;
        const bool key_ok = key < sk.len;
        const float c = p.scale_log2;
        // each warp keeps its own copy of its 64 queries' lse / D (no cross-warp barrier needed)
        float* s_lse = reinterpret_cast<float*>(smem + OFF_VEC + warp * VEC_BYTES);
        float* s_del = s_lse + 64;
        bool ok = true;
        // a tile's lse / D come from global memory one tile ahead, so their latency hides
        // behind the previous tile instead of delaying the wait for S^T
        float nl[2], nd[2];
        Walk at_tile(it0, per_head), ahead = at_tile;
        const int row0 = cb + lane, row1 = row0 + 32, heads = (1 << pack_log2) - 1;
        const int tok_row[2] = {row0 >> pack_log2, row1 >> pack_log2};
        const long long at_row[2] = {static_cast<long long>(row0 & heads) * p.Tq + tok_row[0],
                                     static_cast<long long>(row1 & heads) * p.Tq + tok_row[1]};
        auto load_vec = [&]() {
            const int first = (i_first + ahead.tile) * tokens;
            const long long at = static_cast<long long>(hk * group + (ahead.head << pack_log2)) * p.Tq + sq.begin + first;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool there = first + tok_row[e] < sq.len;
                nl[e] = there ? p.lse[at + at_row[e]] * LOG2E : 0.f;
                nd[e] = there ? p.delta[at + at_row[e]] : 0.f;
            }
            ahead.next();
        };
        if (n > 0) load_vec();
        for (int i = 0; i < n && ok; ++i, at_tile.next()) {
            __syncwarp();                                    // previous tile's values no longer read
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s_lse[e * 32 + lane] = nl[e];
                s_del[e * 32 + lane] = nd[e];
            }
            __syncwarp();
            if (i + 1 < n) load_vec();
            // columns [lo, hi) of this half are rows of the sequence that see this key
            const int first = (i_first + at_tile.tile) * tokens;
            const int rows = (min(sq.len - first, tokens) << pack_log2) - cb;       // rows of this half that exist
            const int hi = key_ok ? rows : 0;
            const int lo = p.causal ? (min(max(key - shift - first, 0), tokens) << pack_log2) - cb : 0;
            const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < 64);

            ok = wait_warp(bar(S_FULL), i & 1, wc);
            if (!ok) break;
            tc_fence_after();
            float pr[64];
            {
                uint32_t* sr = reinterpret_cast<uint32_t*>(pr);
                tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 64; ++e) pr[e] = ex2_approx(fmaf(pr[e], c, -s_lse[e]));
            if (masked) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e < lo || e >= hi) pr[e] = 0.f;
            }
            {
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(pr[2 * e], pr[2 * e + 1]);
                tmem_st32(tS, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            g_arrive(bar(P_READY), lane);

            ok = wait_warp(bar(DP_FULL), i & 1, wc);
            if (!ok) break;
            tc_fence_after();
            uint32_t dsp[32];                                // this half-row's dS^T, bf16 pairs
            {
                uint32_t dp[64];
                tmem_ld32(tDP, *reinterpret_cast<uint32_t(*)[32]>(&dp[0]));
                tmem_ld32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(&dp[32]));
                tmem_wait_ld();
                // dS = P (dP - D), a pair at a time; selected where masked, whatever dP and D hold there
                float* ds = reinterpret_cast<float*>(dp);
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    const float2 dd = fsub2(make_float2(ds[e], ds[e + 1]), make_float2(s_del[e], s_del[e + 1]));
                    const float2 d2 = fmul2(make_float2(pr[e], pr[e + 1]), dd);
                    ds[e] = d2.x;
                    ds[e + 1] = d2.y;
                }
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (e < lo || e >= hi) ds[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) dsp[e] = pack_bf16x2(ds[2 * e], ds[2 * e + 1]);
            }
            tmem_st32(tDP, dsp);
            tmem_wait_st();
            tc_fence_before();
            g_arrive(bar(DS_READY), lane);
            // dS^T row j, queries cb..cb+63 -> the 128-byte swizzled row j of half hq, in dO's
            // buffer: only once dV (the last reader of dO) is done
            ok = wait_warp(bar(DV_DONE), i & 1, wc);
            if (!ok) break;
            const uint32_t half_tile = base + OFF_STAGE + (i & 1) * STAGE_BYTES + TILE_BYTES + hq * HALF_BYTES;
            st_row_sw128(half_tile, j, dsp);
            fence_proxy_async_smem();
            g_arrive(bar(DS_SMEM), lane);

            ok = wait_warp(bar(DQ_FULL), i & 1, wc);
            if (!ok) break;
            tc_fence_after();
            // dQ^T: TMEM lane = d (= j), column = query.  Copy queries cb..cb+63 into the stage as
            // fp32 [query][d] (its Q and dS^T are consumed), free the TMEM columns, and let the
            // reducer warp add the tile into the accumulator by TMA.
            float* stage = reinterpret_cast<float*>(smem + OFF_STAGE + (i & 1) * STAGE_BYTES);
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                uint32_t v[32];
                tmem_ld32(tDP + q * 32, v);
                tmem_wait_ld();
                if (rows < 64) {                             // behind the sequence: add nothing, whatever K holds
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (q * 32 + e >= rows) v[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) stage[(cb + q * 32 + e) * HD + j] = __uint_as_float(v[e]);
            }
            tc_fence_before();
            g_arrive(bar(DQ_DRAINED), lane);
            fence_proxy_async_smem();
            g_arrive(bar(STAGED), lane);
        }
        if (ok && n > 0) ok = wait_warp(bar(FINAL), 0, wc);
        if (ok && p.splits > 1) {
            // stage dV, dK (fp32, unscaled) for the reducer warp's TMA reduce-adds, once it has
            // finished reading the stages for dQ; keys behind the sequence add nothing
            if (n > 0) ok = wait_warp(bar(RED_DONE), 0, wc);
            if (ok && n > 0) {
                tc_fence_after();
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
                    const uint32_t src = tmem + (which ? T_DK : T_DV) + lane_off + cb;
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        uint32_t v[32];
                        tmem_ld32(src + q * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = key_ok ? v[e] : 0u;
                        // sub-tile hq*2+q holds d = 32(hq*2+q) .. +31
                        st_row_sw128(base + OFF_STAGE + which * STAGE_BYTES + (hq * 2 + q) * SUB_BYTES, j, v);
                    }
                }
                fence_proxy_async_smem();
                g_arrive(bar(EPI_STAGED), lane);
            }
        } else if (ok) {
            tc_fence_after();
            const long long row = sk.begin + key;
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const uint32_t src = tmem + (which ? T_DK : T_DV) + lane_off + cb;
                const float mul = which ? p.scale : 1.f;
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? p.dk : p.dv) + row * (which ? p.lddk : p.lddv) +
                                     hk * HD + cb;
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    uint32_t v[32];
                    if (n > 0) {
                        tmem_ld32(src + q * 32, v);
                        tmem_wait_ld();
                    } else {                                 // no query sees any key of the tile
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0u;
                    }
                    uint4 pk[4];
                    uint32_t* pw = reinterpret_cast<uint32_t*>(pk);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pw[e] = pack_bf16x2(__uint_as_float(v[2 * e]) * mul, __uint_as_float(v[2 * e + 1]) * mul);
                    if (key_ok) {
                        uint4* d4 = reinterpret_cast<uint4*>(dst + q * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) d4[e] = pk[e];
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WARP_MMA) tmem_dealloc(tmem, TMEM_COLS);
}

// One block: p.order[0 .. bound) = the key tiles of all sequences as (sequence, tile), those with most Q
// tiles first (a counting sort; tiles with equal work in any order), then (-1, 0).
__device__ void sort_tiles(const VarlenBwdParams& p) {
    constexpr int BUCKETS = 1024;
    __shared__ int count[BUCKETS], sums[8], carry;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int b = tid; b < BUCKETS; b += 256) count[b] = 0;
    if (tid == 0) carry = 0;
    __syncthreads();
    // inclusive block scan of one value per thread, on top of what earlier steps summed to; sums stop at
    // the bound (below 2^26), which offsets that are no offsets would pass, and 2^31 after it
    auto scan = [&](int v) {
        v = min(v, p.tile_bound);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v = min(v + o, p.tile_bound);
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        for (int w = 0; w < warp; ++w) v = min(v + sums[w], p.tile_bound);
        v = min(v + carry, p.tile_bound);
        __syncthreads();
        if (tid == 255) carry = v;
        __syncthreads();
        return v;
    };
    // tile_end[n]: tiles of sequences 0 .. n
    for (int n0 = 0; n0 < p.N; n0 += 256) {
        const int n = n0 + tid;
        const int end = scan(n < p.N ? (span_of(p.cu_k, n, p.Tk).len + BM - 1) / BM : 0);
        if (n < p.N) p.tile_end[n] = end;
    }
    const int total = carry;
    __syncthreads();
    auto place = [&](int x, int& seq, int& tile) {           // the first n with tile_end[n] > x
        int lo = 0, hi = p.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.tile_end[mid] > x) hi = mid;
            else lo = mid + 1;
        }
        seq = lo;
        tile = x - (lo ? p.tile_end[lo - 1] : 0);
        const int work = q_tiles(p, span_of(p.cu_q, lo, p.Tq), span_of(p.cu_k, lo, p.Tk), tile);
        return BUCKETS - 1 - min(work, BUCKETS - 1);         // bucket 0: the most work
    };
    int seq, tile;
    for (int x = tid; x < total; x += 256) atomicAdd(&count[place(x, seq, tile)], 1);
    if (tid == 0) carry = 0;
    __syncthreads();
    for (int b0 = 0; b0 < BUCKETS; b0 += 256) {              // counts -> first positions
        const int c = count[b0 + tid], end = scan(c);
        count[b0 + tid] = end - c;
    }
    __syncthreads();
    for (int x = tid; x < total; x += 256) {
        const int at = atomicAdd(&count[place(x, seq, tile)], 1);
        p.order[at] = make_int2(seq, tile);
    }
    for (int x = total + tid; x < p.tile_bound; x += 256) p.order[x] = make_int2(-1, 0);
}

// D_i = sum_d dO_id * O_id (fp32) for every (token, head) row, and dQ accumulator := 0.
// 16 threads per row, 8 elements (16 bytes) each.  The first block sorts the key tiles instead.
__global__ void __launch_bounds__(256) varlen_prep_kernel(const VarlenBwdParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x == 0) {
        sort_tiles(p);
        return;
    }
    const long long rows = static_cast<long long>(p.Tq) * p.H, total = rows * 16;
    const int lane = threadIdx.x & 31;
    const long long warp0 = static_cast<long long>(blockIdx.x - 1) * blockDim.x + threadIdx.x - lane;
    const long long stride = static_cast<long long>(gridDim.x - 1) * blockDim.x;
    const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(p.o);
    const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(p.dout);
    for (long long t0 = warp0; t0 < total; t0 += stride) {        // warp-uniform trip count
        const long long t = t0 + lane;
        const bool valid = t < total;
        const long long r = t >> 4;               // row index over [Tq, H]
        const int part = static_cast<int>(t & 15);
        float acc = 0.f;
        if (valid) {
            const uint4 ov = *reinterpret_cast<const uint4*>(o + r * HD + part * 8);
            const uint4 dv = *reinterpret_cast<const uint4*>(dout + r * HD + part * 8);
            const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(&ov);
            const __nv_bfloat162* d2 = reinterpret_cast<const __nv_bfloat162*>(&dv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = __bfloat1622float2(o2[e]);
                const float2 c = __bfloat1622float2(d2[e]);
                acc = fmaf(a.x, c.x, acc);
                acc = fmaf(a.y, c.y, acc);
            }
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        if (valid) {
            float4* z = reinterpret_cast<float4*>(p.dq_acc + r * HD + part * 8);
            z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
            z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (part == 0) p.delta[(r % p.H) * p.Tq + r / p.H] = acc;
        }
    }
}

// out[t, h, :] = bf16(acc[t, h, :] * scale) for the tokens from the first sequence's to the last's,
// 8 elements per thread; out has token stride ld.
__global__ void __launch_bounds__(256) varlen_cast_kernel(const float* acc, __nv_bfloat16* out, const int* cu, int N, int T, int H, long long ld,
                                                          float scale) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long row8 = static_cast<long long>(H) * 16;                // 8-element parts to a token
    const long long begin = min(max(cu[0], 0), T) * row8, end = min(max(cu[N], 0), T) * row8;
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long t = begin + static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; t < end; t += stride) {
        const float4 a = reinterpret_cast<const float4*>(acc)[2 * t];
        const float4 c = reinterpret_cast<const float4*>(acc)[2 * t + 1];
        uint4 w;
        w.x = pack_bf16x2(a.x * scale, a.y * scale);
        w.y = pack_bf16x2(a.z * scale, a.w * scale);
        w.z = pack_bf16x2(c.x * scale, c.y * scale);
        w.w = pack_bf16x2(c.z * scale, c.w * scale);
        *reinterpret_cast<uint4*>(out + (t / row8) * ld + (t % row8) * 8) = w;
    }
}

}  // namespace varlen_bwd

int varlen_bwd_tile_bound(int N, int Tk) {
    const long long bound = Tk / varlen_bwd::BM + static_cast<long long>(N);
    return static_cast<int>(bound < Tk ? bound : Tk);
}

// Query heads that share a Q tile: the largest power of two that divides the group (and the tile's rows, so
// that no row of a tile is left over).
int varlen_bwd_pack(int H, int Hkv) {
    const int group = H / Hkv;
    int pack = group & -group;
    return pack < varlen_bwd::BM ? pack : varlen_bwd::BM;
}

// CTAs among which a key tile's Q tiles are split: the number with the least estimated time, in units of
// one Q tile's products (3.4 us measured).  Most work first, the CTAs finish together unless one is longer
// than its SM's share: the larger of the two, with about 3 units of prologue and epilogue for every CTA;
// some of a CTA for the uneven end; and about 5 units of extra launches to clear and cast the fp32 dK, dV
// when there is more than one.  From the sizes alone: sequences of average length, full.  One sequence of
// 2000 and 12 heads takes 70 us unsplit, 106 us in three; one of 4096 with 16 heads over a single kv head
// 0.32 ms split, 1.54 ms unsplit.
int varlen_bwd_splits(int N, int Tq, int Tk, int H, int Hkv) {
    if (Tk == 0) return 1;               // no key tile to split
    const double ctas = static_cast<double>(varlen_bwd_tile_bound(N, Tk)) * Hkv;
    const int pack = varlen_bwd_pack(H, Hkv), tokens = varlen_bwd::BM / pack;
    const double q_tiles = static_cast<double>((static_cast<long long>(Tq) / N + tokens - 1) / tokens) * (H / Hkv / pack);
    int best = 1;
    double least = 0;
    for (int s = 1; s <= 64 && s <= q_tiles; ++s) {
        const double share = ctas * (q_tiles + 3 * s) / 148, one = q_tiles / s + 3;
        const double time = (share > one ? share : one) + 0.15 * one + (s > 1 ? 5 : 0);
        if (s == 1 || time < least) {
            least = time;
            best = s;
        }
    }
    return best;
}

int launch_varlen_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                      const CUtensorMap& tdq, const CUtensorMap& tdk, const CUtensorMap& tdv, const VarlenBwdParams& p,
                      cudaStream_t stream) {
    using namespace varlen_bwd;
    const int blocks = 148 * 8;          // grid-stride elementwise kernels: 8 blocks of 256 per SM
    const long long ctas = static_cast<long long>(p.tile_bound) * p.Hkv * p.splits;
    // Launched early, the main kernel's and the casts' blocks cost a grid of several waves 3 to 4 % (7797 tokens,
    // 536 CTAs: 440 against 423 us) and save a single wave as much as its launches take (3 x 200: 32 against 41).
    const bool early = ctas <= 148;
    auto cast = [&](const float* acc, void* out, const int* cu, int T, int heads, long long ld, float scale) {
        return launch_dependent(varlen_cast_kernel, dim3(blocks), 256, 0, stream, 1, early, acc, static_cast<__nv_bfloat16*>(out), cu,
                                p.N, T, heads, ld, scale);
    };
    if (launch_dependent(varlen_prep_kernel, dim3(1 + blocks), 256, 0, stream, 1, true, p) != 0) return -1;
    if (p.Tk > 0) {
        if (p.splits > 1) {
            const size_t bytes = static_cast<size_t>(p.Tk) * p.Hkv * HD * 4;
            if (cudaMemsetAsync(p.dk_acc, 0, bytes, stream) != cudaSuccess ||
                cudaMemsetAsync(p.dv_acc, 0, bytes, stream) != cudaSuccess)
                return -1;
        }
        if (configure_smem(reinterpret_cast<const void*>(varlen_main_kernel), SMEM_BYTES) != 0) return -1;
        const dim3 grid(static_cast<unsigned>(p.tile_bound) * p.Hkv, 1, p.splits);
        if (launch_dependent(varlen_main_kernel, grid, NTHREADS, SMEM_BYTES, stream, 1, early, tq, tk, tv, tdo, tdq, tdk, tdv,
                             p) != 0)
            return -1;
        if (p.splits > 1 && (cast(p.dk_acc, p.dk, p.cu_k, p.Tk, p.Hkv, p.lddk, p.scale) != 0 ||
                             cast(p.dv_acc, p.dv, p.cu_k, p.Tk, p.Hkv, p.lddv, 1.f) != 0))
            return -1;
    }
    return p.Tq > 0 ? cast(p.dq_acc, p.dq, p.cu_q, p.Tq, p.H, p.lddq, p.scale) : 0;
}

}  // namespace wan
