// Packed attention forward on sm_100a: sequences of different lengths on one token axis, full or
// causal, grouped heads.
//
// For query row i of a sequence with Lq queries and Lk keys (causal: keys j <= i + Lk - Lq)
//     m = max_j s_ij,  l = sum_j 2^(s_ij - m),  o_i = sum_j 2^(s_ij - m) v_j / l,  lse_i = (m + log2 l) ln 2,
// s = q.k log2(e) / sqrt(D), in one pass over the keys with a running m and l (fp32).
//
// How.  A work item is two Q tiles of 128 rows of one sequence and one packed head: a row is a (token,
// query head of the group) pair, `pack` heads to a token, so that heads that read the same keys share
// one walk over them (a single token's group is one tile; without packing its keys would cross the
// memory system once a head).  Within an item, as the dense forward:
//   warp 8      TMA producer: the Q tiles, then K_j / V_j of 128 keys into rings of two stages
//   warp 9      tcgen05 issuer: S_t = Q_t K_j^T (TMEM, fp32), O_t += P_t V_j (P_t in TMEM, bf16)
//   warps 0-3 / 4-7   softmax of tile 0 / 1, one row per thread; epilogue
//   warp 10     scheduler
// Items differ by orders of magnitude (a causal tile's keys, a sequence's length) and the short ones are
// mostly prologue and epilogue, so a CTA goes on to another item without a break: the scheduler asks the
// hardware for a block that has not started yet (cluster launch control), finds its place and its key
// range by a scan over the offsets (item_at: no table, no extra launch), and hands it to the other warps
// through two slots, some key blocks before it is needed.  K and V of the next item load, and its first scores are computed,
// under the epilogue of the last; the two tiles' groups run apart.  A sequence's tiles go backwards, so that
// causal's longest start first, and heads in groups (HeadOrder): 16384 tokens of 40 heads, causal, 2.50 ms
// against 2.61 with all heads in turn.
// What packing sequences adds:
//   - each tile has its own last key block (causal), blocks behind the diagonal are never loaded, and
//     only blocks on the diagonal or at the sequence's end are masked (a count per row)
//   - the last key block may hold the next sequence's rows: its K only meets masked scores, its V rows
//     are zeroed in shared memory before the tensor core reads them (0 x NaN is NaN)
//   - a tile that the sequence does not fill is stored row by row; the rows behind it are not touched
//   - an item with a single Q tile (a generated token, a sequence's last rows) has both groups work on it,
//     each on every other key block with a running m, l and O of its own, joined at the end in TMEM: one
//     group alone would leave the memory idle between its scores and its products
//   - few query rows against many keys: a sequence's keys go to several items, `chunk` key blocks to each, so
//     that sequences of any lengths make items of one size, and a second kernel joins their normalised fp32
//     partial results by their lse
#include <cuda.h>

#include "sm100_ptx.cuh"
#include "varlen.cuh"

namespace wan {
namespace varlen {

constexpr int BM = 128;        // rows per Q tile
constexpr int BN = 128;        // keys per K/V tile
constexpr int HD = 128;        // head dimension
constexpr int TILE_BYTES = BM * HD * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;    // 64 columns of d (one 128-byte swizzle span)

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + 2 * TILE_BYTES;
constexpr int OFF_V = OFF_K + 2 * TILE_BYTES;
constexpr int OFF_WORK = OFF_V + 2 * TILE_BYTES;   // two work slots
constexpr int WORK_BYTES = 64;
constexpr int MAX_PARTS = 64;                      // of a sequence's keys
constexpr int AHEAD = 6;                           // key blocks left of an item when the next one is fetched
constexpr int OFF_CLC = OFF_WORK + 2 * WORK_BYTES; // cluster launch control's answer
constexpr int OFF_ML = OFF_CLC + 16;               // m and l of tile 1's rows, for the join of a shared tile
constexpr int OFF_BAR = OFF_ML + 2 * BM * 4;
enum Bar { Q_FULL = 0, Q_EMPTY = 2, K_FULL = 4, K_EMPTY = 6, V_FULL = 8, V_EMPTY = 10, S_FULL = 12, P_FULL = 14,
           O_FINAL = 16, W_FULL = 18, W_EMPTY = 20, V_TAIL = 22, CLC = 23, NEXT = 24, ML_READY = 25, ML_DONE = 26, DRAIN = 27, NBARS = 28 };
constexpr int OFF_TMEM_SLOT = OFF_BAR + NBARS * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
constexpr int SMEM_BYTES = OFF_ABORT + 8 + 1024;   // slack for 1024-byte alignment of the tiles
constexpr int NTHREADS = 384;                  // three warpgroups; the last warp only makes up the third
constexpr int WARP_TMA = 8, WARP_MMA = 9, WARP_SCHED = 10;
constexpr uint32_t TMEM_COLS = 512;            // S0 S1 O0 O1, 128 columns each
constexpr float RESCALE_THRESHOLD = 8.0f;      // log2 units: keep a stale max while p <= 2^8

// One item, as the scheduler hands it over (WORK_BYTES of shared memory).
struct Work {
    int n;                 // key blocks of this item; -1: there is no more work
    int nt[2];             // key blocks of each tile, 0 for a tile without rows or keys here
    int shared;            // both tiles are the same rows: tile t takes the item's blocks t, t + 2, ...
    int j0;                // first key block
    int h0;                // first query head of the packed group
    int q_begin, q_len;    // the sequence's rows on the query axis
    int k_begin, k_len;    // ... and on the key axis
    int i0;                // first token of the item, within the sequence
    int part, parts;       // of the tile's keys
};
static_assert(sizeof(Work) <= WORK_BYTES, "a work slot");
__device__ __forceinline__ int ld_shared_int(uint32_t addr) {
    int v;
    asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
#define WORK(slot, field) ld_shared_int((slot) + static_cast<uint32_t>(offsetof(Work, field)))
// The same value, computed anew: keeps the epilogue's addresses from being carried through the item loop
// in registers that the scores need.
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+r"(v));
    return v;
}

// The scheduler's waits last as long as an item does (milliseconds for a million keys), unlike all others:
// it gives up when another role has (the abort flag), and by itself only after 64 budgets.
__device__ __forceinline__ bool wait_item(uint32_t bar, uint32_t parity, const WaitCtl& w) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (it & 15u) continue;
        int stop = 0;
        if ((threadIdx.x & 31) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            stop = *w.abort_flag;
            if (!stop && (now - t0) / 64 > w.budget_ns) {
                *w.abort_flag = 1;
                report_status(w.status, kStatusTimeout);
                stop = 1;
            }
        }
        if (__shfl_sync(0xffffffffu, stop, 0)) return false;
    }
}

__global__ void __launch_bounds__(NTHREADS, 1)
varlen_fwd_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo,
                  const VarlenFwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_addr);

    const int warp = warp_id();
    const int lane = lane_id();
    const int tile_tokens = BM / p.pack;
    const uint32_t sQ = base + OFF_Q, sK = base + OFF_K, sV = base + OFF_V;
    const uint32_t bar0 = base + OFF_BAR;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const WaitCtl wc{abort_flag, p.wait_budget_ns, p.status};
    auto slot_of = [&](uint32_t item) { return reinterpret_cast<volatile Work*>(smem + OFF_WORK + (item & 1u) * WORK_BYTES); };

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(Q_FULL + t), 1);
            mbar_init(bar(Q_EMPTY + t), 1);
            mbar_init(bar(K_FULL + t), 1);
            mbar_init(bar(K_EMPTY + t), 1);
            mbar_init(bar(V_FULL + t), 1);
            mbar_init(bar(V_EMPTY + t), 1);
            mbar_init(bar(S_FULL + t), 1);
            mbar_init(bar(P_FULL + t), BM);
            mbar_init(bar(O_FINAL + t), 1);
            mbar_init(bar(W_FULL + t), 1);
            mbar_init(bar(W_EMPTY + t), 10);          // producer, issuer, eight softmax warps
        }
        mbar_init(bar(V_TAIL), 1);
        mbar_init(bar(CLC), 1);
        mbar_init(bar(NEXT), 1);
        mbar_init(bar(ML_READY), 4);
        mbar_init(bar(ML_DONE), 4);
        mbar_init(bar(DRAIN), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    if (warp == WARP_MMA) {
        tmem_alloc(base + OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

    // Registers: the softmax warps hold a row's 128 scores; the launch's 384 x 168 are shared out as
    // 256 x 224 + 128 x 56.
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == WARP_SCHED) {
        // ------------------------------ scheduler ---------------------------------
        const int units = p.order.units;
        int x = blockIdx.x;
        uint32_t asked = 0, item = 0;
        ItemScan scan;
        bool more = true, pending = false;
        while (more) {
            int unit, h0;
            p.order.at(x, unit, h0);
            h0 *= p.pack;
            bool ok = true;
            // a block stands for item `unit`; with split keys, where the grid is an estimate, also for every
            // units-th one after it
            for (int target = unit;; target += units) {
                const ItemAt at = item_at(p.cu_q, p.cu_k, p.N, p.Tq, p.Tk, 2 * tile_tokens, p.chunk * BN, target, scan);
                if (at.seq < 0) break;
                const Span sq = at.q, sk = at.k;
                int tile = at.item, tiles = at.items, part = 0, parts = 1;
                if (p.chunk) {
                    parts = max(parts_of(sk.len, p.chunk * BN), 1);
                    tile /= parts;
                    tiles /= parts;
                    part = at.item - tile * parts;
                }
                const int i0 = (tiles - 1 - tile) * 2 * tile_tokens;
                const int shift = sk.len - sq.len;    // causal: token i sees keys 0 .. i + shift
                int nblk[2];                          // key blocks that tile t needs (its last token sees the most)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int last = min(i0 + (t + 1) * tile_tokens, sq.len) - 1;
                    const int keys = i0 + t * tile_tokens >= sq.len ? 0
                                     : p.causal ? min(max(last + shift + 1, 0), sk.len) : sk.len;
                    nblk[t] = (keys + BN - 1) / BN;
                }
                const int all = max(nblk[0], nblk[1]);
                const int j0 = min(part * p.chunk, all);
                const int n = p.chunk ? min(p.chunk, all - j0) : all;   // blocks j0 .. j0 + n - 1
                ok = wait_item(bar(W_EMPTY + (item & 1u)), ((item >> 1) & 1u) ^ 1u, wc);
                if (!ok) break;
                if (lane == 0) {
                    volatile Work* w = slot_of(item);
                    const bool shared = i0 + tile_tokens >= sq.len && n > 1;
                    w->n = n;
                    w->nt[0] = shared ? (n + 1) / 2 : min(max(nblk[0] - j0, 0), n);
                    w->nt[1] = shared ? n / 2 : min(max(nblk[1] - j0, 0), n);
                    w->shared = shared ? 1 : 0;
                    w->j0 = j0;
                    w->h0 = h0;
                    w->q_begin = sq.begin;
                    w->q_len = sq.len;
                    w->k_begin = sk.begin;
                    w->k_len = sk.len;
                    w->i0 = i0;
                    w->part = part;
                    w->parts = parts;
                    mbar_arrive(bar(W_FULL + (item & 1u)));
                }
                // the producer says when this item nears its end: a block taken earlier could wait here while
                // other SMs run out of work
                ok = wait_item(bar(NEXT), item & 1u, wc);
                if (!ok) break;
                ++item;
                if (!p.chunk) break;
            }
            if (!ok) break;
            pending = true;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(CLC), 16);
                clc_try_cancel(base + OFF_CLC, bar(CLC));
            }
            __syncwarp();
            if (!wait_warp(bar(CLC), asked & 1u, wc)) break;
            pending = false;
            ++asked;
            int y;
            more = clc_answer(base + OFF_CLC, x, y);
            fence_proxy_async_smem();                 // read before the next answer overwrites it
            __syncwarp();
        }
        if (pending) drain_wait(bar(CLC), asked & 1u);    // the answer must not land in memory that is gone
        const bool stopped = __any_sync(0xffffffffu, *abort_flag != 0);      // the same on every lane: wait_item votes
        if (!stopped && wait_item(bar(W_EMPTY + (item & 1u)), ((item >> 1) & 1u) ^ 1u, wc) && lane == 0) {
            slot_of(item)->n = -1;
            mbar_arrive(bar(W_FULL + (item & 1u)));
        }
    } else if (warp == WARP_TMA) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            tma_prefetch_desc(&tmq);
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
        const uint64_t keep = p.streamed ? l2_policy_evict_first() : l2_policy_evict_last();
        const uint32_t qbytes = static_cast<uint32_t>(p.pack * tile_tokens) * 256u;
        uint32_t kv = 0, tails = 0, loads[2] = {0, 0};     // K/V stages, V_TAIL phases and Q tiles used so far
        uint32_t k_out = 0, v_out = 0;                     // copies issued on K_FULL and V_FULL (the last two may be in flight)
        bool ok = true;
        for (uint32_t item = 0; ok; ++item) {
            ok = wait_warp(bar(W_FULL + (item & 1u)), (item >> 1) & 1u, wc);
            if (!ok) break;
            volatile Work* w = slot_of(item);
            const int n = w->n;
            if (n < 0) break;
            const int j0 = w->j0, k_begin = w->k_begin, h0 = w->h0, hk = h0 / (p.H / p.Hkv);
            const int q_tok = w->q_begin + w->i0;
            const int nt[2] = {w->nt[0], w->nt[1]}, tok1 = w->shared ? 0 : tile_tokens;      // tile 1's first token
            // rows of the last block that lie behind the sequence (only a sequence's last block has any)
            const int tail = n > 0 ? max((j0 + n) * BN - w->k_len, 0) : 0;
            const int whole = n - (tail > 0 ? 1 : 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(W_EMPTY + (item & 1u)));
            if (lane == 0) {
                if (n <= AHEAD) mbar_arrive(bar(NEXT));
                for (int i = 0; i < n; ++i, ++kv) {
                    if (i > 0 && i == n - AHEAD) mbar_arrive(bar(NEXT));
                    const uint32_t s = kv & 1u, use = (kv >> 1) & 1u;
                    const int tok = k_begin + (j0 + i) * BN;
                    ok = wait_thread(bar(K_EMPTY + s), use ^ 1u, wc);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(K_FULL + s), TILE_BYTES);
                    tma_load_3d_hint(sK + s * TILE_BYTES, &tmk, bar(K_FULL + s), 0, hk, tok, keep);
                    tma_load_3d_hint(sK + s * TILE_BYTES + HALF_BYTES, &tmk, bar(K_FULL + s), 64, hk, tok, keep);
                    k_out = kv + 1;
                    for (int t = 0; t < 2 && ok && i == 0; ++t) {
                        // behind the first K: a tile's buffer is still the last item's O on its way out
                        if (nt[t] == 0) continue;
                        ok = wait_thread(bar(Q_EMPTY + t), (loads[t] & 1u) ^ 1u, wc);
                        if (!ok) break;
                        mbar_arrive_expect_tx(bar(Q_FULL + t), qbytes);
                        tma_load_3d(sQ + t * TILE_BYTES, &tmq, bar(Q_FULL + t), 0, h0, q_tok + t * tok1);
                        tma_load_3d(sQ + t * TILE_BYTES + HALF_BYTES, &tmq, bar(Q_FULL + t), 64, h0, q_tok + t * tok1);
                        ++loads[t];
                    }
                    if (!ok) break;
                    ok = wait_thread(bar(V_EMPTY + s), use ^ 1u, wc);
                    if (!ok) break;
                    const uint32_t full = bar(i < whole ? V_FULL + s : V_TAIL);
                    mbar_arrive_expect_tx(full, TILE_BYTES);
                    tma_load_3d_hint(sV + s * TILE_BYTES, &tmv, full, 0, hk, tok, keep);
                    tma_load_3d_hint(sV + s * TILE_BYTES + HALF_BYTES, &tmv, full, 64, hk, tok, keep);
                    v_out = kv + 1;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            kv = __shfl_sync(0xffffffffu, kv, 0);
            if (ok && whole < n) {
                // the whole warp zeroes the V rows behind the sequence, then hands the stage over
                const uint32_t s = (kv - 1u) & 1u;
                ok = wait_warp(bar(V_TAIL), tails & 1u, wc);
                if (!ok) {
                    drain_wait(bar(V_TAIL), tails & 1u);
                    break;
                }
                ++tails;
                for (int half = 0; half < 2; ++half) {
                    const uint32_t row0 = sV + s * TILE_BYTES + half * HALF_BYTES + (BN - tail) * 128;
                    for (int c = lane; c < tail * 8; c += 32) st_shared_v4(row0 + c * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(V_FULL + s));
            }
        }
        if (!ok && lane == 0) {
            // let the copies already issued land before the CTA's shared memory goes away
            for (int t = 0; t < 2; ++t)
                if (loads[t]) drain_wait(bar(Q_FULL + t), (loads[t] - 1u) & 1u);
            for (uint32_t i = k_out > 2 ? k_out - 2 : 0; i < k_out; ++i) drain_wait(bar(K_FULL + (i & 1u)), (i >> 1) & 1u);
            for (uint32_t i = v_out > 2 ? v_out - 2 : 0; i < v_out; ++i) drain_wait(bar(V_FULL + (i & 1u)), (i >> 1) & 1u);
        }
    } else if (warp == WARP_MMA) {
        // ------------------------------ MMA issuer --------------------------------
        if (lane == 0) {
            const uint32_t idesc_qk = make_idesc(1, 1, 1, 0, 0, BM, BN);
            const uint32_t idesc_pv = make_idesc(1, 1, 1, 0, 1, BM, HD);
            const uint32_t hi = sdesc_hi();
            const uint32_t q_lo = sdesc_lo(sQ, 16), k_lo = sdesc_lo(sK, 16), v_lo = sdesc_lo(sV, HALF_BYTES);
            constexpr uint32_t TILE16 = TILE_BYTES >> 4;
            auto issue_qk = [&](int t_, uint32_t s_) {
                mma8_f16_ss<HALF_BYTES / 16, 2>(tmem + t_ * BN, q_lo + t_ * TILE16, k_lo + s_ * TILE16, hi, idesc_qk, 0u);
            };
            auto issue_pv = [&](int t_, uint32_t s_, bool acc) {
                mma8_f16_ts<32, 512, 128>(tmem + 256 + t_ * HD, tmem + t_ * BN, v_lo + s_ * TILE16, hi, idesc_pv,
                                          acc ? 1u : 0u);
            };
            uint32_t kv = 0;                               // K/V stages used so far
            uint32_t loads = 0, blocks = 0;                // parities of Q_FULL and P_FULL, a bit per tile
            bool ok = true;
            for (uint32_t item = 0; ok; ++item) {
                ok = wait_thread(bar(W_FULL + (item & 1u)), (item >> 1) & 1u, wc);
                if (!ok) break;
                volatile Work* w = slot_of(item);
                const int n = w->n, nt[2] = {w->nt[0], w->nt[1]}, shared = w->shared;
                if (n < 0) break;
                mbar_arrive(bar(W_EMPTY + (item & 1u)));
                if (n == 0) continue;
                if (shared) {
                    // block i is tile i & 1's alone; a tile's next scores follow its products
                    auto scores = [&](int t, uint32_t at) {
                        if (!wait_thread(bar(K_FULL + (at & 1u)), (at >> 1) & 1u, wc)) return false;
                        tc_fence_after();
                        issue_qk(t, at & 1u);
                        mma_commit(bar(S_FULL + t));
                        mma_commit(bar(K_EMPTY + (at & 1u)));
                        return true;
                    };
                    for (int t = 0; t < 2 && ok; ++t) {
                        ok = wait_thread(bar(Q_FULL + t), (loads >> t) & 1u, wc);
                        loads ^= 1u << t;
                        if (ok) ok = scores(t, kv + t);
                    }
                    for (int i = 0; i < n && ok; ++i, ++kv) {
                        const int t = i & 1;
                        ok = wait_thread(bar(V_FULL + (kv & 1u)), (kv >> 1) & 1u, wc);
                        if (ok) ok = wait_thread(bar(P_FULL + t), (blocks >> t) & 1u, wc);
                        if (!ok) break;
                        blocks ^= 1u << t;
                        tc_fence_after();
                        issue_pv(t, kv & 1u, i > 1);
                        mma_commit(bar(V_EMPTY + (kv & 1u)));
                        if (i + 2 < n) ok = scores(t, kv + 2);
                        else mma_commit(bar(O_FINAL + t));
                    }
                    continue;
                }
                ok = wait_thread(bar(K_FULL + (kv & 1u)), (kv >> 1) & 1u, wc);
                if (!ok) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (nt[t] == 0 || !ok) continue;
                    ok = wait_thread(bar(Q_FULL + t), (loads >> t) & 1u, wc);
                    if (!ok) continue;
                    loads ^= 1u << t;
                    tc_fence_after();
                    issue_qk(t, kv & 1u);
                    mma_commit(bar(S_FULL + t));
                }
                if (!ok) break;
                mma_commit(bar(K_EMPTY + (kv & 1u)));
                for (int i = 0; i < n && ok; ++i, ++kv) {
                    const uint32_t s = kv & 1u, s1 = s ^ 1u;
                    ok = wait_thread(bar(V_FULL + s), (kv >> 1) & 1u, wc);
                    bool k_here = false;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (i >= nt[t] || !ok) continue;
                        ok = wait_thread(bar(P_FULL + t), (blocks >> t) & 1u, wc);
                        if (!ok) continue;
                        blocks ^= 1u << t;
                        tc_fence_after();
                        issue_pv(t, s, i > 0);
                        if (i + 1 == nt[t]) {
                            mma_commit(bar(O_FINAL + t));
                        } else {
                            if (!k_here) {
                                ok = wait_thread(bar(K_FULL + s1), ((kv + 1) >> 1) & 1u, wc);
                                if (!ok) continue;
                                tc_fence_after();
                                k_here = true;
                            }
                            issue_qk(t, s1);
                            mma_commit(bar(S_FULL + t));
                        }
                    }
                    if (!ok) break;
                    mma_commit(bar(V_EMPTY + s));
                    if (i + 1 < n) mma_commit(bar(K_EMPTY + s1));
                }
            }
            // every MMA issued so far completes before TMEM is released
            mma_commit(bar(DRAIN));
            drain_wait(bar(DRAIN), 0);
        }
    }
    } else {
        // ------------------------- softmax / correction / epilogue ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int t = warp >> 2;                 // Q tile of this warpgroup
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + t * BN + lane_off;
        const uint32_t tO = tmem + 256 + t * HD + lane_off;
        const float c = p.scale_log2;
        uint32_t st = 0;                         // parity bits: 1 S_FULL, 2 O_FINAL, 4 ML_*; above: the item's number
        for (;; st += 8u) {
            // the item's slot is kept until its epilogue is done: only what the loop needs is in registers
            bool ok = wait_warp(bar(W_FULL + ((st >> 3) & 1u)), (st >> 4) & 1u, wc);
            // The group's warps go on together or not at all: a warp that gave up set the flag before the barrier.
            // Any other role may set it at any time, so what counts is what they read before, joined.
            if (named_bar_any(1 + t, BM, *abort_flag != 0)) break;
            uint32_t w = base + OFF_WORK + ((st >> 3) & 1u) * WORK_BYTES;
            if (WORK(w, n) < 0) break;
            const int nt = t ? WORK(w, nt[1]) : WORK(w, nt[0]);
            int keys;                            // keys that the row sees, counted from the item's first block
            {
                const int row_tok = fresh(threadIdx.x & 127) / p.pack;
                const int i_tok = WORK(w, i0) + (WORK(w, shared) ? 0 : t * tile_tokens) + row_tok, k_len = WORK(w, k_len), q_len = WORK(w, q_len);
                const bool real = row_tok < tile_tokens && i_tok < q_len;
                keys = !real ? 0 : p.causal ? min(max(i_tok + k_len - q_len + 1, 0), k_len) : k_len;
                keys -= (WORK(w, j0) + (WORK(w, shared) ? t : 0)) * BN;       // ... from the tile's first block
            }
            float m_ref = -INFINITY, l = 0.f;
            for (int i = 0; i < nt; ++i, keys -= WORK(w, shared) ? 2 * BN : BN) {
                ok = wait_warp(bar(S_FULL + t), st & 1u, wc);
                if (!ok) break;
                st ^= 1u;
                tc_fence_after();
                uint32_t sr[128];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[q * 32]));
                tmem_wait_ld();
                float* s = reinterpret_cast<float*>(sr);
                if (__any_sync(0xffffffffu, keys < BN)) {     // the row sees the first `keys` of this block
#pragma unroll
                    for (int q = 0; q < 128; ++q)
                        if (q >= keys) s[q] = -INFINITY;
                }
                // row max: 8 chains of three-input maxima, then a short tree
                float m8[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) m8[q] = fmax3(s[q], s[q + 8], s[q + 16]);
#pragma unroll
                for (int q = 24; q < 128; q += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        m8[e] = (q + 8 + e < 128) ? fmax3(m8[e], s[q + e], s[q + 8 + e]) : fmaxf(m8[e], s[q + e]);
                const float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                const float m_cand = mx * c;
                float alpha = 1.f;
                bool moved = false;
                if (m_cand > m_ref + RESCALE_THRESHOLD) {
                    alpha = ex2_approx(m_ref - m_cand);
                    m_ref = m_cand;
                    moved = true;
                }
                // P = 2^(s c - m) in packed pairs, the row sum in four independent packed accumulators;
                // a row that has seen no key yet keeps m = -inf: its scores are all -inf, its P zero
                const float off = m_ref == -INFINITY ? 0.f : -m_ref;
                const float2 c2 = make_float2(c, c), n2 = make_float2(off, off);
                float2 acc[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) acc[a] = make_float2(0.f, 0.f);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        const float2 x = ffma2(make_float2(s[half * 64 + 2 * q], s[half * 64 + 2 * q + 1]), c2, n2);
                        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                        acc[q & 3] = fadd2(acc[q & 3], e);
                        pk[q] = pack_bf16x2(e.x, e.y);
                    }
                    tmem_st32(tS + half * 32, pk);
                }
                const float2 acc2 = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
                l = l * alpha + (acc2.x + acc2.y);
                if (i > 0 && __any_sync(0xffffffffu, moved)) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[32];
                        tmem_ld32(tO + q * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(tO + q * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(P_FULL + t));
            }
            if (ok && nt > 0) {
                ok = wait_warp(bar(O_FINAL + t), (st >> 1) & 1u, wc);
                st ^= 2u;
            }
            // A whole tile leaves through its Q buffer (every MMA that read it has completed) and two TMA
            // stores; a tile that the sequence does not fill, or a split's partial result, row by row.
            w = base + OFF_WORK + ((static_cast<uint32_t>(fresh(st)) >> 3) & 1u) * WORK_BYTES;
            const int r = fresh(threadIdx.x & 127);       // row within the tile = TMEM lane
            const bool shared = WORK(w, shared) != 0;
            float a0 = 1.f, a1 = 0.f;                     // what the two tiles' O count when a shared tile is joined
            if (shared) {
                float* ml = reinterpret_cast<float*>(smem + OFF_ML) + r;
                if (t == 1) {
                    ml[0] = m_ref;
                    ml[BM] = l;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(ML_READY));
                    if (ok) ok = wait_warp(bar(ML_DONE), (st >> 2) & 1u, wc);
                } else {
                    if (ok) ok = wait_warp(bar(ML_READY), (st >> 2) & 1u, wc);
                    if (ok) {
                        const float m1 = ml[0], m = fmaxf(m_ref, m1);
                        a0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m);
                        a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
                        l = l * a0 + ml[BM] * a1;
                        m_ref = m;
                    }
                }
                st ^= 4u;
            }
            const int row_tok = r / p.pack, i_tile = WORK(w, i0) + (shared ? 0 : t * tile_tokens), q_len = WORK(w, q_len);
            const int head = WORK(w, h0) + r - row_tok * p.pack, token = WORK(w, q_begin) + i_tile + row_tok;
            const bool real = row_tok < tile_tokens && i_tile + row_tok < q_len && !(shared && t == 1);
            const bool empty = l == 0.f;                      // the row saw no key here (a NaN score leaves l NaN: it shows)
            const bool split = WORK(w, parts) > 1;
            const bool by_tma = !split && i_tile + tile_tokens <= q_len && nt > 0 && !shared;
            const uint32_t stage = sQ + t * TILE_BYTES;
            if (ok && !(shared && t == 1)) {
                tc_fence_after();
                const float inv_l = empty ? 0.f : 1.f / l;
                a0 *= inv_l;
                a1 *= inv_l;
                const long long row = static_cast<long long>(token) * p.H + head;
                const long long part = static_cast<long long>(WORK(w, part)) * p.Tq * p.H;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {                 // 32 columns of d at a time
                    uint32_t o[32];
                    if (nt > 0) {
                        tmem_ld32(tO + q * 32, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = empty ? 0u : __float_as_uint(__uint_as_float(o[e]) * a0);
                    if (shared) {
                        uint32_t o1[32];
                        tmem_ld32(tO + HD + q * 32, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (a1 != 0.f) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), a1, __uint_as_float(o[e])));
                    }
                    if (split) {
                        if (real && !empty) {
                            uint4* dst = reinterpret_cast<uint4*>(p.o_part + (part + row) * HD + q * 32);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    } else {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pk[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                        if (by_tma) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                st_shared_v4(sw128_chunk(stage + (q >> 1) * HALF_BYTES, r, (q & 1) * 4 + e), pk[4 * e],
                                             pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                        } else if (real) {
                            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + row * HD + q * 32);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                        }
                    }
                }
                tc_fence_before();                            // O is read: the next item's products may overwrite it
                if (shared) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(ML_DONE));
                }
                fence_proxy_async_smem();
                if (real) {
                    const float lse2 = empty ? -INFINITY : m_ref + log2f(l);
                    const long long at = static_cast<long long>(head) * p.Tq + token;
                    if (p.chunk && head == 0 && WORK(w, part) == 0) p.parts[token] = WORK(w, parts);
                    if (split) p.lse_part[part + at] = lse2;
                    else p.lse[at] = lse2 * 0.69314718055994531f;
                }
            }
            const int q_begin = WORK(w, q_begin), h0 = WORK(w, h0);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(W_EMPTY + ((st >> 3) & 1u)));
            if (named_bar_any(1 + t, BM, *abort_flag != 0)) break;   // every warp of the group, whatever its state
            if (r == 0 && nt > 0) {
                if (by_tma) {
                    tma_store_3d(&tmo, stage, 0, h0, q_begin + i_tile);
                    tma_store_3d(&tmo, stage + HALF_BYTES, 64, h0, q_begin + i_tile);
                    bulk_commit_group();
                    bulk_wait_read_all();             // the buffer is free once the copies have read it
                }
                mbar_arrive(bar(Q_EMPTY + t));
            }
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WARP_MMA) tmem_dealloc(tmem, TMEM_COLS);
}

// o = sum_z 2^(lse_z - lse) o_z, lse = log2 sum_z 2^lse_z over the parts' results: one warp per (token, head)
// row.  They are few (only calls with few query rows are split).
__global__ void __launch_bounds__(128) varlen_join_kernel(const VarlenFwdParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long rows = static_cast<long long>(p.Tq) * p.H;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31, token = static_cast<int>(row / p.H), head = static_cast<int>(row % p.H);
    if (token < p.cu_q[0] || token >= p.cu_q[p.N]) return;       // outside every sequence
    const int parts = parts_to_join(p.parts[token], p.most_parts);
    if (parts == 1) return;                                      // the item wrote its results itself
    // the parts' weights: part z and z + 32 in lane z, then one after the other past every lane's columns
    const float* lse = p.lse_part + static_cast<long long>(head) * p.Tq + token;
    static_assert(MAX_PARTS == 64, "two parts to a lane");
    const float z0 = lane < parts ? lse[lane * rows] : -INFINITY, z1 = lane + 32 < parts ? lse[(lane + 32) * rows] : -INFINITY;
    float m = fmaxf(z0, z1);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float w0 = z0 == -INFINITY ? 0.f : ex2_approx(z0 - m), w1 = z1 == -INFINITY ? 0.f : ex2_approx(z1 - m);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = p.o_part + row * HD + lane * 4;
    for (int g = 0; g < parts; g += 8) {
        float w[8];
        float4 o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = __shfl_sync(0xffffffffu, g < 32 ? w0 : w1, (g + e) & 31);
            // a part of weight 0 may not have been written
            if (w[e] != 0.f) o[e] = *reinterpret_cast<const float4*>(src + (g + e) * rows * HD);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (w[e] == 0.f) continue;
            l += w[e];
            acc = make_float4(fmaf(w[e], o[e].x, acc.x), fmaf(w[e], o[e].y, acc.y), fmaf(w[e], o[e].z, acc.z),
                              fmaf(w[e], o[e].w, acc.w));
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;       // a NaN shows
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + row * HD + lane * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0)
        p.lse[static_cast<long long>(head) * p.Tq + token] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// CTAs along the tile axis, an upper bound from the sizes alone: every sequence wastes less than one tile.
static long long tile_bound(int N, int Tq, int pack) {
    const int per_cta = 2 * (BM / pack);
    const long long bound = static_cast<long long>(Tq) / per_cta + N;
    return bound < Tq ? bound : Tq;
}

}  // namespace varlen

// pack: the most heads of a group that fill at least 120 of a tile's 128 rows (128 / pack tokens of
// `pack` heads each).
// chunk: keys are split when there are fewer than two tiles for every SM, into parts that make two; and when
// the sequences are single tiles on average (generated tokens: memory bound, lengths anything), into parts that
// make four.  Parts of one size rather than a number of parts to each sequence: 40 generated tokens of 8 kv heads
// against 17 to 9806 keys 152 us (5.3 TB/s; calls one by one with a cold L2, below the power cap: a loop of them
// takes 165) against 159, 8 of 4 kv heads against 11,089 keys, one of them 8650, 25 us against 52.  A part has at
// least 4 blocks (its prologue and epilogue take as long as two or three), there are at most 64, and the partial
// results take no more memory than K and V, or 16 MB.  Beyond SPLIT_N sequences the scheduler's scan over the
// offsets would take longer than an item.
VarlenFwdPlan varlen_fwd_plan(int N, int Tq, int Tk, int H, int Hkv) {
    constexpr int SPLIT_N = 256, MIN_CHUNK = 4;
    const int group = H / Hkv;
    int pk = 1;
    for (int d = 1; d <= group && d <= varlen::BM; ++d)
        if (group % d == 0 && (varlen::BM / d) * d >= 120) pk = d;
    const long long tiles = varlen::tile_bound(N, Tq, pk), ctas = tiles * (H / pk);
    const long long blocks = (static_cast<long long>(Tk) + varlen::BN - 1) / varlen::BN;
    const bool single = static_cast<long long>(Tq) <= static_cast<long long>(N) * (varlen::BM / pk);
    VarlenFwdPlan plan{pk, 0, single ? 1 : 0, 1, tiles, {}};
    if (ctas == 0) return plan;
    plan.order = head_order(tiles, H / pk, 512.0 * Tk * Hkv);
    const long long want = (single ? 4 : 2) * 148;
    if (ctas >= want || N > SPLIT_N) return plan;
    // key blocks that one head's items walk in all: a sequence's once for every tile of its queries
    const long long walked = single ? blocks : blocks * ((tiles + N - 1) / N);
    const long long items = (want + H / pk - 1) / (H / pk);            // of one packed head
    long long chunk = (walked + items - 1) / items;
    if (chunk < MIN_CHUNK) chunk = MIN_CHUNK;
    double memory = 256.0 * Tk * Hkv * 2;
    if (memory < 16 << 20) memory = 16 << 20;
    long long most = static_cast<long long>(memory / (516.0 * Tq * H));
    if (most > varlen::MAX_PARTS) most = varlen::MAX_PARTS;
    if (most < 2) return plan;
    if (chunk < (blocks + most - 1) / most) chunk = (blocks + most - 1) / most;
    if (blocks <= chunk) return plan;
    plan.chunk = static_cast<int>(chunk);
    plan.parts = static_cast<int>((blocks + chunk - 1) / chunk);
    plan.units = walked / chunk + tiles;
    plan.order = head_order(plan.units, H / pk, 512.0 * Tk * Hkv);
    return plan;
}

int launch_varlen_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to,
                      const VarlenFwdParams& p, long long units, cudaStream_t stream) {
    if (configure_smem(reinterpret_cast<const void*>(varlen::varlen_fwd_kernel), varlen::SMEM_BYTES) != 0) return -1;
    const dim3 grid(static_cast<unsigned>(units * (p.H / p.pack)));
    // a grid of many waves runs 3 to 4 % longer when launched early (7799 tokens, 1312 blocks: 143 against 137 us;
    // 12 prompts of 100, 192 blocks: 16.3 against 18.5)
    if (launch_dependent(varlen::varlen_fwd_kernel, grid, varlen::NTHREADS, varlen::SMEM_BYTES, stream, 1, grid.x <= 2 * 148, tq,
                         tk, tv, to, p) != 0)
        return -1;
    if (!p.chunk) return 0;
    const long long rows = static_cast<long long>(p.Tq) * p.H;
    return launch_dependent(varlen::varlen_join_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, stream, 1, true, p);
}

}  // namespace wan
