// The int8 linear layer's backward from 8-bit operands on sm_100a:
//     out[r, c] = sum_t a(t, r) x[t, c],   x[t, c] = s[t] codes[t, c]
// with a(t, r) = dY[t, r] for dW (t = tokens; the codes are the activation's checkpoint) and
// a(t, r) = dY[r, t] for dX (t = output channels; the codes are the weight's).
//
// Bound by the bf16 tensor cores.  The codes stay 8 bits until they are on the SM: TMA brings
// [64 t][128 c] bytes, converter warps multiply by the row's scale in fp32 and write bf16 into tensor
// memory, so the dequantised matrix never exists in memory (a pass of its own would write and read 4 bytes
// for every code).  The one rounding on the way, x to bf16 (2^-8 relative at most), is what the tensor
// core's operand type costs; dY is used as it is, sums are fp32.  Byte to float costs one PRMT and half an
// add: the code + 128 goes under the exponent of 2^23.
//
// The MMA's rows (TMEM lanes) are c and its columns r: x, transposed, is the operand that tensor memory can
// hold.  ldmatrix with transposition gives a thread four consecutive t of one c, and the 16x256b store takes
// them in exactly that fragment.  With x converted into a shared-memory operand instead, writing it and the
// MMA reading it back added 32 KB of shared-memory traffic to a stage's 56, past the 64 KB that the products
// leave time for: 1070 TFLOP/s.
//
// Two launches of the same roles (warp 0 TMA of dY, 1 MMA, 2-5 epilogue, 6-13 converters, 14 TMA of the
// codes; a stage holds dY and the codes, 16 + 8 KB, and its x 32 columns of TMEM):
//   PAIR   persistent CTA pairs (cta_group::2) on 256 x 256 tiles: each CTA converts its 128 c and loads
//          its 128 r of the pair's
//   else   one 128 x 128 tile per CTA; a cluster splits t and joins its fp32 partial tiles in rank order
//          (deterministic) through distributed shared memory: sizes whose 256 x 256 tiles leave SMs idle
#include <cuda.h>

#include "sm100_ptx.cuh"
#include "wan_attn_internal.h"

namespace wan {
namespace int8_grad {

constexpr int BT = 64;                                       // terms of the sum per stage
constexpr int STAGES = 8;
constexpr int Y_BYTES = 128 * BT * 2, C_BYTES = 128 * BT;    // dY | codes
constexpr int HALF_BYTES = Y_BYTES / 2;                      // 64 columns of an MN-major tile
constexpr int STAGE_BYTES = Y_BYTES + C_BYTES;
constexpr int X_COLS = BT / 2;                               // TMEM columns of a stage's x (bf16 pairs)
constexpr int OFF_BAR = STAGES * STAGE_BYTES;
enum Bar { FULL = 0, CODES = STAGES, READY = 2 * STAGES, EMPTY = 3 * STAGES, TFULL = 4 * STAGES, TEMPTY = 4 * STAGES + 1,
           DRAIN = 4 * STAGES + 2, NBARS = 4 * STAGES + 3 };
constexpr int OFF_TMEM_SLOT = OFF_BAR + NBARS * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
constexpr int OFF_EPI = (OFF_ABORT + 8 + 15) & ~15;          // per epilogue warp: 32 rows x 64 B
constexpr int EPI_WARP_BYTES = 32 * 64;
constexpr int GROUPS = 2;                                    // of four converter warps
constexpr int WARP_CODES = 6 + 4 * GROUPS, NTHREADS = (WARP_CODES + 1) * 32;
constexpr int SCALE_AHEAD = 3, SCALE_WARP_BYTES = SCALE_AHEAD * BT * 4;     // per converter warp: a stage's scales
constexpr int OFF_SCALES = OFF_EPI + 4 * EPI_WARP_BYTES;
constexpr int SMEM_BYTES = OFF_SCALES + 4 * GROUPS * SCALE_WARP_BYTES + 1024;
constexpr int GROUP = 16;                                    // tile order: row blocks in groups
constexpr uint32_t TMEM_COLS = 512;                          // an fp32 tile, then the stages' x
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");
static_assert(128 * 128 * 4 <= STAGES * STAGE_BYTES, "a partial tile reuses the stages");
static_assert(256 + STAGES * X_COLS <= TMEM_COLS, "tile and stages in TMEM");

struct Params {
    const float* scales;              // fp32 [terms]
    __nv_bfloat16* out;               // [rows, cols]
    int rows, cols, terms;
    unsigned long long wait_budget_ns;
    int* status;
};

__device__ __forceinline__ void mma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Two 16 x 16 byte matrices, transposed: lane L's address is row L % 16 of matrix L / 16; it gets columns
// L / 4 and L / 4 + 8 of each, rows 4 (L % 4) .. + 3, one register each.
__device__ __forceinline__ void ldmatrix_t8_x2(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}
// 16 lanes x 32 columns: registers 4k .. 4k + 3 are columns 8k + 2 (L % 4), + 1 of lane L / 4, then of lane
// L / 4 + 8.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// wait_thread with acquire at cluster scope: what the peer CTA wrote before its arrival is visible.
__device__ __forceinline__ bool wait_thread_cluster(uint32_t bar, uint32_t parity, const WaitCtl& w) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if (t0 == 0) t0 = global_timer_ns();
        if ((it & 15u) == 0 && wait_expired(w, t0)) return false;
    }
}

// After an abort: the last `issued` copies counted on a ring's barriers land before the memory goes away.
__device__ __forceinline__ void drain_ring(uint32_t bar0, Ring<STAGES> at, uint32_t issued) {
    for (uint32_t i = 1; i <= issued; ++i) {
        const int s = at.s >= static_cast<int>(i) ? at.s - i : at.s + STAGES - i;
        drain_wait(bar0 + 8u * s, at.s >= static_cast<int>(i) ? at.use : at.use ^ 1u);
    }
}

// Two codes (bytes of w, biased by 128) times s, as packed bf16.
template <uint32_t SEL0, uint32_t SEL1>
__device__ __forceinline__ uint32_t scale2(uint32_t w, float2 s) {
    const float2 f = make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, SEL0)),
                                 __uint_as_float(__byte_perm(w, 0x4b000000u, SEL1)));     // 2^23 + code + 128
    const float2 c = fadd2(f, make_float2(-8388736.f, -8388736.f));                       // the code, exactly
    const float2 x = fmul2(c, s);
    return pack_bf16x2(x.x, x.y);
}

template <bool Y_MN, bool PAIR>
__device__ __forceinline__ void grad_body(const CUtensorMap& tma_y, const CUtensorMap& tma_c, const Params& p) {
    constexpr int CG = PAIR ? 2 : 1, TILE = 128 * CG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;       // the same offset in every CTA
    uint8_t* smem = smem_raw + (base - raw_addr);
    const int warp = warp_id(), lane = lane_id();
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = !PAIR || rank == 0;
    const uint32_t bar0 = base + OFF_BAR;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const WaitCtl wc{abort_flag, p.wait_budget_ns, p.status};

    const int r_tiles = (p.rows + TILE - 1) / TILE, c_tiles = (p.cols + TILE - 1) / TILE;
    const long long tiles = static_cast<long long>(r_tiles) * c_tiles;
    const int nk_all = (p.terms + BT - 1) / BT;
    // PAIR: tiles first, first + step, ...; else one tile and this rank's share of the terms
    const int splits = PAIR ? 1 : gridDim.x;
    const long long first = PAIR ? blockIdx.x >> 1 : static_cast<long long>(blockIdx.y) + 65535ll * blockIdx.z;
    const long long step = PAIR ? gridDim.x >> 1 : tiles;
    const int k0 = PAIR ? 0 : static_cast<int>(static_cast<long long>(rank) * nk_all / splits);
    const int nk = (PAIR ? nk_all : static_cast<int>(static_cast<long long>(rank + 1) * nk_all / splits)) - k0;
    if (!PAIR && first >= tiles) return;                     // the whole cluster (the grid's y, z may overshoot)
    // row blocks in groups of GROUP, the row block fastest: tiles in flight share both operands in L2
    auto tile_of = [&](long long t, int& r0, int& c0) {
        const long long per_group = static_cast<long long>(GROUP) * c_tiles;
        const int g = static_cast<int>(t / per_group);
        const int rows = min(GROUP, r_tiles - g * GROUP);
        const long long w = t - g * per_group;
        r0 = (g * GROUP + static_cast<int>(w % rows)) * TILE;
        c0 = static_cast<int>(w / rows) * TILE;
        if (PAIR) {                                          // this CTA's r of dY and c of the codes
            r0 += rank * 128;
            c0 += rank * 128;
        }
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(FULL + s), 1);
            mbar_init(bar(CODES + s), 1);
            mbar_init(bar(READY + s), 4 * CG);
            mbar_init(bar(EMPTY + s), 1);
        }
        mbar_init(bar(TFULL), 1);
        mbar_init(bar(TEMPTY), 128 * CG);
        mbar_init(bar(DRAIN), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    if (warp == 1) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + OFF_TMEM_SLOT),
                         "r"(TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            tmem_alloc(base + OFF_TMEM_SLOT, TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR) cluster_sync_all();       // both CTAs' barriers and TMEM exist before any remote use
    else __syncthreads();
    tc_fence_after();
    grid_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

    if (warp == 0) {
        // ------------------------------ TMA producer of dY ------------------------
        if (lane == 0) {
            tma_prefetch_desc(&tma_y);
            const uint32_t full0 = PAIR ? mapa_shared(bar(FULL), 0) : bar(FULL);
            Ring<STAGES> ring;
            uint32_t issued = 0;                             // stages whose copies may be in flight
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
                int r0, c0;
                tile_of(t, r0, c0);
                int t0 = k0 * BT;
                for (int kb = 0; kb < nk; ++kb, ring.next(), t0 += BT) {
                    ok = wait_thread(bar(EMPTY + ring.s), ring.use ^ 1u, wc);
                    if (!ok) break;
                    const uint32_t st = base + ring.s * STAGE_BYTES, full = full0 + 8u * ring.s;
                    if (leader) mbar_arrive_expect_tx(bar(FULL + ring.s), CG * Y_BYTES);
                    // [64 t][2 x 64 r] (dW, MN-major) or [128 r][64 t] (dX, K-major)
                    if (PAIR) {
                        if (Y_MN) {
                            tma_load_2d_pair(st, &tma_y, full, r0, t0);
                            tma_load_2d_pair(st + HALF_BYTES, &tma_y, full, r0 + 64, t0);
                        } else {
                            tma_load_2d_pair(st, &tma_y, full, t0, r0);
                        }
                    } else if (Y_MN) {
                        tma_load_2d(st, &tma_y, full, r0, t0);
                        tma_load_2d(st + HALF_BYTES, &tma_y, full, r0 + 64, t0);
                    } else {
                        tma_load_2d(st, &tma_y, full, t0, r0);
                    }
                    issued = min(issued + 1u, static_cast<uint32_t>(STAGES));
                }
            }
            if (!ok && leader) drain_ring(bar(FULL), ring, issued);
        }
    } else if (warp == WARP_CODES) {
        // ------------------------------ TMA producer of the codes -----------------
        if (lane == 0) {
            tma_prefetch_desc(&tma_c);
            Ring<STAGES> ring;
            uint32_t issued = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
                int r0, c0;
                tile_of(t, r0, c0);
                int t0 = k0 * BT;
                for (int kb = 0; kb < nk; ++kb, ring.next(), t0 += BT) {
                    ok = wait_thread(bar(EMPTY + ring.s), ring.use ^ 1u, wc);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(CODES + ring.s), C_BYTES);
                    tma_load_2d(base + ring.s * STAGE_BYTES + Y_BYTES, &tma_c, bar(CODES + ring.s), c0, t0);
                    issued = min(issued + 1u, static_cast<uint32_t>(STAGES));
                }
            }
            if (!ok) drain_ring(bar(CODES), ring, issued);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer (a pair's leader) --------------
        if (lane == 0 && leader) {
            const uint32_t idesc = make_idesc(1, 1, 1, 0, Y_MN ? 1 : 0, TILE, TILE);
            // K-major: 16 terms are 32 bytes of a row; MN-major: 16 rows of 128 bytes, halves of the other
            // axis HALF_BYTES apart.  The descriptors' high halves are the same, the low ones count 16 bytes.
            constexpr uint32_t Y_STEP = Y_MN ? 128 : 2;
            const uint32_t hi = sdesc_hi(), y_lo = sdesc_lo(base, Y_MN ? HALF_BYTES : 16);
            Ring<STAGES> ring;
            int tc = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step, ++tc) {
                ok = wait_thread(bar(TEMPTY), (tc & 1) ^ 1, wc);
                if (!ok) break;
                tc_fence_after();
                for (int kb = 0; kb < nk; ++kb, ring.next()) {
                    ok = wait_thread(bar(FULL + ring.s), ring.use, wc);
                    if (ok)
                        ok = PAIR ? wait_thread_cluster(bar(READY + ring.s), ring.use, wc)
                                  : wait_thread(bar(READY + ring.s), ring.use, wc);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t x = tmem + TILE + ring.s * X_COLS, y = y_lo + ring.s * (STAGE_BYTES >> 4);
#pragma unroll
                    for (int kk = 0; kk < BT / 16; ++kk) {
                        const uint64_t yd = static_cast<uint64_t>(hi) << 32 | (y + kk * Y_STEP);
                        const uint32_t accumulate = (kb > 0 || kk > 0) ? 1u : 0u;
                        if (PAIR) mma_f16_ts_pair(tmem, x + kk * 8, yd, idesc, accumulate);
                        else mma_f16_ts(tmem, x + kk * 8, yd, idesc, accumulate);
                    }
                    if (PAIR) mma_commit_pair_both(bar(EMPTY + ring.s));     // both CTAs' stage is free
                    else mma_commit(bar(EMPTY + ring.s));
                }
                if (!ok) break;
                if (PAIR) mma_commit_pair_both(bar(TFULL));
                else mma_commit(bar(TFULL));
            }
            if (PAIR) mma_commit_pair(bar(DRAIN));
            else mma_commit(bar(DRAIN));
            drain_wait(bar(DRAIN), 0);
        }
    } else if (warp >= 6) {
        // ------------------------------ converters --------------------------------
        // Groups of four warps take the stages in turn.  A warp takes the 32 c of its TMEM quadrant: two times
        // 16 c, each 64 t as four transposed 16 x 16 matrices.  The codes' rows lie in the 128-byte swizzle, so
        // that eight of them fall on different banks.  The scales come SCALE_AHEAD stages early by cp.async.
        const int cw = warp - 6, quad = warp & 3;
        const uint32_t ready = PAIR ? mapa_shared(bar(READY), 0) : bar(READY);
        const uint32_t ring = base + OFF_SCALES + cw * SCALE_WARP_BYTES;
        const long long total = ((tiles - first + step - 1) / step) * nk;
        auto fetch_scales = [&](long long it, int kb, int slot) {
            if (it < total)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = (k0 + kb) * BT + e * 32 + lane;
                    const float* src = p.scales + min(t, p.terms - 1);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ring + (slot * BT + e * 32 + lane) * 4),
                                 "l"(src), "r"(t < p.terms ? 4 : 0)          // zero behind the last term
                                 : "memory");
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto after = [&](int kb) { return kb + GROUPS < nk ? kb + GROUPS : (kb + GROUPS) % nk; };
        const int g = cw >> 2;
        int kb_next = g % nk;                                // the stage whose scales are fetched next
        for (int a = 0; a < SCALE_AHEAD; ++a, kb_next = after(kb_next)) fetch_scales(g + GROUPS * a, kb_next, a);
        int slot = 0;
        Ring<STAGES> stage;
        for (int i = 0; i < g; ++i) stage.next();
        for (long long it = g; it < total; it += GROUPS) {
            const int s = stage.s;
            asm volatile("cp.async.wait_group %0;" ::"n"(SCALE_AHEAD - 1) : "memory");
            if (!wait_warp(bar(CODES + s), stage.use, wc)) break;
            __syncwarp();                                    // every lane's copies are there for every lane
            const float4* sc = reinterpret_cast<const float4*>(smem + OFF_SCALES + cw * SCALE_WARP_BYTES + slot * BT * 4);
            const uint32_t codes = base + s * STAGE_BYTES + Y_BYTES;
            float4 s4[4];                                    // of terms 16 tb + 4 (lane % 4) .. + 3
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) s4[tb] = sc[tb * 4 + (lane & 3)];
#pragma unroll
            for (int cg = 0; cg < 2; ++cg) {
                uint32_t x[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[4];
                    ldmatrix_t8_x2(sw128_chunk(codes, h * 32 + lane, quad * 2 + cg), v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {            // matrix e / 2, columns lane / 4 (e even) or + 8
                        const uint32_t w = v[e] ^ 0x80808080u;
                        const float4 f = s4[h * 2 + (e >> 1)];
                        x[(h * 2 + (e >> 1)) * 4 + (e & 1) * 2] = scale2<0x7540, 0x7541>(w, make_float2(f.x, f.y));
                        x[(h * 2 + (e >> 1)) * 4 + (e & 1) * 2 + 1] = scale2<0x7542, 0x7543>(w, make_float2(f.z, f.w));
                    }
                }
                tmem_st_16x256b_x4(tmem + TILE + s * X_COLS + (static_cast<uint32_t>(quad * 32 + cg * 16) << 16), x);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_cluster_relaxed_scope(ready + 8u * static_cast<uint32_t>(s));
                else mbar_arrive(ready + 8u * static_cast<uint32_t>(s));
            }
            fetch_scales(it + GROUPS * SCALE_AHEAD, kb_next, slot);
            kb_next = after(kb_next);
            slot = slot + 1 < SCALE_AHEAD ? slot + 1 : 0;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) stage.next();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (PAIR || splits == 1) {
        // ------------------------------ epilogue: this CTA's 128 columns of out ----
        // TMEM lane = c, column = r.  A warp's 32 c by 32 r at a time go through its 2 KB of shared memory,
        // [r][c] as bf16, and leave as 64-byte pieces of 32 rows.
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tempty = PAIR ? mapa_shared(bar(TEMPTY), 0) : bar(TEMPTY);
        const uint32_t wbuf = base + OFF_EPI + (warp - 2) * EPI_WARP_BYTES;
        int tc = 0;
        for (long long t = first; t < tiles; t += step, ++tc) {
            int r0, c0;
            tile_of(t, r0, c0);
            if (PAIR) r0 -= rank * 128;                      // the accumulator spans the pair's r
            if (!wait_warp(bar(TFULL), tc & 1, wc)) break;
            tc_fence_after();
            const int col = c0 + (warp & 3) * 32 + (lane & 3) * 8;
#pragma unroll 1
            for (int c = 0; c < TILE / 32; ++c) {
                if (r0 + c * 32 >= p.rows) break;
                uint32_t v[32];
                tmem_ld32(tmem + lane_off + c * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const uint32_t two = pack_bf16x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(wbuf + e * 64 + lane * 2), "h"(static_cast<uint16_t>(two))
                                 : "memory");
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(wbuf + (e + 1) * 64 + lane * 2),
                                 "h"(static_cast<uint16_t>(two >> 16))
                                 : "memory");
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int rr = 8 * k + (lane >> 2), row = r0 + c * 32 + rr;
                    const uint4 val = *reinterpret_cast<const uint4*>(smem + (wbuf - base) + rr * 64 + (lane & 3) * 16);
                    if (row < p.rows && col < p.cols)        // cols % 16 == 0
                        *reinterpret_cast<uint4*>(p.out + static_cast<long long>(row) * p.cols + col) = val;
                }
                __syncwarp();
            }
            tc_fence_before();
            if (PAIR) mbar_arrive_cluster(tempty);
            else mbar_arrive(tempty);
        }
    } else {
        // ------------------------------ split: partial tile to shared memory ------
        // [r][c] fp32 over the stages (every copy has landed and every MMA has read them)
        if (wait_warp(bar(TFULL), 0, wc)) {
            tc_fence_after();
            const uint32_t at = base + ((warp & 3) * 32 + lane) * 4;
            const uint32_t src = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                tmem_ld32(src + c * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + (c * 32 + e) * 512), "r"(v[e]) : "memory");
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR || splits > 1) cluster_sync_all();              // PAIR: no CTA leaves while its peer may signal it
    tc_fence_after();
    if (!PAIR && splits > 1) {
        // rows rank, rank + splits, ... of the tile: one warp a row, four columns a lane, ranks in order
        int r0, c0;
        tile_of(first, r0, c0);
        const int rows = min(128, p.rows - r0), col = c0 + lane * 4;
        if (!*abort_flag && col < p.cols)
            for (int r = rank + warp * splits; r < rows; r += (NTHREADS / 32) * splits) {
                const uint32_t at = base + r * 512 + lane * 16;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int z = 0; z < splits; ++z) {
                    const uint4 v = ld_shared_cluster_v4(mapa_shared(at, z));
                    acc = make_float4(acc.x + __uint_as_float(v.x), acc.y + __uint_as_float(v.y),
                                      acc.z + __uint_as_float(v.z), acc.w + __uint_as_float(v.w));
                }
                *reinterpret_cast<uint2*>(p.out + static_cast<long long>(r0 + r) * p.cols + col) =
                    make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            }
        __syncthreads();
        cluster_sync_all();                                  // no CTA leaves while a peer reads its partial tile
    }
    if (warp == 1) {
        if (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
        else
            tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <bool Y_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
grad_pair_kernel(const __grid_constant__ CUtensorMap tma_y, const __grid_constant__ CUtensorMap tma_c, const Params p) {
    grad_body<Y_MN, true>(tma_y, tma_c, p);
}
template <bool Y_MN>
__global__ void __launch_bounds__(NTHREADS, 1)
grad_split_kernel(const __grid_constant__ CUtensorMap tma_y, const __grid_constant__ CUtensorMap tma_c, const Params p) {
    grad_body<Y_MN, false>(tma_y, tma_c, p);
}

template <bool Y_MN>
int launch(const CUtensorMap& ta, const CUtensorMap& tc, const Params& p, cudaStream_t stream) {
    auto tiles = [&](long long n) { return ((p.rows + n - 1) / n) * ((p.cols + n - 1) / n); };
    const long long t256 = tiles(256), t128 = tiles(128);
    // A wave of 256 x 256 tiles on the pairs takes about as long as one of 128 x 128 tiles on single CTAs, which
    // read twice the shared memory per product (4096 terms: 33 to 39 us and 30 to 35), so the fewer waves win, and
    // the single CTAs where they are as many: 9600 x 784 in 3 waves of pairs 98 us, in 4 of CTAs 123; 2048 x 2048
    // 39 (1 wave) and 65 (2); 5120 x 784, two waves of each, 68 and 66; 1536 x 1536, one of each, 39 and 35.
    if ((t256 + 73) / 74 < (t128 + 147) / 148) {
        if (configure_smem(reinterpret_cast<const void*>(grad_pair_kernel<Y_MN>), SMEM_BYTES) != 0) return -1;
        return launch_dependent(grad_pair_kernel<Y_MN>, dim3(2 * static_cast<unsigned>(t256 < 74 ? t256 : 74)), NTHREADS,
                                SMEM_BYTES, stream, 1, true, ta, tc, p);
    }
    if (configure_smem(reinterpret_cast<const void*>(grad_split_kernel<Y_MN>), SMEM_BYTES) != 0) return -1;
    // the terms are split while that still fits one CTA per SM and each has eight stages or more
    const int nk = (p.terms + BT - 1) / BT;
    int splits = 1;
    while (splits < 8 && (splits + 1) * t128 <= 148 && nk / (splits + 1) >= 8) ++splits;
    const dim3 grid(splits, static_cast<unsigned>(t128 < 65535 ? t128 : 65535), static_cast<unsigned>((t128 + 65534) / 65535));
    return launch_dependent(grad_split_kernel<Y_MN>, grid, NTHREADS, SMEM_BYTES, stream, splits, true, ta, tc, p);
}

}  // namespace int8_grad

int launch_int8_grad(const CUtensorMap& tdy, const CUtensorMap& tcodes, const float* scales, void* out, int rows, int cols,
                     int terms, bool weight, unsigned long long budget_ns, int* status, cudaStream_t stream) {
    const int8_grad::Params p{scales, static_cast<__nv_bfloat16*>(out), rows, cols, terms, budget_ns, status};
    return weight ? int8_grad::launch<true>(tdy, tcodes, p, stream) : int8_grad::launch<false>(tdy, tcodes, p, stream);
}

}  // namespace wan
