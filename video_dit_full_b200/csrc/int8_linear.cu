// Int8 linear layer on sm_100a: rows to 8 bits and back, and Y = diag(sx) (Cx Cw^T) diag(sw) + bias.
//
//   quant_rows     s = absmax / 127, c = rint(127 x / absmax) per row
//   dequant_rows   x = bf16(s c)
//   gemm_pair      many tokens: CTA pairs (tcgen05 cta_group::2), 256 x 256 tiles, kind::i8 into int32 TMEM
//   gemm_few       few tokens: the weight's 128 channels are the MMA's M, 16 to 128 tokens its N; a cluster
//                  splits K and adds its exact int32 partial sums through distributed shared memory
//   layer_few      the same with the quantiser inside: one launch for a layer of a few tokens
// Sums are exact in int32 (K <= 131072), so neither the tiling nor the split changes a result.
#include <cuda.h>

#include "sm100_ptx.cuh"
#include "wan_attn_internal.h"

namespace wan {
namespace int8 {

// ------------------------------------------------------------------------------------
// rows <-> 8 bits
// ------------------------------------------------------------------------------------
__device__ __forceinline__ float2 bf16x2_floats(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// rint of the exact quotients 127 x / amax, half to even, as the low bytes of the results.  127 x is exact in
// fp32 (7 + 8 bits).  q = 127 x * inv is within an ulp of the quotient, the fma's residual 127 x - q amax is
// exact, and one correction gives the correctly rounded quotient (Markstein's division, inv = RN(1 / amax)).
// A quotient of these 8-bit significands that is not a half-integer stays 2^9 of fp32's half steps or more away from
// one, in every binade (1/64768 at 127 * 255 / (253 * 2^8), next to 1/2; 2^-9 next to 126.5), so rounding it again to
// an integer is rounding the exact quotient; a half-integer is represented exactly.
// In pairs (packed fp32): one value an instruction, the quantiser's arithmetic no longer hid behind memory
// (32760 x 5120: 97 us; 80 us and 6.3 TB/s in pairs).
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, float pre, float amax, float inv) {
    auto pair = [&](uint32_t u) {
        const float2 a = fmul2(bf16x2_floats(u), both(127.f * pre));
        const float2 q = fmul2(a, both(inv));
        const float2 r = ffma2(ffma2(q, both(-amax), a), both(inv), q);
        const float2 c = fadd2(r, both(12582912.f));       // 1.5 * 2^23: the sum's low bits are the integer
        return __byte_perm(__float_as_uint(c.x), __float_as_uint(c.y), 0x0040);
    };
    return __byte_perm(pair(lo), pair(hi), 0x5410);
}
// |x| as bits: the largest finite magnitude orders like an integer, and an infinity or NaN above it.  Of eight
// values, the even and the odd ones apart, with what was seen before.
__device__ __forceinline__ uint32_t most_of(uint32_t seen, uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) asm("max.u16x2 %0, %0, %1;" : "+r"(seen) : "r"(w[e] & 0x7fff7fffu));
    return seen;
}
__device__ __forceinline__ uint32_t most_of_halves(uint32_t seen) { return max(seen & 0xffffu, seen >> 16); }

// What a row's absmax (as bf16 bits; an infinity or NaN is at least 0x7f80) makes of its values.
struct RowScale {
    float scale, pre, amax, inv;
    bool bad;
    __device__ __forceinline__ explicit RowScale(uint32_t amax_bits) {
        const bool zero = amax_bits == 0;
        bad = amax_bits >= 0x7f80u;
        amax = __uint_as_float(amax_bits << 16);
        scale = bad ? __uint_as_float(0x7fc00000u) : zero ? 1.f : __fdiv_rn(amax, 127.f);
        // powers of two keep 127 x and 1 / amax inside fp32's range, and change no quotient
        pre = bad || zero ? 0.f : amax < 0x1p-100f ? 0x1p100f : amax > 0x1p100f ? 0x1p-100f : 1.f;
        amax = bad || zero ? 1.f : amax * pre;
        inv = __frcp_rn(amax);
    }
    __device__ __forceinline__ uint2 codes8(uint4 u) const {
        if (bad) u = make_uint4(0u, 0u, 0u, 0u);           // 0 * inf is not 0
        return make_uint2(codes4(u.x, u.y, pre, amax, inv), codes4(u.z, u.w, pre, amax, inv));
    }
};

// T threads per row (a power of two, 32 to 256), 256 / T rows per block.  Bound by memory: x is read once
// (rows of up to 8 CACHED T elements stay in registers between the absmax and the codes), the codes written
// once.
template <int T, int CACHED>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __nv_bfloat16* x, int8_t* codes, float* scales, int M, int K, long long ldx) {
    grid_dependency_wait();
    grid_launch_dependents();                              // a layer's product may fetch its weight meanwhile
    __shared__ uint32_t top[8];
    const int tid = threadIdx.x % T;
    const long long m = static_cast<long long>(blockIdx.x) * (256 / T) + threadIdx.x / T;
    const bool here = m < M;
    const uint4* row = reinterpret_cast<const uint4*>(x + (here ? m : 0) * ldx);
    const int pieces = here ? K / 8 : 0;
    uint4 kept[CACHED];
    uint32_t amax_bits = 0;
#pragma unroll
    for (int c = 0; c < CACHED; ++c)
        if (c * T + tid < pieces) kept[c] = row[c * T + tid];
#pragma unroll
    for (int c = 0; c < CACHED; ++c)
        if (c * T + tid < pieces) amax_bits = most_of(amax_bits, kept[c]);
    for (int c = CACHED * T + tid; c < pieces; c += T) amax_bits = most_of(amax_bits, row[c]);
    amax_bits = most_of_halves(amax_bits);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax_bits = max(amax_bits, __shfl_xor_sync(0xffffffffu, amax_bits, off));
    if (T > 32) {
        if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = amax_bits;
        __syncthreads();
        const int first = (threadIdx.x / T) * (T / 32);
#pragma unroll
        for (int w = 0; w < T / 32; ++w) amax_bits = max(amax_bits, top[first + w]);
    }
    const RowScale rs(amax_bits);
    if (here && tid == 0) scales[m] = rs.scale;
    uint2* out = reinterpret_cast<uint2*>(codes + (here ? m : 0) * K);
#pragma unroll
    for (int c = 0; c < CACHED; ++c)
        if (c * T + tid < pieces) out[c * T + tid] = rs.codes8(kept[c]);
    for (int c = CACHED * T + tid; c < pieces; c += T) out[c] = rs.codes8(row[c]);
}

// T threads per row, 256 / T rows per block, 8 codes per thread and step (a warp's store is 512 bytes in one
// piece), eight steps' codes in flight.  Bound by memory.
template <int T>
__global__ void __launch_bounds__(256) dequant_rows_kernel(const uint2* codes, const float* scales, uint4* x, int M, int K8) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long m = static_cast<long long>(blockIdx.x) * (256 / T) + threadIdx.x / T;
    if (m >= M) return;
    const float s = scales[m];
    const uint2* src = codes + m * K8;
    uint4* dst = x + m * K8;
    for (int c0 = threadIdx.x % T; c0 < K8; c0 += 8 * T) {
        uint2 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + i * T < K8) u[i] = src[c0 + i * T];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c0 + i * T >= K8) break;
            const int a = static_cast<int>(u[i].x), b = static_cast<int>(u[i].y);
            dst[c0 + i * T] = make_uint4(
                pack_bf16x2(s * static_cast<float>(a << 24 >> 24), s * static_cast<float>(a << 16 >> 24)),
                pack_bf16x2(s * static_cast<float>(a << 8 >> 24), s * static_cast<float>(a >> 24)),
                pack_bf16x2(s * static_cast<float>(b << 24 >> 24), s * static_cast<float>(b << 16 >> 24)),
                pack_bf16x2(s * static_cast<float>(b << 8 >> 24), s * static_cast<float>(b >> 24)));
        }
    }
}

// ------------------------------------------------------------------------------------
// product
// ------------------------------------------------------------------------------------
constexpr int BK = 128;                              // bytes = codes of K per stage
constexpr int NTHREADS = 192;                        // warp 0 TMA, 1 MMA, 2-5 epilogue

// y = acc * (sx * sw) + bias.  int32 -> fp32 rounds at 2^-24, far below the bf16 result's 2^-8.
__device__ __forceinline__ float result(uint32_t acc, float sx, float sw, float bias) {
    return fmaf(static_cast<float>(static_cast<int>(acc)), sx * sw, bias);
}

__device__ __forceinline__ void mma_i8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Many tokens.  Persistent CTA pairs walk 256 x 256 output tiles; CTA r of a pair loads rows 128 r.. of the
// tile's tokens and of its channels (half of each operand), the leader issues M256 N256 K32 MMAs that read
// both CTAs' shared memory, and each CTA's TMEM holds its own 128 rows of two accumulators in turn, so that
// the epilogue of one tile runs under the next one's products.  Tiles go in groups of 16 row blocks with the
// row block fastest: the tiles in flight share a few blocks of each operand in L2.
namespace pair {
constexpr int BN = 256, STAGES = 6, GROUP_M = 16;
constexpr int HALF_BYTES = 128 * BK, STAGE_BYTES = 2 * HALF_BYTES;       // A rows | B half rows
constexpr int OFF_BAR = STAGES * STAGE_BYTES;
enum Bar { FULL = 0, EMPTY = STAGES, TFULL = 2 * STAGES, TEMPTY = 2 * STAGES + 2, DRAIN = 2 * STAGES + 4,
           NBARS = 2 * STAGES + 5 };
constexpr int OFF_TMEM_SLOT = OFF_BAR + NBARS * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
constexpr int OFF_EPI = (OFF_ABORT + 8 + 15) & ~15;                      // per epilogue warp: 32 rows x 64 B
constexpr int EPI_WARP_BYTES = 32 * 64;
constexpr int SMEM_BYTES = OFF_EPI + 4 * EPI_WARP_BYTES + 1024;
constexpr uint32_t TMEM_COLS = 512;                                      // two 256-column int32 accumulators

__device__ __forceinline__ void tile_of(long long t, int m_tiles, int n_tiles, int& mb, int& nb) {
    const long long per_group = static_cast<long long>(GROUP_M) * n_tiles;
    const int g = static_cast<int>(t / per_group);
    const int rows = min(GROUP_M, m_tiles - g * GROUP_M);
    const long long w = t - g * per_group;
    mb = g * GROUP_M + static_cast<int>(w % rows);
    nb = static_cast<int>(w / rows);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
gemm_pair_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                 const Int8GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;     // the same offset in both CTAs
    uint8_t* smem = smem_raw + (base - raw_addr);
    const int warp = warp_id(), lane = lane_id();
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t bar0 = base + OFF_BAR;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const WaitCtl wc{abort_flag, p.wait_budget_ns, p.status};

    const int m_tiles = (p.M + 255) / 256, n_tiles = (p.N + BN - 1) / BN;
    const long long tiles = static_cast<long long>(m_tiles) * n_tiles;
    const int nk = (p.K + BK - 1) / BK;
    const long long pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(FULL + s), 1);
            mbar_init(bar(EMPTY + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(TFULL + b), 1);
            mbar_init(bar(TEMPTY + b), 256);
        }
        mbar_init(bar(DRAIN), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + OFF_TMEM_SLOT),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync_all();                 // both CTAs' barriers and TMEM exist before any remote use
    tc_fence_after();
    grid_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs; bytes counted on the leader's FULL) ----------------
        if (lane == 0) {
            tma_prefetch_desc(&tma_a);
            tma_prefetch_desc(&tma_b);
            int par[STAGES];
            for (int s = 0; s < STAGES; ++s) par[s] = -1;
            long long it = 0;
            bool ok = true;
            for (long long t = pair; t < tiles && ok; t += npairs) {
                int mb, nbk;
                tile_of(t, m_tiles, n_tiles, mb, nbk);
                const int m0 = mb * 256 + static_cast<int>(rank) * 128;
                const int nb = nbk * BN + static_cast<int>(rank) * 128;
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = static_cast<int>(it % STAGES);
                    const int use = static_cast<int>((it / STAGES) & 1);
                    ok = wait_thread(bar(EMPTY + s), use ^ 1, wc);
                    if (!ok) break;
                    if (leader) mbar_arrive_expect_tx(bar(FULL + s), 2 * STAGE_BYTES);
                    const uint32_t full = mapa_shared(bar(FULL + s), 0);
                    const uint32_t st = base + s * STAGE_BYTES;
                    tma_load_2d_pair(st, &tma_a, full, kb * BK, m0);
                    tma_load_2d_pair(st + HALF_BYTES, &tma_b, full, kb * BK, nb);
                    par[s] = use;
                }
            }
            if (!ok && leader)
                for (int s = 0; s < STAGES; ++s)
                    if (par[s] >= 0) drain_wait(bar(FULL + s), par[s]);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader only) ----------------
        if (lane == 0 && leader) {
            const uint32_t idesc = make_idesc(2, 1, 1, 0, 0, 256, BN);       // s32 <- s8 x s8, K-major
            long long it = 0;
            int tc = 0;
            bool ok = true;
            for (long long t = pair; t < tiles && ok; t += npairs, ++tc) {
                const int b = tc & 1;
                ok = wait_thread(bar(TEMPTY + b), ((tc >> 1) & 1) ^ 1, wc);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + b * BN;
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = static_cast<int>(it % STAGES);
                    ok = wait_thread(bar(FULL + s), static_cast<int>((it / STAGES) & 1), wc);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sa = base + s * STAGE_BYTES, sb = sa + HALF_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        mma_i8_ss_pair(acc, sdesc_sw128(sa + kk * 32, 16, 1024), sdesc_sw128(sb + kk * 32, 16, 1024),
                                       idesc, (kb > 0 || kk > 0) ? 1u : 0u);
                    mma_commit_pair(bar(EMPTY + s));                         // both CTAs' stage s is free
                    mma_commit_pair(mapa_shared(bar(EMPTY + s), 1));
                }
                if (!ok) break;
                mma_commit_pair(bar(TFULL + b));
                mma_commit_pair(mapa_shared(bar(TFULL + b), 1));
            }
            mma_commit_pair(bar(DRAIN));
            drain_wait(bar(DRAIN), 0);
        }
    } else {
        // ---------------- epilogue (both CTAs: each its own 128 rows) ----------------
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tempty_leader = mapa_shared(bar(TEMPTY), 0);
        int tc = 0;
        bool ok = true;
        for (long long t = pair; t < tiles && ok; t += npairs, ++tc) {
            int mb, nbk;
            tile_of(t, m_tiles, n_tiles, mb, nbk);
            const int m0 = mb * 256 + static_cast<int>(rank) * 128;
            const int n0 = nbk * BN;
            const int b = tc & 1;
            ok = wait_warp(bar(TFULL + b), (tc >> 1) & 1, wc);
            if (!ok) break;
            tc_fence_after();
            const int m = m0 + r;
            const float sx = m < p.M ? p.a_scales[m] : 0.f;
            // each 32-column chunk goes through the warp's 2 KB of shared memory (16-byte pieces
            // swizzled by row / 2), so that a store writes 8 whole 64-byte row segments
            uint8_t* wbuf = smem + OFF_EPI + (warp - 2) * EPI_WARP_BYTES;
            const int row0 = m0 + (warp & 3) * 32;                           // this warp's 32 rows
#pragma unroll 1
            for (int c = 0; c < BN / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(tmem + b * BN + lane_off + c * 32, v);
                tmem_wait_ld();
                if (n0 + c * 32 >= p.N) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // 8 channels (N % 8 == 0: all there or none); the same addresses in every lane
                    const int n = n0 + c * 32 + q * 8;
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (n < p.N) {
                        float sw[8], bi[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) sw[e] = p.b_scales[n + e];
                        const uint4 u = p.bias ? *reinterpret_cast<const uint4*>(p.bias + n) : w;
                        const uint32_t bw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = bf16x2_floats(bw[e]);
                            bi[2 * e] = f.x;
                            bi[2 * e + 1] = f.y;
                        }
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = pack_bf16x2(result(v[q * 8 + 2 * e], sx, sw[2 * e], bi[2 * e]),
                                               result(v[q * 8 + 2 * e + 1], sx, sw[2 * e + 1], bi[2 * e + 1]));
                        w = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    *reinterpret_cast<uint4*>(wbuf + lane * 64 + ((q ^ ((lane >> 1) & 3)) * 16)) = w;
                }
                __syncwarp();
                const int n = n0 + c * 32 + (lane & 3) * 8;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int rr = 8 * k + (lane >> 2);
                    const uint4 val =
                        *reinterpret_cast<const uint4*>(wbuf + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) * 16));
                    const int mm = row0 + rr;
                    if (mm < p.M && n < p.N)
                        *reinterpret_cast<uint4*>(p.y + static_cast<long long>(mm) * p.N + n) = val;
                }
                __syncwarp();
            }
            tc_fence_before();
            mbar_arrive_cluster(tempty_leader + 8u * static_cast<uint32_t>(b));   // leader's TEMPTY[b]
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                 // no CTA leaves while its peer may still signal it
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                                : "memory");
}
}  // namespace pair

// Few tokens: bound by reading the weight once.  The MMA's M is 128 channels, its N is NT tokens (the tile
// that a row of tokens would leave mostly empty the other way round).  The CTAs of a cluster share a tile
// and split K, so that a layer of a few dozen channel tiles still keeps every SM loading; each keeps its
// int32 partial tile in shared memory, and after a cluster barrier every CTA adds up (exactly) and stores
// its share of the tokens.  Launched behind the quantiser as a dependent launch it fetches its first
// weight stages while the quantiser still runs (p.after_quant).
namespace few {
template <int NT>
struct Cfg {
    static constexpr int A_BYTES = 128 * BK, B_BYTES = NT * BK, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = NT <= 32 ? 5 : NT == 64 ? 4 : 3;           // two CTAs per SM
    static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
    static constexpr int FULL = 0, EMPTY = STAGES, DONE = 2 * STAGES, NBARS = 2 * STAGES + 1;
    static constexpr int OFF_TMEM_SLOT = OFF_BAR + NBARS * 8;
    static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
    static constexpr int SMEM_BYTES = OFF_ABORT + 8 + 1024;
    static constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
    static_assert(NT * 128 * 4 <= STAGES * STAGE_BYTES, "the partial tile reuses the stages");
    static_assert(2 * SMEM_BYTES <= 228 * 1024 - 2048, "two CTAs per SM");
};

// The cluster's partial tiles (at `base` in each CTA, [token][channel] int32) summed, scaled and stored: this
// CTA takes tokens rank, rank + splits, ... of the tile, one warp a token, four channels a lane.
template <int NT>
__device__ __forceinline__ void store_tokens(const Int8GemmParams& p, uint32_t base, const float* sx, bool ok, int n0,
                                             int m0, int rank, int splits, int warps) {
    const int lane = lane_id(), n = n0 + lane * 4;
    if (!ok || n >= p.N) return;
    const float4 sw = make_float4(p.b_scales[n], p.b_scales[n + 1], p.b_scales[n + 2], p.b_scales[n + 3]);
    float2 b01 = make_float2(0.f, 0.f), b23 = b01;
    if (p.bias) {
        const uint2 u = *reinterpret_cast<const uint2*>(p.bias + n);
        b01 = bf16x2_floats(u.x);
        b23 = bf16x2_floats(u.y);
    }
    const int tokens = min(NT, p.M - m0);
    for (int t = rank + (threadIdx.x >> 5) * splits; t < tokens; t += warps * splits) {
        const uint32_t at = base + (t * 128 + lane * 4) * 4;
        uint4 acc = make_uint4(0u, 0u, 0u, 0u);
        for (int z = 0; z < splits; ++z) {
            const uint4 v = ld_shared_cluster_v4(splits > 1 ? mapa_shared(at, z) : at);
            acc = make_uint4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
        }
        *reinterpret_cast<uint2*>(p.y + static_cast<long long>(m0 + t) * p.N + n) =
            make_uint2(pack_bf16x2(result(acc.x, sx[t], sw.x, b01.x), result(acc.y, sx[t], sw.y, b01.y)),
                       pack_bf16x2(result(acc.z, sx[t], sw.z, b23.x), result(acc.w, sx[t], sw.w, b23.y)));
    }
}

template <int NT>
__global__ void __launch_bounds__(NTHREADS, 2)
gemm_few_kernel(const __grid_constant__ CUtensorMap tma_x, const __grid_constant__ CUtensorMap tma_w,
                const Int8GemmParams p) {
    using C = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;     // the same offset in every CTA
    uint8_t* smem = smem_raw + (base - raw_addr);
    const int warp = warp_id(), lane = lane_id();
    const int splits = gridDim.x, rank = blockIdx.x;       // the cluster is the grid's x
    const int n0 = blockIdx.y * 128, m0 = blockIdx.z * NT;
    const int nk_all = (p.K + BK - 1) / BK;
    const int k0 = rank * nk_all / splits, nk = (rank + 1) * nk_all / splits - k0;
    const uint32_t bar0 = base + C::OFF_BAR;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    const WaitCtl wc{abort_flag, p.wait_budget_ns, p.status};

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(bar(C::FULL + s), 1);
            mbar_init(bar(C::EMPTY + s), 1);
        }
        mbar_init(bar(C::DONE), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (!p.after_quant) grid_dependency_wait();
    if (warp == 1) {
        tmem_alloc(base + C::OFF_TMEM_SLOT, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM_SLOT);

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&tma_x);
            tma_prefetch_desc(&tma_w);
            auto load_w = [&](int kb) {
                const int s = kb % C::STAGES;
                mbar_arrive_expect_tx(bar(C::FULL + s), C::STAGE_BYTES);
                tma_load_2d(base + s * C::STAGE_BYTES, &tma_w, bar(C::FULL + s), (k0 + kb) * BK, n0);
            };
            auto load_x = [&](int kb) {
                const int s = kb % C::STAGES;
                tma_load_2d(base + s * C::STAGE_BYTES + C::A_BYTES, &tma_x, bar(C::FULL + s), (k0 + kb) * BK, m0);
            };
            const int early = min(nk, C::STAGES);
            for (int kb = 0; kb < early; ++kb) load_w(kb);
            if (p.after_quant) grid_dependency_wait();     // x's codes are the quantiser's
            for (int kb = 0; kb < early; ++kb) load_x(kb);
            int issued = early;
            bool ok = true;
            for (int kb = early; kb < nk; ++kb) {
                ok = wait_thread(bar(C::EMPTY + kb % C::STAGES), ((kb / C::STAGES) & 1) ^ 1, wc);
                if (!ok) break;
                load_w(kb);
                load_x(kb);
                issued = kb + 1;
            }
            if (!ok)
                for (int kb = max(0, issued - C::STAGES); kb < issued; ++kb)
                    drain_wait(bar(C::FULL + kb % C::STAGES), (kb / C::STAGES) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc(2, 1, 1, 0, 0, 128, NT);       // s32 <- s8 x s8, K-major
            for (int kb = 0; kb < nk; ++kb) {
                const int s = kb % C::STAGES;
                if (!wait_thread(bar(C::FULL + s), (kb / C::STAGES) & 1, wc)) {
                    // what is in flight lands before the CTA's shared memory goes away
                    for (int j = kb; j < min(nk, kb + C::STAGES); ++j)
                        drain_wait(bar(C::FULL + j % C::STAGES), (j / C::STAGES) & 1);
                    break;
                }
                tc_fence_after();
                const uint32_t sa = base + s * C::STAGE_BYTES, sb = sa + C::A_BYTES;
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)
                    mma_i8_ss(tmem, sdesc_sw128(sa + kk * 32, 16, 1024), sdesc_sw128(sb + kk * 32, 16, 1024), idesc,
                              (kb > 0 || kk > 0) ? 1u : 0u);
                mma_commit(bar(C::EMPTY + s));
            }
            mma_commit(bar(C::DONE));                      // all of this CTA's products, also after a time-out
        }
    } else {
        // partial tile [token][channel] (int32) over the stages, which every MMA has read by now
        const bool ok = wait_warp(bar(C::DONE), 0, wc);
        if (ok) {
            tc_fence_after();
            const int ch = (warp & 3) * 32 + lane;
            const uint32_t src = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            int* part = reinterpret_cast<int*>(smem);
#pragma unroll 1
            for (int t = 0; t < NT; t += 16) {
                uint32_t v[16];
                tmem_ld16(src + t, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) part[(t + e) * 128 + ch] = static_cast<int>(v[e]);
            }
        } else {
            drain_wait(bar(C::DONE), 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (splits > 1) cluster_sync_all();
    tc_fence_after();

    if (p.after_quant) grid_dependency_wait();             // the scales are the quantiser's
    store_tokens<NT>(p, base, p.a_scales + m0, *abort_flag == 0, n0, m0, rank, splits, NTHREADS / 32);
    __syncthreads();
    if (splits > 1) cluster_sync_all();                    // no CTA leaves while a peer reads its partial tile
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// The layer for up to 16 tokens in one launch: bound by latency and by the weight's bytes.  While the weight's
// first stages are on their way, each CTA of a cluster turns its own slice of K of the tokens into 8 bits,
// straight into the swizzled operand, which stays for all of the CTA's stages.  A slice is read once and kept in
// registers (LAYER_PIECES of 8 elements a thread); the row's absmax meets through distributed shared memory.
// Every channel tile does so again; the few tokens come from L2.  The first tile's cluster also writes the
// checkpoint, if one is asked for.  One launch less is what it saves: a token of 1536 -> 1536 takes 5.3 us a call
// against 7.2 with a quantiser launched before the product.  In a graph, and where the weight's bytes take
// longer, the two kernels overlap as well (5120 -> 5120, weights from memory: 10.0 us both; in a graph 9.3 and
// 9.1), and with more tokens they win (37 tokens of 1536 -> 8960: 8.2 and 11.4), so it stops at 16.
constexpr int LAYER_TOKENS = 16, LAYER_PIECES = 8;         // pieces of the slice a thread keeps
struct LayerCfg {
    static constexpr int A_BYTES = 128 * BK, STAGES = 5;
    static constexpr int X_BLOCK = LAYER_TOKENS * BK, X_MAX = 24 * 1024;     // a K block of codes; all of them
    static constexpr int OFF_X = STAGES * A_BYTES;
    static constexpr int OFF_ROW = OFF_X + X_MAX;                            // a token's pre, absmax, 1 / absmax, bad
    static constexpr int OFF_TOP = OFF_ROW + LAYER_TOKENS * 16, OFF_SCALE = OFF_TOP + LAYER_TOKENS * 4;
    static constexpr int OFF_BAR = OFF_SCALE + LAYER_TOKENS * 4;
    static constexpr int FULL = 0, EMPTY = STAGES, READY = 2 * STAGES, DONE = 2 * STAGES + 1, NBARS = 2 * STAGES + 2;
    static constexpr int OFF_TMEM_SLOT = OFF_BAR + NBARS * 8;
    static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
    static constexpr int SMEM_BYTES = OFF_ABORT + 8 + 1024;
    static constexpr int NTHREADS = 320, QUANT = 256;                        // warp 0 TMA, 1 MMA, 2-9 quantiser
    static constexpr uint32_t TMEM_COLS = 32;
    static_assert(LAYER_TOKENS * 128 * 4 <= STAGES * A_BYTES, "the partial tile reuses the stages");
    static_assert(2 * SMEM_BYTES <= 228 * 1024 - 2048, "two CTAs per SM");
};

struct LayerParams : Int8GemmParams {
    const __nv_bfloat16* x;           // [M, K], ldx apart
    long long ldx;
    int8_t* codes;                    // [M, K] or null
    float* scales;                    // [M] or null
};

__global__ void __launch_bounds__(LayerCfg::NTHREADS, 2)
layer_few_kernel(const __grid_constant__ CUtensorMap tma_w, const LayerParams p) {
    using C = LayerCfg;
    constexpr int NT = LAYER_TOKENS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;     // the same offset in every CTA
    uint8_t* smem = smem_raw + (base - raw_addr);
    const int warp = warp_id(), lane = lane_id();
    const int splits = gridDim.x, rank = blockIdx.x;       // the cluster is the grid's x
    const int n0 = blockIdx.y * 128;
    const int nk_all = (p.K + BK - 1) / BK;
    const int k0 = rank * nk_all / splits, nk = (rank + 1) * nk_all / splits - k0;
    const uint32_t bar0 = base + C::OFF_BAR;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    const WaitCtl wc{abort_flag, p.wait_budget_ns, p.status};
    uint32_t* top = reinterpret_cast<uint32_t*>(smem + C::OFF_TOP);
    float* scale = reinterpret_cast<float*>(smem + C::OFF_SCALE);
    float4* rows = reinterpret_cast<float4*>(smem + C::OFF_ROW);
    const int pieces = (min(p.K, (k0 + nk) * BK) - k0 * BK) / 8;             // 8-element pieces of the slice

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(bar(C::FULL + s), 1);
            mbar_init(bar(C::EMPTY + s), 1);
        }
        mbar_init(bar(C::READY), C::QUANT / 32);
        mbar_init(bar(C::DONE), 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tma_w);
        // the weight needs nothing of what follows
        grid_dependency_wait();
        for (int kb = 0; kb < min(nk, C::STAGES); ++kb) {
            mbar_arrive_expect_tx(bar(C::FULL + kb), C::A_BYTES);
            tma_load_2d(base + kb * C::A_BYTES, &tma_w, bar(C::FULL + kb), (k0 + kb) * BK, n0);
        }
    }
    grid_dependency_wait();
    if (warp == 1) {
        tmem_alloc(base + C::OFF_TMEM_SLOT, C::TMEM_COLS);
        tmem_relinquish();
    }
    // piece i * QUANT + q of the slice, token by token, is thread q's i-th
    const int q = static_cast<int>(threadIdx.x) - 64;
    auto piece_of = [&](int i, int per_token, int& t, int& c) {
        const int at = i * C::QUANT + q;
        t = at / per_token;
        c = at - t * per_token;
        return t < p.M;
    };
    auto load = [&](int t, int c) { return *reinterpret_cast<const uint4*>(p.x + t * p.ldx + c * 8); };
    // the whole warp: into the token's absmax, with one atomic where its lanes hold one token
    auto fold = [&](bool here, int t, uint32_t most) {
        const int t0 = __shfl_sync(0xffffffffu, t, 0);
        if (__all_sync(0xffffffffu, here && t == t0)) {
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) atomicMax(top + t0, most);
        } else if (here) {
            atomicMax(top + t, most);
        }
    };
    uint4 kept[LAYER_PIECES];
    if (warp >= 2) {
        if (q < NT) top[q] = 0;
#pragma unroll
        for (int i = 0; i < LAYER_PIECES; ++i) {
            int t, c;
            if (piece_of(i, pieces, t, c)) kept[i] = load(t, k0 * (BK / 8) + c);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_launch_dependents();
    if (warp >= 2) {
#pragma unroll
        for (int i = 0; i < LAYER_PIECES; ++i) {
            if (i * C::QUANT >= p.M * pieces) break;       // the same for every thread
            int t, c;
            const bool here = piece_of(i, pieces, t, c);
            fold(here, t, here ? most_of_halves(most_of(0u, kept[i])) : 0u);
        }
    }
    if (splits > 1) cluster_sync_all();        // the slices' absmax are there
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM_SLOT);

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int issued = min(nk, C::STAGES);
            for (int kb = issued; kb < nk; ++kb) {
                const int s = kb % C::STAGES;
                ok = wait_thread(bar(C::EMPTY + s), ((kb / C::STAGES) & 1) ^ 1, wc);
                if (!ok) break;
                mbar_arrive_expect_tx(bar(C::FULL + s), C::A_BYTES);
                tma_load_2d(base + s * C::A_BYTES, &tma_w, bar(C::FULL + s), (k0 + kb) * BK, n0);
                issued = kb + 1;
            }
            if (!ok)
                for (int kb = max(0, issued - C::STAGES); kb < issued; ++kb)
                    drain_wait(bar(C::FULL + kb % C::STAGES), (kb / C::STAGES) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc(2, 1, 1, 0, 0, 128, NT);       // s32 <- s8 x s8, K-major
            const bool ready = wait_thread(bar(C::READY), 0, wc);
            for (int kb = 0; kb < nk; ++kb) {
                const int s = kb % C::STAGES;
                if (!ready || !wait_thread(bar(C::FULL + s), (kb / C::STAGES) & 1, wc)) {
                    // what is in flight lands before the CTA's shared memory goes away
                    for (int j = kb; j < min(nk, kb + C::STAGES); ++j)
                        drain_wait(bar(C::FULL + j % C::STAGES), (j / C::STAGES) & 1);
                    break;
                }
                tc_fence_after();
                const uint32_t sa = base + s * C::A_BYTES, sb = base + C::OFF_X + kb * C::X_BLOCK;
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)
                    mma_i8_ss(tmem, sdesc_sw128(sa + kk * 32, 16, 1024), sdesc_sw128(sb + kk * 32, 16, 1024), idesc,
                              (kb > 0 || kk > 0) ? 1u : 0u);
                mma_commit(bar(C::EMPTY + s));
            }
            mma_commit(bar(C::DONE));                      // all of this CTA's products, also after a time-out
        }
    } else {
        named_bar_sync(1, C::QUANT);
        if (q < p.M) {
            uint32_t most = top[q];
            for (int z = 0; z < splits; ++z)
                if (z != rank) most = max(most, ld_shared_cluster_u32(mapa_shared(smem_u32(top + q), z)));
            const RowScale rs(most);
            scale[q] = rs.scale;
            rows[q] = make_float4(rs.pre, rs.amax, rs.inv, rs.bad ? 1.f : 0.f);
            if (p.scales && blockIdx.y == 0 && rank == 0) p.scales[q] = rs.scale;
        }
        named_bar_sync(1, C::QUANT);
#pragma unroll
        for (int i = 0; i < LAYER_PIECES; ++i) {
            int t, c;
            if (!piece_of(i, pieces, t, c)) break;
            const float4 row = rows[t];
            uint4 u = kept[i];
            if (row.w != 0.f) u = make_uint4(0u, 0u, 0u, 0u);
            const uint2 v = make_uint2(codes4(u.x, u.y, row.x, row.y, row.z), codes4(u.z, u.w, row.x, row.y, row.z));
            // half of 16-byte chunk (c / 2) % 8 of row t of K block c / 16
            const uint32_t at = sw128_chunk(base + C::OFF_X + (c >> 4) * C::X_BLOCK, t, (c >> 1) & 7) + (c & 1) * 8;
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(v.x), "r"(v.y) : "memory");
            if (p.codes && blockIdx.y == 0)
                *reinterpret_cast<uint2*>(p.codes + static_cast<long long>(t) * p.K + k0 * BK + c * 8) = v;
        }
        // rows behind the last token and codes behind K stay whatever they are: they meet other columns of the
        // result, and zeros of the weight
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::READY));
        if (warp < 6) {
            // partial tile [token][channel] (int32) over the stages, which every MMA has read by now
            if (wait_warp(bar(C::DONE), 0, wc)) {
                tc_fence_after();
                const int ch = (warp & 3) * 32 + lane;
                const uint32_t src = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
                int* part = reinterpret_cast<int*>(smem);
#pragma unroll 1
                for (int t = 0; t < NT; t += 16) {
                    uint32_t v[16];
                    tmem_ld16(src + t, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) part[(t + e) * 128 + ch] = static_cast<int>(v[e]);
                }
            } else {
                drain_wait(bar(C::DONE), 0);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (splits > 1) cluster_sync_all();
    tc_fence_after();
    store_tokens<NT>(p, base, scale, *abort_flag == 0, n0, 0, rank, splits, C::NTHREADS / 32);
    __syncthreads();
    if (splits > 1) cluster_sync_all();                    // no CTA leaves while a peer reads its partial tile
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// K is split while the CTAs stay within two per SM and each has two stages of K or more.
int splits_for(int m_tiles, int N, int K) {
    const int n_tiles = (N + 127) / 128, nk = (K + BK - 1) / BK;
    int splits = 1;
    while (splits < 8 && 2ll * splits * n_tiles * m_tiles <= 2 * 148 && nk / (2 * splits) >= 2) splits *= 2;
    return splits;
}

// Whether a layer fits layer_few: the slices stay in registers, their codes in the operand that stays.
bool layer_fits(int M, int N, int K) {
    if (M > LAYER_TOKENS || N > 65535 * 128) return false;
    const int nk = (K + BK - 1) / BK, splits = splits_for(1, N, K), most = (nk + splits - 1) / splits;
    return most * LayerCfg::X_BLOCK <= LayerCfg::X_MAX && M * most * (BK / 8) <= LAYER_PIECES * LayerCfg::QUANT;
}

int launch_layer(const CUtensorMap& tw, const LayerParams& p, cudaStream_t stream) {
    if (configure_smem(reinterpret_cast<const void*>(layer_few_kernel), LayerCfg::SMEM_BYTES) != 0) return -1;
    const int splits = splits_for(1, p.N, p.K);
    return launch_dependent(layer_few_kernel, dim3(splits, (p.N + 127) / 128), LayerCfg::NTHREADS, LayerCfg::SMEM_BYTES,
                            stream, splits, true, tw, p);
}

template <int NT>
int launch(const CUtensorMap& tx, const CUtensorMap& tw, const Int8GemmParams& p, cudaStream_t stream) {
    if (configure_smem(reinterpret_cast<const void*>(gemm_few_kernel<NT>), Cfg<NT>::SMEM_BYTES) != 0) return -1;
    const int n_tiles = (p.N + 127) / 128, m_tiles = (p.M + NT - 1) / NT;
    const int splits = splits_for(m_tiles, p.N, p.K);
    return launch_dependent(gemm_few_kernel<NT>, dim3(splits, n_tiles, m_tiles), NTHREADS, Cfg<NT>::SMEM_BYTES, stream,
                            splits, true, tx, tw, p);
}
}  // namespace few

template <int T, int CACHED>
int launch_quant(const void* x, void* codes, float* scales, int M, int K, long long ldx, cudaStream_t stream) {
    const int rows = 256 / T;
    return launch_dependent(quant_rows_kernel<T, CACHED>, dim3((M + rows - 1) / rows), 256, 0, stream, 1, true,
                            static_cast<const __nv_bfloat16*>(x), static_cast<int8_t*>(codes), scales, M, K, ldx);
}
template <int T>
int launch_dequant(const void* codes, const float* scales, void* x, int M, int K, cudaStream_t stream) {
    const int rows = 256 / T;
    return launch_dependent(dequant_rows_kernel<T>, dim3((M + rows - 1) / rows), 256, 0, stream, 1, true,
                            static_cast<const uint2*>(codes), scales, static_cast<uint4*>(x), M, K / 8);
}

}  // namespace int8

int launch_int8_quant_rows(const void* x, void* codes, float* scales, int M, int K, long long ldx, cudaStream_t stream) {
    // Few rows: all of a block on each, for latency (148 rows of 5120: 8 us, 12 with 32 threads a row).  Else as
    // few threads as keep the row in registers.  32760 rows, us with 32, 64, 128, 256 threads: of 1536 elements
    // 31, 41, 60, 96; of 4096 78, 66, 78, 114; of 5120 98, 94, 88, 121; of 13824 397, 272, 240, 197.  Rows of 512
    // with room for 4 pieces a thread 18 us, for 8 21.
    if (M <= 148) return int8::launch_quant<256, 4>(x, codes, scales, M, K, ldx, stream);
    if (K <= 1024) return int8::launch_quant<32, 4>(x, codes, scales, M, K, ldx, stream);
    if (K <= 2048) return int8::launch_quant<32, 8>(x, codes, scales, M, K, ldx, stream);
    if (K <= 4096) return int8::launch_quant<64, 8>(x, codes, scales, M, K, ldx, stream);
    if (K <= 8192) return int8::launch_quant<128, 8>(x, codes, scales, M, K, ldx, stream);
    return int8::launch_quant<256, 8>(x, codes, scales, M, K, ldx, stream);
}

int launch_int8_dequant_rows(const void* codes, const float* scales, void* x, int M, int K, cudaStream_t stream) {
    // 32760 rows, us with 32, 64, 256 threads a row: of 512 elements 16, 21, 39; of 5120 84, 82, 84; of 13824 219,
    // 217, 207
    if (K <= 2048) return int8::launch_dequant<32>(codes, scales, x, M, K, stream);
    if (K <= 8192) return int8::launch_dequant<64>(codes, scales, x, M, K, stream);
    return int8::launch_dequant<256>(codes, scales, x, M, K, stream);
}

bool int8_layer_fits(int M, int N, int K) { return int8::few::layer_fits(M, N, K); }

int launch_int8_layer(const CUtensorMap& tw, const void* x, long long ldx, void* codes, float* scales,
                      const Int8GemmParams& p, cudaStream_t stream) {
    int8::few::LayerParams q;
    static_cast<Int8GemmParams&>(q) = p;
    q.x = static_cast<const __nv_bfloat16*>(x);
    q.ldx = ldx;
    q.codes = static_cast<int8_t*>(codes);
    q.scales = scales;
    return int8::few::launch_layer(tw, q, stream);
}

int int8_gemm_token_tile(int M, int N) {
    // pairs where their 256 x 256 tiles occupy at least half of the SMs (and where the other kernel's
    // channel tiles would not fit a grid)
    if ((static_cast<long long>((M + 255) / 256) * ((N + 255) / 256) * 2 >= 74 && M > 128) || N > 65535 * 128) return 0;
    return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
}

int launch_int8_gemm(const CUtensorMap& tx, const CUtensorMap& tw, const Int8GemmParams& p, cudaStream_t stream) {
    switch (int8_gemm_token_tile(p.M, p.N)) {
        case 16: return int8::few::launch<16>(tx, tw, p, stream);
        case 32: return int8::few::launch<32>(tx, tw, p, stream);
        case 64: return int8::few::launch<64>(tx, tw, p, stream);
        case 128: return int8::few::launch<128>(tx, tw, p, stream);
    }
    namespace pr = int8::pair;
    if (configure_smem(reinterpret_cast<const void*>(pr::gemm_pair_kernel), pr::SMEM_BYTES) != 0) return -1;
    const long long tiles = static_cast<long long>((p.M + 255) / 256) * ((p.N + pr::BN - 1) / pr::BN);
    const int grid = 2 * static_cast<int>(tiles < 74 ? tiles : 74);
    return launch_dependent(pr::gemm_pair_kernel, dim3(grid), int8::NTHREADS, pr::SMEM_BYTES, stream, 1, true, tx, tw, p);
}

}  // namespace wan
