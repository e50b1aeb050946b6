// C-ABI layer: argument validation, TMA tensor maps, launches, status word.
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <mutex>
#include <set>
#include <utility>

#include "wan_attn.h"
#include "sm100_ptx.cuh"
#include "wan_attn_internal.h"

namespace wan {

__device__ int g_device_status = 0;

int* device_status_word() {
    static std::mutex mu;
    static int* addr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void* a = nullptr;
        if (cudaGetSymbolAddress(&a, g_device_status) != cudaSuccess) return nullptr;
        addr[dev] = static_cast<int*>(a);
    }
    return addr[dev];
}

namespace {

std::atomic<unsigned long long> g_wait_budget_ns{2000000000ull};

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Tensor map over a bf16 [B, S, H, D] tensor viewed as 4-D (D, H, S, B), box
// (64 of D, 1 head, `box_tokens` tokens, 1 batch) with the 128-byte swizzle.
// Coordinates past S read as zero.
bool make_bshd_map(CUtensorMap* m, const void* base, int B, int S, int H, int D, int box_tokens) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2, (cuuint64_t)S * H * D * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_tokens, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over an 8-bit [B*H, S, 128] tensor viewed as 3-D (128, S, B*H), box (128, rows, 1),
// 128-byte swizzle (one 128-byte row per token), tokens past S read as zero.
bool make_bh_s_d8_map(CUtensorMap* m, const void* base, int BH, int S, int rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {128, (cuuint64_t)S, (cuuint64_t)BH};
    const cuuint64_t strides[2] = {128, (cuuint64_t)S * 128};
    const cuuint32_t box[3] = {128, (cuuint32_t)rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over the fp32 dQ accumulator [B, S, H, 128] as 4-D (128, H, S, B), box
// (128, 1, 128, 1) without swizzle: the backward adds [128 query][128 d] tiles into it.
bool make_dq_acc_map(CUtensorMap* m, void* base, int B, int S, int H) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {128, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
    const cuuint64_t strides[3] = {128 * 4, (cuuint64_t)H * 128 * 4, (cuuint64_t)S * H * 128 * 4};
    const cuuint32_t box[4] = {128, 1, 128, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over an fp32 [B, S, H, 128] accumulator as 4-D (128, H, S, B), box (32, 1, 128, 1)
// with the 128-byte swizzle: the split backward adds [128 key][32 d] sub-tiles of dK, dV into it.
bool make_acc_sw_map(CUtensorMap* m, void* base, int B, int S, int H) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {128, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
    const cuuint64_t strides[3] = {128 * 4, (cuuint64_t)H * 128 * 4, (cuuint64_t)S * H * 128 * 4};
    const cuuint32_t box[4] = {32, 1, 128, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over an 8-bit [rows, K] matrix (K contiguous) as 2-D (K, rows), box (128, box_rows),
// 128-byte swizzle; elements past the edges read as zero.
bool make_rows_u8_map(CUtensorMap* m, const void* base, int rows, int K, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shape checks of the FP8 GEMM calls: rows, K >= 1, K % 16 == 0 (16-byte code rows),
// rows * K < 2^40.
int check_fp8_shape(long long rows, long long K) {
    if (rows < 1 || K < 16 || (K & 15) || rows > 0x7fffffffLL || K > 0x7fffffffLL) return WAN_ATTN_ERR_INVALID_ARG;
    if (double(rows) * double(K) >= double(1ull << 40)) return WAN_ATTN_ERR_INVALID_ARG;
    return WAN_ATTN_OK;
}

struct Range {
    uintptr_t lo, hi;
};
Range range_of(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes};
}
bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Shape checks common to every call.  Returns a wan_attn_status.
int check_shape(int B, int S, int H, int D) {
    if (B < 1 || S < 1 || H < 1 || D < 1) return WAN_ATTN_ERR_INVALID_ARG;
    if (D != 128) return WAN_ATTN_ERR_UNSUPPORTED;
    if (B > 65535 || H > 65535) return WAN_ATTN_ERR_INVALID_ARG;       // grid y/z limits
    const double n = double(B) * S * H * D;
    if (n >= double(1ull << 40)) return WAN_ATTN_ERR_INVALID_ARG;
    return WAN_ATTN_OK;
}

}  // namespace

int configure_smem(const void* kernel, int bytes) {
    static std::mutex mu;
    static std::set<std::pair<int, const void*>> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({dev, kernel})) return 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return -1;
    done.insert({dev, kernel});
    return 0;
}

unsigned long long wait_budget_ns() { return g_wait_budget_ns.load(); }

// ---------------------------------------------------------------------------
// bounded-wait self test: one warp waits on a barrier that nobody arrives at
// ---------------------------------------------------------------------------
__global__ void selftest_wait_kernel(unsigned long long budget_ns, int* status) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        mbar_init(b, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const WaitCtl wc{&abort_flag, budget_ns, status};
    (void)wait_warp(b, 0, wc);     // gives up after budget_ns and records the timeout
    __syncthreads();
}

}  // namespace wan

using namespace wan;

namespace {

// Forward of Sq queries against Skv keys (self-attention: Skv = Sq).  The cross-attention call
// with a short key sequence (Skv <= 1024, Sq != Skv: the text embedding) runs the per-tile
// kernel: with a few key blocks per tile, a CTA's prologue and epilogue are much of its time,
// and two CTAs per SM hide each other's.
int fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Sq, int Skv, int H,
             int D, void* stream, bool cross) {
    if (!q || !k || !v || !o || !lse) return WAN_ATTN_ERR_INVALID_ARG;
    int st = check_shape(B, Sq, H, D);
    if (st == WAN_ATTN_OK) st = check_shape(B, Skv, H, D);
    if (st != WAN_ATTN_OK) return st;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return WAN_ATTN_ERR_INVALID_ARG;
    const size_t nq = size_t(B) * Sq * H * D, nkv = size_t(B) * Skv * H * D;
    const Range rq = range_of(q, nq * 2), rk = range_of(k, nkv * 2), rv = range_of(v, nkv * 2);
    const Range ro = range_of(o, nq * 2), rl = range_of(lse, size_t(B) * H * Sq * 4);
    for (const Range& in : {rq, rk, rv})
        if (overlaps(ro, in) || overlaps(rl, in)) return WAN_ATTN_ERR_INVALID_ARG;
    if (overlaps(ro, rl)) return WAN_ATTN_ERR_INVALID_ARG;

    const bool per_tile = cross && Sq != Skv && Skv <= 1024;
    const int kv_box = per_tile ? 64 : 128;
    CUtensorMap tq, tk, tv, to;
    if (!make_bshd_map(&tq, q, B, Sq, H, D, 128) || !make_bshd_map(&tk, k, B, Skv, H, D, kv_box) ||
        !make_bshd_map(&tv, v, B, Skv, H, D, kv_box) || !make_bshd_map(&to, o, B, Sq, H, D, 128))
        return WAN_ATTN_ERR_CUDA;
    FwdParams p{};
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.S = Sq;
    p.Skv = Skv;
    p.H = H;
    p.scale_log2 = static_cast<float>((1.0 / std::sqrt(double(D))) * 1.4426950408889634);
    p.wait_budget_ns = wait_budget_ns();
    p.status = device_status_word();
    if (!p.status) return WAN_ATTN_ERR_CUDA;
    if (per_tile) {
        p.nqb = (Sq + 63) / 64;
        p.nkb = (Skv + 63) / 64;
        p.nctas = (Sq + 127) / 128;
        return launch_fwd_tiles(tq, tk, tv, to, p, static_cast<cudaStream_t>(stream)) == 0 ? WAN_ATTN_OK
                                                                                           : WAN_ATTN_ERR_CUDA;
    }
    return launch_fwd(tq, tk, tv, to, p, static_cast<cudaStream_t>(stream)) == 0 ? WAN_ATTN_OK : WAN_ATTN_ERR_CUDA;
}

// Block-sparse forward: per 128-row Q tile (2 query blocks of 64) the list of attended key
// blocks, int32 [B, H, ntiles, nkb], then the lists' lengths [B, H, ntiles].
size_t sparse_ws_size(int B, int Sq, int Skv, int H, int D) {
    if (check_shape(B, Sq, H, D) != WAN_ATTN_OK || check_shape(B, Skv, H, D) != WAN_ATTN_OK) return 0;
    const size_t ntiles = (size_t(Sq) + 127) / 128, nkb = (size_t(Skv) + 63) / 64;
    return align256(size_t(B) * H * ntiles * nkb * 4) + align256(size_t(B) * H * ntiles * 4);
}

int fwd_block_sparse_impl(const void* q, const void* k, const void* v, void* o, float* lse, const uint8_t* mask,
                          int B, int Sq, int Skv, int H, int D, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (!q || !k || !v || !o || !lse || !mask) return WAN_ATTN_ERR_INVALID_ARG;
    int st = check_shape(B, Sq, H, D);
    if (st == WAN_ATTN_OK) st = check_shape(B, Skv, H, D);
    if (st != WAN_ATTN_OK) return st;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return WAN_ATTN_ERR_INVALID_ARG;
    const size_t need = sparse_ws_size(B, Sq, Skv, H, D);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return WAN_ATTN_ERR_WORKSPACE;
    const int nqb = (Sq + 63) / 64, nkb = (Skv + 63) / 64, ntiles = (Sq + 127) / 128;
    const size_t nq = size_t(B) * Sq * H * D, nkv = size_t(B) * Skv * H * D;
    const Range ins[] = {range_of(q, nq * 2), range_of(k, nkv * 2), range_of(v, nkv * 2),
                         range_of(mask, size_t(B) * H * nqb * nkb)};
    const Range outs[] = {range_of(o, nq * 2), range_of(lse, size_t(B) * H * Sq * 4), range_of(workspace, need)};
    for (size_t a = 0; a < 3; ++a) {
        for (const Range& in : ins)
            if (overlaps(outs[a], in)) return WAN_ATTN_ERR_INVALID_ARG;
        for (size_t c = a + 1; c < 3; ++c)
            if (overlaps(outs[a], outs[c])) return WAN_ATTN_ERR_INVALID_ARG;
    }
    CUtensorMap tq, tk, tv, to;
    if (!make_bshd_map(&tq, q, B, Sq, H, D, 128) || !make_bshd_map(&tk, k, B, Skv, H, D, 64) ||
        !make_bshd_map(&tv, v, B, Skv, H, D, 64) || !make_bshd_map(&to, o, B, Sq, H, D, 128))
        return WAN_ATTN_ERR_CUDA;
    FwdParams p{};
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.S = Sq;
    p.Skv = Skv;
    p.H = H;
    p.mask = mask;
    p.kv_list = static_cast<const int*>(workspace);
    p.kv_count = reinterpret_cast<const int*>(static_cast<char*>(workspace) +
                                              align256(size_t(B) * H * ntiles * nkb * 4));
    p.nqb = nqb;
    p.nkb = nkb;
    p.nctas = ntiles;
    p.scale_log2 = static_cast<float>((1.0 / std::sqrt(double(D))) * 1.4426950408889634);
    p.wait_budget_ns = wait_budget_ns();
    p.status = device_status_word();
    if (!p.status) return WAN_ATTN_ERR_CUDA;
    return launch_fwd_tiles(tq, tk, tv, to, p, static_cast<cudaStream_t>(stream)) == 0 ? WAN_ATTN_OK
                                                                                       : WAN_ATTN_ERR_CUDA;
}

// Backward workspace: fp32 dQ accumulator [B, Sq, H, D], fp32 D_i [B, H, Sq] and, for the
// cross-attention call, fp32 dK and dV accumulators [B, Skv, H, D]; each part 256-byte aligned.
size_t bwd_ws_size(int B, int Sq, int Skv, int H, int D, bool cross) {
    if (check_shape(B, Sq, H, D) != WAN_ATTN_OK || check_shape(B, Skv, H, D) != WAN_ATTN_OK) return 0;
    const size_t nq = size_t(B) * Sq * H * D, nkv = size_t(B) * Skv * H * D;
    size_t bytes = align256(nq * 4) + align256(size_t(B) * H * Sq * 4);
    if (cross) bytes += 2 * align256(nkv * 4);
    return bytes;
}

int bwd_impl(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
             void* dq, void* dk, void* dv, int B, int Sq, int Skv, int H, int D, void* workspace,
             size_t workspace_bytes, void* stream, bool cross) {
    if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return WAN_ATTN_ERR_INVALID_ARG;
    int st = check_shape(B, Sq, H, D);
    if (st == WAN_ATTN_OK) st = check_shape(B, Skv, H, D);
    if (st != WAN_ATTN_OK) return st;
    for (const void* ptr : {q, k, v, o, dO, static_cast<const void*>(lse), static_cast<const void*>(dq),
                            static_cast<const void*>(dk), static_cast<const void*>(dv)})
        if (!aligned16(ptr)) return WAN_ATTN_ERR_INVALID_ARG;
    const size_t need = bwd_ws_size(B, Sq, Skv, H, D, cross);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return WAN_ATTN_ERR_WORKSPACE;
    const size_t nq = size_t(B) * Sq * H * D, nkv = size_t(B) * Skv * H * D;
    const Range ins[] = {range_of(q, nq * 2), range_of(k, nkv * 2), range_of(v, nkv * 2), range_of(o, nq * 2),
                         range_of(dO, nq * 2), range_of(lse, size_t(B) * H * Sq * 4)};
    const Range outs[] = {range_of(dq, nq * 2), range_of(dk, nkv * 2), range_of(dv, nkv * 2),
                          range_of(workspace, need)};
    for (size_t a = 0; a < 4; ++a) {
        for (const Range& in : ins)
            if (overlaps(outs[a], in)) return WAN_ATTN_ERR_INVALID_ARG;
        for (size_t c = a + 1; c < 4; ++c)
            if (overlaps(outs[a], outs[c])) return WAN_ATTN_ERR_INVALID_ARG;
    }

    char* ws = static_cast<char*>(workspace);
    const size_t off_delta = align256(nq * 4);
    const size_t off_dk = off_delta + align256(size_t(B) * H * Sq * 4);
    const size_t off_dv = off_dk + align256(nkv * 4);
    BwdParams p;
    p.lse = lse;
    p.dq_acc = reinterpret_cast<float*>(ws);
    p.delta = reinterpret_cast<float*>(ws + off_delta);
    p.dk_acc = cross ? reinterpret_cast<float*>(ws + off_dk) : nullptr;
    p.dv_acc = cross ? reinterpret_cast<float*>(ws + off_dv) : nullptr;
    CUtensorMap tq, tk, tv, tdo, tdq, tdk, tdv;
    if (!make_bshd_map(&tq, q, B, Sq, H, D, 128) || !make_bshd_map(&tk, k, B, Skv, H, D, 128) ||
        !make_bshd_map(&tv, v, B, Skv, H, D, 128) || !make_bshd_map(&tdo, dO, B, Sq, H, D, 128) ||
        !make_dq_acc_map(&tdq, workspace, B, Sq, H))
        return WAN_ATTN_ERR_CUDA;
    if (cross) {
        if (!make_acc_sw_map(&tdk, p.dk_acc, B, Skv, H) || !make_acc_sw_map(&tdv, p.dv_acc, B, Skv, H))
            return WAN_ATTN_ERR_CUDA;
    } else {
        tdk = tdq;    // never read: self-attention keeps one CTA per key tile (nsplit = 1)
        tdv = tdq;
    }
    p.dk = dk;
    p.dv = dv;
    p.B = B;
    p.Sq = Sq;
    p.Skv = Skv;
    p.H = H;
    p.nsplit = 1;
    p.scale = static_cast<float>(1.0 / std::sqrt(double(D)));
    p.scale_log2 = static_cast<float>((1.0 / std::sqrt(double(D))) * 1.4426950408889634);
    p.wait_budget_ns = wait_budget_ns();
    p.status = device_status_word();
    if (!p.status) return WAN_ATTN_ERR_CUDA;
    return launch_bwd(tq, tk, tv, tdo, tdq, tdk, tdv, p, cross, o, dO, dq, static_cast<cudaStream_t>(stream)) == 0
               ? WAN_ATTN_OK
               : WAN_ATTN_ERR_CUDA;
}

// Tensor map over a bf16 [T, H, 128] tensor of token stride ld (elements) as 3-D (128, H, T), box
// (64 of D, `heads`, `tokens`) with the 128-byte swizzle: rows of the tile are token-major.
bool make_packed_map(CUtensorMap* m, const void* base, int T, int H, long long ld, int heads, int tokens) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {128, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {256, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over an fp32 accumulator [T, H, 128] as 3-D (128, H, T), box (`cols`, `heads`, 128 / `heads`); `swizzle`:
// the 128-byte swizzle (cols = 32).
bool make_packed_acc_map(CUtensorMap* m, void* base, int T, int H, int cols, int heads, bool swizzle) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {128, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {128 * 4, (cuuint64_t)H * 128 * 4};
    const cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)heads, (cuuint32_t)(128 / heads)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shape, stride, alignment and overlap checks of the packed attention calls.  A tensor without
// rows may have a null pointer.
struct Packed {
    const void* ptr;
    long long rows, ld;
    int heads;
    bool out;
    Range range() const {
        return rows > 0 ? range_of(ptr, (size_t(rows - 1) * ld + size_t(heads) * 128) * 2) : Range{0, 0};
    }
};

// Two tensors may interleave (slices of one fused [T, (H + 2 Hkv) D] buffer: the same token stride,
// heads beside each other); otherwise their ranges must be apart.
bool packed_clash(const Packed& a, const Packed& b) {
    if (!overlaps(a.range(), b.range())) return false;
    if (a.ld != b.ld) return true;
    const long long ld = a.ld * 2, da = static_cast<long long>(a.heads) * 256, db = static_cast<long long>(b.heads) * 256;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
    const long long gap = pa <= pb ? static_cast<long long>((pb - pa) % ld)              // a's row, then b's ...
                                   : (ld - static_cast<long long>((pa - pb) % ld)) % ld;
    return gap < da || gap + db > ld;                                                    // ... then a's next row
}

int check_packed(int N, int Tq, int Tk, int H, int Hkv, int D) {
    if (N < 1 || Tq < 0 || Tk < 0 || H < 1 || Hkv < 1 || D < 1 || H % Hkv) return WAN_ATTN_ERR_INVALID_ARG;
    if (D != 128) return WAN_ATTN_ERR_UNSUPPORTED;
    // token coordinates and grids stay in 32 bits
    if (H > 65535 || Tq > 0x7fff0000 || Tk > 0x7fff0000 || N > (1 << 24) || double(N) * H >= double(1 << 30))
        return WAN_ATTN_ERR_INVALID_ARG;
    const double lim = double(1ull << 40);
    if (double(Tq) * H * D >= lim || double(Tk) * Hkv * D >= lim) return WAN_ATTN_ERR_INVALID_ARG;
    return WAN_ATTN_OK;
}

int check_packed_tensors(const Packed* t, int n, const Range* plain_in, int n_in, const Range* plain_out, int n_out) {
    for (int i = 0; i < n; ++i) {
        if (t[i].rows == 0) continue;
        if (!t[i].ptr || !aligned16(t[i].ptr)) return WAN_ATTN_ERR_INVALID_ARG;
        if (t[i].ld < static_cast<long long>(t[i].heads) * 128 || (t[i].ld & 7)) return WAN_ATTN_ERR_INVALID_ARG;
        if (double(t[i].ld) * t[i].rows >= double(1ull << 40)) return WAN_ATTN_ERR_INVALID_ARG;
    }
    for (int i = 0; i < n; ++i) {
        if (!t[i].rows) continue;
        for (int j = 0; j < n; ++j)
            if (j != i && t[j].rows && (t[i].out || t[j].out) && packed_clash(t[i], t[j])) return WAN_ATTN_ERR_INVALID_ARG;
        for (int j = 0; j < n_out; ++j)
            if (overlaps(t[i].range(), plain_out[j])) return WAN_ATTN_ERR_INVALID_ARG;
        for (int j = 0; t[i].out && j < n_in; ++j)
            if (overlaps(t[i].range(), plain_in[j])) return WAN_ATTN_ERR_INVALID_ARG;
    }
    for (int a = 0; a < n_out; ++a) {
        for (int j = 0; j < n_in; ++j)
            if (overlaps(plain_out[a], plain_in[j])) return WAN_ATTN_ERR_INVALID_ARG;
        for (int c = a + 1; c < n_out; ++c)
            if (overlaps(plain_out[a], plain_out[c])) return WAN_ATTN_ERR_INVALID_ARG;
    }
    return WAN_ATTN_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Fields that the packed forward and backward share.  False if there is no status word.
bool fill_packed(VarlenParams& p, const void* q, const void* k, const void* v, const int* cu_q, const int* cu_k, int N,
                 int Tq, int Tk, int H, int Hkv, long long ldq, long long ldk, long long ldv, int causal) {
    p.q = q;
    p.k = k;
    p.v = v;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.N = N;
    p.Tq = Tq;
    p.Tk = Tk;
    p.H = H;
    p.Hkv = Hkv;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.causal = causal ? 1 : 0;
    p.scale = static_cast<float>(1.0 / std::sqrt(128.0));
    p.scale_log2 = static_cast<float>((1.0 / std::sqrt(128.0)) * 1.4426950408889634);
    p.wait_budget_ns = wait_budget_ns();
    p.status = device_status_word();
    return p.status != nullptr;
}

// Shapes of the int8 linear calls: M >= 0 rows, K % 16 == 0, 16 <= K <= 131072, N % 8 == 0 (>= 8); M and N leave
// room for rounding up to a tile in 32 bits.
int check_int8_shape(int M, int N, int K) {
    if (M > 0x7fff0000 || N > 0x7fff0000 || M < 0 || K < 16 || (K & 15) || K > 131072 || N < 8 || (N & 7)) return WAN_ATTN_ERR_INVALID_ARG;
    const double lim = double(1ull << 40);
    if (double(M) * K >= lim || double(N) * K >= lim || double(M) * N >= lim) return WAN_ATTN_ERR_INVALID_ARG;
    return WAN_ATTN_OK;
}

// No null pointer, alignment `mask` + 1 each, and no output range over any other range.
struct Arg {
    const void* ptr;
    size_t bytes;
    unsigned mask;
    bool out;
};
int check_args(const Arg* a, int n) {
    for (int i = 0; i < n; ++i)
        if (!a[i].ptr || (reinterpret_cast<uintptr_t>(a[i].ptr) & a[i].mask)) return WAN_ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && a[i].out && overlaps(range_of(a[i].ptr, a[i].bytes), range_of(a[j].ptr, a[j].bytes)))
                return WAN_ATTN_ERR_INVALID_ARG;
    return WAN_ATTN_OK;
}

Int8GemmParams int8_params(const float* a_scales, const float* b_scales, const void* bias, void* y, int M, int N, int K) {
    Int8GemmParams p;
    p.a_scales = a_scales;
    p.b_scales = b_scales;
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.y = static_cast<__nv_bfloat16*>(y);
    p.M = M;
    p.N = N;
    p.K = K;
    p.after_quant = 0;
    p.wait_budget_ns = wait_budget_ns();
    p.status = device_status_word();
    return p;
}

// The int8 product on validated arguments.
int int8_product(const void* a_codes, const float* a_scales, const void* b_codes, const float* b_scales,
                 const void* bias, void* y, int M, int N, int K, bool after_quant, cudaStream_t stream) {
    Int8GemmParams p = int8_params(a_scales, b_scales, bias, y, M, N, K);
    p.after_quant = after_quant ? 1 : 0;
    if (!p.status) return WAN_ATTN_ERR_CUDA;
    const int tokens = int8_gemm_token_tile(M, N);
    CUtensorMap tx, tw;
    if (!make_rows_u8_map(&tx, a_codes, M, K, tokens ? tokens : 128) || !make_rows_u8_map(&tw, b_codes, N, K, 128))
        return WAN_ATTN_ERR_CUDA;
    return launch_int8_gemm(tx, tw, p, stream) == 0 ? WAN_ATTN_OK : WAN_ATTN_ERR_CUDA;
}

// The products of the int8 layer's backward on validated arguments (dy bf16 [M, N]; codes [terms, K]).
int int8_grad_product(const void* dy, const void* codes, const float* scales, void* out, int M, int N, int K, bool weight,
                      cudaStream_t stream) {
    auto enc = tensor_map_encoder();
    int* status = device_status_word();
    if (!enc || !status) return WAN_ATTN_ERR_CUDA;
    const int terms = weight ? M : N;
    CUtensorMap tdy, tcodes;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M}, strides[1] = {(cuuint64_t)N * 2};
    const cuuint32_t box[2] = {64, weight ? 64u : 128u}, estr[2] = {1, 1};
    const cuuint64_t cdims[2] = {(cuuint64_t)K, (cuuint64_t)terms}, cstrides[1] = {(cuuint64_t)K};
    const cuuint32_t cbox[2] = {128, 64};
    if (enc(&tdy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(dy), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        enc(&tcodes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), cdims, cstrides, cbox, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return WAN_ATTN_ERR_CUDA;
    return launch_int8_grad(tdy, tcodes, scales, out, weight ? N : M, K, terms, weight, wait_budget_ns(), status, stream) == 0
               ? WAN_ATTN_OK
               : WAN_ATTN_ERR_CUDA;
}

int as_status(int rc) { return rc == 0 ? WAN_ATTN_OK : WAN_ATTN_ERR_CUDA; }

}  // namespace

extern "C" {

int wan_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int S, int H, int D,
                 void* stream) {
    return fwd_impl(q, k, v, o, lse, B, S, S, H, D, stream, false);
}

int wan_attn_cross_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Sq, int Skv,
                       int H, int D, void* stream) {
    return fwd_impl(q, k, v, o, lse, B, Sq, Skv, H, D, stream, true);
}

size_t wan_attn_bwd_workspace_size(int B, int S, int H, int D) { return bwd_ws_size(B, S, S, H, D, false); }

size_t wan_attn_fwd_block_sparse_workspace_size(int B, int Sq, int Skv, int H, int D) {
    return sparse_ws_size(B, Sq, Skv, H, D);
}

int wan_attn_fwd_block_sparse(const void* q, const void* k, const void* v, void* o, float* lse,
                              const uint8_t* block_mask, int B, int Sq, int Skv, int H, int D, void* workspace,
                              size_t workspace_bytes, void* stream) {
    return fwd_block_sparse_impl(q, k, v, o, lse, block_mask, B, Sq, Skv, H, D, workspace, workspace_bytes, stream);
}

int wan_attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                 void* dq, void* dk, void* dv, int B, int S, int H, int D, void* workspace,
                 size_t workspace_bytes, void* stream) {
    return bwd_impl(q, k, v, o, dO, lse, dq, dk, dv, B, S, S, H, D, workspace, workspace_bytes, stream, false);
}

size_t wan_attn_cross_bwd_workspace_size(int B, int Sq, int Skv, int H, int D) {
    return bwd_ws_size(B, Sq, Skv, H, D, true);
}

int wan_attn_cross_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
                       const float* lse, void* dq, void* dk, void* dv, int B, int Sq, int Skv, int H, int D,
                       void* workspace, size_t workspace_bytes, void* stream) {
    return bwd_impl(q, k, v, o, dO, lse, dq, dk, dv, B, Sq, Skv, H, D, workspace, workspace_bytes, stream, true);
}

size_t wan_attn_fwd_q8_workspace_size(int B, int S, int H, int D) {
    if (check_shape(B, S, H, D) != WAN_ATTN_OK) return 0;
    const size_t n = size_t(B) * S * H * D;
    const size_t nblk = (size_t(S) + 63) / 64;
    return 3 * align256(n) + 3 * align256(size_t(B) * H * nblk * 4);
}

int wan_attn_fwd_q8(const void* q, const void* k, const void* v, void* o, float* lse, int B, int S, int H, int D,
                    void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !k || !v || !o || !lse) return WAN_ATTN_ERR_INVALID_ARG;
    const int st = check_shape(B, S, H, D);
    if (st != WAN_ATTN_OK) return st;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return WAN_ATTN_ERR_INVALID_ARG;
    const size_t need = wan_attn_fwd_q8_workspace_size(B, S, H, D);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return WAN_ATTN_ERR_WORKSPACE;
    const size_t n = size_t(B) * S * H * D;
    const Range ins[] = {range_of(q, n * 2), range_of(k, n * 2), range_of(v, n * 2)};
    const Range outs[] = {range_of(o, n * 2), range_of(lse, size_t(B) * H * S * 4), range_of(workspace, need)};
    for (size_t a = 0; a < 3; ++a) {
        for (const Range& in : ins)
            if (overlaps(outs[a], in)) return WAN_ATTN_ERR_INVALID_ARG;
        for (size_t c = a + 1; c < 3; ++c)
            if (overlaps(outs[a], outs[c])) return WAN_ATTN_ERR_INVALID_ARG;
    }
    const int nblk = (S + 63) / 64;
    char* ws = static_cast<char*>(workspace);
    const size_t code_bytes = align256(n), scale_bytes = align256(size_t(B) * H * nblk * 4);
    Q8QuantParams qp;
    qp.q = static_cast<const __nv_bfloat16*>(q);
    qp.k = static_cast<const __nv_bfloat16*>(k);
    qp.v = static_cast<const __nv_bfloat16*>(v);
    qp.q8 = reinterpret_cast<int8_t*>(ws);
    qp.k8 = reinterpret_cast<int8_t*>(ws + code_bytes);
    qp.v8 = reinterpret_cast<uint8_t*>(ws + 2 * code_bytes);
    qp.sq = reinterpret_cast<float*>(ws + 3 * code_bytes);
    qp.sk = reinterpret_cast<float*>(ws + 3 * code_bytes + scale_bytes);
    qp.sv = reinterpret_cast<float*>(ws + 3 * code_bytes + 2 * scale_bytes);
    qp.B = B;
    qp.S = S;
    qp.H = H;
    qp.nblk = nblk;
    CUtensorMap tq, tk, tv, to;
    if (!make_bh_s_d8_map(&tq, qp.q8, B * H, S, 128) || !make_bh_s_d8_map(&tk, qp.k8, B * H, S, 64) ||
        !make_bh_s_d8_map(&tv, qp.v8, B * H, S, 64) || !make_bshd_map(&to, o, B, S, H, D, 128))
        return WAN_ATTN_ERR_CUDA;
    Q8AttnParams p;
    p.o = o;
    p.lse = lse;
    p.sq = qp.sq;
    p.sk = qp.sk;
    p.sv = qp.sv;
    p.B = B;
    p.S = S;
    p.H = H;
    p.nblk = nblk;
    p.scale_log2 = static_cast<float>((1.0 / std::sqrt(double(D))) * 1.4426950408889634);
    p.wait_budget_ns = wait_budget_ns();
    p.status = device_status_word();
    if (!p.status) return WAN_ATTN_ERR_CUDA;
    return launch_q8(qp, tq, tk, tv, to, p, static_cast<cudaStream_t>(stream)) == 0 ? WAN_ATTN_OK
                                                                                    : WAN_ATTN_ERR_CUDA;
}

int wan_attn_cp_merge(float* o_acc, float* lse_acc, const void* o_part, const float* lse_part, void* o_out, int B,
                      int S, int H, int D, int first, void* stream) {
    if (!o_acc || !lse_acc || !o_part || !lse_part) return WAN_ATTN_ERR_INVALID_ARG;
    const int st = check_shape(B, S, H, D);
    if (st != WAN_ATTN_OK) return st;
    for (const void* ptr : {static_cast<const void*>(o_acc), static_cast<const void*>(lse_acc), o_part,
                            static_cast<const void*>(lse_part), static_cast<const void*>(o_out)})
        if (ptr && !aligned16(ptr)) return WAN_ATTN_ERR_INVALID_ARG;
    const size_t n = size_t(B) * S * H * D, nl = size_t(B) * H * S;
    const Range ra = range_of(o_acc, n * 4), rl = range_of(lse_acc, nl * 4);
    const Range ins[] = {range_of(o_part, n * 2), range_of(lse_part, nl * 4)};
    for (const Range& in : ins)
        if (overlaps(ra, in) || overlaps(rl, in)) return WAN_ATTN_ERR_INVALID_ARG;
    if (overlaps(ra, rl)) return WAN_ATTN_ERR_INVALID_ARG;
    if (o_out) {
        const Range ro = range_of(o_out, n * 2);
        if (overlaps(ro, ra) || overlaps(ro, rl) || overlaps(ro, ins[0]) || overlaps(ro, ins[1]))
            return WAN_ATTN_ERR_INVALID_ARG;
    }
    return launch_cp_merge(o_acc, lse_acc, o_part, lse_part, o_out, B, S, H, first ? 1 : 0,
                           static_cast<cudaStream_t>(stream)) == 0
               ? WAN_ATTN_OK
               : WAN_ATTN_ERR_CUDA;
}

int wan_attn_cp_accumulate(float* acc, const void* part, void* out, size_t n, int first, void* stream) {
    if (!acc || !part || n == 0 || (n & 7u)) return WAN_ATTN_ERR_INVALID_ARG;
    if (!aligned16(acc) || !aligned16(part) || (out && !aligned16(out))) return WAN_ATTN_ERR_INVALID_ARG;
    const Range ra = range_of(acc, n * 4), rp = range_of(part, n * 2);
    if (overlaps(ra, rp)) return WAN_ATTN_ERR_INVALID_ARG;
    if (out) {
        const Range ro = range_of(out, n * 2);
        if (overlaps(ro, ra) || overlaps(ro, rp)) return WAN_ATTN_ERR_INVALID_ARG;
    }
    return launch_cp_accumulate(acc, part, out, static_cast<long long>(n / 8), first ? 1 : 0,
                                static_cast<cudaStream_t>(stream)) == 0
               ? WAN_ATTN_OK
               : WAN_ATTN_ERR_CUDA;
}

int wan_attn_cp_layout(void* dst, const void* src, int B, int S_loc, int G, int Hg, int D, int which,
                       void* stream) {
    if (!dst || !src || G < 1 || Hg < 1 || which < WAN_ATTN_CP_SEQ_TO_SEND || which > WAN_ATTN_CP_RECV_TO_SEQ)
        return WAN_ATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(G) * Hg > 65535) return WAN_ATTN_ERR_INVALID_ARG;
    const int st = check_shape(B, S_loc, G * Hg, D);
    if (st != WAN_ATTN_OK) return st;
    if (double(B) * S_loc * G * Hg * D >= double(1ull << 40) / G) return WAN_ATTN_ERR_INVALID_ARG;
    if (!aligned16(dst) || !aligned16(src)) return WAN_ATTN_ERR_INVALID_ARG;
    const size_t bytes = size_t(B) * S_loc * G * Hg * D * 2;
    if (overlaps(range_of(dst, bytes), range_of(src, bytes))) return WAN_ATTN_ERR_INVALID_ARG;
    return launch_cp_layout(dst, src, B, S_loc, G, Hg * D * 2 / 16, which, static_cast<cudaStream_t>(stream)) == 0
               ? WAN_ATTN_OK
               : WAN_ATTN_ERR_CUDA;
}

int wan_fp8_quantize_rows(const void* x, void* codes, float* scales, int M, int K, void* stream) {
    if (!x || !codes || !scales) return WAN_ATTN_ERR_INVALID_ARG;
    const int st = check_fp8_shape(M, K);
    if (st != WAN_ATTN_OK) return st;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return WAN_ATTN_ERR_INVALID_ARG;
    const size_t n = size_t(M) * K;
    const Range rx = range_of(x, n * 2), rc = range_of(codes, n), rs = range_of(scales, size_t(M) * 4);
    if (overlaps(rx, rc) || overlaps(rx, rs) || overlaps(rc, rs)) return WAN_ATTN_ERR_INVALID_ARG;
    return launch_fp8_quant_rows(x, codes, scales, M, K, static_cast<cudaStream_t>(stream)) == 0 ? WAN_ATTN_OK
                                                                                               : WAN_ATTN_ERR_CUDA;
}

int wan_fp8_quantize_tensor(const void* w, void* codes, float* scale2, int N, int K, void* stream) {
    if (!w || !codes || !scale2) return WAN_ATTN_ERR_INVALID_ARG;
    const int st = check_fp8_shape(N, K);
    if (st != WAN_ATTN_OK) return st;
    if (!aligned16(w) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scale2) & 7u))
        return WAN_ATTN_ERR_INVALID_ARG;
    const size_t n = size_t(N) * K;
    const Range rw = range_of(w, n * 2), rc = range_of(codes, n), rs = range_of(scale2, 8);
    if (overlaps(rw, rc) || overlaps(rw, rs) || overlaps(rc, rs)) return WAN_ATTN_ERR_INVALID_ARG;
    return launch_fp8_quant_tensor(w, codes, scale2, static_cast<long long>(n), static_cast<cudaStream_t>(stream)) == 0
               ? WAN_ATTN_OK
               : WAN_ATTN_ERR_CUDA;
}

int wan_fp8_gemm(const void* a_codes, const float* a_scales, const void* b_codes, const float* b_scale, void* y,
                 int M, int N, int K, void* stream) {
    if (!a_codes || !a_scales || !b_codes || !b_scale || !y) return WAN_ATTN_ERR_INVALID_ARG;
    int st = check_fp8_shape(M, K);
    if (st == WAN_ATTN_OK) st = check_fp8_shape(N, K);
    if (st != WAN_ATTN_OK) return st;
    if ((N & 7) || double(M) * N >= double(1ull << 40)) return WAN_ATTN_ERR_INVALID_ARG;
    if (!aligned16(a_codes) || !aligned16(b_codes) || !aligned16(y) || (reinterpret_cast<uintptr_t>(a_scales) & 3u) ||
        (reinterpret_cast<uintptr_t>(b_scale) & 3u))
        return WAN_ATTN_ERR_INVALID_ARG;
    const Range ry = range_of(y, size_t(M) * N * 2);
    const Range ins[] = {range_of(a_codes, size_t(M) * K), range_of(a_scales, size_t(M) * 4),
                         range_of(b_codes, size_t(N) * K), range_of(b_scale, 4)};
    for (const Range& in : ins)
        if (overlaps(ry, in)) return WAN_ATTN_ERR_INVALID_ARG;
    CUtensorMap ta, tb, tb_half;
    if (!make_rows_u8_map(&ta, a_codes, M, K, 128) || !make_rows_u8_map(&tb, b_codes, N, K, 256) ||
        !make_rows_u8_map(&tb_half, b_codes, N, K, 128))
        return WAN_ATTN_ERR_CUDA;
    Fp8GemmParams p;
    p.a_scales = a_scales;
    p.b_scale = b_scale;
    p.y = y;
    p.M = M;
    p.N = N;
    p.K = K;
    p.wait_budget_ns = wait_budget_ns();
    p.status = device_status_word();
    if (!p.status) return WAN_ATTN_ERR_CUDA;
    return launch_fp8_gemm(ta, tb, tb_half, p, static_cast<cudaStream_t>(stream)) == 0 ? WAN_ATTN_OK
                                                                                     : WAN_ATTN_ERR_CUDA;
}

size_t wan_attn_varlen_fwd_workspace_size(int N, int Tq, int Tk, int H, int Hkv, int D) {
    if (check_packed(N, Tq, Tk, H, Hkv, D) != WAN_ATTN_OK) return 0;
    const VarlenFwdPlan plan = varlen_fwd_plan(N, Tq, Tk, H, Hkv);
    if (plan.chunk == 0) return 0;
    const size_t rows = size_t(plan.parts) * Tq * H;
    return align256(rows * 128 * 4) + align256(rows * 4) + align256(size_t(Tq) * 4);
}

int wan_attn_varlen_fwd(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_q,
                        const int* cu_k, int N, int Tq, int Tk, int H, int Hkv, int D, int64_t ldq, int64_t ldk,
                        int64_t ldv, int causal, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_packed(N, Tq, Tk, H, Hkv, D);
    if (st != WAN_ATTN_OK) return st;
    if (!cu_q || !cu_k || !aligned4(cu_q) || !aligned4(cu_k)) return WAN_ATTN_ERR_INVALID_ARG;
    if (Tq == 0) return WAN_ATTN_OK;
    if (!lse || !aligned16(lse)) return WAN_ATTN_ERR_INVALID_ARG;
    const Packed t[] = {{q, Tq, ldq, H, false}, {k, Tk, ldk, Hkv, false}, {v, Tk, ldv, Hkv, false},
                        {o, Tq, static_cast<long long>(H) * 128, H, true}};
    const Range ins[] = {range_of(cu_q, size_t(N + 1) * 4), range_of(cu_k, size_t(N + 1) * 4)};
    const size_t need = wan_attn_varlen_fwd_workspace_size(N, Tq, Tk, H, Hkv, D);
    if (need && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return WAN_ATTN_ERR_WORKSPACE;
    const Range outs[] = {range_of(lse, size_t(H) * Tq * 4), range_of(workspace, need)};
    st = check_packed_tensors(t, 4, ins, 2, outs, need ? 2 : 1);
    if (st != WAN_ATTN_OK) return st;
    VarlenFwdParams p{};
    if (!fill_packed(p, q, k, v, cu_q, cu_k, N, Tq, Tk, H, Hkv, ldq, ldk, ldv, causal)) return WAN_ATTN_ERR_CUDA;
    p.o = o;
    p.lse = lse;
    const VarlenFwdPlan plan = varlen_fwd_plan(N, Tq, Tk, H, Hkv);
    p.pack = plan.pack;
    p.chunk = plan.chunk;
    p.streamed = plan.streamed;
    p.order = plan.order;
    p.most_parts = plan.parts;
    if (need) {
        const size_t rows = size_t(plan.parts) * Tq * H;
        char* ws = static_cast<char*>(workspace);
        p.o_part = reinterpret_cast<float*>(ws);
        p.lse_part = reinterpret_cast<float*>(ws + align256(rows * 128 * 4));
        p.parts = reinterpret_cast<int*>(ws + align256(rows * 128 * 4) + align256(rows * 4));
    }
    CUtensorMap tq, tk, tv, to;
    if (!make_packed_map(&tq, q, Tq, H, ldq, p.pack, 128 / p.pack) ||
        !make_packed_map(&to, o, Tq, H, static_cast<long long>(H) * 128, p.pack, 128 / p.pack))
        return WAN_ATTN_ERR_CUDA;
    if (Tk > 0) {
        if (!make_packed_map(&tk, k, Tk, Hkv, ldk, 1, 128) || !make_packed_map(&tv, v, Tk, Hkv, ldv, 1, 128))
            return WAN_ATTN_ERR_CUDA;
    } else {
        tk = tv = tq;                     // never read: without keys no tile has a key block
    }
    return as_status(launch_varlen_fwd(tq, tk, tv, to, p, plan.units, static_cast<cudaStream_t>(stream)));
}

size_t wan_attn_varlen_bwd_workspace_size(int N, int Tq, int Tk, int H, int Hkv, int D) {
    if (check_packed(N, Tq, Tk, H, Hkv, D) != WAN_ATTN_OK) return 0;
    size_t bytes = align256(size_t(Tq) * H * 128 * 4) + align256(size_t(Tq) * H * 4) +
                   align256(size_t(varlen_bwd_tile_bound(N, Tk)) * 8) + align256(size_t(N) * 4);
    if (varlen_bwd_splits(N, Tq, Tk, H, Hkv) > 1) bytes += 2 * align256(size_t(Tk) * Hkv * 128 * 4);
    return bytes;
}

int wan_attn_varlen_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                        void* dq, void* dk, void* dv, const int* cu_q, const int* cu_k, int N, int Tq, int Tk, int H,
                        int Hkv, int D, int64_t ldq, int64_t ldk, int64_t ldv, int64_t lddq, int64_t lddk,
                        int64_t lddv, int causal, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_packed(N, Tq, Tk, H, Hkv, D);
    if (st != WAN_ATTN_OK) return st;
    if (!cu_q || !cu_k || !aligned4(cu_q) || !aligned4(cu_k)) return WAN_ATTN_ERR_INVALID_ARG;
    if (Tq == 0 && Tk == 0) return WAN_ATTN_OK;
    if (Tq > 0 && (!lse || !aligned16(lse))) return WAN_ATTN_ERR_INVALID_ARG;
    const size_t need = wan_attn_varlen_bwd_workspace_size(N, Tq, Tk, H, Hkv, D);
    if (need && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return WAN_ATTN_ERR_WORKSPACE;
    const long long hd = static_cast<long long>(H) * 128;
    const Packed t[] = {{q, Tq, ldq, H, false},  {k, Tk, ldk, Hkv, false},  {v, Tk, ldv, Hkv, false},
                        {o, Tq, hd, H, false},   {dO, Tq, hd, H, false},    {dq, Tq, lddq, H, true},
                        {dk, Tk, lddk, Hkv, true}, {dv, Tk, lddv, Hkv, true}};
    const Range ins[] = {range_of(cu_q, size_t(N + 1) * 4), range_of(cu_k, size_t(N + 1) * 4),
                         range_of(lse, size_t(H) * Tq * 4)};
    const Range outs[] = {range_of(workspace, need)};
    st = check_packed_tensors(t, 8, ins, 3, outs, 1);
    if (st != WAN_ATTN_OK) return st;
    VarlenBwdParams p{};
    if (!fill_packed(p, q, k, v, cu_q, cu_k, N, Tq, Tk, H, Hkv, ldq, ldk, ldv, causal)) return WAN_ATTN_ERR_CUDA;
    p.o = o;
    p.dout = dO;
    p.lse = lse;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.lddq = lddq;
    p.lddk = lddk;
    p.lddv = lddv;
    p.splits = varlen_bwd_splits(N, Tq, Tk, H, Hkv);
    char* ws = static_cast<char*>(workspace);
    p.tile_bound = varlen_bwd_tile_bound(N, Tk);
    if (Tk > 0) p.heads = head_order(p.tile_bound, Hkv, 1024.0 * Tq * H);       // Q, dO and the fp32 dQ
    const int pack = varlen_bwd_pack(H, Hkv);
    while ((1 << p.pack_log2) < pack) ++p.pack_log2;
    const size_t off_delta = align256(size_t(Tq) * H * 128 * 4), off_order = off_delta + align256(size_t(Tq) * H * 4);
    const size_t off_end = off_order + align256(size_t(p.tile_bound) * 8), off_dk = off_end + align256(size_t(N) * 4);
    p.dq_acc = reinterpret_cast<float*>(ws);
    p.delta = reinterpret_cast<float*>(ws + off_delta);
    p.order = reinterpret_cast<int2*>(ws + off_order);
    p.tile_end = reinterpret_cast<int*>(ws + off_end);
    if (p.splits > 1) {
        p.dk_acc = reinterpret_cast<float*>(ws + off_dk);
        p.dv_acc = reinterpret_cast<float*>(ws + off_dk + align256(size_t(Tk) * Hkv * 128 * 4));
    }
    CUtensorMap tq{}, tk{}, tv{}, tdo{}, tdq{}, tdk{}, tdv{};        // those of an empty axis are never read
    if (Tq > 0 && (!make_packed_map(&tq, q, Tq, H, ldq, pack, 128 / pack) ||
                   !make_packed_map(&tdo, dO, Tq, H, hd, pack, 128 / pack) ||
                   !make_packed_acc_map(&tdq, p.dq_acc, Tq, H, 128, pack, false)))
        return WAN_ATTN_ERR_CUDA;
    if (Tk > 0 && (!make_packed_map(&tk, k, Tk, Hkv, ldk, 1, 128) || !make_packed_map(&tv, v, Tk, Hkv, ldv, 1, 128)))
        return WAN_ATTN_ERR_CUDA;
    if (p.splits > 1 && (!make_packed_acc_map(&tdk, p.dk_acc, Tk, Hkv, 32, 1, true) ||
                         !make_packed_acc_map(&tdv, p.dv_acc, Tk, Hkv, 32, 1, true)))
        return WAN_ATTN_ERR_CUDA;
    return as_status(launch_varlen_bwd(tq, tk, tv, tdo, tdq, tdk, tdv, p, static_cast<cudaStream_t>(stream)));
}

int wan_int8_quantize_rows(const void* x, void* codes, float* scales, int M, int K, int64_t ldx, void* stream) {
    const int st = check_int8_shape(M, 8, K);
    if (st != WAN_ATTN_OK || ldx < K || (ldx & 7) || double(ldx) * M >= double(1ull << 40)) return WAN_ATTN_ERR_INVALID_ARG;
    if (M == 0) return WAN_ATTN_OK;
    const Arg a[] = {{x, (size_t(M - 1) * ldx + K) * 2, 15, false}, {codes, size_t(M) * K, 15, true},
                     {scales, size_t(M) * 4, 3, true}};
    const int sa = check_args(a, 3);
    if (sa != WAN_ATTN_OK) return sa;
    return as_status(launch_int8_quant_rows(x, codes, scales, M, K, ldx, static_cast<cudaStream_t>(stream)));
}

int wan_int8_dequantize_rows(const void* codes, const float* scales, void* x, int M, int K, void* stream) {
    const int st = check_int8_shape(M, 8, K);
    if (st != WAN_ATTN_OK) return st;
    if (M == 0) return WAN_ATTN_OK;
    const Arg a[] = {{codes, size_t(M) * K, 15, false}, {scales, size_t(M) * 4, 3, false}, {x, size_t(M) * K * 2, 15, true}};
    const int sa = check_args(a, 3);
    if (sa != WAN_ATTN_OK) return sa;
    return as_status(launch_int8_dequant_rows(codes, scales, x, M, K, static_cast<cudaStream_t>(stream)));
}

int wan_int8_gemm(const void* a_codes, const float* a_scales, const void* b_codes, const float* b_scales,
                  const void* bias, void* y, int M, int N, int K, void* stream) {
    const int st = check_int8_shape(M, N, K);
    if (st != WAN_ATTN_OK) return st;
    if (M == 0) return WAN_ATTN_OK;
    const Arg a[] = {{a_codes, size_t(M) * K, 15, false}, {a_scales, size_t(M) * 4, 3, false},
                     {b_codes, size_t(N) * K, 15, false}, {b_scales, size_t(N) * 4, 3, false},
                     {y, size_t(M) * N * 2, 15, true},    {bias, size_t(N) * 2, 15, false}};
    const int sa = check_args(a, bias ? 6 : 5);
    if (sa != WAN_ATTN_OK) return sa;
    return int8_product(a_codes, a_scales, b_codes, b_scales, bias, y, M, N, K, false, static_cast<cudaStream_t>(stream));
}

int wan_int8_linear(const void* x, const void* w_codes, const float* w_scales, const void* bias, void* y, void* codes,
                    float* scales, int M, int N, int K, int64_t ldx, void* stream) {
    const int st = check_int8_shape(M, N, K);
    if (st != WAN_ATTN_OK || ldx < K || (ldx & 7) || double(ldx) * M >= double(1ull << 40)) return WAN_ATTN_ERR_INVALID_ARG;
    if (M == 0) return WAN_ATTN_OK;
    const Arg a[] = {{x, (size_t(M - 1) * ldx + K) * 2, 15, false}, {w_codes, size_t(N) * K, 15, false},
                     {w_scales, size_t(N) * 4, 3, false},           {y, size_t(M) * N * 2, 15, true},
                     {codes, size_t(M) * K, 15, true},              {scales, size_t(M) * 4, 3, true},
                     {bias, size_t(N) * 2, 15, false}};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int8_layer_fits(M, N, K)) {
        // one launch; codes and scales are outputs only if they are given
        Arg b[7] = {a[0], a[1], a[2], a[3]};
        int n = 4;
        if (codes) b[n++] = a[4];
        if (scales) b[n++] = a[5];
        if (bias) b[n++] = a[6];
        const int sa = check_args(b, n);
        if (sa != WAN_ATTN_OK) return sa;
        const Int8GemmParams p = int8_params(nullptr, w_scales, bias, y, M, N, K);
        CUtensorMap tw;
        if (!p.status || !make_rows_u8_map(&tw, w_codes, N, K, 128)) return WAN_ATTN_ERR_CUDA;
        return launch_int8_layer(tw, x, ldx, codes, scales, p, s) == 0 ? WAN_ATTN_OK : WAN_ATTN_ERR_CUDA;
    }
    if (!codes && !scales) return WAN_ATTN_ERR_WORKSPACE;
    const int sa = check_args(a, bias ? 7 : 6);
    if (sa != WAN_ATTN_OK) return sa;
    if (launch_int8_quant_rows(x, codes, scales, M, K, ldx, s) != 0) return WAN_ATTN_ERR_CUDA;
    return int8_product(codes, scales, w_codes, w_scales, bias, y, M, N, K, true, s);
}

int wan_int8_grad_weight(const void* dy, const void* codes, const float* scales, void* dw, int M, int N, int K,
                         void* stream) {
    const int st = check_int8_shape(M, N, K);
    if (st != WAN_ATTN_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (!dw || !aligned16(dw)) return WAN_ATTN_ERR_INVALID_ARG;
        return cudaMemsetAsync(dw, 0, size_t(N) * K * 2, s) == cudaSuccess ? WAN_ATTN_OK : WAN_ATTN_ERR_CUDA;
    }
    const Arg a[] = {{dy, size_t(M) * N * 2, 15, false}, {codes, size_t(M) * K, 15, false},
                     {scales, size_t(M) * 4, 3, false}, {dw, size_t(N) * K * 2, 15, true}};
    const int sa = check_args(a, 4);
    if (sa != WAN_ATTN_OK) return sa;
    return int8_grad_product(dy, codes, scales, dw, M, N, K, true, s);
}

int wan_int8_grad_input(const void* dy, const void* w_codes, const float* w_scales, void* dx, int M, int N, int K,
                        void* stream) {
    const int st = check_int8_shape(M, N, K);
    if (st != WAN_ATTN_OK) return st;
    if (M == 0) return WAN_ATTN_OK;
    const Arg a[] = {{dy, size_t(M) * N * 2, 15, false}, {w_codes, size_t(N) * K, 15, false},
                     {w_scales, size_t(N) * 4, 3, false}, {dx, size_t(M) * K * 2, 15, true}};
    const int sa = check_args(a, 4);
    if (sa != WAN_ATTN_OK) return sa;
    return int8_grad_product(dy, w_codes, w_scales, dx, M, N, K, false, static_cast<cudaStream_t>(stream));
}

int wan_attn_sync_status(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return WAN_ATTN_ERR_CUDA;
    int h = 0;
    if (cudaMemcpyFromSymbol(&h, g_device_status, sizeof(int)) != cudaSuccess) return WAN_ATTN_ERR_CUDA;
    if (h != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess) return WAN_ATTN_ERR_CUDA;
    }
    return h;
}

const char* wan_attn_status_string(int status) {
    switch (status) {
        case WAN_ATTN_OK: return "ok";
        case WAN_ATTN_ERR_INVALID_ARG: return "invalid argument";
        case WAN_ATTN_ERR_UNSUPPORTED: return "unsupported (head dim must be 128)";
        case WAN_ATTN_ERR_CUDA: return "CUDA error";
        case WAN_ATTN_ERR_TIMEOUT: return "a kernel wait ran out of time";
        case WAN_ATTN_ERR_WORKSPACE: return "workspace missing or too small";
        default: return "unknown status";
    }
}

uint64_t wan_attn_set_wait_budget_ns(uint64_t ns) {
    if (ns < 1000) ns = 1000;
    return g_wait_budget_ns.exchange(ns);
}

int wan_attn_selftest_wait_timeout(uint64_t budget_ns, void* stream) {
    if (budget_ns < 1000) budget_ns = 1000;
    int* status = device_status_word();
    if (!status) return WAN_ATTN_ERR_CUDA;
    selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(budget_ns, status);
    return cudaGetLastError() == cudaSuccess ? WAN_ATTN_OK : WAN_ATTN_ERR_CUDA;
}

}  // extern "C"
