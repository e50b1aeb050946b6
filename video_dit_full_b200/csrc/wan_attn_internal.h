// Internal declarations shared by the C-ABI layer and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace wan {

struct FwdParams {
    void* o;                    // bf16 [B, S, H, 128]
    float* lse;                 // fp32 [B, H, S], natural log
    int B, S, H;                // S = query tokens
    int Skv;                    // key / value tokens (= S for self-attention)
    // block-sparse forward only: 64 x 64 block mask uint8 [B, H, nqb, nkb], and per 128-row Q
    // tile (2 query blocks) the ascending list of key blocks either attends
    // (kv_list [B, H, nctas, nkb] int32, nctas = the number of Q tiles; each entry the key block
    // with bit 30 set if the tile's first query block attends it, bit 31 if the second does)
    // with its length (kv_count [B, H, nctas])
    const uint8_t* mask;
    const int* kv_list;
    const int* kv_count;
    int nqb, nkb, nctas;
    float scale_log2;           // (1 / sqrt(D)) * log2(e)
    unsigned long long wait_budget_ns;
    int* status;                // device status word (see wan_attn_sync_status)
};

struct BwdParams {
    const float* lse;           // fp32 [B, H, Sq] from the forward (natural log)
    float* delta;               // workspace fp32 [B, H, Sq]: rowsum(dO * O)
    float* dq_acc;              // workspace fp32 [B, Sq, H, 128]: unscaled dS K
    float* dk_acc;              // workspace fp32 [B, Skv, H, 128] (split query ranges only)
    float* dv_acc;              // workspace fp32 [B, Skv, H, 128] (split query ranges only)
    void* dk;                   // bf16 [B, Skv, H, 128]
    void* dv;                   // bf16 [B, Skv, H, 128]
    int B, Sq, Skv, H;
    int nsplit;                 // CTAs sharing one key tile, each over its own range of Q tiles
    float scale;                // 1 / sqrt(D)
    float scale_log2;           // scale * log2(e)
    unsigned long long wait_budget_ns;
    int* status;
};

struct Q8QuantParams {
    const __nv_bfloat16 *q, *k, *v;   // bf16 [B, S, H, 128]
    int8_t *q8, *k8;                  // int8 [B, H, S, 128]
    uint8_t* v8;                      // e4m3 [B, H, S, 128]
    float *sq, *sk, *sv;              // fp32 [B, H, nblk]
    int B, S, H, nblk;
};

struct Q8AttnParams {
    void* o;                          // bf16 [B, S, H, 128]
    float* lse;                       // fp32 [B, H, S]
    const float *sq, *sk, *sv;        // fp32 [B, H, nblk]
    int B, S, H, nblk;
    float scale_log2;
    unsigned long long wait_budget_ns;
    int* status;
};

struct Fp8GemmParams {
    const float* a_scales;            // fp32 [M]: per-row (token) scales of the activation codes
    const float* b_scale;             // fp32 [1]: the weight's per-tensor scale (device memory)
    void* y;                          // bf16 [M, N]
    int M, N, K;
    unsigned long long wait_budget_ns;
    int* status;
};

// Packed attention: sequence n owns query rows [cu_q[n], cu_q[n+1]) and key rows [cu_k[n], cu_k[n+1]).
struct VarlenParams {
    const void *q, *k, *v;            // bf16 [Tq, H, 128], [Tk, Hkv, 128] with the token strides below
    const int *cu_q, *cu_k;           // int32 [N + 1], device
    int N, Tq, Tk, H, Hkv;
    long long ldq, ldk, ldv;          // elements from one token to the next
    int causal;
    float scale, scale_log2;          // 1 / sqrt(D); the same times log2(e)
    unsigned long long wait_budget_ns;
    int* status;
};
// The order in which a packed kernel's blocks take (unit, head) pairs, units being a head's items, longest
// first.  Head by head, the blocks of a wave share a head's keys (or queries) in L2; with all heads in turn, the
// longest units of every head start first and the blocks end together.  So the first heads go in groups of about
// one wave, the last ones in one group of three; all in one where what they share fits L2 anyway.
struct HeadOrder {
    int units, heads, group, last;    // heads to a group; heads of the last group
#ifdef __CUDACC__
    __device__ __forceinline__ void at(int x, int& unit, int& head) const {
        int first = heads - last, n = last, y = x - first * units;
        if (y < 0) {
            const int g = x / (group * units);
            n = min(group, first - g * group);
            first = g * group;
            y = x - first * units;
        }
        unit = y / n;
        head = first + (y - unit * n);
    }
#endif
};
inline HeadOrder head_order(long long units, int heads, double shared_bytes) {
    const long long wave = (148 + units - 1) / units, tail = (3 * 148 + units - 1) / units;
    const int last = shared_bytes <= 100e6 || tail > heads ? heads : static_cast<int>(tail);
    return {static_cast<int>(units), heads, static_cast<int>(wave < heads ? wave : heads), last};
}

struct VarlenFwdParams : VarlenParams {
    void* o;                          // bf16 [Tq, H, 128]
    float* lse;                       // fp32 [H, Tq]
    int pack;                         // query heads that share a Q tile (a divisor of H / Hkv)
    int chunk;                        // key blocks of a part where a sequence's keys are split, 0: they are not
    int streamed;                     // K and V are read about once
    HeadOrder order;                  // of packed heads
    float* o_part;                    // workspace fp32 [most parts, Tq, H, 128], where split
    float* lse_part;                  // workspace fp32 [most parts, H, Tq] (base-2 log)
    int* parts;                       // workspace [Tq]: parts of the token's sequence
    int most_parts;                   // that the workspace has room for
};
struct VarlenBwdParams : VarlenParams {
    const void *o, *dout;             // bf16 [Tq, H, 128]
    const float* lse;                 // fp32 [H, Tq]
    void *dq, *dk, *dv;               // bf16, token strides below
    long long lddq, lddk, lddv;
    int splits;                       // CTAs sharing one key tile, each over its own run of Q tiles
    HeadOrder heads;                  // of kv heads
    float* dq_acc;                    // workspace fp32 [Tq, H, 128]: unscaled dS K
    float* delta;                     // workspace fp32 [H, Tq]: rowsum(dO * O)
    float *dk_acc, *dv_acc;           // workspace fp32 [Tk, Hkv, 128], splits > 1 only
    int pack_log2;                    // log2 of the query heads that share a Q tile
    int tile_bound;                   // key tiles, an upper bound
    int2* order;                      // workspace [tile_bound]: key tiles as (sequence, tile), most work first
    int* tile_end;                    // workspace [N]: key tiles up to and including each sequence
};

struct Int8GemmParams {
    const float *a_scales, *b_scales; // fp32 [M], [N]
    const __nv_bfloat16* bias;        // [N] or null
    __nv_bfloat16* y;                 // [M, N]
    int M, N, K;
    int after_quant;                  // launched as the dependent of the quantiser that writes x's codes and scales
    unsigned long long wait_budget_ns;
    int* status;
};

// Device address of the status word on the current device (nullptr on failure).
int* device_status_word();
unsigned long long wait_budget_ns();

// Sets the dynamic shared-memory limit of a kernel once per device.  0 on success.
int configure_smem(const void* kernel, int bytes);

// Launches a kernel that starts while the stream's kernel before it may still run (programmatic dependent
// launch), `cluster` CTAs along x to a cluster.  What its CTAs set up before grid_dependency_wait overlaps
// that kernel's end; nothing that kernel may have written is read before it (and no pointer is __restrict__,
// which would let the compiler move a load of const data there).  Such a kernel allocates TMEM
// only behind that wait (a waiting CTA then holds none that the kernel before it still has to get), and lets
// the next one start, by grid_launch_dependents, only once it has it.
// `early` false: an ordinary launch.
template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, int cluster, bool early,
                     A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = early ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...) == cudaSuccess ? 0 : -1;
}

// `to`: a map over O with the layout and box of tq (the epilogue TMA-stores O through it).
int launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to,
               const FwdParams& p, cudaStream_t stream);
// Forward with one CTA per 128-row Q tile (p.nctas = the number of Q tiles); tk64 / tv64 are
// K / V maps with 64-token boxes.  Block-sparse (p.kv_list set): builds each tile's
// key-block list in p.kv_list / p.kv_count (device workspace) from p.mask, then runs the
// pair-step kernel over the lists.  p.kv_list null: every key block, no mask, on the per-tile
// kernel with 64-key steps.
int launch_fwd_tiles(const CUtensorMap& tq, const CUtensorMap& tk64, const CUtensorMap& tv64, const CUtensorMap& to,
                     const FwdParams& p, cudaStream_t stream);

// Chooses p.nsplit (1 unless allow_split and the key tiles alone fill too few waves of the
// GPU), then launches the backward's kernels.  tdk / tdv (fp32 accumulators, as tdq) are only
// read when p.nsplit > 1.
int launch_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
               const CUtensorMap& tdq, const CUtensorMap& tdk, const CUtensorMap& tdv, BwdParams p,
               bool allow_split, const void* o, const void* dout, void* dq, cudaStream_t stream);

// Context-parallel helpers (cp_kernels.cu).  0 on success.
int launch_cp_merge(float* o_acc, float* lse_acc, const void* o_part, const float* lse_part, void* o_out, int B,
                    int S, int H, int first, cudaStream_t stream);
int launch_cp_accumulate(float* acc, const void* part, void* out, long long n8, int first, cudaStream_t stream);
int launch_cp_layout(void* dst, const void* src, int B, int S, int G, int blk16, int which, cudaStream_t stream);

// FP8 GEMM of the linear layers (fp8_gemm.cu).  0 on success.
int launch_fp8_quant_rows(const void* x, void* codes, float* scales, int M, int K, cudaStream_t stream);
int launch_fp8_quant_tensor(const void* w, void* codes, float* scale2, long long n, cudaStream_t stream);
// tb: W's map with 256-row boxes (1-CTA kernel); tb_half: 128-row boxes (CTA pairs).
int launch_fp8_gemm(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tb_half, const Fp8GemmParams& p,
                    cudaStream_t stream);

// Packed attention (attn_varlen_fwd.cu, attn_varlen_bwd.cu).  0 on success.
// tq, to: maps over q and o (128, H, Tq) with boxes (64, pack, 128 / pack); tk, tv: (128, Hkv, Tk), (64, 1, 128).
int launch_varlen_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to,
                      const VarlenFwdParams& p, long long units, cudaStream_t stream);
// How the forward lays out a call: heads per Q tile and splits of the keys (see VarlenFwdParams).
struct VarlenFwdPlan {
    int pack, chunk, streamed;        // as in VarlenFwdParams
    int parts;                        // most parts of a sequence
    long long units;                  // the grid: units x (H / pack), in `order`
    HeadOrder order;
};
VarlenFwdPlan varlen_fwd_plan(int N, int Tq, int Tk, int H, int Hkv);
// tk, tv: boxes (64, 1, 128); tq, tdo: (64, pack, 128 / pack); tdq: fp32 [Tq, H, 128], (128, pack, 128 / pack); tdk, tdv: fp32
// [Tk, Hkv, 128], boxes (32, 1, 128) with the 128-byte swizzle, only read when p.splits > 1.
int launch_varlen_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                      const CUtensorMap& tdq, const CUtensorMap& tdk, const CUtensorMap& tdv, const VarlenBwdParams& p,
                      cudaStream_t stream);
int varlen_bwd_splits(int N, int Tq, int Tk, int H, int Hkv);
int varlen_bwd_tile_bound(int N, int Tk);
int varlen_bwd_pack(int H, int Hkv);

// Int8 linear layer (int8_linear.cu) and its backward (int8_grad.cu).  0 on success.
int launch_int8_quant_rows(const void* x, void* codes, float* scales, int M, int K, long long ldx, cudaStream_t stream);
int launch_int8_dequant_rows(const void* codes, const float* scales, void* x, int M, int K, cudaStream_t stream);
// Whether a layer of this size runs in one launch (quantiser included; codes and scales may then be null),
// and that launch.  tw: the weight's codes, boxes of 128 rows.
bool int8_layer_fits(int M, int N, int K);
int launch_int8_layer(const CUtensorMap& tw, const void* x, long long ldx, void* codes, float* scales,
                      const Int8GemmParams& p, cudaStream_t stream);
// Tokens of one tile of the few-token kernel for this size, or 0 for the CTA-pair kernel.
int int8_gemm_token_tile(int M, int N);
// tx: x's codes, boxes of the token tile's rows (128 for pairs); tw: the weight's codes, boxes of 128 rows.
int launch_int8_gemm(const CUtensorMap& tx, const CUtensorMap& tw, const Int8GemmParams& p, cudaStream_t stream);
// out[r, c] = sum_t a(t, r) scales[t] codes[t, c].  weight: a(t, r) = dy[t, r] (rows = N, terms = M), tdy with
// boxes of (64, 64); else a(t, r) = dy[r, t] (rows = M, terms = N), boxes (64, 128).  tcodes: boxes (128, 64).
int launch_int8_grad(const CUtensorMap& tdy, const CUtensorMap& tcodes, const float* scales, void* out, int rows, int cols,
                     int terms, bool weight, unsigned long long budget_ns, int* status, cudaStream_t stream);

// `to`: a map over the bf16 O [B, S, H, D] with 128-token boxes (the epilogue TMA-stores O through it).
int launch_q8(const Q8QuantParams& qp, const CUtensorMap& tq8, const CUtensorMap& tk8, const CUtensorMap& tv8,
              const CUtensorMap& to, const Q8AttnParams& p, cudaStream_t stream);

}  // namespace wan
