// Packed attention forward: one warp per (query row, head), four dims per lane.
#include "sm100_ptx.cuh"
#include "varlen.cuh"

namespace wan {
namespace varlen {

__device__ __forceinline__ float4 ld4(const void* base, long long elem) {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + elem);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(128) varlen_fwd_kernel(const VarlenFwdParams p) {
    const long long id = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (id >= static_cast<long long>(p.Tq) * p.H) return;
    const int lane = threadIdx.x & 31, t = static_cast<int>(id / p.H), h = static_cast<int>(id % p.H);
    const int n = sequence_of(p.cu_q, p.N, t);
    if (n < 0) return;
    const Span sq = span_of(p.cu_q, n, p.Tq), sk = span_of(p.cu_k, n, p.Tk);
    const int hk = h / (p.H / p.Hkv);
    const int seen = p.causal ? min(sk.len, max(0, t - sq.begin + sk.len - sq.len + 1)) : sk.len;
    const float4 q = ld4(p.q, t * p.ldq + h * 128 + lane * 4);
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < seen; ++j) {
        const long long row = sk.begin + j;
        const float4 k = ld4(p.k, row * p.ldk + hk * 128 + lane * 4);
        float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), alpha = ex2_approx(m - mn), e = ex2_approx(s - mn);
        const float4 v = ld4(p.v, row * p.ldv + hk * 128 + lane * 4);
        acc = make_float4(acc.x * alpha + e * v.x, acc.y * alpha + e * v.y, acc.z * alpha + e * v.z,
                          acc.w * alpha + e * v.w);
        l = l * alpha + e;
        m = mn;
    }
    const float inv = seen ? 1.f / l : 0.f;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (static_cast<long long>(t) * p.H + h) * 128 + lane * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0)
        p.lse[static_cast<long long>(h) * p.Tq + t] = seen ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace varlen

int launch_varlen_fwd(const VarlenFwdParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.Tq) * p.H;
    varlen::varlen_fwd_kernel<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace wan
