// Packed attention backward: one warp per (query row, head) for dQ, one per (key row, kv head) for dK and dV.
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
__device__ __forceinline__ float dot(float4 a, float4 b) {
    float s = a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}
__device__ __forceinline__ void axpy(float4& a, float s, float4 b) {
    a = make_float4(a.x + s * b.x, a.y + s * b.y, a.z + s * b.z, a.w + s * b.w);
}
__device__ __forceinline__ void st4(void* base, long long elem, float4 a, float mul) {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + elem) =
        make_uint2(pack_bf16x2(a.x * mul, a.y * mul), pack_bf16x2(a.z * mul, a.w * mul));
}

__global__ void __launch_bounds__(128) varlen_dq_kernel(const VarlenBwdParams p) {
    const long long id = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (id >= static_cast<long long>(p.Tq) * p.H) return;
    const int lane = threadIdx.x & 31, t = static_cast<int>(id / p.H), h = static_cast<int>(id % p.H);
    const int n = sequence_of(p.cu_q, p.N, t);
    if (n < 0) return;
    const Span sq = span_of(p.cu_q, n, p.Tq), sk = span_of(p.cu_k, n, p.Tk);
    const int hk = h / (p.H / p.Hkv);
    const int seen = p.causal ? min(sk.len, max(0, t - sq.begin + sk.len - sq.len + 1)) : sk.len;
    const long long at = (static_cast<long long>(t) * p.H + h) * 128 + lane * 4;
    const float4 q = ld4(p.q, t * p.ldq + h * 128 + lane * 4), o = ld4(p.o, at), g = ld4(p.dout, at);
    const float delta = dot(o, g), lse = p.lse[static_cast<long long>(h) * p.Tq + t] * 1.4426950408889634f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < seen; ++j) {
        const long long row = sk.begin + j;
        const float4 k = ld4(p.k, row * p.ldk + hk * 128 + lane * 4), v = ld4(p.v, row * p.ldv + hk * 128 + lane * 4);
        const float pr = ex2_approx(dot(q, k) * p.scale_log2 - lse);
        axpy(acc, pr * (dot(g, v) - delta), k);
    }
    st4(p.dq, t * p.lddq + h * 128 + lane * 4, acc, p.scale);
}

__global__ void __launch_bounds__(128) varlen_dkv_kernel(const VarlenBwdParams p) {
    const long long id = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (id >= static_cast<long long>(p.Tk) * p.Hkv) return;
    const int lane = threadIdx.x & 31, t = static_cast<int>(id / p.Hkv), hk = static_cast<int>(id % p.Hkv);
    const int n = sequence_of(p.cu_k, p.N, t);
    if (n < 0) return;
    const Span sq = span_of(p.cu_q, n, p.Tq), sk = span_of(p.cu_k, n, p.Tk);
    const int group = p.H / p.Hkv;
    const int first = p.causal ? max(0, t - sk.begin - (sk.len - sq.len)) : 0;
    const float4 k = ld4(p.k, t * p.ldk + hk * 128 + lane * 4), v = ld4(p.v, t * p.ldv + hk * 128 + lane * 4);
    float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
    for (int h = hk * group; h < (hk + 1) * group; ++h)
        for (int i = first; i < sq.len; ++i) {
            const long long row = sq.begin + i, at = (row * p.H + h) * 128 + lane * 4;
            const float4 q = ld4(p.q, row * p.ldq + h * 128 + lane * 4), o = ld4(p.o, at), g = ld4(p.dout, at);
            const float lse = p.lse[static_cast<long long>(h) * p.Tq + row] * 1.4426950408889634f;
            const float pr = ex2_approx(dot(q, k) * p.scale_log2 - lse);
            axpy(dv, pr, g);
            axpy(dk, pr * (dot(g, v) - dot(o, g)), q);
        }
    st4(p.dk, t * p.lddk + hk * 128 + lane * 4, dk, p.scale);
    st4(p.dv, t * p.lddv + hk * 128 + lane * 4, dv, 1.f);
}

}  // namespace varlen

int launch_varlen_bwd(const VarlenBwdParams& p, cudaStream_t stream) {
    const long long rq = static_cast<long long>(p.Tq) * p.H, rk = static_cast<long long>(p.Tk) * p.Hkv;
    if (rq) varlen::varlen_dq_kernel<<<static_cast<unsigned>((rq + 3) / 4), 128, 0, stream>>>(p);
    if (rk) varlen::varlen_dkv_kernel<<<static_cast<unsigned>((rk + 3) / 4), 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace wan
