// Int8 linear layer: row quantiser, its inverse, and Y = diag(sx) (Cx Cw^T) diag(sw) + bias.
#include "sm100_ptx.cuh"
#include "wan_attn_internal.h"

namespace wan {
namespace int8 {

// One warp per row.  Codes are rint of the exact quotient 127 x / absmax: 127 x is exact in fp32
// (7 + 8 bits) and the division is correctly rounded; a quotient that is not a half-integer is at
// least 2^-9 away from one (its denominator has 8 bits), far more than the rounding error.
__global__ void __launch_bounds__(256) quant_rows_kernel(const __nv_bfloat16* __restrict__ x, int8_t* __restrict__ codes,
                                                         float* __restrict__ scales, int M, int K, long long ldx) {
    const int lane = threadIdx.x & 31;
    const long long m = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (m >= M) return;
    float amax = 0.f;
    bool bad = false;
    for (int k = lane; k < K; k += 32) {
        const float f = fabsf(__bfloat162float(x[m * ldx + k]));
        bad |= !(f <= 3.4e38f);
        amax = fmaxf(amax, f);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) scales[m] = bad ? NAN : amax > 0.f ? __fdiv_rn(amax, 127.f) : 1.f;
    const float pre = amax > 1e30f ? 0x1p-32f : 1.f;          // 127 x must not overflow; exact, as the powers of two are
    for (int k = lane; k < K; k += 32)
        codes[m * K + k] = (bad || !(amax > 0.f)) ? 0
                               : static_cast<int8_t>(__float2int_rn(
                                     __fdiv_rn(127.f * (pre * __bfloat162float(x[m * ldx + k])), pre * amax)));
}

__global__ void __launch_bounds__(256) dequant_rows_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                           __nv_bfloat16* __restrict__ x, int K, long long n) {
    for (long long t = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; t < n; t += 256ll * gridDim.x)
        x[t] = __float2bfloat16_rn(scales[t / K] * codes[t]);
}

__global__ void __launch_bounds__(256) gemm_kernel(const int8_t* __restrict__ a, const float* __restrict__ sa,
                                                   const int8_t* __restrict__ b, const float* __restrict__ sb,
                                                   const __nv_bfloat16* __restrict__ bias, __nv_bfloat16* __restrict__ y,
                                                   int M, int N, int K) {
    __shared__ int as[16][17], bs[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long m = blockIdx.x * 16ll + ty;
    const int n = blockIdx.y * 16 + tx, nb = blockIdx.y * 16 + ty;
    int acc = 0;
    for (int k = 0; k < K; k += 64) {
        const int kk = k + tx * 4;
        as[ty][tx] = (m < M && kk < K) ? *reinterpret_cast<const int*>(a + m * K + kk) : 0;
        bs[ty][tx] = (nb < N && kk < K) ? *reinterpret_cast<const int*>(b + static_cast<long long>(nb) * K + kk) : 0;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) acc = __dp4a(as[ty][e], bs[tx][e], acc);
        __syncthreads();
    }
    if (m < M && n < N) {
        const float f = static_cast<float>(acc) * (sa[m] * sb[n]) + (bias ? __bfloat162float(bias[n]) : 0.f);
        y[m * N + n] = __float2bfloat16_rn(f);
    }
}

}  // namespace int8

int launch_int8_quant_rows(const void* x, void* codes, float* scales, int M, int K, long long ldx, cudaStream_t stream) {
    int8::quant_rows_kernel<<<(M + 7) / 8, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(x),
                                                             static_cast<int8_t*>(codes), scales, M, K, ldx);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_int8_dequant_rows(const void* codes, const float* scales, void* x, int M, int K, cudaStream_t stream) {
    int8::dequant_rows_kernel<<<148 * 8, 256, 0, stream>>>(static_cast<const int8_t*>(codes), scales,
                                                           static_cast<__nv_bfloat16*>(x), K, static_cast<long long>(M) * K);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_int8_gemm(const void* a_codes, const float* a_scales, const void* b_codes, const float* b_scales,
                     const void* bias, void* y, int M, int N, int K, cudaStream_t stream) {
    const dim3 grid((M + 15) / 16, (N + 15) / 16);
    int8::gemm_kernel<<<grid, 256, 0, stream>>>(static_cast<const int8_t*>(a_codes), a_scales,
                                                static_cast<const int8_t*>(b_codes), b_scales,
                                                static_cast<const __nv_bfloat16*>(bias), static_cast<__nv_bfloat16*>(y),
                                                M, N, K);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace wan
