// The int8 linear layer's backward: out[r, c] = sum_t a(t, r) s[t] codes[t, c] (dW and dX).
#include "sm100_ptx.cuh"
#include "wan_attn_internal.h"

namespace wan {
namespace int8 {

__global__ void __launch_bounds__(256) grad_kernel(const __nv_bfloat16* __restrict__ dy, const int8_t* __restrict__ codes,
                                                   const float* __restrict__ s, __nv_bfloat16* __restrict__ out, int rows,
                                                   int cols, int terms, int a_by_row) {
    __shared__ float as[16][17], bs[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long r0 = blockIdx.x * 16ll, c = blockIdx.y * 16ll + tx;
    float acc = 0.f;
    for (int t0 = 0; t0 < terms; t0 += 16) {
        // as[term][row]
        const long long r = a_by_row ? r0 + ty : r0 + tx, t = a_by_row ? t0 + tx : t0 + ty;
        const float av = (r < rows && t < terms) ? __bfloat162float(a_by_row ? dy[r * terms + t] : dy[t * rows + r]) : 0.f;
        if (a_by_row) as[tx][ty] = av;
        else as[ty][tx] = av;
        bs[ty][tx] = (t0 + ty < terms && c < cols) ? s[t0 + ty] * codes[static_cast<long long>(t0 + ty) * cols + c] : 0.f;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) acc = fmaf(as[e][ty], bs[e][tx], acc);
        __syncthreads();
    }
    if (r0 + ty < rows && c < cols) out[(r0 + ty) * cols + c] = __float2bfloat16_rn(acc);
}

}  // namespace int8

int launch_int8_grad(const void* dy, const void* codes, const float* scales, void* out, int rows, int cols, int terms,
                     int a_by_row, cudaStream_t stream) {
    const dim3 grid((rows + 15) / 16, (cols + 15) / 16);
    int8::grad_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(dy), static_cast<const int8_t*>(codes),
                                                scales, static_cast<__nv_bfloat16*>(out), rows, cols, terms, a_by_row);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace wan
