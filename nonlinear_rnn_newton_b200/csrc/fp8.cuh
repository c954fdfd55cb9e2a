// 8-bit product with a scale for each block of 128:
//   u[m][n] = sum over blocks k of xs[m][k] ws[n / 128][k] (x[m] . w[n] over
//   the 128 columns of block k)  (+ bias[n]),
// x [M][K] and w [N][K] in e4m3, one fp32 scale per row of x and per 128 rows
// of w in each block.
#pragma once

#include "norm.cuh"

namespace pararnn {

__device__ __forceinline__ float from_e4m3(uint8_t b)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

struct Fp8Params {
    const uint8_t *x, *w;
    const float *xs, *ws, *bias;
    void* u;
    long long M, N, K, KB;
    int u_bf16;
};

// 64 x 64 outputs a CTA, 4 x 4 a thread, 32 columns of K at a time
__global__ void __launch_bounds__(256) fp8_project_kernel(const Fp8Params p)
{
    __shared__ float sx[32][65], sw[32][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long m0 = (long long)blockIdx.y * 64, n0 = (long long)blockIdx.x * 64;
    float acc[4][4] = {};
    for (long long k0 = 0; k0 < p.K; k0 += 32) {
        const long long kb = k0 / 128;
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * 32; i += 256) {
            const int r = i >> 5, c = i & 31;
            const bool ck = k0 + c < p.K;
            sx[c][r] = ck && m0 + r < p.M ? from_e4m3(p.x[(m0 + r) * p.K + k0 + c]) * p.xs[(m0 + r) * p.KB + kb] : 0.f;
            sw[c][r] = ck && n0 + r < p.N ? from_e4m3(p.w[(n0 + r) * p.K + k0 + c]) * p.ws[(n0 + r) / 128 * p.KB + kb] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 32; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sx[c][ty * 4 + i], sw[c][tx * 4 + j], acc[i][j]);
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= p.M || n >= p.N) continue;
            const float v = acc[i][j] + (p.bias ? p.bias[n] : 0.f);
            if (p.u_bf16) static_cast<uint16_t*>(p.u)[m * p.N + n] = uint16_t(pack_bf16x2(v, 0.f));
            else static_cast<float*>(p.u)[m * p.N + n] = v;
        }
}

}  // namespace pararnn
