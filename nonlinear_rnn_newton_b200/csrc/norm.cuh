// RMS norm with the residual's addition before it and an 8-bit output with
// scales behind it, and its adjoint.
//
//   v = x + residual,  sum = v in the residual's type,
//   rstd = 1 / sqrt(mean(v^2) + eps),  y = v rstd w;
//   8 bits: per block of 128 columns scale = max(amax / 448, 2^-126) and
//   q = e4m3(y / scale).
// Adjoint, with n = v rstd and g = dy w:
//   dx = dsum + rstd (g - n mean(g n)),  dw = sum over rows of dy n.
//
// Both are bound by HBM: a row is read once into registers (8 columns a
// vector, NV vectors a thread) and everything else happens there.  A row
// belongs to `tpr` threads (a multiple of 32); 16 neighbouring lanes hold one
// block of 128 columns, so its scale needs four shuffles.
#pragma once

#include <cuda_fp8.h>

#include "device_common.cuh"

namespace pararnn {

constexpr int kNormThreads = 512;      // most threads of a CTA (and of a row)
constexpr int kNormVectors = 4;        // most vectors of 8 columns a thread keeps
constexpr long long kNormMaxD = 8ll * kNormThreads * kNormVectors;
constexpr float kE4m3Max = 448.0f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126, the smallest normal number

// eight consecutive values as loaded (16 bytes of bf16, 32 of fp32)
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    uint4 w;
    __device__ __forceinline__ void load(const void* p, long long i)
    {
        w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(x[i] << 16);
            v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p, long long i)
    {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        a = __ldg(q);
        b = __ldg(q + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <>
struct Raw8<void> {  // absent: zeros
    __device__ __forceinline__ void load(const void*, long long) {}
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
};

// two bf16, rounded to nearest even, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void store8(void* p, long long i, bool bf16, const float (&v)[8])
{
    if (bf16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// eight e4m3, rounded to nearest even, NaN kept
__device__ __forceinline__ uint2 pack_e4m3x8(const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ float amax8(const float (&v)[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_keep_nan(m, fabsf(v[i]));
    return m;
}

// the scale of a block with that largest magnitude (NaN and inf are kept: such
// a block stands for NaN throughout)
__device__ __forceinline__ float scale_of(float amax) { return max_keep_nan(amax / kE4m3Max, kLeastScale); }

// the largest of 16 neighbouring lanes
__device__ __forceinline__ float max16(float m)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_keep_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// Sum of v over the tpr threads of this row; every thread gets it.  s: one
// float per warp of the CTA.  Every thread of the CTA calls it.
__device__ __forceinline__ float row_sum(float v, int tpr, float* s)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    const int w = threadIdx.x >> 5, per = tpr >> 5, first = w / per * per;
    if ((threadIdx.x & 31) == 0) s[w] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < per; ++i) v += s[first + i];
    return v;
}

struct NormParams {
    const void *x, *res;
    const float* w;
    void* sum;
    void* y;
    float* scale;
    float* rstd;
    long long T, D;
    float eps;
    int tpr;
    int sum_bf16;
    int y_dtype;
};

template <class XT, class RT, int NV>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const NormParams p)
{
    __shared__ float s_red[32];
    const int tpr = p.tpr, rows = blockDim.x / tpr;
    const int lane = threadIdx.x % tpr;
    const long long t = (long long)blockIdx.x * rows + threadIdx.x / tpr;
    const bool live = t < p.T;
    const long long D = p.D, base = t * D;
    Raw8<XT> rx[NV];
    Raw8<RT> rr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const long long c = 8ll * (lane + k * tpr);
        if (live && c < D) {
            rx[k].load(p.x, base + c);
            rr[k].load(p.res, base + c);
        }
    }
    float v[NV][8], ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const long long c = 8ll * (lane + k * tpr);
        const bool in = live && c < D;
        float r[8];
        rx[k].get(v[k]);
        rr[k].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[k][j] = in ? v[k][j] + r[j] : 0.f;
            ss = fmaf(v[k][j], v[k][j], ss);
        }
        if (in && p.sum) store8(p.sum, base + c, p.sum_bf16, v[k]);
    }
    ss = row_sum(ss, tpr, s_red);
    const float rstd = 1.0f / sqrtf(ss / float(D) + p.eps);
    if (live && lane == 0 && p.rstd) p.rstd[t] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const long long c = 8ll * (lane + k * tpr);
        const bool in = live && c < D;
        float y[8];
        if (in) {
            Raw8<float> rw;
            rw.load(p.w, c);
            rw.get(y);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = in ? v[k][j] * rstd * y[j] : 0.f;
        if (p.y_dtype == PARARNN_E4M3) {
            const float sc = scale_of(max16(amax8(y)));
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = y[j] / sc;
            if (in) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + base + c) = pack_e4m3x8(y);
                if ((lane & 15) == 0) p.scale[t * ((D + 127) / 128) + c / 128] = sc;
            }
        } else if (in) {
            store8(p.y, base + c, p.y_dtype == PARARNN_BF16, y);
        }
    }
}

struct NormAdjParams {
    const void *dy, *v;
    const float *w, *rstd;
    const void* dv;  // or NULL
    void* dx;
    float* part;  // [gridDim.x][D]
    long long T, D;
    int tpr;
};

// A CTA takes rows blockIdx.x * rows + k * gridDim.x * rows; dw of its rows
// stays in registers and leaves once, one row of `part` a CTA.
template <class YT, class VT, int NV>
__global__ void __launch_bounds__(kNormThreads) rms_norm_adjoint_kernel(const NormAdjParams p)
{
    __shared__ float s_red[2][32];
    extern __shared__ float s_dw[];  // [rows][D] where a CTA has several rows
    const int tpr = p.tpr, rows = blockDim.x / tpr, row = threadIdx.x / tpr;
    const int lane = threadIdx.x % tpr;
    const long long D = p.D;
    float dw[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
    int turn = 0;
    for (long long t0 = (long long)blockIdx.x * rows; t0 < p.T; t0 += (long long)gridDim.x * rows, turn ^= 1) {
        const long long t = t0 + row, base = t * D;
        const bool live = t < p.T;
        Raw8<YT> ry[NV];
        Raw8<VT> rv[NV], rd[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long c = 8ll * (lane + k * tpr);
            if (live && c < D) {
                ry[k].load(p.dy, base + c);
                rv[k].load(p.v, base + c);
                if (p.dv) rd[k].load(p.dv, base + c);
            }
        }
        const float rstd = live ? p.rstd[t] : 0.f;
        float g[NV][8], n[NV][8], gn = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long c = 8ll * (lane + k * tpr);
            const bool in = live && c < D;
            ry[k].get(g[k]);
            rv[k].get(n[k]);
            float w[8];
            if (in) {
                Raw8<float> rw;
                rw.load(p.w, c);
                rw.get(w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[k][j] = in ? n[k][j] * rstd : 0.f;
                const float dy = in ? g[k][j] : 0.f;
                dw[k][j] = fmaf(dy, n[k][j], dw[k][j]);
                g[k][j] = in ? dy * w[j] : 0.f;
                gn = fmaf(g[k][j], n[k][j], gn);
            }
        }
        // two buffers in turn: a warp may be a row ahead of one still summing
        gn = row_sum(gn, tpr, s_red[turn]) / float(D);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long c = 8ll * (lane + k * tpr);
            if (live && c < D) {
                float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (p.dv) rd[k].get(o);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = fmaf(rstd, fmaf(-n[k][j], gn, g[k][j]), o[j]);
                store8(p.dx, base + c, sizeof(VT) == 2, o);
            }
        }
    }
    if (rows > 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long c = 8ll * (lane + k * tpr);
            if (c < D)
                for (int j = 0; j < 8; ++j) s_dw[row * D + c + j] = dw[k][j];
        }
        __syncthreads();
        for (long long c = threadIdx.x; c < D; c += blockDim.x) {
            float a = 0.f;
            for (int r = 0; r < rows; ++r) a += s_dw[r * D + c];
            p.part[(long long)blockIdx.x * D + c] = a;
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long c = 8ll * (lane + k * tpr);
            if (c < D) store8(p.part, (long long)blockIdx.x * D + c, false, dw[k]);
        }
    }
}

// ------------------------------------------------------- 8-bit quantisation

// One scale per row and 128 columns: 16 lanes a block, 8 columns a lane.
template <class XT>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const void* x, uint8_t* q, float* scale, long long M,
                                                                long long K, long long KB)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // 8 columns of a row filled up to whole blocks
    const long long m = i / (KB * 16), c = 8 * (i - m * KB * 16);
    const bool in = m < M && c < K;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
        Raw8<XT> r;
        r.load(x, m * K + c);
        r.get(v);
    }
    const float sc = scale_of(max16(amax8(v)));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] / sc;
    if (in) {
        *reinterpret_cast<uint2*>(q + m * K + c) = pack_e4m3x8(v);
        if ((threadIdx.x & 15) == 0) scale[m * KB + c / 128] = sc;
    }
}

// One scale per 128 rows and 128 columns: a CTA a block, kept in registers.
template <class XT>
__global__ void __launch_bounds__(256) fp8_quantize_blocks_kernel(const void* x, uint8_t* q, float* scale, long long M,
                                                                  long long K, long long KB)
{
    __shared__ float s_max[8];
    const long long mb = blockIdx.x / KB, kb = blockIdx.x - mb * KB;
    const long long c = kb * 128 + 8 * (threadIdx.x & 15), m0 = mb * 128 + (threadIdx.x >> 4);
    Raw8<XT> r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (m0 + 16 * i < M && c < K) r[i].load(x, (m0 + 16 * i) * K + c);
    float v[8][8], most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (m0 + 16 * i < M && c < K) {
            r[i].get(v[i]);
            most = max_keep_nan(most, amax8(v[i]));
        }
    most = max16(most);
    most = max_keep_nan(most, __shfl_xor_sync(0xffffffffu, most, 16));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max_keep_nan(most, s_max[i]);
    const float sc = scale_of(most);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (m0 + 16 * i < M && c < K) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] / sc;
            *reinterpret_cast<uint2*>(q + (m0 + 16 * i) * K + c) = pack_e4m3x8(v[i]);
        }
    if (threadIdx.x == 0) scale[blockIdx.x] = sc;
}

}  // namespace pararnn
