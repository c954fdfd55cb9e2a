// RMS norm with the residual's addition before it and an 8-bit output with
// scales behind it, and its adjoint.
//
//   v = x + residual,  sum = v in the residual's type,
//   rstd = 1 / sqrt(mean(v^2) + eps),  y = v rstd w;
//   8 bits: per block of 128 columns scale = max(amax / 448, 2^-126) and
//   q = e4m3(y / scale), the same bits that the quantiser makes of an fp32 y.
// Adjoint, with n = v rstd and g = dy w:
//   dx = dsum + rstd (g - n mean(g n)),  dw = sum over rows of dy n.
//
// Both are bound by HBM: a row is read once into registers (8 columns a
// vector, NV vectors a thread) and everything else happens there.  A row
// belongs to `tpr` threads (a multiple of 32); 16 neighbouring lanes hold one
// block of 128 columns, so its scale needs four shuffles.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "device_common.cuh"

namespace pararnn {

constexpr int kNormThreads = 512;      // most threads of a CTA (and of a row)
constexpr int kNormVectors = 4;        // most vectors of 8 columns a thread keeps
constexpr long long kNormMaxD = 8ll * kNormThreads * kNormVectors;
constexpr float kE4m3Max = 448.0f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126, the smallest normal number

// eight consecutive values as loaded (16 bytes of bf16, 32 of fp32); plain
// loads, not those of read-only data: an output may stand in its input's place
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    uint4 w;
    __device__ __forceinline__ void load(const void* p, long long i)
    {
        w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
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
        a = q[0];
        b = q[1];
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

// Arithmetic on pairs of neighbouring columns, in the packed fp32 instructions.
struct P8 {
    float2 v[4];
};

__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

template <class R>
__device__ __forceinline__ P8 pairs(const R& raw)
{
    float x[8];
    raw.get(x);
    P8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = make_float2(x[2 * i], x[2 * i + 1]);
    return r;
}

// two bf16, rounded to nearest even, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void store8(void* p, long long i, bool bf16, const P8& x)
{
    if (bf16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(pack_bf16x2(x.v[0].x, x.v[0].y), pack_bf16x2(x.v[1].x, x.v[1].y), pack_bf16x2(x.v[2].x, x.v[2].y),
                       pack_bf16x2(x.v[3].x, x.v[3].y));
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
        q[1] = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
    }
}

// eight e4m3, rounded to nearest even, NaN kept
__device__ __forceinline__ uint2 pack_e4m3x8(const P8& x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __nv_cvt_float2_to_fp8x2(x.v[i], __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ float amax8(const P8& x)
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_keep_nan(max_keep_nan(m, fabsf(x.v[i].x)), fabsf(x.v[i].y));
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

// v / sc rounded to fp32, for the norm and the quantiser: bf16 values often lie
// halfway between two e4m3 ones, and the rounded quotient then decides, so a
// product with 1 / sc alone will not do.  Markstein's correction (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000", 1990): with y = 1 / sc rounded and q = v y, the
// residual v - q sc is exact in one fused multiply-add, and q + residual y
// rounds to the quotient.  The residual must not underflow, so small blocks are
// scaled up by 2^64 first, which is exact.  Tested bit for bit against IEEE
// division.  The quantiser, M 16384 K 4096, bf16: 41 us (4.9 TB/s; fp32 51, 6.6 TB/s); with a
// division each 55; a reciprocal with divisions only beside the middles 81, for
// its branches.
__device__ __forceinline__ P8 quotients(const P8& v, float sc)
{
    const float up = sc < 1e-25f ? 18446744073709551616.0f : 1.0f;
    const float s = sc * up;
    const float2 y = twice(1.0f / s), ns = twice(-s);
    P8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __fmul2_rn(v.v[i], twice(up));
        const float2 q = __fmul2_rn(x, y);
        r.v[i] = __ffma2_rn(__ffma2_rn(q, ns, x), y, q);
    }
    return r;
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

// T 32768 D 2048 (fp32 in, bf16 residual, e4m3 out): 96 us, 6.3 TB/s, from a
// graph; with a product by the scale's rounded reciprocal for the quotient the
// same.  48 registers let ten CTAs of 128 threads on an SM; the quotients took
// 50, nine CTAs and 98 us (T 16384 D 4096: 106.5 against 98).
template <class XT, class RT, int NV>
__global__ void __maxnreg__(NV <= 2 ? 48 : 128) rms_norm_kernel(const NormParams p)
{
    __shared__ float s_red[32];
    const int tpr = p.tpr, rows = blockDim.x / tpr;
    const int lane = threadIdx.x % tpr;
    const long long t = (long long)blockIdx.x * rows + threadIdx.x / tpr;
    const long long D = p.D, base = t * D;
    const int left = t < p.T ? int(D) - 8 * lane : 0;  // vector k is in the row where 8 k tpr < left
    Raw8<XT> rx[NV];
    Raw8<RT> rr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (8 * k * tpr < left) {
            rx[k].load(p.x, base + 8 * (lane + k * tpr));
            rr[k].load(p.res, base + 8 * (lane + k * tpr));
        }
    }
    P8 v[NV];
    float2 ss = twice(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const bool in = 8 * k * tpr < left;
        v[k] = pairs(rx[k]);
        if constexpr (!std::is_void<RT>::value) {
            const P8 r = pairs(rr[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[k].v[j] = __fadd2_rn(v[k].v[j], r.v[j]);
        }
        if (in) {
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = __ffma2_rn(v[k].v[j], v[k].v[j], ss);
            if (p.sum) store8(p.sum, base + 8 * (lane + k * tpr), p.sum_bf16, v[k]);
        }
    }
    const float all = row_sum(ss.x + ss.y, tpr, s_red);
    const float rstd = 1.0f / sqrtf(all / float(D) + p.eps);
    if (left > 0 && lane == 0 && p.rstd) p.rstd[t] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = 8 * (lane + k * tpr);
        const bool in = 8 * k * tpr < left;
        P8 y;
        if (in) {
            Raw8<float> rw;
            rw.load(p.w, c);
            y = pairs(rw);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) y.v[j] = in ? __fmul2_rn(__fmul2_rn(v[k].v[j], twice(rstd)), y.v[j]) : twice(0.f);
        if (p.y_dtype == PARARNN_E4M3) {
            const float sc = scale_of(max16(amax8(y)));
            if (in) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + base + c) = pack_e4m3x8(quotients(y, sc));
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

// A CTA takes rows blockIdx.x * rows + k * gridDim.x * rows, and asks for its
// next row before it works on this one; dw of its rows stays in registers and
// leaves once, one row of `part` a CTA.  T 32768 D 2048, bf16: 94 to 96 us, 5.6
// TB/s (without the loads ahead 120 us, one vector a thread 108); 125 registers
// leave four CTAs an SM, whose loads of three arrays are 48 KB in flight.  Four
// vectors a thread (D above 8192) do not fit into the 128 registers that 512
// threads leave: T 4096 D 16384 takes 172 us in bf16 (540 bytes of spills read a
// thread) and 458 in fp32 (1236), where 82 and 164 are the memory's.
template <class YT, class VT, int NV>
__global__ void __launch_bounds__(kNormThreads) rms_norm_adjoint_kernel(const NormAdjParams p)
{
    __shared__ float s_red[2][32];
    extern __shared__ __align__(16) float s_dw[];  // [rows][D] where a CTA has several rows
    const int tpr = p.tpr, rows = blockDim.x / tpr, row = threadIdx.x / tpr;
    const int lane = threadIdx.x % tpr;
    const long long D = p.D, step = (long long)gridDim.x * rows;
    const int left = int(D) - 8 * lane;
    P8 dw[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k].v[j] = twice(0.f);
    Raw8<YT> ry[NV];
    Raw8<VT> rv[NV], rd[NV];
    float rstd = 0.f;
    auto load = [&](long long t) {
        if (t >= p.T) return;
        rstd = __ldg(p.rstd + t);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long c = t * D + 8 * (lane + k * tpr);
            if (8 * k * tpr < left) {
                ry[k].load(p.dy, c);
                rv[k].load(p.v, c);
                if (p.dv) rd[k].load(p.dv, c);
            }
        }
    };
    // four vectors a thread leave no registers for a second row's loads
    constexpr bool kAhead = NV <= 2;
    int turn = 0;
    long long t0 = (long long)blockIdx.x * rows;
    if (kAhead) load(t0 + row);
    for (; t0 < p.T; t0 += step, turn ^= 1) {
        const long long t = t0 + row, base = t * D;
        const bool live = t < p.T;
        if (!kAhead) load(t);
        const float rs = live ? rstd : 0.f;
        P8 g[NV], n[NV], d[NV];
        float2 gn2 = twice(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            g[k] = pairs(ry[k]);
            n[k] = pairs(rv[k]);
            if (p.dv) d[k] = pairs(rd[k]);
        }
        if (kAhead) load(t + step);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (live && 8 * k * tpr < left) {
                Raw8<float> rw;
                rw.load(p.w, 8 * (lane + k * tpr));
                const P8 w = pairs(rw);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[k].v[j] = __fmul2_rn(n[k].v[j], twice(rs));
                    dw[k].v[j] = __ffma2_rn(g[k].v[j], n[k].v[j], dw[k].v[j]);
                    g[k].v[j] = __fmul2_rn(g[k].v[j], w.v[j]);
                    gn2 = __ffma2_rn(g[k].v[j], n[k].v[j], gn2);
                }
            }
        }
        // two buffers in turn: a warp may be a row ahead of one still summing
        const float mean = row_sum(gn2.x + gn2.y, tpr, s_red[turn]) / float(D);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (live && 8 * k * tpr < left) {
                P8 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o.v[j] = __ffma2_rn(n[k].v[j], twice(-mean), g[k].v[j]);
                    o.v[j] = p.dv ? __ffma2_rn(twice(rs), o.v[j], d[k].v[j]) : __fmul2_rn(twice(rs), o.v[j]);
                }
                store8(p.dx, base + 8 * (lane + k * tpr), sizeof(VT) == 2, o);
            }
        }
    }
    if (rows > 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (8 * k * tpr < left) store8(s_dw, row * D + 8 * (lane + k * tpr), false, dw[k]);
        __syncthreads();
        for (long long c = threadIdx.x; c < D; c += blockDim.x) {
            float a = 0.f;
            for (int r = 0; r < rows; ++r) a += s_dw[r * D + c];
            p.part[(long long)blockIdx.x * D + c] = a;
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (8 * k * tpr < left) store8(p.part, (long long)blockIdx.x * D + 8 * (lane + k * tpr), false, dw[k]);
    }
}

// ------------------------------------------------------- 8-bit quantisation

// One scale per row and 128 columns: 16 lanes a block, 8 columns a lane.  A CTA
// takes 2^shift vectors of 8 columns of kQuantRows times 256 / 2^shift rows, so
// no thread has to divide for its place, and asks for all of its vectors first.
constexpr int kQuantRows = 2;
template <class XT>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const void* x, uint8_t* q, float* scale, long long M,
                                                                long long K, long long KB, int shift)
{
    const int rows = 256 >> shift;
    const long long m0 = (long long)blockIdx.x * (kQuantRows * rows) + (threadIdx.x >> shift);
    const long long c = 8ll * (((long long)blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1)));
    Raw8<XT> r[kQuantRows];
#pragma unroll
    for (int i = 0; i < kQuantRows; ++i)
        if (m0 + i * rows < M && c < K) r[i].load(x, (m0 + i * rows) * K + c);
#pragma unroll
    for (int i = 0; i < kQuantRows; ++i) {
        const long long m = m0 + i * rows;
        const bool in = m < M && c < K;
        P8 v = {{twice(0.f), twice(0.f), twice(0.f), twice(0.f)}};
        if (in) v = pairs(r[i]);
        const float sc = scale_of(max16(amax8(v)));
        if (in) {
            *reinterpret_cast<uint2*>(q + m * K + c) = pack_e4m3x8(quotients(v, sc));
            if ((threadIdx.x & 15) == 0) scale[m * KB + c / 128] = sc;
        }
    }
}

// One scale per 128 rows and 128 columns: a CTA a block, kept in registers.
template <class XT>
__global__ void __launch_bounds__(512) fp8_quantize_blocks_kernel(const void* x, uint8_t* q, float* scale, long long M,
                                                                  long long K, long long KB)
{
    __shared__ float s_max[16];
    const long long mb = blockIdx.x / KB, kb = blockIdx.x - mb * KB;
    const long long c = kb * 128 + 8 * (threadIdx.x & 15), m0 = mb * 128 + (threadIdx.x >> 4);
    Raw8<XT> r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m0 + 32 * i < M && c < K) r[i].load(x, (m0 + 32 * i) * K + c);
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m0 + 32 * i < M && c < K) most = max_keep_nan(most, amax8(pairs(r[i])));
    most = max16(most);
    most = max_keep_nan(most, __shfl_xor_sync(0xffffffffu, most, 16));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) most = max_keep_nan(most, s_max[i]);
    const float sc = scale_of(most);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m0 + 32 * i < M && c < K)
            *reinterpret_cast<uint2*>(q + (m0 + 32 * i) * K + c) = pack_e4m3x8(quotients(pairs(r[i]), sc));
    if (threadIdx.x == 0) scale[blockIdx.x] = sc;
}

}  // namespace pararnn
