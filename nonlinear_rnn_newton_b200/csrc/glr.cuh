// Gated linear recurrence: the diagonal linear SSM of "O compromisso que SSMs
// fizeram" (h_l = A_l h_{l-1} + B_l x_l, page "ParaRNN: Apple destrava treino
// paralelo de RNNs não-lineares e escala pra 7B parâmetros") with both terms
// gated by the input, its adjoint and its decode step.
//
// Per channel, with gates u = (r, i, x) and a rate s >= 0:
//   l = s sig(r),  a = e^-l,  p = 1 - a,  m = sqrt(1 - a^2) = sqrt(p (2 - p)),
//   h_t = a_t h_{t-1} + m_t sig(i_t) x_t.
// m keeps the state's variance at that of the input whatever the decay.
// Adjoint, lam_t = dh_t + a_{t+1} lam_{t+1}, carried as G_t = a_t lam_t so
// that a step needs its own row alone:
//   dx = lam m sig(i),  di = dx x (1 - sig(i)),
//   dl = lam (sig(i) x a^2 / m - a h_{t-1}),
//   dr = dl l (1 - sig(r)),  ds = sum dl sig(r),  dh0 = G of the first row.
#pragma once

#include "device_common.cuh"

namespace pararnn {

// ------------------------------------------------------------------ numerics

// s(x) = 1 / (1 + e^-x) with its own reciprocal: e^-x = inf gives exactly 0,
// so a gate at the type's lowest value (or -inf) is shut and not nearly shut.
__device__ __forceinline__ float logistic(float x) { return rcp_approx(1.0f + ex2_approx(-kLog2e * x)); }

// 1 - e^-l for l >= 0.  Below 1/4 from its series up to l^6 (the first term
// left out is l^7/5040, 5e-8 of the value), since 1 - ex2.approx would keep
// only the bits of e^-l below 1: at l = 1e-3, a common decay, four digits.
__device__ __forceinline__ float one_minus_exp(float l)
{
    float t = fmaf(l, -1.0f / 720, 1.0f / 120);
    t = fmaf(l, t, -1.0f / 24);
    t = fmaf(l, t, 1.0f / 6);
    t = fmaf(l, t, -0.5f);
    t = fmaf(l, t, 1.0f);
    const float far = 1.0f - ex2_approx(-kLog2e * l);
    return l < 0.25f ? l * t : far;
}

struct GlrStep {
    float sr, si, l, a, q;  // q = m^2
};

__device__ __forceinline__ GlrStep glr_gates(float r, float i, float rate)
{
    GlrStep g;
    g.sr = logistic(r);
    g.si = logistic(i);
    g.l = rate * g.sr;
    const float p = one_minus_exp(g.l);
    g.a = 1.0f - p;
    g.q = p * (2.0f - p);
    return g;
}

__device__ __forceinline__ float sqrt_approx(float x)
{
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rsqrt_approx(float x)
{
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }

// ------------------------------------------------- sequences in packed rows

// Rows [lo, hi) of sequence s among T packed rows: seq_starts[s] and [s + 1]
// held to 0..T, or equal lengths where seq_starts is NULL.
__device__ __forceinline__ void seq_rows(const int* starts, long long T, long long n_seq, long long s, long long& lo,
                                         long long& hi)
{
    if (starts) {
        lo = min(max((long long)starts[s], 0ll), T);
        hi = min(max((long long)starts[s + 1], lo), T);
    } else {
        lo = s * (T / n_seq);
        hi = lo + T / n_seq;
    }
}

// ------------------------------------------------------------------ kernels

template <class UT>
__global__ void __launch_bounds__(64) glr_scan_seq_kernel(const UT* __restrict__ u, const float* __restrict__ rate,
                                                          const float* __restrict__ h0, const int* __restrict__ starts,
                                                          float* __restrict__ h, float* __restrict__ h_last,
                                                          long long T, long long n_seq, long long D)
{
    const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= n_seq * D) return;
    const long long s = c / D, d = c - s * D;
    long long lo, hi;
    seq_rows(starts, T, n_seq, s, lo, hi);
    float y = h0 ? h0[c] : 0.f;
    const float sp = rate[d];
    for (long long t = lo; t < hi; ++t) {
        const UT* p = u + t * 3 * D + d;
        const GlrStep g = glr_gates(widen(p[0]), widen(p[D]), sp);
        y = fmaf(g.a, y, sqrt_approx(g.q) * g.si * widen(p[2 * D]));
        h[t * D + d] = y;
    }
    if (h_last) h_last[c] = y;
}

struct GlrGrad {
    float dr, di, dx, ds;
};

__device__ __forceinline__ GlrGrad glr_grad(const GlrStep& g, float x, float before, float lam)
{
    // where l = 0 (a shut gate) the square root has no slope: its term is 0
    const float im = g.q > 1e-37f ? rsqrt_approx(g.q) : 0.f;
    GlrGrad o;
    o.dx = lam * (g.q * im) * g.si;
    o.di = o.dx * x * (1.0f - g.si);
    const float dl = lam * (g.si * x * (g.a * g.a * im) - g.a * before);
    o.dr = dl * g.l * (1.0f - g.sr);
    o.ds = dl * g.sr;
    return o;
}

template <class UT>
__global__ void __launch_bounds__(64)
    glr_adjoint_seq_kernel(const UT* __restrict__ u, const float* __restrict__ rate, const float* __restrict__ h0,
                           const int* __restrict__ starts, const float* __restrict__ h, const float* __restrict__ dh,
                           const float* __restrict__ dh_last, float* __restrict__ du, float* __restrict__ dh0,
                           float* __restrict__ part, long long T, long long n_seq, long long D)
{
    const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= n_seq * D) return;
    const long long s = c / D, d = c - s * D;
    long long lo, hi;
    seq_rows(starts, T, n_seq, s, lo, hi);
    float G = dh_last ? dh_last[c] : 0.f, ds = 0.f;
    const float sp = rate[d];
    for (long long t = hi - 1; t >= lo; --t) {
        const UT* p = u + t * 3 * D + d;
        const float x = widen(p[2 * D]);
        const GlrStep g = glr_gates(widen(p[0]), widen(p[D]), sp);
        const float before = t > lo ? h[(t - 1) * D + d] : h0 ? h0[c] : 0.f;
        const float lam = dh[t * D + d] + G;
        const GlrGrad o = glr_grad(g, x, before, lam);
        float* q = du + t * 3 * D + d;
        q[0] = o.dr;
        q[D] = o.di;
        q[2 * D] = o.dx;
        ds += o.ds;
        G = g.a * lam;
    }
    if (dh0) dh0[c] = G;
    part[c] = ds;
}

// out[d] = sum of part[k][d] over k in 0..n-1, in a fixed order: 32 columns a
// CTA, 8 interleaved runs of rows joined in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                         long long n, long long D)
{
    __shared__ float s[8][33];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const long long d = (long long)blockIdx.x * 32 + c;
    float v = 0.f;
    if (d < D)
        for (long long k = g; k < n; k += 8) v += part[k * D + d];
    s[g][c] = v;
    __syncthreads();
    if (g == 0 && d < D) {
#pragma unroll
        for (int k = 1; k < 8; ++k) v += s[k][c];
        out[d] = v;
    }
}

// One step for B sequences: four channels a thread, as the solves' cells'
// decode step; every input is read before the state is written.
template <class UT>
__global__ void __launch_bounds__(256) glr_step_kernel(const UT* __restrict__ u, const float* __restrict__ rate,
                                                       const float* prev, float* next, long long B, long long D)
{
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long D4 = D >> 2;
    if (i >= B * D4) return;
    const long long b = i / D4, d = (i - b * D4) << 2;
    const F4 r = load4(u + b * 3 * D + d), g = load4(u + (b * 3 + 1) * D + d), x = load4(u + (b * 3 + 2) * D + d);
    const F4 s = load4(rate + d);
    F4 y = {{0.f, 0.f, 0.f, 0.f}};
    if (prev) y = load4(prev + b * D + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const GlrStep k = glr_gates(r.v[j], g.v[j], s.v[j]);
        y.v[j] = fmaf(k.a, y.v[j], sqrt_approx(k.q) * k.si * x.v[j]);
    }
    store4(next + b * D + d, y.v);
}

}  // namespace pararnn
