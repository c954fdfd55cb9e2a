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

#include "fp8.cuh"  // bounded waits counted in clocks

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

// from sr = s(r)
__device__ __forceinline__ GlrStep glr_open(float sr, float i, float rate)
{
    GlrStep g;
    g.sr = sr;
    g.si = logistic(i);
    g.l = rate * g.sr;
    const float p = one_minus_exp(g.l);
    g.a = 1.0f - p;
    g.q = p * (2.0f - p);
    return g;
}

__device__ __forceinline__ GlrStep glr_gates(float r, float i, float rate) { return glr_open(logistic(r), i, rate); }

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

// ------------------------------------------------- sequences in packed rows

// The sequence that row t belongs to, or -1, and whether t is its first or its
// last row.  Offsets are held to 0..T.  Without offsets: equal lengths.
struct RowSeq {
    int owner;
    bool first, last;
};

__device__ __forceinline__ RowSeq row_seq(const int* starts, int T, int n_seq, int L, int t)
{
    RowSeq r{-1, false, false};
    if (t < 0 || t >= T) return r;
    if (!starts) {
        r.owner = t / L;
        r.first = t == r.owner * L;
        r.last = t + 1 == (r.owner + 1) * L;
        return r;
    }
    // the last sequence that starts at or before t (empty ones end there too)
    int lo = -1, hi = n_seq + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(starts + mid) <= t) lo = mid;
        else hi = mid;
    }
    if (lo < 0 || lo >= n_seq) return r;
    r.owner = lo;
    r.first = max(__ldg(starts + lo), 0) == t;
    r.last = min(__ldg(starts + lo + 1), T) == t + 1;
    return r;
}

// Sequences without rows: `out` gets `in` (or zeros).  The CTAs of the grid
// share them.
__device__ __forceinline__ void copy_empty(const int* starts, int T, int n_seq, long long D, const float* in, float* out)
{
    if (!starts || !out) return;
    for (int s = blockIdx.x; s < n_seq; s += gridDim.x) {
        const int lo = min(max(__ldg(starts + s), 0), T);
        if (min(max(__ldg(starts + s + 1), lo), T) > lo) continue;
        for (long long d = threadIdx.x; d < D; d += blockDim.x) out[s * D + d] = in ? in[s * D + d] : 0.f;
    }
}

// ------------------------------------------------------------------ the scans
//
// Both scans run over the packed rows as one line of T rows, whatever the
// sequences: a sequence's first row (for the adjoint: its last) takes its
// state from h0 (dh_last) and cuts what came before.  Cut means selected, not
// multiplied by 0, so nothing non-finite gets across.
//
// A slab of 64 channels belongs to P CTAs, which take its tiles of rows in
// turn.  A tile's rows fold to one affine map a channel (A, B), which does not
// depend on the state entering it, so a CTA publishes its tile's map as soon
// as it has read the tile, and finds the state entering its next tile by
// applying the P - 1 maps of the tiles between to the state that its own last
// tile ended with: no chain of CTAs waiting for one another's states, and a
// fixed order of operations (the same bits every run).  Warp w of a CTA takes
// rows w kRows .. of a tile, lane l channels 2 l and 2 l + 1.

constexpr int kGD = 64;        // channels of a slab
constexpr int kGWarps = 8;
constexpr int kGThreads = 32 * kGWarps;
constexpr int kGMaxP = 33;     // CTAs of a slab: one lane for each of the others

struct GlrParams {
    const float *rate, *h0;
    const int* starts;
    float *h, *h_last;                    // scan
    const float *states, *dh, *dh_last;   // adjoint
    float *du, *dh0, *part;
    long long D;
    int T, n_seq, L, S, P, tiles;
    WsHeader* hdr;
    unsigned* flags;  // [tiles][S]: 0, or 1 + whether the tile holds a cut
    float4* maps;     // [tiles][S][32]: (A, B) of channel 2 l, of 2 l + 1
    unsigned long long wait_ns;
};

// One channel pair's map y -> A y + B, or y -> B (cut).
struct Map2 {
    float2 a, b;
    bool cut;
};

__device__ __forceinline__ float2 apply(const Map2& m, float2 y)
{
    return m.cut ? m.b : make_float2(fmaf(m.a.x, y.x, m.b.x), fmaf(m.a.y, y.y, m.b.y));
}

// The shared parts of both scans' shared memory behind the stages.
struct GlrShared {
    float4 agg[kGWarps][32];   // the warps' maps
    float2 enter[kGWarps][32]; // the state entering each warp's rows
    int cut[kGWarps];
    int failed;
    uint64_t full[2];
};

// Warp 0, after the warps' maps are in sh.agg: the tile's map to the other
// CTAs, the state entering the tile, and from it that entering each warp's
// rows.  `own` is the state the CTA's last tile ended with; it becomes this
// tile's.  W(i) is the warp that comes i-th in the scan's direction.
template <bool Reverse>
__device__ __forceinline__ void glr_carry(const GlrParams& p, GlrShared& sh, int slab, int k, int lane, float2& own)
{
    auto warp_at = [](int i) { return Reverse ? kGWarps - 1 - i : i; };
    Map2 m[kGWarps];
#pragma unroll
    for (int i = 0; i < kGWarps; ++i) {
        const float4 v = sh.agg[warp_at(i)][lane];
        m[i] = Map2{make_float2(v.x, v.z), make_float2(v.y, v.w), sh.cut[warp_at(i)] != 0};
    }
    bool ok = true;
    if (p.P > 1) {
        Map2 all = m[0];
#pragma unroll
        for (int i = 1; i < kGWarps; ++i) {
            all.b = apply(m[i], all.b);
            all.a = make_float2(m[i].a.x * all.a.x, m[i].a.y * all.a.y);
            all.cut |= m[i].cut;
        }
        const size_t at = size_t(k) * p.S + slab;
        __stcg(p.maps + at * 32 + lane, make_float4(all.a.x, all.b.x, all.a.y, all.b.y));
        __threadfence();
        __syncwarp();
        if (lane == 0)
            asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p.flags + at), "r"(all.cut ? 2u : 1u) : "memory");
        // the tiles since this CTA's last one (all of them in its first turn)
        const int first = max(k - p.P + 1, 0), n = k - first;
        unsigned f = 1;
        if (lane < n) {
            const unsigned* q = p.flags + size_t(first + lane) * p.S + slab;
            f = ld_acquire_gpu_u32(q);
            if (f == 0) {
                const long long t0 = clock64();
                while ((f = ld_acquire_gpu_u32(q)) == 0) {
                    if (clock64() - t0 > (long long)(2 * p.wait_ns) || error_raised(&p.hdr->error)) {
                        raise_error(&p.hdr->error, PARARNN_ERR_TIMEOUT);
                        break;
                    }
                }
            }
        }
        ok = __all_sync(0xffffffffu, f != 0);
        const unsigned cuts = __ballot_sync(0xffffffffu, lane < n && f == 2);
        if (ok) {
            // nothing before the last cut matters
            int i = cuts ? 31 - __clz(cuts) : 0;
            for (; i < n; i += 8) {
                float4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i + j < n) v[j] = __ldcg(p.maps + (size_t(first + i + j) * p.S + slab) * 32 + lane);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i + j < n)
                        own = apply(Map2{make_float2(v[j].x, v[j].z), make_float2(v[j].y, v[j].w),
                                         ((cuts >> (i + j)) & 1u) != 0},
                                    own);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kGWarps; ++i) {
        sh.enter[warp_at(i)][lane] = own;
        own = apply(m[i], own);
    }
    if (lane == 0 && !ok) sh.failed = 1;
}

template <class UT>
__device__ __forceinline__ float2 pair_of(const UT* p)
{
    const FV<2> v = loadv<2>(p);
    return make_float2(v.v[0], v.v[1]);
}

template <class UT>
struct GlrScanLayout {
    static constexpr int kRows = sizeof(UT) == 2 ? 16 : 8;  // of a warp
    static constexpr int kTile = kRows * kGWarps;
    static constexpr size_t stage_bytes = size_t(kTile) * 3 * kGD * sizeof(UT);
    static constexpr size_t smem_bytes = 2 * stage_bytes + sizeof(GlrShared) + 128;
};

template <class UT>
__global__ void __launch_bounds__(kGThreads, 2) glr_scan_kernel(const __grid_constant__ CUtensorMap tm_u, const GlrParams p)
{
    using LY = GlrScanLayout<UT>;
    constexpr int R = LY::kRows;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
    GlrShared& sh = *reinterpret_cast<GlrShared*>(smem + 2 * LY::stage_bytes);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slab = blockIdx.x % p.S, turn = blockIdx.x / p.S;
    const int d = slab * kGD + 2 * lane;
    const bool in = d < p.D;
    if (threadIdx.x == 0) {
        if (p.P == 1 && blockIdx.x == 0) clear_outcome(p.hdr);
        sh.failed = 0;
        mbar_init(&sh.full[0], 1);
        mbar_init(&sh.full[1], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto load = [&](int k, int s) {
        mbar_arrive_expect_tx(&sh.full[s], uint32_t(LY::stage_bytes));
        tma_load_3d(smem + s * LY::stage_bytes, &tm_u, slab * kGD, 0, k * LY::kTile, &sh.full[s]);
    };
    if (threadIdx.x == 0) {
        if (turn < p.tiles) load(turn, 0);
        if (turn + p.P < p.tiles) load(turn + p.P, 1);
    }
    copy_empty(p.starts, p.T, p.n_seq, p.D, p.h0, p.h_last);
    const float2 rate = in ? pair_of(p.rate + d) : make_float2(0.f, 0.f);
    float2 own = make_float2(0.f, 0.f);  // warp 0's: the state this CTA's last tile ended with
    bool ok = true;
    int n = 0;
    for (int k = turn; k < p.tiles; k += p.P, ++n) {
        const int s = n & 1, t0 = k * LY::kTile + w * R;
        // this warp's rows: lane i looks at row i
        const RowSeq rs = row_seq(p.starts, p.T, p.n_seq, p.L, lane < R ? t0 + lane : -1);
        const unsigned firsts = __ballot_sync(0xffffffffu, rs.first), lasts = __ballot_sync(0xffffffffu, rs.last);
        const unsigned mine = __ballot_sync(0xffffffffu, rs.owner >= 0);
        ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.full[s], uint32_t(n >> 1) & 1u, &p.hdr->error, p.wait_ns));
        const UT* src = reinterpret_cast<const UT*>(smem + s * LY::stage_bytes) + size_t(w) * R * 3 * kGD + 2 * lane;
        float2 a[R], b[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 r = pair_of(src + i * 3 * kGD), g = pair_of(src + (i * 3 + 1) * kGD),
                         x = pair_of(src + (i * 3 + 2) * kGD);
            const GlrStep g0 = glr_gates(r.x, g.x, rate.x), g1 = glr_gates(r.y, g.y, rate.y);
            a[i] = make_float2(g0.a, g1.a);
            b[i] = make_float2(sqrt_approx(g0.q) * g0.si * x.x, sqrt_approx(g1.q) * g1.si * x.y);
        }
        if (firsts) {  // the states before the sequences that start here
#pragma unroll
            for (int i = 0; i < R; ++i)
                if ((firsts >> i) & 1u) {
                    const long long o = __shfl_sync(0xffffffffu, rs.owner, i);
                    if (p.h0 && in) {
                        const float2 h = pair_of(p.h0 + o * p.D + d);
                        b[i] = make_float2(fmaf(a[i].x, h.x, b[i].x), fmaf(a[i].y, h.y, b[i].y));
                    }
                }
        }
        float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool cut = (firsts >> i) & 1u;
            B = apply(Map2{a[i], b[i], cut}, B);
            A = make_float2(A.x * a[i].x, A.y * a[i].y);
        }
        sh.agg[w][lane] = make_float4(A.x, B.x, A.y, B.y);
        if (lane == 0) sh.cut[w] = firsts != 0;
        ok = !__syncthreads_or(!ok);  // the stage is read, the maps are there
        if (!ok) break;
        if (threadIdx.x == 0 && k + 2 * p.P < p.tiles) load(k + 2 * p.P, s);
        if (w == 0) glr_carry<false>(p, sh, slab, k, lane, own);
        __syncthreads();
        if (sh.failed) {  // written between the two barriers alone
            ok = false;
            break;
        }
        float2 y = sh.enter[w][lane];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            y = apply(Map2{a[i], b[i], ((firsts >> i) & 1u) != 0}, y);
            if (in && ((mine >> i) & 1u)) *reinterpret_cast<float2*>(p.h + (long long)(t0 + i) * p.D + d) = y;
            if ((lasts >> i) & 1u) {
                const long long o = __shfl_sync(0xffffffffu, rs.owner, i);
                if (p.h_last && in) *reinterpret_cast<float2*>(p.h_last + o * p.D + d) = y;
            }
        }
    }
    if (!ok) let_copies_land();
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
struct GlrAdjointLayout {
    static constexpr int kRows = sizeof(UT) == 2 ? 7 : 5;  // of a warp: two CTAs of two stages on an SM
    static constexpr int kTile = kRows * kGWarps;
    static constexpr size_t u_bytes = size_t(kTile) * 3 * kGD * sizeof(UT), f_bytes = size_t(kTile) * kGD * 4;
    static constexpr size_t stage_bytes = u_bytes + 2 * f_bytes;
    static constexpr size_t smem_bytes = 2 * stage_bytes + sizeof(GlrShared) + 128;
};

// Tiles are counted from the last row: tile k holds rows T - (k + 1) kTile ..
// T - k kTile - 1 (tile after tile towards the first row; the last tile may
// start before row 0, where there is nothing).  The stage stays until the
// second sweep has read it again.
template <class UT>
__global__ void __launch_bounds__(kGThreads, 2)
    glr_adjoint_kernel(const __grid_constant__ CUtensorMap tm_u, const __grid_constant__ CUtensorMap tm_h,
                       const __grid_constant__ CUtensorMap tm_dh, const GlrParams p)
{
    using LY = GlrAdjointLayout<UT>;
    constexpr int R = LY::kRows;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
    GlrShared& sh = *reinterpret_cast<GlrShared*>(smem + 2 * LY::stage_bytes);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slab = blockIdx.x % p.S, turn = blockIdx.x / p.S;
    const int d = slab * kGD + 2 * lane;
    const bool in = d < p.D;
    if (threadIdx.x == 0) {
        if (p.P == 1 && blockIdx.x == 0) clear_outcome(p.hdr);
        sh.failed = 0;
        mbar_init(&sh.full[0], 1);
        mbar_init(&sh.full[1], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto load = [&](int k, int s) {
        unsigned char* to = smem + s * LY::stage_bytes;
        const int t = p.T - (k + 1) * LY::kTile;
        mbar_arrive_expect_tx(&sh.full[s], uint32_t(LY::stage_bytes));
        tma_load_3d(to, &tm_u, slab * kGD, 0, t, &sh.full[s]);
        tma_load_2d(to + LY::u_bytes, &tm_h, slab * kGD, t - 1, &sh.full[s]);  // the states before the rows
        tma_load_2d(to + LY::u_bytes + LY::f_bytes, &tm_dh, slab * kGD, t, &sh.full[s]);
    };
    if (threadIdx.x == 0) {
        if (turn < p.tiles) load(turn, 0);
        if (turn + p.P < p.tiles) load(turn + p.P, 1);
    }
    copy_empty(p.starts, p.T, p.n_seq, p.D, p.dh_last, p.dh0);
    const float2 rate = in ? pair_of(p.rate + d) : make_float2(0.f, 0.f);
    float2 own = make_float2(0.f, 0.f), ds = make_float2(0.f, 0.f);
    bool ok = true;
    int n = 0;
    for (int k = turn; k < p.tiles; k += p.P, ++n) {
        const int s = n & 1, t0 = p.T - (k + 1) * LY::kTile + w * R;
        const RowSeq rs = row_seq(p.starts, p.T, p.n_seq, p.L, lane < R ? t0 + lane : -1);
        const unsigned firsts = __ballot_sync(0xffffffffu, rs.first), lasts = __ballot_sync(0xffffffffu, rs.last);
        const unsigned mine = __ballot_sync(0xffffffffu, rs.owner >= 0);
        ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.full[s], uint32_t(n >> 1) & 1u, &p.hdr->error, p.wait_ns));
        const unsigned char* stage = smem + s * LY::stage_bytes;
        const UT* su = reinterpret_cast<const UT*>(stage) + size_t(w) * R * 3 * kGD + 2 * lane;
        const float* sb = reinterpret_cast<const float*>(stage + LY::u_bytes) + w * R * kGD + 2 * lane;
        const float* sd = reinterpret_cast<const float*>(stage + LY::u_bytes + LY::f_bytes) + w * R * kGD + 2 * lane;
        // G = a (up + G of the row behind): the map of a row is (a, a up)
        float2 sr[R], up[R];
        float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            const float2 r = pair_of(su + i * 3 * kGD);
            sr[i] = make_float2(logistic(r.x), logistic(r.y));
            up[i] = pair_of(sd + i * kGD);
            const bool cut = (lasts >> i) & 1u;
            if (cut && p.dh_last) {
                const long long o = __shfl_sync(0xffffffffu, rs.owner, i);
                if (in) {
                    const float2 e = pair_of(p.dh_last + o * p.D + d);
                    up[i] = make_float2(up[i].x + e.x, up[i].y + e.y);
                }
            }
            const float2 a = make_float2(1.0f - one_minus_exp(rate.x * sr[i].x), 1.0f - one_minus_exp(rate.y * sr[i].y));
            B = apply(Map2{a, make_float2(a.x * up[i].x, a.y * up[i].y), cut}, B);
            A = make_float2(A.x * a.x, A.y * a.y);
        }
        sh.agg[w][lane] = make_float4(A.x, B.x, A.y, B.y);
        if (lane == 0) sh.cut[w] = lasts != 0;
        ok = !__syncthreads_or(!ok);
        if (!ok) break;
        if (w == 0) glr_carry<true>(p, sh, slab, k, lane, own);
        __syncthreads();
        if (sh.failed) {
            ok = false;
            break;
        }
        float2 G = sh.enter[w][lane];
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            const float2 g = pair_of(su + (i * 3 + 1) * kGD), x = pair_of(su + (i * 3 + 2) * kGD);
            float2 before = pair_of(sb + i * kGD);
            if ((firsts >> i) & 1u) {
                const long long o = __shfl_sync(0xffffffffu, rs.owner, i);
                before = p.h0 && in ? pair_of(p.h0 + o * p.D + d) : make_float2(0.f, 0.f);
            }
            const bool cut = (lasts >> i) & 1u;
            const float2 lam = cut ? up[i] : make_float2(up[i].x + G.x, up[i].y + G.y);
            const GlrStep s0 = glr_open(sr[i].x, g.x, rate.x), s1 = glr_open(sr[i].y, g.y, rate.y);
            G = make_float2(s0.a * lam.x, s1.a * lam.y);
            if (!((mine >> i) & 1u)) continue;
            const GlrGrad o0 = glr_grad(s0, x.x, before.x, lam.x), o1 = glr_grad(s1, x.y, before.y, lam.y);
            ds.x += o0.ds;
            ds.y += o1.ds;
            if (in) {
                float* q = p.du + (long long)(t0 + i) * 3 * p.D + d;
                *reinterpret_cast<float2*>(q) = make_float2(o0.dr, o1.dr);
                *reinterpret_cast<float2*>(q + p.D) = make_float2(o0.di, o1.di);
                *reinterpret_cast<float2*>(q + 2 * p.D) = make_float2(o0.dx, o1.dx);
            }
            if ((firsts >> i) & 1u) {
                const long long o = __shfl_sync(0xffffffffu, rs.owner, i);
                if (p.dh0 && in) *reinterpret_cast<float2*>(p.dh0 + o * p.D + d) = G;
            }
        }
        __syncthreads();  // the stage is read
        if (threadIdx.x == 0 && k + 2 * p.P < p.tiles) load(k + 2 * p.P, s);
    }
    if (!ok) let_copies_land();
    // this CTA's part of the rates' gradients, the warps in order
    __syncthreads();
    sh.enter[w][lane] = ds;
    __syncthreads();
    if (w == 0 && in) {
        float2 v = sh.enter[0][lane];
#pragma unroll
        for (int i = 1; i < kGWarps; ++i) {
            v.x += sh.enter[i][lane].x;
            v.y += sh.enter[i][lane].y;
        }
        *reinterpret_cast<float2*>(p.part + (long long)turn * p.D + d) = v;
    }
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
