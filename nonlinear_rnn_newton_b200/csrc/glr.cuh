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

#include <type_traits>

#include "fp8.cuh"  // bounded waits counted in clocks

namespace pararnn {

// ------------------------------------------------------------------ numerics

// s(x) = 1 / (1 + e^-x) takes a reciprocal of its own: e^-x = inf then gives
// exactly 0, so a gate at the type's lowest value (or -inf) is shut and not
// nearly shut.
//
// p = 1 - e^-l for l >= 0: below 1/8 from its series up to l^5 (the first term
// left out is l^6/720, 4e-8 of the value), since 1 - ex2.approx would keep
// only the bits of e^-l below 1: at l = 1e-3, a common decay, four digits.

// Pairs of neighbouring channels: the packed fp32 instructions of this
// architecture take both at once.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg(float2 x) { return make_float2(-x.x, -x.y); }

__device__ __forceinline__ float2 logistic(float2 x)
{
    const float2 y = __fmul2_rn(x, both(-kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2_approx(y.x), ex2_approx(y.y)), both(1.0f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
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

// -l = -s sr, a = e^-l, nq = a^2 - 1
struct Decay2 {
    float2 nl, a, nq;
};

// nrate: the rates' negatives.  Near: every rate of the warp is below 1/8, so l <=
// rate is too and the far branch (with its special-function use) is left out.
// Loops over rows are built for both: a branch in each row would keep the rows'
// arithmetic from overlapping.  One fast channel makes its slab's warps take the
// far branch: scan B8 L4096 D1024 95 against 88 us, adjoint B4 L8192 D2048 355
// against 309.  The far branch takes a from the exponential
// itself: 1 + (a - 1) would keep only the bits of a small a above 2^-24, and the
// gradients of fast decays are multiples of a.
template <bool Near>
__device__ __forceinline__ Decay2 glr_decay(float2 sr, float2 nrate)
{
    Decay2 g;
    g.nl = __fmul2_rn(nrate, sr);
    float2 np = __ffma2_rn(g.nl, both(1.0f / 120), both(1.0f / 24));  // a - 1 = -p
    np = __ffma2_rn(g.nl, np, both(1.0f / 6));
    np = __ffma2_rn(g.nl, np, both(0.5f));
    np = __ffma2_rn(g.nl, np, both(1.0f));
    np = __fmul2_rn(g.nl, np);
    g.a = __fadd2_rn(np, both(1.0f));
    if constexpr (!Near) {
        const float2 y = __fmul2_rn(g.nl, both(kLog2e));
        const float2 ex = make_float2(ex2_approx(y.x), ex2_approx(y.y)), far = __fadd2_rn(ex, both(-1.0f));
        const bool sx = g.nl.x > -0.125f, sy = g.nl.y > -0.125f;
        g.a = make_float2(sx ? g.a.x : ex.x, sy ? g.a.y : ex.y);
        np = make_float2(sx ? np.x : far.x, sy ? np.y : far.y);
    }
    g.nq = __fmul2_rn(np, __fadd2_rn(np, both(2.0f)));
    return g;
}

// a and b = m s(i) x of one row
template <bool Near>
__device__ __forceinline__ void glr_row(float2 r, float2 i, float2 x, float2 nrate, float2& a, float2& b)
{
    const Decay2 g = glr_decay<Near>(logistic(r), nrate);
    a = g.a;
    b = __fmul2_rn(__fmul2_rn(make_float2(sqrt_approx(-g.nq.x), sqrt_approx(-g.nq.y)), logistic(i)), x);
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
        if (starts[mid] <= t) lo = mid;
        else hi = mid;
    }
    if (lo < 0 || lo >= n_seq) return r;
    r.owner = lo;
    r.first = max(starts[lo], 0) == t;
    r.last = min(starts[lo + 1], T) == t + 1;
    return r;
}

constexpr int kGD = 64;        // channels of a slab
constexpr int kGMaxP = 33;     // most CTAs of a slab

// Sequences without rows: `out` gets `in` (or zeros).  The computing warps (W a
// CTA) of the grid share them, 32 a look.
template <int W>
__device__ __forceinline__ void copy_empty(const int* starts, int T, int n_seq, long long D, const float* in, float* out)
{
    if (!starts || !out) return;
    const int lane = threadIdx.x & 31;
    for (long long s0 = 32ll * (blockIdx.x * W + (threadIdx.x >> 5)); s0 < n_seq; s0 += 32ll * W * gridDim.x) {
        bool empty = false;
        if (s0 + lane < n_seq) {
            const int lo = min(max(__ldg(starts + s0 + lane), 0), T);
            empty = min(max(__ldg(starts + s0 + lane + 1), lo), T) == lo;
        }
        for (unsigned left = __ballot_sync(0xffffffffu, empty); left; left &= left - 1) {
            const long long at = (s0 + __ffs(left) - 1) * D;
            for (long long d = 4 * lane; d < D; d += 128)
                *reinterpret_cast<float4*>(out + at + d) =
                    in ? *reinterpret_cast<const float4*>(in + at + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
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
// fixed order of operations (the same bits every run).
//
// Ten warps of a CTA compute: warp w takes rows w kRows .. of a tile, lane l
// channels 2 l and 2 l + 1.  They fold one tile (scan) or two (adjoint) ahead
// of the tile that they run through, so that the way of a map to the other CTAs
// and of theirs to here, about 2 us under load, passes behind their work.  Two
// more warps take the tiles in turn: they load them (TMA), join the warps'
// maps, publish, look up the others' and hand each warp the state entering its
// rows; with one such warp its own trips to L2 set the pace (adjoint B4 L16384
// D2048: 0.83 against 0.60 ms).
//
// The scan keeps a and b of the folded rows in registers (12 rows a warp, 4
// registers each, twice) and so gives a stage back at once; the adjoint keeps
// s(r) and the upstream gradients and reads the rest again.  Measured at B1
// L65536 D2048, bf16, scan: 12 rows a warp and one tile ahead 0.311 ms; 6 rows
// and two ahead 0.331; 14 warps of 9 rows 0.364; b kept in the stages' place
// instead 0.332.  With every channel slab a CTA's own (no maps to wait for) a
// scan runs at 5.3 TB/s, and the adjoint at 6.3.
//
// A published map needs no flag: the maps' memory starts as words of all ones,
// a written word is never that, and a reader takes a map when none of its
// words is.  The sign of A (a product of decays, not negative) says whether
// the tile holds a cut.

struct GlrParams {
    const float *rate, *h0;
    const int* starts;
    float *h, *h_last;                    // scan
    const float *states, *dh, *dh_last;   // adjoint
    float *du, *dh0, *part;
    long long D;
    int T, n_seq, L, S, P, tiles;
    WsHeader* hdr;
    uint4* maps;      // [tiles][S][32]: (A, B) of channel 2 l, of 2 l + 1
    unsigned long long wait_ns;
};

// One channel pair's map y -> a y + b, or y -> b (cut).
struct Map2 {
    float2 a, b;
    bool cut;
};

__device__ __forceinline__ float2 apply(const Map2& m, float2 y)
{
    return m.cut ? m.b : __ffma2_rn(m.a, y, m.b);
}

constexpr int kGStarts = 1025;  // offsets kept in shared memory

// The shared parts of both scans' shared memory behind the stages.
//
// What lets a slot be written again: a warp folds tile n + NS, and so arrives on
// its agg_full, only after it has run through tile n (NS = tiles ahead + 1), and
// that needs `entered` of tile n.  So with NS slots each of agg, cut, enter and
// their barriers, tile n + NS finds those of tile n read by every warp, without
// a wait of its own; fewer of enter would be written while a late warp reads.
// own and passed go between the control warps alone: the one of tile n + 2
// waits for tile n + 1's, which comes after its look at tile n's.
constexpr int kGMaxStages = 5;
template <int W, int NS>  // computing warps, folded tiles at a time
struct GlrShared {
    float4 agg[NS][W][32];  // the warps' maps of the CTA's tile n, at n % NS
    float2 enter[NS][W][32];  // the state entering each warp's rows, at n % NS
    int cut[NS][W];
    uint64_t full[kGMaxStages], empty[kGMaxStages];
    float2 own[2][32];            // the state that tile n ended with, at n % 2
    uint64_t agg_full[NS], entered[NS], passed[2];
    int starts[kGStarts];         // the sequences' offsets, where they fit
};

// The sequences' offsets go to shared memory if there are few enough: a search
// in global memory (some trips to L2 one after another) at every new sequence
// took a tenth of the time at T 16384, 37 sequences (adjoint, D 1024: 112 us
// against 84 for one sequence; 101 with the copy).  A barrier must follow.
__device__ __forceinline__ bool starts_fit(int n_seq) { return n_seq + 1 <= kGStarts; }

template <class Shared>
__device__ __forceinline__ void keep_starts(Shared& sh, const int* starts, int n_seq)
{
    if (!starts || !starts_fit(n_seq)) return;
    for (int i = threadIdx.x; i <= n_seq; i += blockDim.x) sh.starts[i] = __ldg(starts + i);
}

template <int W, int NS>
__device__ __forceinline__ void glr_init(GlrShared<W, NS>& sh)
{
    for (int i = 0; i < kGMaxStages; ++i) {
        mbar_init(&sh.full[i], 1);
        mbar_init(&sh.empty[i], W);
    }
    for (int i = 0; i < NS; ++i) {
        mbar_init(&sh.agg_full[i], W);
        mbar_init(&sh.entered[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sh.passed[i], 1);
    fence_mbar_init();
}

// The bits of a published word: never all ones.
__device__ __forceinline__ unsigned map_word(float x)
{
    const unsigned u = __float_as_uint(x);
    return x != x ? 0x7fc00000u : u;
}

__device__ __forceinline__ uint4 ld_map(const uint4* p)
{
    uint4 v;
    asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <bool Reverse, int W, int NS>
__device__ __forceinline__ Map2 warp_map(const GlrShared<W, NS>& sh, int n, int i, int lane)
{
    const int w = Reverse ? W - 1 - i : i;  // the warp that comes i-th
    const float4 v = sh.agg[n % NS][w][lane];
    return Map2{make_float2(v.x, v.z), make_float2(v.y, v.w), sh.cut[n % NS][w] != 0};
}

// The control warp, with the warps' maps of tile k (the CTA's n-th) in shared
// memory: joins them and publishes the tile's map.
template <bool Reverse, int W, int NS>
__device__ __forceinline__ void glr_publish(const GlrParams& p, const GlrShared<W, NS>& sh, int slab, int k, int n, int lane)
{
    Map2 all = warp_map<Reverse>(sh, n, 0, lane);
#pragma unroll
    for (int i = 1; i < W; ++i) {
        const Map2 m = warp_map<Reverse>(sh, n, i, lane);
        all.b = apply(m, all.b);
        all.a = __fmul2_rn(m.a, all.a);
        all.cut |= m.cut;
    }
    uint4 out = make_uint4(map_word(all.a.x), map_word(all.b.x), map_word(all.a.y), map_word(all.b.y));
    out.x = all.cut ? out.x | 0x80000000u : out.x & 0x7fffffffu;
    asm volatile("st.relaxed.gpu.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p.maps + (size_t(k) * p.S + slab) * 32 + lane),
                 "r"(out.x), "r"(out.y), "r"(out.z), "r"(out.w)
                 : "memory");
}

// Maps of `cnt` tiles (as many as eight are taken), `step` apart, once all of
// them are there.  False when the wait ran out.
__device__ __forceinline__ bool look_up(const uint4* from, size_t step, int cnt, uint4 (&v)[8], int* err, uint64_t limit_ns)
{
    long long t0 = 0;
    for (;;) {
        bool there = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < cnt ? ld_map(from + j * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) there = there && v[j].x != ~0u && v[j].y != ~0u && v[j].z != ~0u && v[j].w != ~0u;
        if (__all_sync(0xffffffffu, there)) return true;
        if (t0 == 0) t0 = clock64();
        if (__any_sync(0xffffffffu, clock64() - t0 > (long long)(2 * limit_ns))) {
            raise_error(err, PARARNN_ERR_TIMEOUT);
            return false;
        }
    }
}

// Self test: a look at maps that nobody publishes gives up.
__global__ void selftest_look_up_kernel(const uint4* maps, int* err, unsigned long long limit_ns)
{
    uint4 v[8];
    if (!look_up(maps + threadIdx.x, 32, 3, v, err, limit_ns)) give_up();
}

// Then the state entering tile k, from the one the CTA's tile before ended with
// (the other control warp passes it on), and from it the state entering each
// warp's rows.  False when a wait ran out.
template <bool Reverse, int W, int NS>
__device__ __forceinline__ bool glr_carry(const GlrParams& p, GlrShared<W, NS>& sh, int slab, int k, int n, int lane)
{
    // the tiles since this CTA's last one (all of them in its first turn)
    const int first = max(k - p.P + 1, 0), cnt = p.P > 1 ? k - first : 0;
    const uint4* from = p.maps + (size_t(first) * p.S + slab) * 32 + lane;
    Map2 all{both(1.f), both(0.f), false};
    for (int i = 0; i < cnt; i += 8) {
        uint4 v[8];
        if (!look_up(from + size_t(i) * p.S * 32, size_t(p.S) * 32, cnt - i, v, &p.hdr->error, p.wait_ns)) return false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (i + j < cnt) {
                const Map2 m{make_float2(__uint_as_float(v[j].x & 0x7fffffffu), __uint_as_float(v[j].z)),
                             make_float2(__uint_as_float(v[j].y), __uint_as_float(v[j].w)), (v[j].x >> 31) != 0};
                all.b = apply(m, all.b);
                all.a = __fmul2_rn(m.a, all.a);
                all.cut |= m.cut;
            }
        }
    }
    float2 own = both(0.f);
    if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait_clocked(&sh.passed[(n - 1) & 1], uint32_t((n - 1) >> 1) & 1u, &p.hdr->error,
                                                       p.wait_ns)))
            return false;
        own = sh.own[(n - 1) & 1][lane];
    }
    if (cnt) own = apply(all, own);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        sh.enter[n % NS][Reverse ? W - 1 - i : i][lane] = own;
        own = apply(warp_map<Reverse>(sh, n, i, lane), own);
    }
    sh.own[n & 1][lane] = own;
    __syncwarp();
    if (lane == 0) {
        mbar_arrive(&sh.passed[n & 1]);
        mbar_arrive(&sh.entered[n % NS]);
    }
    return true;
}

template <class UT>
__device__ __forceinline__ float2 pair_of(const UT* p)
{
    const FV<2> v = loadv<2>(p);
    return make_float2(v.v[0], v.v[1]);
}

// What a warp has to know of its rows: bit i for row i, the owners in the lanes.
struct RowMasks {
    unsigned firsts, lasts, mine;
    int owner;
    // rows within one sequence, none its first or last
    __device__ __forceinline__ bool plain() const { return (firsts | lasts | ~mine) == 0; }
};

// The rows strictly inside the sequence that a warp met last: tiles within them
// need no look at the sequences.
struct PlainRows {
    int lo = 0, hi = 0;  // first row behind the sequence's first, its last row
};

__device__ __forceinline__ RowMasks row_masks(const GlrParams& p, const int* kept, int t0, int rows, int lane, PlainRows& plain)
{
    RowMasks m{0u, 0u, ~0u, 0};
    if (t0 >= plain.lo && t0 + rows <= plain.hi) return m;
    const int* starts = p.starts && starts_fit(p.n_seq) ? kept : p.starts;
    const RowSeq rs = row_seq(starts, p.T, p.n_seq, p.L, lane < rows ? t0 + lane : -1);
    m.firsts = __ballot_sync(0xffffffffu, rs.first);
    m.lasts = __ballot_sync(0xffffffffu, rs.last);
    m.mine = __ballot_sync(0xffffffffu, rs.owner >= 0) | (~0u << rows);
    m.owner = rs.owner;
    // the sequence of the last row of any
    const unsigned any = m.mine & ((1u << rows) - 1u);
    if (any) {
        const int o = __shfl_sync(0xffffffffu, rs.owner, 31 - __clz(any));
        plain.lo = (starts ? max(starts[o], 0) : o * p.L) + 1;
        plain.hi = (starts ? min(starts[o + 1], p.T) : (o + 1) * p.L) - 1;
    }
    return m;
}

template <class UT>
struct GlrScanLayout {
    static constexpr int kWarps = 10;  // that compute; two more control
    static constexpr int kThreads = 32 * (kWarps + 2);
    static constexpr int kAhead = 1, kSets = kAhead + 1;  // tiles folded ahead of the one run through
    static constexpr int kRows = sizeof(UT) == 2 ? 12 : 6;  // of a warp
    static constexpr int kStages = 4;
    static constexpr int kTile = kRows * kWarps;
    static constexpr size_t stage_bytes = size_t(kTile) * 3 * kGD * sizeof(UT);
    static constexpr size_t smem_bytes = kStages * stage_bytes + sizeof(GlrShared<kWarps, kSets>) + 128;
    static_assert(smem_bytes <= 232448, "shared memory");
};

template <class UT>
__global__ void __launch_bounds__(GlrScanLayout<UT>::kThreads, 1)
    glr_scan_kernel(const __grid_constant__ CUtensorMap tm_u, const GlrParams p)
{
    using LY = GlrScanLayout<UT>;
    constexpr int R = LY::kRows, W = LY::kWarps, NS = LY::kSets, ahead = LY::kAhead;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
    GlrShared<W, NS>& sh = *reinterpret_cast<GlrShared<W, NS>*>(smem + LY::kStages * LY::stage_bytes);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slab = blockIdx.x % p.S, turn = blockIdx.x / p.S;
    const int d = slab * kGD + 2 * lane;
    const bool in = d < p.D;
    const int mine = turn < p.tiles ? (p.tiles - 1 - turn) / p.P + 1 : 0;  // tiles turn, turn + P, ..
    int* err = &p.hdr->error;
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) clear_outcome(p.hdr);
        glr_init(sh);
    }
    keep_starts(sh, p.starts, p.n_seq);
    __syncthreads();
    bool ok = true;
    if (w >= W) {
        auto load = [&](int n) {
            const int s = n % LY::kStages;
            mbar_arrive_expect_tx(&sh.full[s], uint32_t(LY::stage_bytes));
            tma_load_3d(smem + s * LY::stage_bytes, &tm_u, slab * kGD, 0, (turn + n * p.P) * LY::kTile, &sh.full[s]);
        };
        if (w == W && lane == 0)
            for (int n = 0; n < min(mine, LY::kStages); ++n) load(n);
        // the two control warps take the tiles in turn
        for (int n = w - W; n < mine && ok; n += 2) {
            ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.agg_full[n % NS], uint32_t(n / NS) & 1u, err, p.wait_ns));
            if (!ok) break;
            if (p.P > 1) glr_publish<false>(p, sh, slab, turn + n * p.P, n, lane);
            if (lane == 0 && n + LY::kStages < mine) load(n + LY::kStages);  // every warp has read the stage
            ok = glr_carry<false>(p, sh, slab, turn + n * p.P, n, lane);
        }
    } else {
        const float2 nrate = in ? neg(pair_of(p.rate + d)) : both(0.f);
        const bool near = __all_sync(0xffffffffu, nrate.x > -0.125f && nrate.y > -0.125f);
        PlainRows plain;
        // fold tile n: its rows' a and b into registers, the warp's map out
        auto fold = [&](int n, float2(&a)[R], float2(&b)[R], RowMasks& rm) {
            const int s = n % LY::kStages;
            rm = row_masks(p, sh.starts, (turn + n * p.P) * LY::kTile + w * R, R, lane, plain);
            ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.full[s], uint32_t(n / LY::kStages) & 1u, err, p.wait_ns));
            const UT* src = reinterpret_cast<const UT*>(smem + s * LY::stage_bytes) + size_t(w) * R * 3 * kGD + 2 * lane;
            auto rows = [&](auto is_near) {
#pragma unroll
                for (int i = 0; i < R; ++i)
                    glr_row<decltype(is_near)::value>(pair_of(src + i * 3 * kGD), pair_of(src + (i * 3 + 1) * kGD),
                                                      pair_of(src + (i * 3 + 2) * kGD), nrate, a[i], b[i]);
            };
            if (near) rows(std::true_type());
            else rows(std::false_type());
            float2 A = both(1.f), B = both(0.f);
            if (rm.firsts == 0) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    B = __ffma2_rn(a[i], B, b[i]);
                    A = __fmul2_rn(A, a[i]);
                }
            } else {  // the states before the sequences that start here; what came before is cut
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const bool cut = (rm.firsts >> i) & 1u;
                    const long long o = __shfl_sync(0xffffffffu, rm.owner, i);
                    if (cut && p.h0 && in) b[i] = __ffma2_rn(a[i], pair_of(p.h0 + o * p.D + d), b[i]);
                    B = apply(Map2{a[i], b[i], cut}, B);
                    A = __fmul2_rn(A, a[i]);
                }
            }
            sh.agg[n % NS][w][lane] = make_float4(A.x, B.x, A.y, B.y);
            if (lane == 0) sh.cut[n % NS][w] = rm.firsts != 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.agg_full[n % NS]);
        };
        // run through tile n from the state entering this warp's rows
        auto finish = [&](int n, const float2(&a)[R], const float2(&b)[R], const RowMasks& rm) {
            ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.entered[n % NS], uint32_t(n / NS) & 1u, err, p.wait_ns));
            if (!ok) return;
            const int t0 = (turn + n * p.P) * LY::kTile + w * R;
            float2 y = sh.enter[n % NS][w][lane];
            float* h = p.h + (long long)t0 * p.D + d;
            if (rm.plain()) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    y = __ffma2_rn(a[i], y, b[i]);
                    if (in) *reinterpret_cast<float2*>(h) = y;
                    h += p.D;
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                y = apply(Map2{a[i], b[i], ((rm.firsts >> i) & 1u) != 0}, y);
                if (in && ((rm.mine >> i) & 1u)) *reinterpret_cast<float2*>(h) = y;
                h += p.D;
                if ((rm.lasts >> i) & 1u) {
                    const long long o = __shfl_sync(0xffffffffu, rm.owner, i);
                    if (p.h_last && in) *reinterpret_cast<float2*>(p.h_last + o * p.D + d) = y;
                }
            }
        };
        float2 a[NS][R], b[NS][R];
        RowMasks rm[NS];
        if (mine > 0) fold(0, a[0], b[0], rm[0]);
        if (ahead > 1 && mine > 1 && ok) fold(1, a[1], b[1], rm[1]);
        for (int n = 0; n < mine && ok; n += NS) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                if (n + i >= mine || !ok) break;
                if (n + i + ahead < mine) fold(n + i + ahead, a[(i + ahead) % NS], b[(i + ahead) % NS], rm[(i + ahead) % NS]);
                if (ok) finish(n + i, a[i], b[i], rm[i]);
            }
        }
        copy_empty<W>(p.starts, p.T, p.n_seq, p.D, p.h0, p.h_last);
    }
    if (!ok) give_up();
}

template <class UT>
struct GlrAdjointLayout {
    static constexpr int kWarps = 10;  // that compute; two more control
    static constexpr int kThreads = 32 * (kWarps + 2);
    static constexpr int kAhead = 2, kSets = kAhead + 1;  // tiles folded ahead of the one run through
    static constexpr int kRows = sizeof(UT) == 2 ? 4 : 3;  // of a warp
    static constexpr int kStages = 5;
    static constexpr int kTile = kRows * kWarps;
    static constexpr size_t u_bytes = size_t(kTile) * 3 * kGD * sizeof(UT), f_bytes = size_t(kTile) * kGD * 4;
    static constexpr size_t stage_bytes = u_bytes + 2 * f_bytes;
    static constexpr size_t smem_bytes = kStages * stage_bytes + sizeof(GlrShared<kWarps, kSets>) + 128;
    static_assert(smem_bytes <= 232448, "shared memory");
};

// Tiles are counted from the last row: tile k holds rows T - (k + 1) kTile ..
// T - k kTile - 1 (tile after tile towards the first row; the last tile may
// start before row 0, where there is nothing).  A stage stays until its tile
// has been run through.
template <class UT>
__global__ void __launch_bounds__(GlrAdjointLayout<UT>::kThreads, 1)
    glr_adjoint_kernel(const __grid_constant__ CUtensorMap tm_u, const __grid_constant__ CUtensorMap tm_h,
                       const __grid_constant__ CUtensorMap tm_dh, const GlrParams p)
{
    using LY = GlrAdjointLayout<UT>;
    constexpr int R = LY::kRows, W = LY::kWarps, NS = LY::kSets, ahead = LY::kAhead;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
    GlrShared<W, NS>& sh = *reinterpret_cast<GlrShared<W, NS>*>(smem + LY::kStages * LY::stage_bytes);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slab = blockIdx.x % p.S, turn = blockIdx.x / p.S;
    const int d = slab * kGD + 2 * lane;
    const bool in = d < p.D;
    const int mine = turn < p.tiles ? (p.tiles - 1 - turn) / p.P + 1 : 0;
    int* err = &p.hdr->error;
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) clear_outcome(p.hdr);
        glr_init(sh);
    }
    keep_starts(sh, p.starts, p.n_seq);
    __syncthreads();
    bool ok = true;
    // Minus the rates' gradients: sums of terms of either sign over all of the
    // thread's rows, one or two thousand.  A tile's rows are added up, then joined
    // by compensated summation (W. Kahan, "Further remarks on reducing truncation
    // errors", 1965): 2 EPS of the terms' magnitudes however many there are.  The
    // warps' and the CTAs' sums, 10 and 33 at most, are then added plainly.
    float2 nds = both(0.f), rest = both(0.f);
    if (w >= W) {
        auto load = [&](int n) {
            const int s = n % LY::kStages, t = p.T - (turn + n * p.P + 1) * LY::kTile;
            unsigned char* to = smem + s * LY::stage_bytes;
            mbar_arrive_expect_tx(&sh.full[s], uint32_t(LY::stage_bytes));
            tma_load_3d(to, &tm_u, slab * kGD, 0, t, &sh.full[s]);
            tma_load_2d(to + LY::u_bytes, &tm_h, slab * kGD, t - 1, &sh.full[s]);  // the states before the rows
            tma_load_2d(to + LY::u_bytes + LY::f_bytes, &tm_dh, slab * kGD, t, &sh.full[s]);
        };
        if (w == W && lane == 0)
            for (int n = 0; n < min(mine, LY::kStages); ++n) load(n);
        // the two control warps take the tiles in turn
        for (int n = w - W; n < mine && ok; n += 2) {
            ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.agg_full[n % NS], uint32_t(n / NS) & 1u, err, p.wait_ns));
            if (!ok) break;
            if (p.P > 1) glr_publish<true>(p, sh, slab, turn + n * p.P, n, lane);
            // the warps run through tile n - kAhead next, and fold tile n + 1 then
            if (n >= ahead && n - ahead + LY::kStages < mine) {
                const int s = (n - ahead) % LY::kStages;
                ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.empty[s], uint32_t((n - ahead) / LY::kStages) & 1u, err, p.wait_ns));
                if (!ok) break;
                if (lane == 0) load(n - ahead + LY::kStages);
            }
            ok = glr_carry<true>(p, sh, slab, turn + n * p.P, n, lane);
        }
    } else {
        const float2 nrate = in ? neg(pair_of(p.rate + d)) : both(0.f);
        const bool near = __all_sync(0xffffffffu, nrate.x > -0.125f && nrate.y > -0.125f);
        PlainRows plain;
        // G = a (up + G of the row behind): the map of a row is (a, a up)
        auto fold = [&](int n, float2(&sr)[R], float2(&up)[R], RowMasks& rm) {
            const int s = n % LY::kStages;
            rm = row_masks(p, sh.starts, p.T - (turn + n * p.P + 1) * LY::kTile + w * R, R, lane, plain);
            ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.full[s], uint32_t(n / LY::kStages) & 1u, err, p.wait_ns));
            const unsigned char* stage = smem + s * LY::stage_bytes;
            const UT* su = reinterpret_cast<const UT*>(stage) + size_t(w) * R * 3 * kGD + 2 * lane;
            const float* sd = reinterpret_cast<const float*>(stage + LY::u_bytes + LY::f_bytes) + w * R * kGD + 2 * lane;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                sr[i] = logistic(pair_of(su + i * 3 * kGD));
                up[i] = pair_of(sd + i * kGD);
            }
            if (rm.lasts && p.dh_last) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const long long o = __shfl_sync(0xffffffffu, rm.owner, i);
                    if (((rm.lasts >> i) & 1u) && in) up[i] = __fadd2_rn(up[i], pair_of(p.dh_last + o * p.D + d));
                }
            }
            float2 A = both(1.f), B = both(0.f);
            auto rows = [&](auto is_near) {
#pragma unroll
                for (int i = R - 1; i >= 0; --i) {
                    const float2 a = glr_decay<decltype(is_near)::value>(sr[i], nrate).a;
                    const bool cut = (rm.lasts >> i) & 1u;
                    B = __fmul2_rn(a, cut ? up[i] : __fadd2_rn(up[i], B));
                    A = __fmul2_rn(A, a);
                }
            };
            if (near) rows(std::true_type());
            else rows(std::false_type());
            sh.agg[n % NS][w][lane] = make_float4(A.x, B.x, A.y, B.y);
            if (lane == 0) sh.cut[n % NS][w] = rm.lasts != 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.agg_full[n % NS]);
        };
        auto finish = [&](int n, const float2(&sr)[R], const float2(&up)[R], const RowMasks& rm) {
            ok = __all_sync(0xffffffffu, mbar_wait_clocked(&sh.entered[n % NS], uint32_t(n / NS) & 1u, err, p.wait_ns));
            if (!ok) return;
            const int s = n % LY::kStages, t0 = p.T - (turn + n * p.P + 1) * LY::kTile + w * R;
            const unsigned char* stage = smem + s * LY::stage_bytes;
            const UT* su = reinterpret_cast<const UT*>(stage) + size_t(w) * R * 3 * kGD + 2 * lane;
            const float* sb = reinterpret_cast<const float*>(stage + LY::u_bytes) + w * R * kGD + 2 * lane;
            float2 G = sh.enter[n % NS][w][lane], tile_nds = both(0.f);
            auto run = [&](auto is_near, auto is_plain) {
#pragma unroll
                for (int i = R - 1; i >= 0; --i) {
                    const float2 si = logistic(pair_of(su + (i * 3 + 1) * kGD)), x = pair_of(su + (i * 3 + 2) * kGD);
                    float2 before = pair_of(sb + i * kGD);
                    if (!decltype(is_plain)::value && ((rm.firsts >> i) & 1u)) {
                        const long long o = __shfl_sync(0xffffffffu, rm.owner, i);
                        before = p.h0 && in ? pair_of(p.h0 + o * p.D + d) : both(0.f);
                    }
                    const float2 lam = !decltype(is_plain)::value && ((rm.lasts >> i) & 1u) ? up[i] : __fadd2_rn(up[i], G);
                    const Decay2 g = glr_decay<decltype(is_near)::value>(sr[i], nrate);
                    G = __fmul2_rn(g.a, lam);
                    if (!decltype(is_plain)::value && !((rm.mine >> i) & 1u)) continue;
                    // -1 / m; where l = 0 (a shut gate) the root has no slope: its terms are 0
                    const float2 nim = make_float2(g.nq.x < -1e-37f ? -rsqrt_approx(-g.nq.x) : 0.f,
                                                   g.nq.y < -1e-37f ? -rsqrt_approx(-g.nq.y) : 0.f);
                    const float2 lsi = __fmul2_rn(lam, si), lx = __fmul2_rn(lsi, x);
                    const float2 dx = __fmul2_rn(lsi, __fmul2_rn(g.nq, nim));
                    const float2 di = __fmul2_rn(__fmul2_rn(dx, x), __ffma2_rn(si, both(-1.f), both(1.f)));
                    // dl = lam (s(i) x a^2 / m - a h), negated
                    const float2 ndl = __ffma2_rn(G, before, __fmul2_rn(__fmul2_rn(lx, __fmul2_rn(g.a, g.a)), nim));
                    const float2 dr = __fmul2_rn(__fmul2_rn(ndl, g.nl), __ffma2_rn(sr[i], both(-1.f), both(1.f)));
                    tile_nds = __ffma2_rn(ndl, sr[i], tile_nds);
                    if (in) {
                        float* q = p.du + (long long)(t0 + i) * 3 * p.D + d;
                        *reinterpret_cast<float2*>(q) = dr;
                        *reinterpret_cast<float2*>(q + p.D) = di;
                        *reinterpret_cast<float2*>(q + 2 * p.D) = dx;
                    }
                    if (!decltype(is_plain)::value && ((rm.firsts >> i) & 1u)) {
                        const long long o = __shfl_sync(0xffffffffu, rm.owner, i);
                        if (p.dh0 && in) *reinterpret_cast<float2*>(p.dh0 + o * p.D + d) = G;
                    }
                }
            };
            if (__builtin_expect(near && rm.plain(), 1)) run(std::true_type(), std::true_type());
            else if (rm.plain()) run(std::false_type(), std::true_type());
            else run(std::false_type(), std::false_type());
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[s]);
            const float2 y = __fadd2_rn(tile_nds, neg(rest)), all = __fadd2_rn(nds, y);
            rest = __fadd2_rn(__fadd2_rn(all, neg(nds)), neg(y));
            // an infinite sum stays one: what is left of it is no number
            rest = make_float2(fabsf(all.x) <= 3.4e38f ? rest.x : 0.f, fabsf(all.y) <= 3.4e38f ? rest.y : 0.f);
            nds = all;
        };
        float2 sr[NS][R], up[NS][R];
        RowMasks rm[NS];
        if (mine > 0) fold(0, sr[0], up[0], rm[0]);
        if (ahead > 1 && mine > 1 && ok) fold(1, sr[1], up[1], rm[1]);
        for (int n = 0; n < mine && ok; n += NS) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                if (n + i >= mine || !ok) break;
                if (n + i + ahead < mine) fold(n + i + ahead, sr[(i + ahead) % NS], up[(i + ahead) % NS], rm[(i + ahead) % NS]);
                if (ok) finish(n + i, sr[i], up[i], rm[i]);
            }
        }
        copy_empty<W>(p.starts, p.T, p.n_seq, p.D, p.dh_last, p.dh0);
    }
    if (!ok) give_up();
    // this CTA's part of the rates' gradients, the warps in order
    __syncthreads();
    if (w < W) sh.enter[0][w][lane] = neg(nds);
    __syncthreads();
    if (w == 0 && in) {
        float2 v = sh.enter[0][0][lane];
#pragma unroll
        for (int i = 1; i < W; ++i) v = __fadd2_rn(v, sh.enter[0][i][lane]);
        *reinterpret_cast<float2*>(p.part + (long long)turn * p.D + d) = v;
    }
}

// out[d] = sum of part[k][d] over k in 0..n-1, in a fixed order: 32 columns a
// CTA, 32 interleaved runs of rows (four loads of a run in flight) joined in
// order.
constexpr int kSumRuns = 32;
__global__ void __launch_bounds__(32 * kSumRuns) column_sum_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                                   long long n, long long D)
{
    __shared__ float s[kSumRuns][33];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const long long d = (long long)blockIdx.x * 32 + c;
    float v = 0.f;
    if (d < D) {
#pragma unroll 4
        for (long long k = g; k < n; k += kSumRuns) v += __ldg(part + k * D + d);
    }
    s[g][c] = v;
    __syncthreads();
    if (g == 0 && d < D) {
#pragma unroll
        for (int k = 1; k < kSumRuns; ++k) v += s[k][c];
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
    for (int j = 0; j < 4; j += 2) {
        float2 ka, kb;
        glr_row<false>(make_float2(r.v[j], r.v[j + 1]), make_float2(g.v[j], g.v[j + 1]), make_float2(x.v[j], x.v[j + 1]),
                       make_float2(-s.v[j], -s.v[j + 1]), ka, kb);
        y.v[j] = fmaf(ka.x, y.v[j], kb.x);
        y.v[j + 1] = fmaf(ka.y, y.v[j + 1], kb.y);
    }
    store4(next + b * D + d, y.v);
}

}  // namespace pararnn
