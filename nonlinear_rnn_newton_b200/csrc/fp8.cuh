// 8-bit product with a scale for each block of 128 columns:
//   u[m][n] = sum over blocks b of xs[m][b] ws[n / 128][b] (x[m] . w[n] over
//   the 128 columns of block b)  (+ bias[n]),
// x [M][K] and w [N][K] in e4m3, one fp32 scale per row of x and per 128 rows
// of w in each block.
//
// The tensor cores (tcgen05, kind::f8f6f4) form each block's product on its
// own: the scales are any fp32 numbers, so a block's accumulator leaves
// tensor memory before the next block's scale can join, and the sum over
// blocks is kept in registers, acc += (xs ws) t.  Two accumulators in tensor
// memory let the next block's product run while this one is read.
//
// A block is one 128-byte row of the 128-byte swizzle: a stage holds one
// block of every row of the tile, and four products of K = 32 read it.
#pragma once

#include "norm.cuh"
#include "project.cuh"  // tcgen05 wrappers, smem_desc_sw128

namespace pararnn {

constexpr int kQK = 128;  // columns (bytes) of a block

// kind::f8f6f4: fp32 accumulator, e4m3 A and B, both K-major
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// ------------------------------------------------- PTX of one CTA and of pairs

template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* dst_smem, uint32_t ncols)
{
    if constexpr (CG == 1) {
        tmem_alloc(dst_smem, ncols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)),
                     "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t ncols)
{
    if constexpr (CG == 1) tmem_dealloc(taddr, ncols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

template <int CG>
__device__ __forceinline__ void umma_e4m3(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate)
{
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
            : "memory");
}

// arrive on the barrier at this offset in both CTAs of the pair once every
// product issued so far is done
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(uint16_t(3))
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// the shared::cluster address of this CTA's `p` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t mapa(const void* p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Arrives on a barrier of the cluster without ordering this thread's memory
// accesses: what it announces is that registers have been read from tensor
// memory (tcgen05.wait::ld, tcgen05.fence::before_thread_sync).  The releasing
// form waits for every outstanding access first, and stalled the reading warps
// for more than the product took.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Bounded wait on a barrier of this CTA (arrivals may come from the cluster).
// The limit is counted in SM clocks, whose reading costs less than that of
// %globaltimer: a wait here often finds its barrier not ready.
__device__ __forceinline__ bool mbar_wait_clocked(uint64_t* bar, uint32_t parity, int* err, uint64_t limit_ns)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > (long long)(2 * limit_ns)) {  // an SM clock is about half a nanosecond
            raise_error(err, PARARNN_ERR_TIMEOUT);
            return false;
        }
    }
}

// A tiled load into this CTA's shared memory that completes on a barrier of
// either CTA of the pair (no multicast).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* tm, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(tm), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// After a wait that ran out: give the copies in flight into this CTA's shared
// memory time to land (a copy takes microseconds) before the CTA ends.
__device__ __forceinline__ void let_copies_land()
{
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
}

// 32 consecutive fp32 columns of this warp's 32 TMEM lanes (one per thread)
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 of them
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// (a0, a1) + s (t0, t1) in one packed instruction
__device__ __forceinline__ void fma2(float& a0, float& a1, float t0, float t1, float s0, float s1)
{
    asm("{\n\t.reg .b64 a, t, s;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 t, {%2, %3};\n\t"
        "mov.b64 s, {%4, %5};\n\t"
        "fma.rn.f32x2 a, t, s, a;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(t0), "f"(t1), "f"(s0), "f"(s1));
}

struct Fp8Params {
    const float *xs, *ws, *bias;
    void* u;
    long long M, N, K;
    int KB, n_tiles, tiles_n;
    int u_bf16;
    int splits;  // CTAs of a cluster that share a tile's blocks (narrow form)
    WsHeader* hdr;
    unsigned long long wait_ns;
};

// The outcome starts as OK; a wait that runs out does so seconds later.
__device__ __forceinline__ void clear_outcome(WsHeader* hdr)
{
    hdr->error = 0;
    hdr->passes = 0;
    hdr->result.status = PARARNN_OK;
    hdr->result.iters = 0;
    hdr->result.residual = 0.f;
    hdr->result.residual0 = 0.f;
}

// ------------------------------------------------------------------ wide form
//
// Many rows: a pair of CTAs (cta_group::2, M = 256, N = 256) owns a tile of 256
// rows x 256 columns; each CTA loads its 128 rows of x and 128 of the 256 rows
// of w and ends up with its own rows' sums.  Warps: 0 loads, 1 issues the
// products (in the leading CTA), 4..11 read the accumulators, a row a thread
// and 128 columns a warp: 128 running sums and two loads of 32 columns in
// registers, for which the other warps hand theirs over (setmaxnreg: 128 x 40
// + 256 x 232 = 384 x 168, what the kernel is launched with).
constexpr int kQM = 128;       // rows of x a CTA (256 a pair)
constexpr int kQN = 256;       // columns of a pair's tile
constexpr int kQThreads = 384;
constexpr int kQAhead = 4;     // blocks that a thread fetches its scales ahead
constexpr int kQStages = 5;
constexpr size_t kQStageBytes = size_t(kQM + kQN / 2) * kQK;
constexpr size_t kQOut = kQStages * kQStageBytes;  // 2 x 4 KB a reading warp
constexpr size_t kQBar = kQOut + 8 * 8192;
constexpr size_t kQSmem = kQBar + (2 * kQStages + 4) * 8 + 16 + 1024;
static_assert(kQSmem <= 232448, "shared memory");

// Stores a tile of this CTA's shared memory (written by the generic proxy,
// fenced) to a tensor; rows and columns beyond it are clipped.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, const void* src, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tm), "r"(c0),
                 "r"(c1), "r"(smem_addr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// all but the last `Left` stores issued have read their shared memory
template <int Left>
__device__ __forceinline__ void tma_store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(Left) : "memory");
}

// A warp's 32 rows x 128 columns of sums, a row a thread, to rows m0 and
// columns n0 of u: by pieces of 128 bytes a row through 4 KB of shared memory
// (two in turn) in the 128-byte swizzle (16-byte piece i of row r at i ^ (r %
// 8): eight rows' writes fall in distinct banks) and a bulk store of the
// piece.  Writing the rows from registers, 16 bytes a row and instruction,
// took 250 of 650 us at M 32768, N 6144, K 2048.  Lane l holds the bias of
// columns 4 l .. 4 l + 3.
template <bool Bf16>
__device__ __forceinline__ void store_sums(const Fp8Params& p, const CUtensorMap* tm_u, unsigned char* stage, int m0,
                                           int n0, int lane, float4 bias, float (&acc)[128])
{
    constexpr int kCols = Bf16 ? 64 : 32;  // columns of a piece
    constexpr int kPer = kCols / 8;        // columns of 16 bytes
    if (p.bias) {
#pragma unroll
        for (int j = 0; j < 128; j += 4) {
            acc[j] += __shfl_sync(0xffffffffu, bias.x, j / 4);
            acc[j + 1] += __shfl_sync(0xffffffffu, bias.y, j / 4);
            acc[j + 2] += __shfl_sync(0xffffffffu, bias.z, j / 4);
            acc[j + 3] += __shfl_sync(0xffffffffu, bias.w, j / 4);
        }
    }
#pragma unroll
    for (int c = 0; c < 128; c += kCols) {
        if (n0 + c >= p.N) break;
        unsigned char* buf = stage + (c / kCols & 1) * 4096;
        if (lane == 0) tma_store_wait_read<1>();  // the piece before the last has left
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* v = acc + c + i * kPer;
            uint4 o;
            if constexpr (Bf16)
                o = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                               pack_bf16x2(v[6], v[7]));
            else
                o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) = o;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) tma_store_2d(tm_u, buf, n0 + c, m0);
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kQThreads, 1)
    fp8_project_wide_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                            const __grid_constant__ CUtensorMap tm_u, const Fp8Params p)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kQBar);  // the leading CTA's: both CTAs' loads
    uint64_t* empty = full + kQStages;                           // each CTA's: the products that read a stage are done
    uint64_t* tfull = empty + kQStages;                          // [2] each CTA's: an accumulator is written
    uint64_t* tempty = tfull + 2;                                // [2] the leading CTA's: both CTAs have read it
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + 2);

    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    int* err = &p.hdr->error;
    bool ok = true;

    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) clear_outcome(p.hdr);
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * 8);
        }
        fence_mbar_init();
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_w);
    }
    if (w == 0) tmem_alloc_cg<2>(s_tmem, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (w < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (w == 0 && lane == 0) {
            int q = 0;
            for (int t = pair; t < p.n_tiles && ok; t += pairs) {
                const int tm = t / p.tiles_n, tn = t - tm * p.tiles_n;
                for (int kb = 0; kb < p.KB; ++kb, ++q) {
                    const int s = q % kQStages;
                    if (q >= kQStages && !mbar_wait_clocked(&empty[s], uint32_t(q / kQStages - 1) & 1u, err, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    unsigned char* sp = smem + s * kQStageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], uint32_t(2 * kQStageBytes));
                    const uint32_t bar = mapa(&full[s], 0);
                    tma_load_2d_pair(sp, &tm_x, kb * kQK, tm * 2 * kQM + int(rank) * kQM, bar);
                    tma_load_2d_pair(sp + kQM * kQK, &tm_w, kb * kQK, tn * kQN + int(rank) * (kQN / 2), bar);
                }
            }
        } else if (w == 1 && lane == 0 && rank == 0) {
            constexpr uint32_t kIdesc = idesc_e4m3(2 * kQM, kQN);
            int q = 0;
            for (int t = pair; t < p.n_tiles && ok; t += pairs) {
                for (int kb = 0; kb < p.KB && ok; ++kb, ++q) {
                    const int s = q % kQStages;
                    const int b = q & 1;
                    if ((q >= 2 && !mbar_wait_clocked(&tempty[b], uint32_t(q / 2 - 1) & 1u, err, p.wait_ns)) ||
                        !mbar_wait_clocked(&full[s], uint32_t(q / kQStages) & 1u, err, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const unsigned char* sp = smem + s * kQStageBytes;
                    const uint64_t ad = smem_desc_sw128(sp), bd = smem_desc_sw128(sp + kQM * kQK);
#pragma unroll
                    for (int k = 0; k < kQK / 32; ++k)  // 32 bytes apart inside the swizzle atom
                        umma_e4m3<2>(tmem + uint32_t(b) * kQN, ad + uint64_t(2 * k), bd + uint64_t(2 * k), kIdesc, k != 0);
                    umma_commit_pair(&empty[s]);
                    umma_commit_pair(&tfull[b]);
                }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int lq = w & 3, half = (w >> 2) - 1;
        const uint32_t ta = tmem + (uint32_t(32 * lq) << 16) + uint32_t(half) * 128;
        unsigned char* out = smem + kQOut + (w - 4) * 8192;
        int q = 0;
        for (int t = pair; t < p.n_tiles && ok; t += pairs) {
            const int tm = t / p.tiles_n, tn = t - tm * p.tiles_n;
            const long long m = (long long)tm * 2 * kQM + rank * kQM + 32 * lq + lane;
            const long long n = (long long)tn * kQN + half * 128;
            const bool in = m < p.M && n < p.N;
            const float* xs = p.xs + m * p.KB;
            const float* ws = p.ws + n / 128 * p.KB;
            float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.bias && n + 4 * lane < p.N) bias = __ldg(reinterpret_cast<const float4*>(p.bias + n) + lane);
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            float sx[kQAhead], sw[kQAhead];  // scales of the blocks from kb on
#pragma unroll
            for (int i = 0; i < kQAhead; ++i) {
                sx[i] = in && i < p.KB ? __ldg(xs + i) : 0.f;
                sw[i] = in && i < p.KB ? __ldg(ws + i) : 0.f;
            }
            for (int kb = 0; kb < p.KB; ++kb, ++q) {
                const int b = q & 1;
                const float sc = sx[0] * sw[0];
#pragma unroll
                for (int i = 0; i + 1 < kQAhead; ++i) {
                    sx[i] = sx[i + 1];
                    sw[i] = sw[i + 1];
                }
                const bool more = in && kb + kQAhead < p.KB;
                sx[kQAhead - 1] = more ? __ldg(xs + kb + kQAhead) : 0.f;
                sw[kQAhead - 1] = more ? __ldg(ws + kb + kQAhead) : 0.f;
                ok = __all_sync(0xffffffffu, mbar_wait_clocked(&tfull[b], uint32_t(q / 2) & 1u, err, p.wait_ns));
                if (!ok) break;
                tc_fence_after();
                float v[2][32];
                const uint32_t tb = ta + uint32_t(q & 1) * 256;
                tmem_ld(tb, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_wait_ld();
                    if (c < 3) {
                        tmem_ld(tb + 32 * (c + 1), v[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa(&tempty[b], 0));
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        { acc[32*c+j]=fmaf(v[c&1][j],sc,acc[32*c+j]); acc[32*c+j+1]=fmaf(v[c&1][j+1],sc,acc[32*c+j+1]); }
                }
            }
            if (ok) {
                const int m0 = tm * 2 * kQM + int(rank) * kQM + 32 * lq;
                if (m0 < p.M && n < p.N) {
                    if (p.u_bf16) store_sums<true>(p, &tm_u, out, m0, int(n), lane, bias, acc);
                    else store_sums<false>(p, &tm_u, out, m0, int(n), lane, bias, acc);
                }
            }
        }
        if (lane == 0) tma_store_wait_read<0>();
    }
    if (!ok) let_copies_land();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (w == 0) tmem_dealloc_cg<2>(tmem, 512);
}

// ---------------------------------------------------------------- narrow form
//
// Few rows: the weight is what has to be read, so its 128 rows are the
// accumulator's lanes and up to NT rows of x its columns (M = 128, N = NT),
// and `splits` CTAs of a cluster share the tile's blocks of K to put enough
// loads in flight.  Their sums meet in shared memory (each CTA adds a slice of
// the tile over the cluster's CTAs in rank order, so the order is fixed).
// Warps: 0 loads, 1 issues the products, 2..5 read the accumulators.
constexpr int kNThreads = 32 * 6;
constexpr int kNScaleBlocks = 16;  // blocks whose scales are in shared memory at a time

template <int NT>
struct NarrowLayout {
    static constexpr size_t stage_bytes = size_t(128 + NT) * kQK;
    static constexpr int kStages = NT >= 128 ? 6 : NT >= 64 ? 4 : 5;
    static constexpr size_t off_scale = kStages * stage_bytes;  // [kNScaleBlocks][NT] xs ws
    static constexpr size_t off_bar = off_scale + size_t(kNScaleBlocks) * NT * 4;
    static constexpr size_t smem_bytes = off_bar + (2 * kStages + 4) * 8 + 16 + 1024;
    static constexpr uint32_t tmem_cols = 2 * NT < 32 ? 32 : 2 * NT;
    static_assert(size_t(NT) * 512 <= off_scale, "the sums fit where the stages were");
};

template <int NT>
__global__ void __launch_bounds__(kNThreads)
    fp8_project_narrow_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                              const Fp8Params p)
{
    using LY = NarrowLayout<NT>;
    constexpr int S = LY::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    float* scales = reinterpret_cast<float*>(smem + LY::off_scale);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + LY::off_bar);
    uint64_t* empty = full + S;
    uint64_t* tfull = empty + S;
    uint64_t* tempty = tfull + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + 2);

    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(cluster_rank());
    const int t = blockIdx.x / p.splits;
    const int tm = t / p.tiles_n, tn = t - tm * p.tiles_n;
    const long long m0 = (long long)tm * NT, n0 = (long long)tn * 128;
    const int kb0 = int((long long)p.KB * rank / p.splits), kb1 = int((long long)p.KB * (rank + 1) / p.splits);
    int* err = &p.hdr->error;
    bool ok = true;

    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) clear_outcome(p.hdr);
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 4);
        }
        fence_mbar_init();
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_w);
    }
    if (w == 1) tmem_alloc_cg<1>(s_tmem, LY::tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    float acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = 0.f;

    if (w == 0) {
        if (lane == 0) {
            for (int q = 0; q < kb1 - kb0; ++q) {
                const int s = q % S;
                if (q >= S && !mbar_wait_clocked(&empty[s], uint32_t(q / S - 1) & 1u, err, p.wait_ns)) {
                    ok = false;
                    break;
                }
                unsigned char* sp = smem + s * LY::stage_bytes;
                mbar_arrive_expect_tx(&full[s], uint32_t(LY::stage_bytes));
                tma_load_2d(sp, &tm_w, (kb0 + q) * kQK, int(n0), &full[s]);
                tma_load_2d(sp + 128 * kQK, &tm_x, (kb0 + q) * kQK, int(m0), &full[s]);
            }
        }
    } else if (w == 1) {
        if (lane == 0) {
            constexpr uint32_t kIdesc = idesc_e4m3(128, NT);
            for (int q = 0; q < kb1 - kb0; ++q) {
                const int s = q % S, b = q & 1;
                if ((q >= 2 && !mbar_wait_clocked(&tempty[b], uint32_t(q / 2 - 1) & 1u, err, p.wait_ns)) ||
                    !mbar_wait_clocked(&full[s], uint32_t(q / S) & 1u, err, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const unsigned char* sp = smem + s * LY::stage_bytes;
                const uint64_t ad = smem_desc_sw128(sp), bd = smem_desc_sw128(sp + 128 * kQK);
#pragma unroll
                for (int k = 0; k < kQK / 32; ++k)
                    umma_e4m3<1>(tmem + uint32_t(b) * NT, ad + uint64_t(2 * k), bd + uint64_t(2 * k), kIdesc, k != 0);
                umma_commit(&empty[s]);
                umma_commit(&tfull[b]);
            }
        }
    } else {
        const int lq = w & 3, et = threadIdx.x - 64;
        const uint32_t ta = tmem + (uint32_t(32 * lq) << 16);
        const float* ws = p.ws + n0 / 128 * p.KB;
        for (int q = 0; q < kb1 - kb0; ++q) {
            const int b = q & 1;
            if (q % kNScaleBlocks == 0) {
                asm volatile("bar.sync 1, 128;" ::: "memory");  // the last batch's scales are read
                const int nb = min(kNScaleBlocks, kb1 - kb0 - q);
                for (int i = et; i < NT * kNScaleBlocks; i += 128) {
                    const int n = i / kNScaleBlocks, k = i % kNScaleBlocks;
                    if (k < nb)
                        scales[k * NT + n] =
                            m0 + n < p.M ? __ldg(p.xs + (m0 + n) * p.KB + kb0 + q + k) * __ldg(ws + kb0 + q + k) : 0.f;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            // after a wait that ran out the loop goes on without waiting: the
            // four warps share the barrier above
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_clocked(&tfull[b], uint32_t(q / 2) & 1u, err, p.wait_ns));
            tc_fence_after();
            const float* sc = scales + (q % kNScaleBlocks) * NT;
#pragma unroll
            for (int c = 0; c < NT / 16; ++c) {
                float v[16];
                tmem_ld(ta + uint32_t(b) * NT + 16 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(sc + 16 * c + j);
                    fma2(acc[16 * c + j], acc[16 * c + j + 1], v[j], v[j + 1], s4.x, s4.y);
                    fma2(acc[16 * c + j + 2], acc[16 * c + j + 3], v[j + 2], v[j + 3], s4.z, s4.w);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[b]);
        }
        // every product has read its stage: the sums take the stages' place
        float* red = reinterpret_cast<float*>(smem);
        if (ok) {
#pragma unroll
            for (int j = 0; j < NT; ++j) red[j * 128 + 32 * lq + lane] = acc[j];
        }
    }
    if (!ok) let_copies_land();
    tc_fence_before();
    __syncthreads();
    if (w == 1) tmem_dealloc_cg<1>(tmem, LY::tmem_cols);
    cluster_sync_all();
    {
        const int j0 = NT * rank / p.splits, j1 = NT * (rank + 1) / p.splits;
        const long long n = n0 + 4 * lane;
        float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.bias && n < p.N) bias = __ldg(reinterpret_cast<const float4*>(p.bias + n));
        for (int j = j0 + w; j < j1 && m0 + j < p.M; j += kNThreads / 32) {
            const float* src = reinterpret_cast<const float*>(smem) + j * 128 + 4 * lane;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < p.splits; ++r) {
                const float4 v = ld_cluster_f4(mapa(src, uint32_t(r)));
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
            if (n < p.N) {  // N is a multiple of 8
                a.x += bias.x;
                a.y += bias.y;
                a.z += bias.z;
                a.w += bias.w;
                if (p.u_bf16)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.u) + (m0 + j) * p.N + n) =
                        make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(p.u) + (m0 + j) * p.N + n) = a;
            }
        }
    }
    cluster_sync_all();  // this CTA's sums stay until every CTA has read them
}

}  // namespace pararnn
