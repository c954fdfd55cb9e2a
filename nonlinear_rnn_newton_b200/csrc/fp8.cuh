// 8-bit product with a scale for each block of 128 columns:
//   u[m][n] = sum over blocks b of xs[m][b] ws[n / 128][b] (x[m] . w[n] over
//   the 128 columns of block b)  (+ bias[n]),
// x [M][K] and w [N][K] in e4m3, one fp32 scale per row of x and per 128 rows
// of w in each block.
//
// The tensor cores (tcgen05, kind::f8f6f4) form each block's product on its
// own: the scales are any fp32 numbers, so a block's accumulator leaves
// tensor memory before the next block's scale can join, and the sum over
// blocks is kept in registers, acc += (xs ws) t.  xs ws is rounded to fp32 first.
// Where it is below 2^-126 that is off by up to 2^-150, and the term by 2^-125 (a
// block's sum is below 2^25); the interface says so.  Taking such a block's two
// factors one after the other, behind a vote of the warp, cost M 32768 N 6144
// K 2048 8 % (442 -> 477 us), and 39 % where half of the rows are zeros.  Two accumulators in tensor
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

// Whether a wait of a layer operator has run out on this device since the host
// last asked: callers may drop the workspace that holds a call's own outcome.
__device__ int g_layer_failure = 0;

// After a wait that ran out: mark the device, and give the copies in flight into
// this CTA's shared memory time to land (a copy takes microseconds) before the
// CTA ends.
__device__ __forceinline__ void give_up()
{
    raise_error(&g_layer_failure, PARARNN_ERR_TIMEOUT);
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
}

// Self test: a wait on a barrier that nothing arrives on gives up.
__global__ void selftest_clocked_wait_kernel(int* err, unsigned long long limit_ns)
{
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (!mbar_wait_clocked(&bar, 0, err, limit_ns)) give_up();
    __syncthreads();
    if (threadIdx.x == 0) mbar_inval(&bar);
}

// 16 consecutive fp32 columns of this warp's 32 TMEM lanes (one per thread)
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
// products (in the leading CTA), 4..19 read the accumulators, a row a thread
// and 64 columns a warp: 64 running sums and two loads of 16 columns in
// registers, for which the other warps hand theirs over (setmaxnreg: 128 x 32
// + 512 x 112 = 640 x 96, what the kernel is launched with).
//
// What bounds it: reading and scaling the accumulators.  M 32768 N 6144 K 2048
// takes 448 us (1.84 PFLOP/s, 1.1 of a bf16 product's measured peak); the same
// kernel that only multiplies, without waiting for its accumulators to be read,
// takes 333.  Eight reading warps of 128 columns: 474 us; products of 128
// columns with four accumulators: 500; one CTA with 128 x 256 tiles: 472.
constexpr int kQM = 128;       // rows of x a CTA (256 a pair)
constexpr int kQN = 256;       // columns of a pair's tile
constexpr int kQEpi = 16;                // warps that read accumulators
constexpr int kQCols = kQN * 4 / kQEpi;  // columns a warp
constexpr int kQChunk = 16;              // of which a load brings this many
constexpr int kQThreads = 32 * (4 + kQEpi);
constexpr int kQAhead = 4;     // blocks that a thread fetches its scales ahead
constexpr int kQStages = 5;
constexpr size_t kQStageBytes = size_t(kQM + kQN / 2) * kQK;
constexpr size_t kQOut = kQStages * kQStageBytes;  // 4 KB a reading warp
constexpr size_t kQBar = kQOut + kQEpi * 4096;
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

// the stores issued so far have read their shared memory
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// A warp's 32 rows x 64 columns of sums, a row a thread, to rows m0 and columns
// n0 of u: by pieces of 128 bytes a row through 4 KB of shared memory in the
// 128-byte swizzle (16-byte piece i of row r at i ^ (r % 8): eight rows' writes
// fall in distinct banks) and a bulk store of the piece.  Writing the rows from registers, 16 bytes a row and instruction,
// took 250 of 650 us at M 32768, N 6144, K 2048.
template <bool Bf16>
__device__ __forceinline__ void store_sums(const Fp8Params& p, const CUtensorMap* tm_u, unsigned char* stage, int m0,
                                           int n0, int lane, const float2 (&acc)[kQCols / 2])
{
    constexpr int kCols = Bf16 ? 64 : 32;  // columns of a piece
    constexpr int kPer = kCols / 8;        // columns of 16 bytes
#pragma unroll
    for (int c = 0; c < kQCols; c += kCols) {
        if (n0 + c >= p.N) break;
        if (lane == 0) tma_store_wait_read();  // the piece before has left
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2* v = acc + (c + i * kPer) / 2;
            uint4 o;
            if constexpr (Bf16)
                o = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                               pack_bf16x2(v[3].x, v[3].y));
            else
                o = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                               __float_as_uint(v[1].y));
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = o;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) tma_store_2d(tm_u, stage, n0 + c, m0);
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
            mbar_init(&tempty[i], 2 * kQEpi);
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(32));
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(112));
        const int lq = w & 3, part = (w >> 2) - 1;
        const uint32_t ta = tmem + (uint32_t(32 * lq) << 16) + uint32_t(part) * kQCols;
        unsigned char* out = smem + kQOut + (w - 4) * 4096;
        int q = 0;
        for (int t = pair; t < p.n_tiles && ok; t += pairs) {
            const int tm = t / p.tiles_n, tn = t - tm * p.tiles_n;
            const long long m = (long long)tm * 2 * kQM + rank * kQM + 32 * lq + lane;
            const long long n = (long long)tn * kQN + part * kQCols;
            const bool in = m < p.M && n < p.N;
            const float* xs = p.xs + m * p.KB;
            const float* ws = p.ws + n / 128 * p.KB;
            float2 acc[kQCols / 2];  // from the bias on
#pragma unroll
            for (int j = 0; j < kQCols; j += 4) {
                float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p.bias && n + j < p.N) bias = __ldg(reinterpret_cast<const float4*>(p.bias + n + j));
                acc[j / 2] = make_float2(bias.x, bias.y);
                acc[j / 2 + 1] = make_float2(bias.z, bias.w);
            }
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
                float v[2][kQChunk];
                const uint32_t tb = ta + uint32_t(q & 1) * kQN;
                constexpr int kChunks = kQCols / kQChunk;
                tmem_ld(tb, v[0]);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    tmem_wait_ld();
                    if (c + 1 < kChunks) tmem_ld(tb + kQChunk * (c + 1), v[(c + 1) & 1]);
                    if (c + 1 == kChunks) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa(&tempty[b], 0));
                    }
#pragma unroll
                    for (int j = 0; j < kQChunk; j += 2) {
                        float2& s = acc[(kQChunk * c + j) / 2];
                        s = __ffma2_rn(make_float2(v[c & 1][j], v[c & 1][j + 1]), make_float2(sc, sc), s);
                    }
                }
            }
            if (ok) {
                const int m0 = tm * 2 * kQM + int(rank) * kQM + 32 * lq;
                if (m0 < p.M && n < p.N) {
                    if (p.u_bf16) store_sums<true>(p, &tm_u, out, m0, int(n), lane, acc);
                    else store_sums<false>(p, &tm_u, out, m0, int(n), lane, acc);
                }
            }
        }
        if (lane == 0) tma_store_wait_read();
    }
    if (!ok) give_up();
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
// M 16 N 6144 K 2048 takes 6.6 us of which its 12.6 MB need 1.9; N 2048 K 8192
// 8.2 us (16.8 MB, 2.6 us): the launch, the first loads' way and the cluster's
// two meetings are about 5 us.
constexpr int kNThreads = 32 * 6;
constexpr int kNScaleBlocks = 16;  // blocks whose scales are in shared memory at a time

template <int NT>
struct NarrowLayout {
    static constexpr size_t stage_bytes = size_t(128 + NT) * kQK;
    static constexpr int kStages = NT >= 64 ? 4 : 5;  // two CTAs fit on an SM
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

    float2 acc[NT / 2];
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) acc[j] = make_float2(0.f, 0.f);

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
                    float2* s = acc + (16 * c + j) / 2;
                    s[0] = __ffma2_rn(make_float2(v[j], v[j + 1]), make_float2(s4.x, s4.y), s[0]);
                    s[1] = __ffma2_rn(make_float2(v[j + 2], v[j + 3]), make_float2(s4.z, s4.w), s[1]);
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
            for (int j = 0; j < NT; ++j) red[j * 128 + 32 * lq + lane] = j & 1 ? acc[j / 2].y : acc[j / 2].x;
        }
    }
    if (!ok) give_up();
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
