// Host side of the layer operators: the gated linear recurrence, the RMS norm
// and the 8-bit product -- argument checks, workspace layouts and launches.
// Included at the end of pararnn_capi.cu: it uses that file's helpers (fail,
// TRY, check_ptr, the tensor-map encoder, resident_grid, ...).
#pragma once

#include "fp8.cuh"
#include "glr.cuh"
#include "norm.cuh"

namespace {

constexpr double kMaxBytes = 1099511627776.0;  // 2^40

size_t dtype_bytes(pararnn_dtype dt) { return dt == PARARNN_F32 ? 4 : dt == PARARNN_BF16 ? 2 : 1; }

pararnn_status check_wide_dtype(pararnn_dtype dt, const char* name)
{
    if (dt != PARARNN_F32 && dt != PARARNN_BF16)
        return fail(PARARNN_ERR_INVALID_ARG, "%s must be PARARNN_F32 or PARARNN_BF16 (got %d)", name, int(dt));
    return PARARNN_OK;
}

// do the byte ranges [x, x + nx) and [y, y + ny) meet?
bool meet(const void* x, size_t nx, const void* y, size_t ny)
{
    if (!x || !y) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return a < b + ny && b < a + nx;
}

struct Range {
    const char* name;
    const void* p;
    size_t bytes;
};

// no output (nor the workspace, where there is one) may meet an input or another
// output; `in_place`: where an output may be the very buffer of an input
template <int NI, int NO>
pararnn_status check_apart(const Range (&in)[NI], const Range (&out)[NO], const void* in_place,
                           const Range& space = Range{"workspace", nullptr, 0})
{
    for (int j = 0; j < NI; ++j)
        if (meet(in[j].p, in[j].bytes, space.p, space.bytes))
            return fail(PARARNN_ERR_INVALID_ARG, "workspace overlaps input %s", in[j].name);
    for (int j = 0; j < NO; ++j)
        if (meet(out[j].p, out[j].bytes, space.p, space.bytes))
            return fail(PARARNN_ERR_INVALID_ARG, "workspace overlaps output %s", out[j].name);
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (meet(in[j].p, in[j].bytes, out[i].p, out[i].bytes) &&
                !(in_place && out[i].p == in_place && in[j].p == in_place && in[j].bytes == out[i].bytes))
                return fail(PARARNN_ERR_INVALID_ARG, "output %s overlaps input %s", out[i].name, in[j].name);
        for (int j = 0; j < i; ++j)
            if (meet(out[j].p, out[j].bytes, out[i].p, out[i].bytes))
                return fail(PARARNN_ERR_INVALID_ARG, "outputs %s and %s overlap", out[j].name, out[i].name);
    }
    return PARARNN_OK;
}

pararnn_status launched()
{
    CUDA_TRY(cudaGetLastError());
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return PARARNN_OK;
}

// ------------------------------------------------ gated linear recurrence

pararnn_status glr_shape(long long T, long long n_seq, long long D, const void* starts)
{
    if (T < 1 || n_seq < 1 || D < 1)
        return fail(PARARNN_ERR_INVALID_ARG, "T, n_seq, D must be >= 1 (got %lld, %lld, %lld)", T, n_seq, D);
    if (D % 8 != 0) return fail(PARARNN_ERR_UNSUPPORTED, "D must be a multiple of 8 (got %lld)", D);
    if (T > INT_MAX / 2 || n_seq > INT_MAX / 2 || D > INT_MAX / 2)
        return fail(PARARNN_ERR_INVALID_ARG, "dimension too large");
    if ((double)T * (double)D * 12.0 >= kMaxBytes || (double)n_seq * (double)D * 4.0 >= kMaxBytes)
        return fail(PARARNN_ERR_INVALID_ARG, "T*D or n_seq*D too large (arrays must stay below 2^40 bytes)");
    if (!starts && T % n_seq != 0)
        return fail(PARARNN_ERR_INVALID_ARG, "without seq_starts T must be a multiple of n_seq (got %lld, %lld)", T, n_seq);
    return PARARNN_OK;
}

pararnn_status check_starts(const void* starts)
{
    if (starts && (reinterpret_cast<uintptr_t>(starts) & 3u) != 0)
        return fail(PARARNN_ERR_INVALID_ARG, "seq_starts is not 4-byte aligned");
    return PARARNN_OK;
}

// header | maps [tiles][S][32] (16 bytes each) | parts of the rates' gradients
// [P][D].  Where CTAs share a slab the maps are set to ones before each launch.
struct GlrLayout {
    size_t maps, part, total;
    int S, tiles;
};

GlrLayout glr_layout(long long T, long long D, int tile)
{
    GlrLayout ly;
    ly.S = int((D + kGD - 1) / kGD);
    ly.tiles = int((T + tile - 1) / tile);
    ly.maps = sizeof(WsHeader);
    ly.part = ly.maps + size_t(ly.tiles) * ly.S * 512;
    ly.total = align256(ly.part + size_t(kGMaxP) * D * 4);
    return ly;
}

size_t glr_ws_bytes(bool adjoint, long long T, long long n_seq, long long D)
{
    if (T < 1 || n_seq < 1 || D < 1 || D % 8 != 0 || T > INT_MAX / 2 || n_seq > INT_MAX / 2 || D > INT_MAX / 2 ||
        (double)T * (double)D * 12.0 >= kMaxBytes || (double)n_seq * (double)D * 4.0 >= kMaxBytes)
        return 0;
    // fp32 gates have the shorter tiles
    return glr_layout(T, D, adjoint ? GlrAdjointLayout<float>::kTile : GlrScanLayout<float>::kTile).total;
}

// rows [T][width] (u: width 3 D, as [T][3][D]) -> box of `rows` rows of 64
// channels (all three gates)
pararnn_status map_glr(CUtensorMap* m, const void* x, pararnn_dtype dt, int gates, long long T, long long D, int rows)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return fail(PARARNN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const cuuint64_t es = dtype_bytes(dt);
    const bool u = gates > 1;
    cuuint64_t dims[3] = {cuuint64_t(D), u ? cuuint64_t(gates) : cuuint64_t(T), cuuint64_t(T)};
    cuuint64_t strides[2] = {cuuint64_t(D) * es, cuuint64_t(D) * es * gates};
    cuuint32_t box[3] = {cuuint32_t(kGD), u ? cuuint32_t(gates) : cuuint32_t(rows), cuuint32_t(rows)};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    CUresult r = enc(m, dt == PARARNN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                     u ? 3 : 2, const_cast<void*>(x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PARARNN_ERR_CUDA, "cuTensorMapEncodeTiled(recurrence) failed: %d", int(r));
    return PARARNN_OK;
}

// How many CTAs share a slab: what fits on the device at once (one an SM, by its
// shared memory), at most one CTA a tile and kGMaxP.  They wait for one another
// only if there are several; the launch is then a cooperative one.
template <class K>
pararnn_status launch_glr(K kern, int threads, size_t smem, const GlrLayout& ly, GlrParams* p, void** args, void* ws,
                          cudaStream_t st)
{
    int sms = 0;
    TRY(device_info(&sms));
    const void* f = reinterpret_cast<const void*>(kern);
    CUDA_TRY(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
    unsigned char* base = static_cast<unsigned char*>(ws);
    p->S = ly.S;
    p->tiles = ly.tiles;
    p->P = std::max(1, std::min({sms / ly.S, ly.tiles, kGMaxP}));
    p->hdr = reinterpret_cast<WsHeader*>(base);
    p->maps = reinterpret_cast<uint4*>(base + ly.maps);
    p->part = reinterpret_cast<float*>(base + ly.part);
    p->wait_ns = kWaitLimitNs;
    const dim3 grid(unsigned(ly.S) * p->P);
    if (p->P > 1) {
        CUDA_TRY(cudaMemsetAsync(base + ly.maps, 0xff, ly.part - ly.maps, st));
        CUDA_TRY(cudaLaunchCooperativeKernel(f, grid, dim3(threads), args, smem, st));
    } else {
        CUDA_TRY(cudaLaunchKernel(f, grid, dim3(threads), args, smem, st));
    }
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return PARARNN_OK;
}

template <class UT>
pararnn_status launch_glr_scan(const UT* u, GlrParams p, long long D, void* ws, cudaStream_t st)
{
    using LY = GlrScanLayout<UT>;
    CUtensorMap tu;
    TRY(map_glr(&tu, u, sizeof(UT) == 2 ? PARARNN_BF16 : PARARNN_F32, 3, p.T, D, LY::kTile));
    void* args[] = {(void*)&tu, (void*)&p};
    return launch_glr(glr_scan_kernel<UT>, LY::kThreads, LY::smem_bytes, glr_layout(p.T, D, LY::kTile), &p, args, ws, st);
}

template <class UT>
pararnn_status launch_glr_adjoint(const UT* u, GlrParams p, float* drate, long long D, void* ws, cudaStream_t st)
{
    using LY = GlrAdjointLayout<UT>;
    CUtensorMap tu, th, td;
    TRY(map_glr(&tu, u, sizeof(UT) == 2 ? PARARNN_BF16 : PARARNN_F32, 3, p.T, D, LY::kTile));
    TRY(map_glr(&th, p.states, PARARNN_F32, 1, p.T, D, LY::kTile));
    TRY(map_glr(&td, p.dh, PARARNN_F32, 1, p.T, D, LY::kTile));
    void* args[] = {(void*)&tu, (void*)&th, (void*)&td, (void*)&p};
    TRY(launch_glr(glr_adjoint_kernel<UT>, LY::kThreads, LY::smem_bytes, glr_layout(p.T, D, LY::kTile), &p, args, ws, st));
    column_sum_kernel<<<unsigned((D + 31) / 32), 32 * kSumRuns, 0, st>>>(p.part, drate, p.P, D);
    return launched();
}

// --------------------------------------------------------------- RMS norm

// Vectors of 8 columns a thread keeps: two (more where D needs it).  Measured at
// T 32768 D 2048, norm: two 92 us, four 96; adjoint: two 98 us, one 108.
constexpr int kNormVecs = 2, kNormAdjVecs = 2;
constexpr int kNormMaxParts = 148 * 8;  // most CTAs of the adjoint: eight on each of a B200's 148 SMs

struct NormShape {
    int tpr, nv, threads, rows;
};

// vectors: how many of 8 columns a thread may keep (kNormVectors where D needs it)
pararnn_status norm_shape(long long T, long long D, int vectors, NormShape* s)
{
    if (T < 1 || D < 1) return fail(PARARNN_ERR_INVALID_ARG, "T, D must be >= 1 (got %lld, %lld)", T, D);
    if (D % 8 != 0) return fail(PARARNN_ERR_UNSUPPORTED, "D must be a multiple of 8 (got %lld)", D);
    if (D > kNormMaxD) return fail(PARARNN_ERR_UNSUPPORTED, "D must be at most %lld (got %lld)", kNormMaxD, D);
    if (T > INT_MAX / 2 || (double)T * (double)D * 4.0 >= kMaxBytes)
        return fail(PARARNN_ERR_INVALID_ARG, "T too large (got %lld)", T);
    const int d8 = int(D / 8);
    // the fewest threads a row that keep it within `vectors` vectors each
    int tpr = 32;
    while (tpr < kNormThreads && tpr * vectors < d8) tpr *= 2;
    // with few rows the chip (148 SMs) is far from full: spread each over more threads
    while (tpr < kNormThreads && tpr < d8 && T * tpr < 148 * 512) tpr *= 2;
    s->tpr = tpr;
    s->nv = 1;
    while (s->nv * tpr < d8) s->nv *= 2;
    s->threads = std::max(tpr, 128);
    s->rows = s->threads / tpr;
    return PARARNN_OK;
}

int norm_adjoint_parts(long long T, const NormShape& s) { return int(std::min<long long>((T + s.rows - 1) / s.rows, kNormMaxParts)); }

template <class XT, class RT>
pararnn_status launch_norm(const NormParams& p, const NormShape& s, cudaStream_t st)
{
    const unsigned grid = unsigned((p.T + s.rows - 1) / s.rows);
    switch (s.nv) {
    case 1: rms_norm_kernel<XT, RT, 1><<<grid, s.threads, 0, st>>>(p); break;
    case 2: rms_norm_kernel<XT, RT, 2><<<grid, s.threads, 0, st>>>(p); break;
    default: rms_norm_kernel<XT, RT, 4><<<grid, s.threads, 0, st>>>(p); break;
    }
    return launched();
}

// As many CTAs as run at once: each takes rows in turn.
template <class YT, class VT, int NV>
pararnn_status launch_norm_adjoint_nv(const NormAdjParams& p, const NormShape& s, int* grid, cudaStream_t st)
{
    auto kern = rms_norm_adjoint_kernel<YT, VT, NV>;
    const size_t smem = s.rows > 1 ? size_t(s.rows) * p.D * 4 : 0;  // at most 4 rows of 512 columns
    int sms = 0, occ = 0;
    TRY(device_info(&sms));
    CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, s.threads, smem));
    *grid = std::max(1, std::min(norm_adjoint_parts(p.T, s), sms * occ));
    kern<<<*grid, s.threads, smem, st>>>(p);
    return launched();
}

template <class YT, class VT>
pararnn_status launch_norm_adjoint(const NormAdjParams& p, const NormShape& s, int* grid, cudaStream_t st)
{
    switch (s.nv) {
    case 1: return launch_norm_adjoint_nv<YT, VT, 1>(p, s, grid, st);
    case 2: return launch_norm_adjoint_nv<YT, VT, 2>(p, s, grid, st);
    default: return launch_norm_adjoint_nv<YT, VT, 4>(p, s, grid, st);
    }
}

// ----------------------------------------------------------- 8-bit product

pararnn_status fp8_dims(long long M, long long N, long long K)
{
    if (M < 1 || N < 1 || K < 1)
        return fail(PARARNN_ERR_INVALID_ARG, "M, N, K must be >= 1 (got %lld, %lld, %lld)", M, N, K);
    if (K % 16 != 0) return fail(PARARNN_ERR_UNSUPPORTED, "K must be a multiple of 16 (got %lld)", K);
    if (N % 8 != 0) return fail(PARARNN_ERR_UNSUPPORTED, "N must be a multiple of 8 (got %lld)", N);
    if (M > INT_MAX / 2 || N > INT_MAX / 2 || K > INT_MAX / 2 || (double)M * (double)K * 4.0 >= kMaxBytes ||
        (double)M * (double)N * 4.0 >= kMaxBytes || (double)N * (double)K * 4.0 >= kMaxBytes)
        return fail(PARARNN_ERR_INVALID_ARG, "dimension too large");
    return PARARNN_OK;
}

long long blocks128(long long n) { return (n + 127) / 128; }

// e4m3 [rows][K] -> box [box_rows][128] with the 128-byte swizzle; K a multiple
// of 16, columns and rows beyond the array read as zeros.
pararnn_status map_e4m3_sw128(CUtensorMap* m, const void* p, long long rows, long long K, int box_rows)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return fail(PARARNN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
    cuuint64_t strides[1] = {cuuint64_t(K)};
    cuuint32_t box[2] = {cuuint32_t(kQK), cuuint32_t(box_rows)};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PARARNN_ERR_CUDA, "cuTensorMapEncodeTiled(8-bit operand) failed: %d", int(r));
    return PARARNN_OK;
}

// u [M][N] -> box of 32 rows x 128 bytes with the 128-byte swizzle
pararnn_status map_sums_sw128(CUtensorMap* m, void* u, long long M, long long N, bool bf16)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return fail(PARARNN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const cuuint64_t es = bf16 ? 2 : 4;
    cuuint64_t dims[2] = {cuuint64_t(N), cuuint64_t(M)};
    cuuint64_t strides[1] = {cuuint64_t(N) * es};
    cuuint32_t box[2] = {cuuint32_t(128 / es), 32u};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, u, dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PARARNN_ERR_CUDA, "cuTensorMapEncodeTiled(output) failed: %d", int(r));
    return PARARNN_OK;
}

template <class K>
pararnn_status launch_clusters(K kern, int grid, int threads, int cluster, size_t smem, cudaStream_t st, void** args)
{
    CUDA_TRY(cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = unsigned(cluster);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    CUDA_TRY(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kern), args));
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return PARARNN_OK;
}

// How many CTAs of the narrow form share a tile's blocks of K: as long as all
// of them run at once (two on each of 148 SMs, less what clusters of up to eight leave over:
// 288 in clusters of four took two rounds, 256 one).
constexpr long long kNarrowRoom = 256;

int narrow_splits(long long tiles, long long KB)
{
    int splits = 1;
    while (splits < 8 && splits * 2 <= KB && tiles * splits * 2 <= kNarrowRoom) splits *= 2;
    return splits;
}

template <int NT>
pararnn_status launch_narrow(const uint8_t* x, const uint8_t* w, Fp8Params p, cudaStream_t st)
{
    using LY = NarrowLayout<NT>;
    CUtensorMap tx, tw;
    TRY(map_e4m3_sw128(&tx, x, p.M, p.K, NT));
    TRY(map_e4m3_sw128(&tw, w, p.N, p.K, 128));
    p.tiles_n = int(blocks128(p.N));
    const long long tiles = (p.M + NT - 1) / NT * p.tiles_n;
    if (tiles > INT_MAX / 8) return fail(PARARNN_ERR_INVALID_ARG, "too many tiles");
    p.n_tiles = int(tiles);
    p.splits = narrow_splits(tiles, p.KB);
    void* args[] = {(void*)&tx, (void*)&tw, (void*)&p};
    return launch_clusters(fp8_project_narrow_kernel<NT>, p.n_tiles * p.splits, kNThreads, p.splits, LY::smem_bytes, st, args);
}

pararnn_status launch_wide(const uint8_t* x, const uint8_t* w, Fp8Params p, int sms, cudaStream_t st)
{
    CUtensorMap tx, tw, tu;
    TRY(map_e4m3_sw128(&tx, x, p.M, p.K, kQM));
    TRY(map_e4m3_sw128(&tw, w, p.N, p.K, kQN / 2));
    TRY(map_sums_sw128(&tu, p.u, p.M, p.N, p.u_bf16));
    p.tiles_n = int((p.N + kQN - 1) / kQN);
    const long long tiles = (p.M + 2 * kQM - 1) / (2 * kQM) * p.tiles_n;
    if (tiles > INT_MAX / 8) return fail(PARARNN_ERR_INVALID_ARG, "too many tiles");
    p.n_tiles = int(tiles);
    p.splits = 1;
    void* args[] = {(void*)&tx, (void*)&tw, (void*)&tu, (void*)&p};
    return launch_clusters(fp8_project_wide_kernel, 2 * std::min(p.n_tiles, sms / 2), kQThreads, 2, kQSmem, st, args);
}

}  // namespace

extern "C" {

pararnn_status pararnn_take_failure(pararnn_stream_t stream)
{
    t_err[0] = '\0';
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void* at = nullptr;
    int code = 0;
    CUDA_TRY(cudaGetSymbolAddress(&at, g_layer_failure));
    CUDA_TRY(cudaMemcpyAsync(&code, at, sizeof(code), cudaMemcpyDeviceToHost, st));
    CUDA_TRY(cudaStreamSynchronize(st));
    if (code == 0) return PARARNN_OK;
    CUDA_TRY(cudaMemsetAsync(at, 0, sizeof(code), st));
    CUDA_TRY(cudaStreamSynchronize(st));
    return fail(pararnn_status(code), "a bounded wait of a layer operator ran out since the last look: its outputs are not valid");
}

size_t pararnn_glr_workspace_size(int64_t T, int64_t n_seq, int64_t D) { return glr_ws_bytes(false, T, n_seq, D); }
size_t pararnn_glr_adjoint_workspace_size(int64_t T, int64_t n_seq, int64_t D) { return glr_ws_bytes(true, T, n_seq, D); }

pararnn_status pararnn_glr_scan(const void* u, pararnn_dtype u_dtype, const float* rate, const float* h0,
                                const int32_t* seq_starts, float* h, float* h_last, int64_t T, int64_t n_seq, int64_t D,
                                void* workspace, size_t workspace_bytes, pararnn_stream_t stream)
{
    t_err[0] = '\0';
    TRY(check_wide_dtype(u_dtype, "u_dtype"));
    TRY(check_ptr(u, "u", true));
    TRY(check_ptr(rate, "rate", true));
    TRY(check_ptr(h0, "h0", false));
    TRY(check_starts(seq_starts));
    TRY(check_ptr(h, "h", true));
    TRY(check_ptr(h_last, "h_last", false));
    TRY(glr_shape(T, n_seq, D, seq_starts));
    const size_t rows = size_t(T) * D, ends = size_t(n_seq) * D * 4;
    const size_t need = glr_ws_bytes(false, T, n_seq, D);
    TRY((check_apart<4, 2>({{"u", u, rows * 3 * dtype_bytes(u_dtype)}, {"rate", rate, size_t(D) * 4}, {"h0", h0, ends},
                           {"seq_starts", seq_starts, size_t(n_seq + 1) * 4}},
                          {{"h", h, rows * 4}, {"h_last", h_last, ends}}, nullptr, {"workspace", workspace, need})));
    TRY(check_workspace(workspace, workspace_bytes, need));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    GlrParams p = {};
    p.rate = rate;
    p.h0 = h0;
    p.starts = seq_starts;
    p.h = h;
    p.h_last = h_last;
    p.D = D;
    p.T = int(T);
    p.n_seq = int(n_seq);
    p.L = int(T / n_seq);
    if (u_dtype == PARARNN_BF16) return launch_glr_scan(static_cast<const uint16_t*>(u), p, D, workspace, st);
    return launch_glr_scan(static_cast<const float*>(u), p, D, workspace, st);
}

pararnn_status pararnn_glr_adjoint(const void* u, pararnn_dtype u_dtype, const float* rate, const float* h0,
                                   const int32_t* seq_starts, const float* h, const float* dh, const float* dh_last,
                                   float* du, float* drate, float* dh0, int64_t T, int64_t n_seq, int64_t D,
                                   void* workspace, size_t workspace_bytes, pararnn_stream_t stream)
{
    t_err[0] = '\0';
    TRY(check_wide_dtype(u_dtype, "u_dtype"));
    TRY(check_ptr(u, "u", true));
    TRY(check_ptr(rate, "rate", true));
    TRY(check_ptr(h0, "h0", false));
    TRY(check_starts(seq_starts));
    TRY(check_ptr(h, "h", true));
    TRY(check_ptr(dh, "dh", true));
    TRY(check_ptr(dh_last, "dh_last", false));
    TRY(check_ptr(du, "du", true));
    TRY(check_ptr(drate, "drate", true));
    TRY(check_ptr(dh0, "dh0", false));
    TRY(glr_shape(T, n_seq, D, seq_starts));
    const size_t rows = size_t(T) * D, ends = size_t(n_seq) * D * 4;
    const size_t need = glr_ws_bytes(true, T, n_seq, D);
    TRY((check_apart<7, 3>({{"u", u, rows * 3 * dtype_bytes(u_dtype)}, {"rate", rate, size_t(D) * 4}, {"h0", h0, ends},
                           {"seq_starts", seq_starts, size_t(n_seq + 1) * 4}, {"h", h, rows * 4}, {"dh", dh, rows * 4},
                           {"dh_last", dh_last, ends}},
                          {{"du", du, rows * 12}, {"drate", drate, size_t(D) * 4}, {"dh0", dh0, ends}}, nullptr,
                          {"workspace", workspace, need})));
    TRY(check_workspace(workspace, workspace_bytes, need));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    GlrParams p = {};
    p.rate = rate;
    p.h0 = h0;
    p.starts = seq_starts;
    p.states = h;
    p.dh = dh;
    p.dh_last = dh_last;
    p.du = du;
    p.dh0 = dh0;
    p.D = D;
    p.T = int(T);
    p.n_seq = int(n_seq);
    p.L = int(T / n_seq);
    if (u_dtype == PARARNN_BF16) return launch_glr_adjoint(static_cast<const uint16_t*>(u), p, drate, D, workspace, st);
    return launch_glr_adjoint(static_cast<const float*>(u), p, drate, D, workspace, st);
}

pararnn_status pararnn_glr_step(const void* u, pararnn_dtype u_dtype, const float* rate, const float* h_prev,
                                float* h_next, int64_t B, int64_t D, pararnn_stream_t stream)
{
    t_err[0] = '\0';
    TRY(check_wide_dtype(u_dtype, "u_dtype"));
    TRY(check_ptr(u, "u", true));
    TRY(check_ptr(rate, "rate", true));
    TRY(check_ptr(h_prev, "h_prev", false));
    TRY(check_ptr(h_next, "h_next", true));
    TRY(check_step_shape(B, D));
    const size_t n = size_t(B) * D;
    TRY((check_apart<3, 1>({{"u", u, n * 3 * dtype_bytes(u_dtype)}, {"rate", rate, size_t(D) * 4}, {"h_prev", h_prev, n * 4}},
                          {{"h_next", h_next, n * 4}}, h_prev)));
    const unsigned grid = unsigned((n / 4 + 255) / 256);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (u_dtype == PARARNN_BF16)
        glr_step_kernel<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(u), rate, h_prev, h_next, B, D);
    else
        glr_step_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(u), rate, h_prev, h_next, B, D);
    return launched();
}

pararnn_status pararnn_rms_norm(const void* x, pararnn_dtype x_dtype, const void* residual, pararnn_dtype sum_dtype,
                                const float* w, float eps, void* sum, void* y, pararnn_dtype y_dtype, float* y_scale,
                                float* rstd, int64_t T, int64_t D, pararnn_stream_t stream)
{
    t_err[0] = '\0';
    TRY(check_wide_dtype(x_dtype, "x_dtype"));
    TRY(check_wide_dtype(sum_dtype, "sum_dtype"));
    if (y_dtype != PARARNN_F32 && y_dtype != PARARNN_BF16 && y_dtype != PARARNN_E4M3)
        return fail(PARARNN_ERR_INVALID_ARG, "unknown y dtype %d", int(y_dtype));
    TRY(check_ptr(x, "x", true));
    TRY(check_ptr(residual, "residual", false));
    TRY(check_ptr(w, "w", true));
    TRY(check_ptr(sum, "sum", false));
    TRY(check_ptr(y, "y", true));
    TRY(check_ptr(y_scale, "y_scale", y_dtype == PARARNN_E4M3));
    TRY(check_ptr(rstd, "rstd", false));
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(PARARNN_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    NormShape s;
    TRY(norm_shape(T, D, kNormVecs, &s));
    if (y_dtype == PARARNN_E4M3 && D % 16 != 0)
        return fail(PARARNN_ERR_UNSUPPORTED, "D must be a multiple of 16 for an 8-bit output (got %lld)", (long long)D);
    const size_t n = size_t(T) * D;
    TRY((check_apart<3, 4>({{"x", x, n * dtype_bytes(x_dtype)}, {"residual", residual, n * dtype_bytes(sum_dtype)},
                           {"w", w, size_t(D) * 4}},
                          {{"sum", sum, n * dtype_bytes(sum_dtype)}, {"y", y, n * dtype_bytes(y_dtype)},
                           {"y_scale", y_dtype == PARARNN_E4M3 ? y_scale : nullptr, size_t(T) * blocks128(D) * 4},
                           {"rstd", rstd, size_t(T) * 4}},
                          residual && residual == sum ? residual : nullptr)));
    NormParams p;
    p.x = x;
    p.res = residual;
    p.w = w;
    p.sum = sum;
    p.y = y;
    p.scale = y_scale;
    p.rstd = rstd;
    p.T = T;
    p.D = D;
    p.eps = eps;
    p.tpr = s.tpr;
    p.sum_bf16 = sum_dtype == PARARNN_BF16;
    p.y_dtype = y_dtype;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (x_dtype == PARARNN_BF16) {
        if (!residual) return launch_norm<uint16_t, void>(p, s, st);
        return p.sum_bf16 ? launch_norm<uint16_t, uint16_t>(p, s, st) : launch_norm<uint16_t, float>(p, s, st);
    }
    if (!residual) return launch_norm<float, void>(p, s, st);
    return p.sum_bf16 ? launch_norm<float, uint16_t>(p, s, st) : launch_norm<float, float>(p, s, st);
}

size_t pararnn_rms_norm_adjoint_workspace_size(int64_t T, int64_t D)
{
    NormShape s;
    if (norm_shape(T, D, kNormAdjVecs, &s) != PARARNN_OK) return 0;
    return align256(size_t(norm_adjoint_parts(T, s)) * D * 4);
}

pararnn_status pararnn_rms_norm_adjoint(const void* dy, pararnn_dtype dy_dtype, const void* sum, pararnn_dtype sum_dtype,
                                        const float* w, const float* rstd, const void* dsum, void* dx, float* dw,
                                        int64_t T, int64_t D, void* workspace, size_t workspace_bytes,
                                        pararnn_stream_t stream)
{
    t_err[0] = '\0';
    TRY(check_wide_dtype(dy_dtype, "dy_dtype"));
    TRY(check_wide_dtype(sum_dtype, "sum_dtype"));
    TRY(check_ptr(dy, "dy", true));
    TRY(check_ptr(sum, "sum", true));
    TRY(check_ptr(w, "w", true));
    TRY(check_ptr(rstd, "rstd", true));
    TRY(check_ptr(dsum, "dsum", false));
    TRY(check_ptr(dx, "dx", true));
    TRY(check_ptr(dw, "dw", true));
    NormShape s;
    TRY(norm_shape(T, D, kNormAdjVecs, &s));
    const size_t n = size_t(T) * D, es = dtype_bytes(sum_dtype);
    const size_t need = align256(size_t(norm_adjoint_parts(T, s)) * D * 4);
    TRY((check_apart<5, 2>({{"dy", dy, n * dtype_bytes(dy_dtype)}, {"sum", sum, n * es}, {"w", w, size_t(D) * 4},
                           {"rstd", rstd, size_t(T) * 4}, {"dsum", dsum, n * es}},
                          {{"dx", dx, n * es}, {"dw", dw, size_t(D) * 4}}, dsum && dsum == dx ? dsum : nullptr,
                          {"workspace", workspace, need})));
    TRY(check_workspace(workspace, workspace_bytes, need));
    NormAdjParams p;
    p.dy = dy;
    p.v = sum;
    p.w = w;
    p.rstd = rstd;
    p.dv = dsum;
    p.dx = dx;
    p.part = static_cast<float*>(workspace);
    p.T = T;
    p.D = D;
    p.tpr = s.tpr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int grid = 0;
    if (dy_dtype == PARARNN_BF16)
        TRY((sum_dtype == PARARNN_BF16 ? launch_norm_adjoint<uint16_t, uint16_t>(p, s, &grid, st)
                                       : launch_norm_adjoint<uint16_t, float>(p, s, &grid, st)));
    else
        TRY((sum_dtype == PARARNN_BF16 ? launch_norm_adjoint<float, uint16_t>(p, s, &grid, st)
                                       : launch_norm_adjoint<float, float>(p, s, &grid, st)));
    column_sum_kernel<<<unsigned((D + 31) / 32), 32 * kSumRuns, 0, st>>>(p.part, dw, grid, D);
    return launched();
}

pararnn_status pararnn_fp8_quantize(const void* x, pararnn_dtype x_dtype, int block_rows, void* q, float* scale, int64_t M,
                                    int64_t K, pararnn_stream_t stream)
{
    t_err[0] = '\0';
    TRY(check_wide_dtype(x_dtype, "x_dtype"));
    TRY(check_ptr(x, "x", true));
    TRY(check_ptr(q, "q", true));
    TRY(check_ptr(scale, "scale", true));
    if (block_rows != 1 && block_rows != 128)
        return fail(PARARNN_ERR_INVALID_ARG, "block_rows must be 1 or 128 (got %d)", block_rows);
    TRY(fp8_dims(M, 8, K));
    const long long KB = blocks128(K);
    // rows: as many blocks of a row side by side as divide it, up to 16
    int shift = 4;
    while (shift < 8 && KB % (2ll << (shift - 4)) == 0) ++shift;
    const int per = kQuantRows * (256 >> shift);
    const dim3 rows_grid(unsigned((M + per - 1) / per), unsigned(KB >> (shift - 4)));
    const long long sets = blocks128(M) * KB;
    if (block_rows == 1 ? (KB >> (shift - 4)) > 65535 : sets > INT_MAX) return fail(PARARNN_ERR_INVALID_ARG, "too many blocks");
    TRY((check_apart<1, 2>({{"x", x, size_t(M) * K * dtype_bytes(x_dtype)}},
                          {{"q", q, size_t(M) * K},
                           {"scale", scale, size_t(block_rows == 1 ? M : blocks128(M)) * KB * 4}}, nullptr)));
    const unsigned grid = unsigned(sets);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* out = static_cast<uint8_t*>(q);
    if (block_rows == 1) {
        if (x_dtype == PARARNN_BF16) fp8_quantize_rows_kernel<uint16_t><<<rows_grid, 256, 0, st>>>(x, out, scale, M, K, KB, shift);
        else fp8_quantize_rows_kernel<float><<<rows_grid, 256, 0, st>>>(x, out, scale, M, K, KB, shift);
    } else {
        if (x_dtype == PARARNN_BF16) fp8_quantize_blocks_kernel<uint16_t><<<grid, 512, 0, st>>>(x, out, scale, M, K, KB);
        else fp8_quantize_blocks_kernel<float><<<grid, 512, 0, st>>>(x, out, scale, M, K, KB);
    }
    return launched();
}

size_t pararnn_fp8_project_workspace_size(int64_t M, int64_t N, int64_t K)
{
    return fp8_dims(M, N, K) == PARARNN_OK ? sizeof(WsHeader) : 0;
}

pararnn_status pararnn_fp8_project(const void* x, const float* x_scale, const void* w, const float* w_scale,
                                   const float* bias, void* u, pararnn_dtype u_dtype, int64_t M, int64_t N, int64_t K,
                                   void* workspace, size_t workspace_bytes, pararnn_stream_t stream)
{
    t_err[0] = '\0';
    TRY(check_wide_dtype(u_dtype, "u_dtype"));
    TRY(check_ptr(x, "x", true));
    TRY(check_ptr(x_scale, "x_scale", true));
    TRY(check_ptr(w, "w", true));
    TRY(check_ptr(w_scale, "w_scale", true));
    TRY(check_ptr(bias, "bias", false));
    TRY(check_ptr(u, "u", true));
    TRY(fp8_dims(M, N, K));
    const long long KB = blocks128(K);
    TRY((check_apart<5, 1>({{"x", x, size_t(M) * K}, {"x_scale", x_scale, size_t(M) * KB * 4}, {"w", w, size_t(N) * K},
                            {"w_scale", w_scale, size_t(blocks128(N)) * KB * 4}, {"bias", bias, size_t(N) * 4}},
                           {{"u", u, size_t(M) * N * dtype_bytes(u_dtype)}}, nullptr,
                           {"workspace", workspace, sizeof(WsHeader)})));
    TRY(check_workspace(workspace, workspace_bytes, sizeof(WsHeader)));
    int sms = 0;
    TRY(device_info(&sms));
    Fp8Params p;
    p.xs = x_scale;
    p.ws = w_scale;
    p.bias = bias;
    p.u = u;
    p.M = M;
    p.N = N;
    p.K = K;
    p.KB = int(KB);
    p.u_bf16 = u_dtype == PARARNN_BF16;
    p.hdr = static_cast<WsHeader*>(workspace);
    p.wait_ns = kWaitLimitNs;
    const uint8_t *xb = static_cast<const uint8_t*>(x), *wb = static_cast<const uint8_t*>(w);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // Blocks of K one after another in the fullest CTA, and what one costs: a
    // pair's 0.53 us each and 5.5 us before and after, the narrow form's (64
    // rows) 0.65 and 6.  Both forms were measured at eleven M from 65 to 4096 for
    // ten weights from N 64 K 2048 to N 12288 K 4096, bf16 and fp32 out: what is
    // chosen is the faster one or within 8 % of it, but for M 512 N 1304 K 512
    // (narrow 9.4 us, wide 8.1).  N 6144 K 2048: 12.6 (narrow) against 14.2 us at
    // M 128, 16.5 against 14.2 at M 256; N 2048 K 8192: 25.9 against 39.3 at
    // M 512, 43.0 against 39.6 at M 768; N 264 K 1104: 9.2 against 10.9 at M 1024,
    // 13.2 against 10.9 at M 4096; N 2048 K 128: 8.0 against 6.0 at M 65.
    const long long pairs = std::max(1, sms / 2);
    const long long wide_tiles = (M + 2 * kQM - 1) / (2 * kQM) * ((N + kQN - 1) / kQN);
    const long long tiles = (M + 63) / 64 * blocks128(N);
    const int splits = narrow_splits(tiles, KB);
    const double wide_us = 5.5 + 0.53 * double((wide_tiles + pairs - 1) / pairs * KB);
    const double narrow_us = 6.0 + 0.65 * double((tiles * splits + kNarrowRoom - 1) / kNarrowRoom * ((KB + splits - 1) / splits));
    if (M > 64 && wide_us < narrow_us) return launch_wide(xb, wb, p, sms, st);
    if (M > 64) return launch_narrow<64>(xb, wb, p, st);
    // up to 64 rows: 32 a CTA also for 33 to 64 (N 2048 K 8192, M 64: 10.7 against 12.0 us)
    if (M > 16) return launch_narrow<32>(xb, wb, p, st);
    return launch_narrow<16>(xb, wb, p, st);
}

}  // extern "C"
