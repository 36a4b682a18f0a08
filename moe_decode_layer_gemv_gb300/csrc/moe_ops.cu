// moe_ops.cu -- the C ABI of the grouped products and the NVFP4 operators
// (declared in include/moe.h): argument checks, the choice of a kernel and
// its launch.  Kernels: moe_grouped.cuh and moe_nvfp4.cuh.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "moe.h"
#include "moe_grouped.cuh"
#include "moe_host.cuh"
#include "moe_nvfp4.cuh"

namespace moe {

// A tensor map over a row-major tensor [outer2, outer1, inner] (outer2 = 0:
// two dimensions) with boxes of box_bytes x box_rows (128 or 64 bytes, the
// swizzle of that width); elements outside the tensor read as zeros.
static bool encode_map(CUtensorMap* map, const void* base, int elem, uint64_t inner, uint64_t outer1, uint64_t outer2,
                       uint32_t box_rows, uint32_t box_bytes = 128) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const uint64_t pitch = inner * elem;
    const cuuint64_t dims[3] = {inner, outer1, outer2};
    const cuuint64_t strides[2] = {pitch, pitch * outer1};
    const cuuint32_t box[3] = {box_bytes / (uint32_t)elem, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, outer2 ? 3 : 2,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map over bf16 [outer2, outer1, inner] (outer2 = 0: [outer1, inner]) whose
// boxes are 64 rows x two 64-column blocks: inner % 64 == 0.
static bool encode_blocked(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer1, uint64_t outer2) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, outer1, inner / 64, outer2};
    const cuuint64_t strides[3] = {inner * 2, 128, inner * outer1 * 2};
    const cuuint32_t box[4] = {64, 64, 2, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, outer2 ? 4 : 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int check_grouped(int R, int N, int K, int E, int dtype) {
    if (R < 0 || R > MOE_MAX_ROWS || E < 1 || E > MOE_MAX_E) return MOE_ERR_INVALID_ARG;
    if (N < 8 || N > 2 * MOE_MAX_DIM || (N & 7) || K < 8 || K > MOE_MAX_DIM || (K & 7)) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DT_F32 && dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// A persistent kernel on every SM, in clusters of CG CTAs.
template <int CG, typename K, typename P>
static int launch_persistent(K kernel, const P& p, int threads, int sms, cudaStream_t st) {
    const int rc = allow_smem(kernel, kGgSmem);
    if (rc) return rc;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)(sms / CG * CG));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = kGgSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    return launch_ex(cfg, kernel, p);
}

// The paired tile (256 x 256) from so many rows a segment on average, where
// the output is wider than a single CTA's tile.  Measured on 64 experts of
// 1536 x 2048, single and paired, at 96 / 128 / 256 rows: forward to bf16 80 /
// 85 / 113 and 82 / 85 / 98 us, to fp32 82 / 88 / 120 and 83 / 86 / 106, dx to
// bf16 72 / 82 / 116 and 73 / 75 / 99.
// Weight gradients of few rows are all stores: in bf16 the pair's larger tiles
// are always ahead (16 rows: 101 and 96 us), in fp32 late (192 rows: 157 and
// 161; 256: 180 and 159; 1024: 425 and 300; of 2048 x 768, 192 rows: 82 and 88,
// 256: 94 and 89).
constexpr int kGgPairRows = 128, kGgPairRowsDw = 0, kGgPairRowsDwF32 = 256;

static bool gg_pairs(int R, int M, int E, int rows = kGgPairRows) { return M > 128 && (int64_t)R >= (int64_t)rows * E; }

// dw: with fewer tiles than CTAs (or pairs) the segments' rows are cut into
// parts, of 512 rows on average at least, whose sums are joined afterwards.
static int gg_split(int R, int N, int K, int E, int sms) {
    const int cg = gg_pairs(R, K, E, kGgPairRowsDwF32) ? 2 : 1;
    const int64_t tiles = (int64_t)E * ceil_div(N, 128 * cg) * ceil_div(K, 128 * cg);
    int64_t parts = sms / cg / tiles;
    if (parts > (int64_t)R / E / 512) parts = (int64_t)R / E / 512;
    return parts < 2 ? 1 : (int)parts;
}

template <int MODE, bool F32>
static int run_gg(GgParams& p, const void* a, const void* b, int R, int N, int K, int E, cudaStream_t st) {
    bool ok;
    p.a_blocked = K % 64 == 0;
    p.b_blocked = N % 64 == 0;
    if (MODE == kGgFwd)
        ok = encode_map(&p.ta, a, 2, K, N, E, 128) && encode_map(&p.tb, b, 2, K, R, 0, kGgBoxN) &&
             encode_map(&p.tb_all, b, 2, K, R, 0, 128);
    else if (MODE == kGgDx)
        ok = (p.a_blocked ? encode_blocked(&p.ta, a, K, N, E) : encode_map(&p.ta, a, 2, K, N, E, 64)) &&
             encode_map(&p.tb, b, 2, N, R, 0, kGgBoxN) &&
             encode_map(&p.tb_all, b, 2, N, R, 0, 128);
    else
        ok = (p.a_blocked ? encode_blocked(&p.ta, a, K, R, 0) : encode_map(&p.ta, a, 2, K, R, 0, 64)) &&
             (p.b_blocked ? encode_blocked(&p.tb, b, N, R, 0) : encode_map(&p.tb, b, 2, N, R, 0, 64));
    for (int i = 0; MODE == kGgDw && ok && i < 4; ++i) ok = encode_map(&p.zero[i], a, 2, K, R, 0, 8 >> i);
    if (!ok) return MOE_ERR_UNSUPPORTED;
    p.E = E;
    p.R = R;
    p.M = MODE == kGgFwd ? N : K;
    p.C = MODE == kGgFwd ? K : N;
    p.NW = N;
    const int sms = sm_count();
    if (sms < 2) return MOE_ERR_CUDA;
    return gg_pairs(R, p.M, E, MODE != kGgDw ? kGgPairRows : F32 ? kGgPairRowsDwF32 : kGgPairRowsDw)
               ? launch_persistent<2>(gg_kernel<MODE, 2, F32>, p, GgCfg<MODE, 2, F32>::kThreads, sms, st)
               : launch_persistent<1>(gg_kernel<MODE, 1, F32>, p, GgCfg<MODE, 1, F32>::kThreads, sms, st);
}

template <bool BF16, int T>
static int launch_rows(const void* x, int G, int nb, uint8_t* q, uint8_t* bs, float* gs, int32_t* status, cudaStream_t st) {
    const int per = 128 / T, bpt = (nb + T - 1) / T;
    const unsigned grid = (unsigned)((G + per - 1) / per);
    if (bpt <= 1) return launch_pdl(nv4_rows_kernel<BF16, T, 1>, grid, 128, 0, st, x, G, nb, q, bs, gs, status);
    if (bpt <= 2) return launch_pdl(nv4_rows_kernel<BF16, T, 2>, grid, 128, 0, st, x, G, nb, q, bs, gs, status);
    if (bpt <= 4) return launch_pdl(nv4_rows_kernel<BF16, T, 4>, grid, 128, 0, st, x, G, nb, q, bs, gs, status);
    return launch_pdl(nv4_rows_kernel<BF16, T, 8>, grid, 128, 0, st, x, G, nb, q, bs, gs, status);
}

template <bool BF16>
static int run_quantize(const void* x, int G, int rows, int cols, uint8_t* q, uint8_t* bs, float* gs, unsigned* ws,
                        int32_t* status, cudaStream_t st) {
    const int nb = cols / 16;
    if (rows == 1)
        return nb <= 32 ? launch_rows<BF16, 32>(x, G, nb, q, bs, gs, status, st)
                        : launch_rows<BF16, 128>(x, G, nb, q, bs, gs, status, st);
    const size_t per = (size_t)rows * nb;
    const unsigned cpm = (unsigned)((per + nv4_chunk<BF16>() - 1) / nv4_chunk<BF16>());
    const int sms = sm_count();
    if (sms < 1) return MOE_ERR_CUDA;
    const unsigned chunks = cpm * (unsigned)G;
    unsigned grid = (unsigned)sms * kNv4CtasPerSm;
    if (grid > chunks) grid = chunks;
    int rc = to_status(cudaMemsetAsync(ws, 0, sizeof(unsigned) * (4 + (size_t)chunks), st));
    if (rc) return rc;
    return launch_pdl(nv4_matrices_kernel<BF16>, grid, 256, 0, st, x, per, cpm, chunks, q, bs, gs, ws, status);
}

static int check_nvfp4(int G, int rows, int cols, int dtype) {
    if (G < 0 || rows < 1 || cols < 32 || cols > MOE_MAX_DIM || (cols & 31)) return MOE_ERR_INVALID_ARG;
    if (rows == 1 ? G > MOE_MAX_ROWS : (G > 65535 || rows > 2 * MOE_MAX_DIM)) return MOE_ERR_INVALID_ARG;
    if (rows > 1 && (int64_t)G * rows * (cols / 16) > MOE_MAX_BLOCKS) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DT_F32 && dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

constexpr int kMaxSms = 152;  // sizes a workspace where no device is visible

static bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

}  // namespace moe

using namespace moe;

extern "C" {

int moe_grouped_gemm(const uint16_t* x, const uint16_t* w, const int32_t* offsets, int R, int N, int K, int E, void* y,
                     int y_dtype, int32_t* dev_status, void* stream) {
    int rc = check_grouped(R, N, K, E, y_dtype);
    if (rc) return rc;
    if (R == 0) return MOE_OK;
    MOE_REQ(x);
    MOE_REQ(w);
    MOE_REQ(offsets);
    MOE_REQ(y);
    MOE_OPT(dev_status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    // fewer tiles than SMs: a few rows' weights stream faster through a warp
    // per weight row on the whole GPU (1536 x 2048, a row an expert: 4 rows 7.1
    // and 10.1 us, 12 rows 15 and 16; beyond, the tiles are ahead)
    if (R <= 32 && R * ceil_div(N, 128) < sms) {
        const dim3 grid((unsigned)ceil_div(N, 8), (unsigned)R);
        const int f32 = y_dtype == MOE_DT_F32;
        return K <= 1024 ? launch_pdl(gg_gemv_kernel<4>, grid, 256, 0, st, x, w, offsets, R, N, K, E, y, f32, dev_status)
                         : launch_pdl(gg_gemv_kernel<8>, grid, 256, 0, st, x, w, offsets, R, N, K, E, y, f32, dev_status);
    }
    GgParams p;
    memset(&p, 0, sizeof p);
    p.offsets = offsets;
    p.out = y;
    p.status = dev_status;
    return y_dtype == MOE_DT_F32 ? run_gg<kGgFwd, true>(p, w, x, R, N, K, E, st)
                                 : run_gg<kGgFwd, false>(p, w, x, R, N, K, E, st);
}

int moe_grouped_gemm_dx(const uint16_t* dy, const uint16_t* w, const int32_t* offsets, int R, int N, int K, int E,
                        void* dx, int dx_dtype, int32_t* dev_status, void* stream) {
    int rc = check_grouped(R, N, K, E, dx_dtype);
    if (rc) return rc;
    if (R == 0) return MOE_OK;
    MOE_REQ(dy);
    MOE_REQ(w);
    MOE_REQ(offsets);
    MOE_REQ(dx);
    MOE_OPT(dev_status);
    GgParams p;
    memset(&p, 0, sizeof p);
    p.offsets = offsets;
    p.out = dx;
    p.status = dev_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dx_dtype == MOE_DT_F32 ? run_gg<kGgDx, true>(p, w, dy, R, N, K, E, st)
                                  : run_gg<kGgDx, false>(p, w, dy, R, N, K, E, st);
}

int moe_grouped_gemm_dw_workspace_bytes(int R, int N, int K, int E, size_t* bytes) {
    const int rc = check_grouped(R, N, K, E, MOE_DT_F32);
    if (rc) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const int sms = sm_count();
    const int split = gg_split(R, N, K, E, sms > 1 ? sms : kMaxSms);
    *bytes = split > 1 ? sizeof(float) * (size_t)split * E * N * K : 0;
    return MOE_OK;
}

int moe_grouped_gemm_dw(const uint16_t* dy, const uint16_t* x, const int32_t* offsets, int R, int N, int K, int E,
                        void* dw, int dw_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                        void* stream) {
    int rc = check_grouped(R, N, K, E, dw_dtype);
    if (rc) return rc;
    MOE_REQ(dw);
    MOE_OPT(dev_status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t n = (size_t)E * N * K;
    if (R == 0) return to_status(cudaMemsetAsync(dw, 0, n * (dw_dtype == MOE_DT_F32 ? 4 : 2), st));
    MOE_REQ(dy);
    MOE_REQ(x);
    MOE_REQ(offsets);
    const int sms = sm_count();
    const int split = gg_split(R, N, K, E, sms > 1 ? sms : kMaxSms);
    if (split > 1) {
        if (!workspace || workspace_bytes < sizeof(float) * split * n) return MOE_ERR_WORKSPACE;
        MOE_REQ(workspace);
    }
    GgParams p;
    memset(&p, 0, sizeof p);
    p.offsets = offsets;
    p.out = split > 1 ? workspace : dw;
    p.split = split;
    p.status = dev_status;
    rc = split > 1 || dw_dtype == MOE_DT_F32 ? run_gg<kGgDw, true>(p, x, dy, R, N, K, E, st)
                                             : run_gg<kGgDw, false>(p, x, dy, R, N, K, E, st);
    if (rc) return rc;
    if (split == 1) return MOE_OK;
    size_t grid = (n / 4 + 31) / 32;
    if (grid > (size_t)sms * 8) grid = (size_t)sms * 8;
    return launch_pdl(gg_join_kernel, (unsigned)grid, 256, 0, st, static_cast<const float4*>(workspace), n / 4, split, dw,
                      (int)(dw_dtype == MOE_DT_F32));
}

int moe_quantize_nvfp4_workspace_bytes(int G, int rows, int cols, size_t* bytes) {
    const int rc = check_nvfp4(G, rows, cols, MOE_DT_F32);
    if (rc) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = rows == 1 ? 0 : align_up(nv4_workspace(G, (size_t)rows * (cols / 16)), 256);
    return MOE_OK;
}

int moe_quantize_nvfp4(const void* x, int x_dtype, int G, int rows, int cols, uint8_t* q, uint8_t* bs, float* gs,
                       void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    int rc = check_nvfp4(G, rows, cols, x_dtype);
    if (rc) return rc;
    if (G == 0) return MOE_OK;
    MOE_REQ(x);
    MOE_REQ(q);
    MOE_REQ(bs);
    MOE_REQ(gs);
    MOE_OPT(dev_status);
    if (!aligned32(x)) return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    if ((rc = moe_quantize_nvfp4_workspace_bytes(G, rows, cols, &need))) return rc;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return MOE_ERR_WORKSPACE;
        MOE_REQ(workspace);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned* ws = static_cast<unsigned*>(workspace);
    return x_dtype == MOE_DT_BF16 ? run_quantize<true>(x, G, rows, cols, q, bs, gs, ws, dev_status, st)
                                  : run_quantize<false>(x, G, rows, cols, q, bs, gs, ws, dev_status, st);
}

int moe_dequantize_nvfp4(const uint8_t* q, const uint8_t* bs, const float* gs, int G, int rows, int cols, void* x,
                         int x_dtype, void* stream) {
    const int rc = check_nvfp4(G, rows, cols, x_dtype);
    if (rc) return rc;
    if (G == 0) return MOE_OK;
    MOE_REQ(q);
    MOE_REQ(bs);
    MOE_REQ(gs);
    MOE_REQ(x);
    if (!aligned32(x)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t per = (size_t)rows * (cols / 16), n = per * G;
    const int sms = sm_count();
    size_t grid = (n + 255) / 256;
    if (grid > (size_t)sms * 64) grid = (size_t)sms * 64;
    return x_dtype == MOE_DT_BF16 ? launch_pdl(nv4_decode_kernel<true>, (unsigned)grid, 256, 0, st, q, bs, gs, per, n, x)
                                  : launch_pdl(nv4_decode_kernel<false>, (unsigned)grid, 256, 0, st, q, bs, gs, per, n, x);
}

int moe_grouped_gemm_nvfp4(const uint8_t* xq, const uint8_t* xbs, const float* xgs, const uint8_t* wq, const uint8_t* wbs,
                           const float* wgs, const int32_t* offsets, int R, int N, int K, int E, void* y, int y_dtype,
                           int32_t* dev_status, void* stream) {
    int rc = check_grouped(R, N, K, E, y_dtype);
    if (rc) return rc;
    if (K & 31) return MOE_ERR_INVALID_ARG;  // rows of codes in whole 16-byte pieces
    if (R == 0) return MOE_OK;
    MOE_REQ(xq);
    MOE_REQ(xbs);
    MOE_REQ(xgs);
    MOE_REQ(wq);
    MOE_REQ(wbs);
    MOE_REQ(wgs);
    MOE_REQ(offsets);
    MOE_REQ(y);
    MOE_OPT(dev_status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 2) return MOE_ERR_CUDA;
    // a few rows: as in moe_grouped_gemm, but the codes cost more instructions
    // than bf16 weights a byte, so the tiles are ahead earlier (1536 x 2048, a
    // row an expert: 2 rows 3.1 and 6.7 us, 8 rows 6.9 and 7.3, 12 rows 9.4 and 7.7)
    if (R <= 32 && 3 * R * ceil_div(N, 128) < 2 * sms) {
        const dim3 grid((unsigned)ceil_div(N, 8 * kG4vRows), (unsigned)R);
        const int f32 = y_dtype == MOE_DT_F32;
        return K <= 1024 ? launch_pdl(g4_gemv_kernel<1>, grid, 256, 0, st, xq, xbs, xgs, wq, wbs, wgs, offsets, R, N, K, E,
                                      y, f32, dev_status)
                         : launch_pdl(g4_gemv_kernel<2>, grid, 256, 0, st, xq, xbs, xgs, wq, wbs, wgs, offsets, R, N, K, E,
                                      y, f32, dev_status);
    }
    G4Params p;
    memset(&p, 0, sizeof p);
    if (!encode_map(&p.ta, wq, 1, K / 2, N, E, 128) || !encode_map(&p.tb, xq, 1, K / 2, R, 0, kGgBoxN) ||
        !encode_map(&p.tb_all, xq, 1, K / 2, R, 0, 128))
        return MOE_ERR_UNSUPPORTED;
    if (K % 256 == 0 && (!encode_map(&p.tsa, wbs, 1, K / 16, N, E, 128, 64) ||
                         !encode_map(&p.tsb, xbs, 1, K / 16, R, 0, kGgBoxN, 64)))
        return MOE_ERR_UNSUPPORTED;
    p.wbs = wbs;
    p.xbs = xbs;
    p.wgs = wgs;
    p.xgs = xgs;
    p.offsets = offsets;
    p.E = E;
    p.R = R;
    p.M = N;
    p.K = K;
    p.out = y;
    p.out_f32 = y_dtype == MOE_DT_F32;
    p.status = dev_status;
    return gg_pairs(R, N, E) ? launch_persistent<2>(g4_kernel<2>, p, kG4Threads, sms, st)
                                                  : launch_persistent<1>(g4_kernel<1>, p, kG4Threads, sms, st);
}

}  // extern "C"
