// moe_launch.cuh -- host-side helpers of the grouped products' launches,
// shared by the translation units that instantiate them: tensor maps,
// argument limits, the pairing rule, the persistent launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "moe.h"
#include "moe_grouped.cuh"
#include "moe_host.cuh"

namespace moe {

// A tensor map over a row-major tensor [outer2, outer1, inner] (outer2 = 0:
// two dimensions) with boxes of box_bytes x box_rows (128 or 64 bytes, the
// swizzle of that width); elements outside the tensor read as zeros.
inline bool encode_map(CUtensorMap* map, const void* base, int elem, uint64_t inner, uint64_t outer1, uint64_t outer2,
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
inline bool encode_blocked(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer1, uint64_t outer2) {
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

// A 16-bit tensor [rows, cols] in boxes of box_rows x 128 columns: inputs of an epilogue.
inline bool encode_input(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * 2};
    const cuuint32_t box[2] = {128, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int check_grouped(int R, int N, int K, int E, int dtype) {
    if (R < 0 || R > MOE_MAX_ROWS || E < 1 || E > MOE_MAX_E) return MOE_ERR_INVALID_ARG;
    if (N < 8 || N > 2 * MOE_MAX_DIM || (N & 7) || K < 8 || K > MOE_MAX_DIM || (K & 7)) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DT_F32 && dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// The launch itself, of a kernel whose shared memory is allowed already.
template <int CG, typename K, typename P>
inline int launch_clusters(K kernel, const P& p, int threads, int sms, cudaStream_t st) {
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

// A persistent kernel on `sms` SMs, in clusters of CG CTAs.
template <int CG, typename K, typename P>
inline int launch_persistent(K kernel, const P& p, int threads, int sms, cudaStream_t st) {
    const int rc = allow_smem(kernel, kGgSmem);
    return rc ? rc : launch_clusters<CG>(kernel, p, threads, sms, st);
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
// The gated unit and its gradient store more, and the unit in fp32 drains its accumulators more often.  64 experts of
// 1536 x 2048 and 2048 x 768, single and paired, at 128 / 192 / 256 / 512 rows: to bf16 85 / 99 / 107 / 177 and 99 / 103
// / 107 / 150 us, to fp32 91 / 113 / 119 / 205 and 119 / 123 / 130 / 203 (1024 rows: 381 and 351), the gradient 56 / 76
// / 80 / 130 and 60 / 66 / 72 / 117 (144 rows: 70 and 62).  128 experts are ahead a little earlier (144 rows to bf16:
// 177 and 168), 16, whose larger tiles leave some SMs without any, later (512 rows to bf16: 58 and 56, uneven 58 and
// 64; the gradient at 144 rows 33 and 31).
constexpr int kGgPairRowsGlu = 256, kGgPairRowsGluF32 = 512, kGgPairRowsGluBack = 144;

inline bool gg_pairs(int R, int M, int E, int rows = kGgPairRows) { return M > 128 && (int64_t)R >= (int64_t)rows * E; }

}  // namespace moe
