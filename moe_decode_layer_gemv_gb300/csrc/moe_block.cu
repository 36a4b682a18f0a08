// moe_block.cu -- the C ABI of the operators around the grouped products
// (declared in include/moe.h): the experts' gated unit and its gradient.
// Argument checks, the choice of a kernel and its launch.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "moe.h"
#include "moe_glu.cuh"
#include "moe_grouped.cuh"
#include "moe_host.cuh"
#include "moe_launch.cuh"

namespace moe {

// gate_up [E, 2, I / 8, 8, H] in boxes of 64 columns x 64 gate and 64 up rows,
// in alternating groups of eight.
static bool encode_gate_up(CUtensorMap* map, const void* base, uint64_t H, uint64_t I, uint64_t E) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[5] = {H, 8, 2, I / 8, E};
    const cuuint64_t strides[4] = {H * 2, I * H * 2, 8 * H * 2, 2 * I * H * 2};
    const cuuint32_t box[5] = {64, 8, 2, 8, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int glu_coefficients(int act, float* c0, float* c1) {
    if (act == MOE_ACT_SILU) {
        *c0 = 1.0f;
        *c1 = 0.0f;
    } else if (act == MOE_ACT_GELU) {
        *c0 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
        *c1 = 0.07135481627260025f;  // 0.044715 of it
    } else {
        return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

template <bool F32>
static int run_glu(GgParams& p, const void* gate_up, const void* x, int R, int I, int H, int E, int sms, cudaStream_t st) {
    if (!encode_gate_up(&p.ta, gate_up, H, I, E) || !encode_map(&p.tb, x, 2, H, R, 0, kGgBoxN) ||
        !encode_map(&p.tb_all, x, 2, H, R, 0, 128))
        return MOE_ERR_UNSUPPORTED;
    p.C = H;
    return gg_pairs(R, 2 * I, E)
               ? launch_persistent<2>(gg_kernel<kGgFwd, 2, F32, kGgGlu>, p, GgCfg<kGgFwd, 2, F32>::kThreads, sms, st)
               : launch_persistent<1>(gg_kernel<kGgFwd, 1, F32, kGgGlu>, p, GgCfg<kGgFwd, 1, F32>::kThreads, sms, st);
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_grouped_glu(const uint16_t* x, const uint16_t* gate_up, const int32_t* offsets, int R, int H, int I, int E, int act,
                    void* h, int h_dtype, uint16_t* gu, int32_t* dev_status, void* stream) {
    if (I < 1 || I > MOE_MAX_DIM) return MOE_ERR_INVALID_ARG;
    int rc = check_grouped(R, I, H, E, h_dtype);
    if (rc) return rc;
    GgParams p;
    memset(&p, 0, sizeof p);
    if ((rc = glu_coefficients(act, &p.c0, &p.c1))) return rc;
    if (R == 0) return MOE_OK;
    MOE_REQ(x);
    MOE_REQ(gate_up);
    MOE_REQ(offsets);
    MOE_REQ(h);
    MOE_OPT(gu);
    MOE_OPT(dev_status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 2) return MOE_ERR_CUDA;
    const int f32 = h_dtype == MOE_DT_F32;
    // a few rows: as in moe_grouped_gemm
    if (R <= 32 && R * ceil_div(2 * I, 128) < sms) {
        const dim3 grid((unsigned)ceil_div(I, 8), (unsigned)R);
        return H <= 1024 ? launch_pdl(glu_gemv_kernel<4>, grid, 256, 0, st, x, gate_up, offsets, R, I, H, E, h, f32, gu, p.c0,
                                      p.c1, dev_status)
                         : launch_pdl(glu_gemv_kernel<8>, grid, 256, 0, st, x, gate_up, offsets, R, I, H, E, h, f32, gu, p.c0,
                                      p.c1, dev_status);
    }
    p.offsets = offsets;
    p.E = E;
    p.R = R;
    p.M = I;
    p.out = h;
    p.out2 = gu;
    p.status = dev_status;
    return f32 ? run_glu<true>(p, gate_up, x, R, I, H, E, sms, st) : run_glu<false>(p, gate_up, x, R, I, H, E, sms, st);
}

int moe_grouped_glu_backward(const uint16_t* dy, const uint16_t* down, const uint16_t* gu, const int32_t* offsets, int R,
                             int H, int I, int E, int act, uint16_t* dgu, uint16_t* h, int32_t* dev_status, void* stream) {
    if (H > MOE_MAX_DIM) return MOE_ERR_INVALID_ARG;
    int rc = check_grouped(R, H, I, E, MOE_DT_BF16);
    if (rc) return rc;
    GgParams p;
    memset(&p, 0, sizeof p);
    if ((rc = glu_coefficients(act, &p.c0, &p.c1))) return rc;
    if (R == 0) return MOE_OK;
    MOE_REQ(dy);
    MOE_REQ(down);
    MOE_REQ(gu);
    MOE_REQ(offsets);
    MOE_REQ(dgu);
    MOE_REQ(h);
    MOE_OPT(dev_status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 2) return MOE_ERR_CUDA;
    p.a_blocked = I % 64 == 0;
    if (!(p.a_blocked ? encode_blocked(&p.ta, down, I, H, E) : encode_map(&p.ta, down, 2, I, H, E, 64)) ||
        !encode_map(&p.tb, dy, 2, H, R, 0, kGgBoxN) || !encode_map(&p.tb_all, dy, 2, H, R, 0, 128))
        return MOE_ERR_UNSUPPORTED;
    p.offsets = offsets;
    p.E = E;
    p.R = R;
    p.M = I;
    p.C = H;
    p.out = dgu;
    p.out2 = h;
    p.in = gu;
    p.status = dev_status;
    return gg_pairs(R, I, E)
               ? launch_persistent<2>(gg_kernel<kGgDx, 2, false, kGgGluBack>, p, GgCfg<kGgDx, 2, false>::kThreads, sms, st)
               : launch_persistent<1>(gg_kernel<kGgDx, 1, false, kGgGluBack>, p, GgCfg<kGgDx, 1, false>::kThreads, sms, st);
}

}  // extern "C"
