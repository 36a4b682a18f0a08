// moe_host.cuh -- host-side helpers shared by the library's translation
// units: argument checks, counted kernel launches, the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "moe.h"

namespace moe {

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define MOE_REQ(p) \
    do {           \
        if (!(p) || !aligned16(p)) return MOE_ERR_INVALID_ARG; \
    } while (0)
#define MOE_OPT(p) \
    do {           \
        if ((p) && !aligned16(p)) return MOE_ERR_INVALID_ARG; \
    } while (0)

inline int to_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    return MOE_ERR_CUDA;
}

// Kernels this library has launched in the process (every launch site goes
// through launch_ex or launch_pdl), for measurement: moe_launch_count().
inline std::atomic<unsigned long long> g_launches{0};

template <typename K, typename... Args>
inline int launch_ex(const cudaLaunchConfig_t& cfg, K kernel, Args... args) {
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return to_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// A launch that may start while the kernel ahead of it on the stream is
// finishing (programmatic stream serialization): the kernel's setup overlaps
// the previous kernel's tail; its first read of earlier results waits in
// grid_dep_wait().  Used for the chain of phase kernels of one layer.
template <typename K, typename... Args>
inline int launch_pdl(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_ex(cfg, kernel, args...);
}

// dynamic shared memory above 48 KB needs an opt-in per kernel and device
template <typename K>
inline int allow_smem(K kernel, size_t bytes) {
    if (bytes <= 48 * 1024) return MOE_OK;
    return to_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (a function-local static
// is initialised exactly once even when several host threads call first).
inline EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(f);
        return nullptr;
    }();
    return fn;
}

inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

}  // namespace moe
