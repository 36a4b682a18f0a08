// moe_nvfp4.cuh -- NVFP4 (E2M1 codes, an E4M3 scale per 16 elements of a
// row, one fp32 scale a matrix or a row): quantisation, its inverse, and the
// product of two NVFP4 operands grouped by expert.
#pragma once

#include "moe_grouped.cuh"

namespace moe {

// ------------------------------------------------------------ quantisation
// For a group (a matrix, or one row) with the finite magnitudes' maximum a:
//   gs = a / 2688 (448 * 6, the largest E4M3 times the largest E2M1),
//        rounded up to 8 significant bits, at least 2^-100
//   bs = E4M3 nearest to (block maximum) / (6 gs)
//   q  = E2M1 nearest to x / (bs gs), both ties to even
// With 8 bits in gs and 4 in bs the divisors 6 gs and bs gs are exact in
// fp32, and a quotient of fp32 numbers by a divisor of at most 12 bits that
// is not on a rounding border of the coarse formats does not round onto one:
// the results are those of exact arithmetic.
constexpr float kNv4Top = 2688.0f;
constexpr float kNv4MinScale = 7.888609052210118e-31f;  // 2^-100
constexpr uint32_t kNv4MaxScaleBits = 0x79c30000u;      // the largest 8-bit scale with 2688 gs finite

__device__ __forceinline__ float nv4_scale(float amax) {
    const float f = __fdiv_ru(amax, kNv4Top);
    const uint32_t up = (__float_as_uint(f) + 0xffffu) & 0xffff0000u;
    return fmaxf(__uint_as_float(min(up, kNv4MaxScaleBits)), kNv4MinScale);
}

// A reciprocal to about one step (the quotients made with it are corrected
// by their remainders; s is normal and so is 1 / s).
__device__ __forceinline__ float nv4_rcp(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}

struct Nv4Scale {
    float gs, six, inv6;  // 6 gs and its reciprocal
    __device__ __forceinline__ explicit Nv4Scale(float amax) {
        gs = nv4_scale(amax);
        six = 6.0f * gs;
        inv6 = nv4_rcp(six);
    }
};

// 32 bytes of global memory in one load or store (both 32-byte aligned).
struct alignas(32) Words8 {
    uint32_t w[8];
};
__device__ __forceinline__ Words8 ld_words8(const void* p) {
    Words8 r;
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(p));
    return r;
}
__device__ __forceinline__ void st_words8(void* p, const Words8& r) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
                 "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                 : "memory");
}

// One 16-element block as loaded: bf16 pairs (8 words) or fp32 (16 words).
template <bool BF16>
struct Nv4Block {
    Words8 w[BF16 ? 1 : 2];

    __device__ __forceinline__ void load(const void* x, size_t block) {
        const char* p = static_cast<const char*>(x) + block * (BF16 ? 32 : 64);
        w[0] = ld_words8(p);
        if (!BF16) w[1] = ld_words8(p + 32);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[0].w[i] = 0;
        if (!BF16)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[1].w[i] = 0;
    }
    // the largest magnitude among the finite elements; `bad` if any is not finite
    __device__ __forceinline__ float amax(bool& bad) const {
        if (BF16) {
            // magnitudes of bf16 numbers order like their bits: two a word
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[0].w[i] & 0x7fff7fffu);
            uint32_t t = max(m & 0xffffu, m >> 16);
            bad = t >= 0x7f80u;
            if (bad) {
                t = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t lo = w[0].w[i] & 0x7fffu, hi = (w[0].w[i] >> 16) & 0x7fffu;
                    if (lo < 0x7f80u) t = max(t, lo);
                    if (hi < 0x7f80u) t = max(t, hi);
                }
            }
            return __uint_as_float(t << 16);
        }
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < (BF16 ? 1 : 2); ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) t = max(t, w[j].w[i] & 0x7fffffffu);
        bad = t >= 0x7f800000u;
        if (bad) {
            t = 0;
#pragma unroll
            for (int j = 0; j < (BF16 ? 1 : 2); ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t b = w[j].w[i] & 0x7fffffffu;
                    if (b < 0x7f800000u) t = max(t, b);
                }
        }
        return __uint_as_float(t);
    }
    // elements 2i and 2i + 1
    __device__ __forceinline__ float2 pair(int i) const {
        if (BF16) return bf16x2_to_f2(w[0].w[i]);
        const Words8& v = w[BF16 ? 0 : i >> 2];
        return make_float2(__uint_as_float(v.w[(2 * i) & 7]), __uint_as_float(v.w[(2 * i + 1) & 7]));
    }
    // codes (8 bytes) and block scale (1 byte) under the group's scale, for a
    // block whose finite maximum is m; a block with an element that is not
    // finite (bad) decodes to NaN throughout
    __device__ __forceinline__ void encode(float m, bool bad, const Nv4Scale& g, uint8_t* q, uint8_t* bs,
                                           size_t block) const {
        const float q0 = m * g.inv6;
        const uint32_t b =
            __nv_cvt_float_to_fp8(fmaf(fmaf(q0, g.six, -m), -g.inv6, q0), __NV_SATFINITE, __NV_E4M3);
        const float s = f8_to_f(b) * g.gs;
        const float inv = s > 0.0f && !bad ? nv4_rcp(s) : 0.0f;
        const float2 s2 = make_float2(s, s), inv2 = make_float2(inv, inv), ninv2 = make_float2(-inv, -inv);
        uint32_t out[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // x / s to nearest: the product with the reciprocal, corrected
                // once by its exact remainder t s - x (written this way round a
                // zero keeps its sign)
                const float2 x = pair(4 * h + i), t = __fmul2_rn(x, inv2);
                v[i] = __ffma2_rn(__ffma2_rn(t, s2, make_float2(-x.x, -x.y)), ninv2, t);
            }
            asm("{\n\t.reg .b8 a, b, c, d;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
                "mov.b32 %0, {a, b, c, d};\n\t}"
                : "=r"(out[h])
                : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
        }
        if (bad) out[0] = out[1] = 0;
        *reinterpret_cast<uint2*>(q + block * 8) = make_uint2(out[0], out[1]);
        bs[block] = (uint8_t)(bad ? 0x7fu : b);
    }
};

// (Rows of 2048: bf16 6.2 TB/s, fp32 7.1 TB/s read and written.)
// One scale a row: T threads hold a row's blocks in registers (up to BPT
// each), find its maximum and write its codes -- x is read once.
template <bool BF16, int T, int BPT>
__global__ void __launch_bounds__(128) nv4_rows_kernel(const void* x, int G, int nb, uint8_t* q, uint8_t* bs,
                                                       float* gs, int32_t* status) {
    __shared__ float s_max[4];
    grid_dep_wait();
    const int sub = threadIdx.x / T, t = threadIdx.x % T;
    const size_t row = (size_t)blockIdx.x * (128 / T) + sub;
    const bool live = row < (size_t)G;
    Nv4Block<BF16> blk[BPT];
    float m = 0.0f, mine[BPT];
    bool any_bad = false, bad[BPT];
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
        const int b = j * T + t;
        if (live && b < nb)
            blk[j].load(x, row * nb + b);
        else
            blk[j].clear();
    }
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
        mine[j] = blk[j].amax(bad[j]);
        m = fmaxf(m, mine[j]);
        any_bad |= bad[j];
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // magnitudes order like their bits
    if (T > 32) {
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
        __syncthreads();
        m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    }
    const Nv4Scale scale(m);
    if (any_bad) set_status(status, MOE_DEV_NONFINITE);
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
        const int b = j * T + t;
        if (live && b < nb) blk[j].encode(mine[j], bad[j], scale, q, bs, row * nb + b);
    }
    if (live && t == 0) gs[row] = scale.gs;
}

// One scale a matrix.  The matrices are cut into chunks of 32 KB, numbered
// through; step t reads chunk t for its maximum and writes the codes of chunk
// t - lag, whose matrix's maxima are all known by then and which is still in
// L2 (lag: a matrix, and the steps in flight): x comes from HBM once.  Steps
// are claimed in order, so that the chunks a step waits for belong to steps
// claimed before it, whose maxima wait for nothing.  Workspace (zeroed):
// claimed steps, then per chunk its maximum's bits with the sign bit set --
// the word is its own flag, no fence orders it.
// Measured: 256 matrices of 2048 x 768 bf16, 195 us (5.3 TB/s of bytes that
// count; reading x twice from HBM 290); instruction issue is 58 % busy, the
// steps' barriers are the rest.
constexpr int kNv4CtasPerSm = 4;
template <bool BF16>
__host__ __device__ constexpr int nv4_bpt() {  // blocks a thread
    return BF16 ? 4 : 2;
}
template <bool BF16>
__host__ __device__ constexpr int nv4_chunk() {
    return 256 * nv4_bpt<BF16>();
}
// words of workspace for G matrices of `per` blocks, whatever x's type
static inline size_t nv4_workspace(int G, size_t per) {
    return sizeof(unsigned) * (4 + (size_t)G * ((per + nv4_chunk<false>() - 1) / nv4_chunk<false>()));
}

__device__ __forceinline__ unsigned ld_relaxed_gpu(const unsigned* p) {
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_relaxed_gpu(unsigned* p, unsigned v) {
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

template <bool BF16>
__global__ void __launch_bounds__(256, kNv4CtasPerSm) nv4_matrices_kernel(const void* x, size_t per,
                                                                          unsigned cpm, unsigned chunks, uint8_t* q,
                                                                          uint8_t* bs, float* gs, unsigned* ws,
                                                                          int32_t* status) {
    constexpr int BPT = nv4_bpt<BF16>();
    constexpr unsigned kFlag = 0x80000000u;
    __shared__ unsigned s_step, s_max[8], s_all[8];
    unsigned* amax = ws + 4;
    grid_dep_wait();
    const unsigned lag = cpm + gridDim.x;
    if (threadIdx.x == 0) s_step = atomicAdd(ws, 1u);
    for (;;) {
        __syncthreads();
        const unsigned t = s_step;
        if (t >= chunks + lag) return;
        unsigned next = 0;
        if (threadIdx.x == 0) next = atomicAdd(ws, 1u);  // on its way while this step runs
        Nv4Block<BF16> blk[BPT];
        if (t < chunks) {
            const unsigned g = t / cpm, c = t - g * cpm;
            const size_t b0 = (size_t)c * nv4_chunk<BF16>() + threadIdx.x;
            float m = 0.0f;
            bool any_bad = false;
#pragma unroll
            for (int j = 0; j < BPT; ++j) {
                if (b0 + j * 256 < per)
                    blk[j].load(x, g * per + b0 + j * 256);
                else
                    blk[j].clear();
            }
#pragma unroll
            for (int j = 0; j < BPT; ++j) {
                bool bad;
                m = fmaxf(m, blk[j].amax(bad));
                any_bad |= bad;
            }
            const unsigned w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));  // magnitudes order like their bits
            if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = w;
            if (any_bad) set_status(status, MOE_DEV_NONFINITE);
        }
        __syncthreads();
        if (t < chunks && threadIdx.x == 0) {
            unsigned v = s_max[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) v = max(v, s_max[i]);
            st_relaxed_gpu(amax + t, v | kFlag);
        }
        if (t >= lag) {
            const unsigned u = t - lag, g = u / cpm, c = u - g * cpm;
            const size_t b0 = (size_t)c * nv4_chunk<BF16>() + threadIdx.x;
#pragma unroll
            for (int j = 0; j < BPT; ++j) {
                if (b0 + j * 256 < per)
                    blk[j].load(x, g * per + b0 + j * 256);
                else
                    blk[j].clear();
            }
            unsigned top = 0;
            for (unsigned i = threadIdx.x; i < cpm; i += 256) {
                unsigned v = ld_relaxed_gpu(amax + (size_t)g * cpm + i);
                for (unsigned n = 0; !(v & kFlag) && n < (1u << 22); ++n) {
                    __nanosleep(64);
                    v = ld_relaxed_gpu(amax + (size_t)g * cpm + i);
                }
                if (!(v & kFlag)) set_status(status, MOE_DEV_TIMEOUT);
                top = max(top, v & ~kFlag);
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if ((threadIdx.x & 31) == 0) s_all[threadIdx.x >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, s_all[i]);
            const Nv4Scale scale(__uint_as_float(top));
#pragma unroll
            for (int j = 0; j < BPT; ++j) {
                bool bad;
                const float m = blk[j].amax(bad);
                if (b0 + j * 256 < per) blk[j].encode(m, bad, scale, q, bs, g * per + b0 + j * 256);
            }
            if (c == 0 && threadIdx.x == 0) gs[g] = scale.gs;
        }
        if (threadIdx.x == 0) s_step = next;
    }
}

// Values e2m1(q) * e4m3(bs) * gs: a thread per block (the first two factors'
// product is exact, the rounding is that of the last product, and of bf16).
// 6.7 TB/s: HBM.
template <bool BF16>
__global__ void __launch_bounds__(256) nv4_decode_kernel(const uint8_t* q, const uint8_t* bs,
                                                         const float* gs, size_t per, size_t n, void* x) {
    grid_dep_wait();
    for (size_t b = (size_t)blockIdx.x * blockDim.x + threadIdx.x; b < n; b += (size_t)gridDim.x * blockDim.x) {
        const uint2 c = reinterpret_cast<const uint2*>(q)[b];
        const float s = f8_to_f(bs[b]), g = gs[b / per];
        Words8 o[BF16 ? 1 : 2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = f4x2_to_f2(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xffu);
            const float lo = v.x * s * g, hi = v.y * s * g;
            if (BF16) {
                o[0].w[i] = (uint32_t)f2bf_bits(lo) | ((uint32_t)f2bf_bits(hi) << 16);
            } else {
                o[BF16 ? 0 : i >> 2].w[(2 * i) & 7] = __float_as_uint(lo);
                o[BF16 ? 0 : i >> 2].w[(2 * i + 1) & 7] = __float_as_uint(hi);
            }
        }
        char* at = static_cast<char*>(x) + b * (BF16 ? 32 : 64);
        st_words8(at, o[0]);
        if (!BF16) st_words8(at + 32, o[BF16 ? 0 : 1]);
    }
}

// ------------------------------------------------------------- the product
// y[r, n] = xgs[r] wgs[e] sum_k (xq bs)(wq bs): tcgen05.mma block-scaled
// (kind::mxf4nvf4, one E4M3 scale per 16 elements), fp32 accumulation.  The
// codes go to shared memory by TMA like the bf16 operands (a 128-byte row
// holds 256 elements, one stage).  An MMA of 64 elements takes a row's four
// scale bytes as one 32-bit word of tensor memory, row 32 j + i at lane i of
// column j, the same in all four lane quarters: four warps, one a quarter,
// read 16 bytes a row (a stage's 16 blocks) from shared memory and write
// tensor memory themselves.  A lane that reads rows i, i + 32, ... holds
// exactly its column words of every 64-element step, so nothing is exchanged.
// (tcgen05.cp does the same copy on the tensor pipe, in line with the MMAs:
// it took 0.3 of the large product's time.)
// A sum is not cut into parts as those of bf16 operands are: K <= MOE_MAX_DIM
// is at most 256 additions, and what they truncate is bounded.  Sums of one
// sign lose up to 1.3e-6 at K = 4096 and 5.3e-6 at 16384, the most where the
// block scales differ widely (2.4e-6 at 16384 where they do not).  Parts of
// 4096 terms take that to 1.2e-6, but beside the scales there is room for one
// accumulator and the sums of a pair's tile spill: 16384 rows of K = 8192 to
// fp32 took 125 us instead of 92.
// Measured: 65536 rows over 64 experts of 1536 x 2048, 104 us (4.0 PFLOP/s).
// At the nominal 4-bit rate its operations are 31 us (not measured; the tensor
// pipe is active 36 % of the time).  Without the copies, scale reads and
// stores, the MMAs and a stage's hand-overs (8 stages a tile) still took 86 of
// 108 us: the hand-overs bound it, then the accumulator's drain.  32 rows over 256 experts: 16.5
// us, 8 of them the bytes.
constexpr int kG4Epi = 8;                 // epilogue warps: lane quarter w & 3, half of the columns w >> 2
constexpr int kG4Threads = 32 * (kG4Epi + 6);  // warp 8 TMA, 9 MMA, 10-13 scales
constexpr int kG4A = 128 * 128;           // codes of 128 rows x 256 elements
constexpr int kG4SfStages = 4;            // stages whose scales one copy brings: 64 bytes a row
constexpr int kG4MaxStages = 8;
constexpr uint32_t kG4SfCol = 256;        // tensor-memory column of the scales, behind the accumulators

// CG = 1: 128 x 128 tiles, two accumulators.  CG = 2 (a CTA pair): 256 x 256
// tiles, one accumulator -- the other 256 columns hold scales; eight epilogue
// warps take it to registers in two steps, so that the next tile's MMAs start
// some hundred cycles later.
template <int CG>
struct G4Cfg {
    static constexpr int BN = 128 * CG;
    static constexpr int ACC = CG == 1 ? 2 : 1;
    static constexpr int SFA = 16, SFB = BN / 32 * 4;        // columns a stage
    static constexpr int S = 256 / (SFA + SFB);              // stages whose scales tensor memory holds (8, 5)
};

template <int V>
struct IntC {
    static constexpr int value = V;
};

struct G4Params {
    CUtensorMap ta, tb;    // wq [E, N, K/2], xq [R, K/2] bytes
    CUtensorMap tb_all;    // tb with boxes of 128 rows
    CUtensorMap tsa, tsb;  // wbs [E, N, K/16], xbs [R, K/16] bytes (K % 256 == 0)
    const uint8_t *wbs, *xbs;
    const float *wgs, *xgs;
    const int32_t* offsets;
    int E, R, M, K;
    void* out;
    int out_f32;
    int32_t* status;
};

struct G4Shared {
    GgShared g;
    alignas(16) float xg[kG4Epi][128];  // the epilogue warps' row scales
    uint64_t cfull[2], cempty[2];  // a copy of scales is in shared memory; the scale warps have read it
};
constexpr int kG4Control = 8192;
static_assert(sizeof(G4Shared) <= kG4Control, "control block");

// Instruction descriptor, kind::mxf4nvf4: E2M1 A and B, E4M3 scales.
__device__ __forceinline__ uint32_t umma_idesc_nvfp4(int M, int N) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void umma_nvfp4(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// 16 words of this lane to 16 consecutive columns
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The 16 scale bytes of a row from block k0 on, from global memory; blocks
// from nb on read as 0 (nb is even: K % 32 == 0).
__device__ __forceinline__ uint4 g4_row_scales(const uint8_t* row, int k0, int nb) {
    const uint8_t* p = row + k0;
    uint32_t w[4] = {0, 0, 0, 0};
    if ((nb & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k0 + 4 * i < nb) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k0 + 2 * i < nb)
                w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 2 * i) << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int CG>
__global__ void __launch_bounds__(kG4Threads, 1) g4_kernel(const __grid_constant__ G4Params p) {
    using Cfg = G4Cfg<CG>;
    extern __shared__ __align__(1024) unsigned char gg_smem_raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(gg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    G4Shared* s4 = reinterpret_cast<G4Shared*>(base);
    GgShared* sh = &s4->g;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const int unit = (int)blockIdx.x / CG, units = (int)gridDim.x / CG;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kG4MaxStages; ++s) {
            mbar_init(&sh->full[s], 1 + 4 * CG);  // the tiles, and the four scale warps (of both CTAs)
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], kG4Epi * CG);
            mbar_init(&s4->cfull[a], 1);
            mbar_init(&s4->cempty[a], 4);
        }
        mbar_init(&sh->mma_done, 1);
        sh->abort = 0;
        fence_mbar_init();
        prefetch_map(&p.ta);
        prefetch_map(&p.tb);
        prefetch_map(&p.tb_all);
        if ((p.K & 255) == 0) {
            prefetch_map(&p.tsa);
            prefetch_map(&p.tsb);
        }
    }
    if (warp == 9) gg_tmem_alloc<CG>(&sh->tmem_slot, kGgTmemCols);
    grid_dep_wait();
    const int mtiles = (p.M + 128 * CG - 1) / (128 * CG);
    gg_segments(sh, p.offsets, 0, p.E, p.R, Cfg::BN, p.status);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_slot;

    // shared memory: two copies of scales (128 weight rows, then the tile's
    // rows, 64 bytes each), then the ring of codes (128 weight rows, then this
    // CTA's share of the tile's rows).  One CTA's tiles hold as many rows as
    // the largest segment needs.
    const int nrows = CG == 2 ? Cfg::BN : min(Cfg::BN, max(kGgBoxN, (sh->nmax + kGgBoxN - 1) / kGgBoxN * kGgBoxN));
    const bool sf_tma = (p.K & 255) == 0;
    const uint32_t sf_bytes = sf_tma ? (128u + (uint32_t)nrows) * 64u : 0u;
    unsigned char* sfbuf = base + kG4Control;
    unsigned char* ring = sfbuf + 2 * sf_bytes;
    const uint32_t stage_bytes = kG4A + (uint32_t)(nrows / CG) * 128u;
    const uint32_t S = min((uint32_t)Cfg::S, ((uint32_t)kGgSmem - 1023u - (uint32_t)kG4Control - 2u * sf_bytes) / stage_bytes);
    const int nk = (p.K + 255) / 256, nb = p.K / 16;

    auto walk = [&](auto f) {
        int e = 0;
        const int rows = sh->start[p.E];
        for (GgWalk w(unit, units, mtiles); w.outer < rows; w.next()) {
            e = gg_seek(sh->start, p.E, w.outer, e);
            const int m0 = w.inner * 128 * CG + (int)rank * 128, n0 = (w.outer - sh->start[e]) * Cfg::BN;
            if (!f(e, sh->p0[e] + n0, min(Cfg::BN, sh->cnt[e] - n0), m0)) break;
        }
    };
    // rows of the tile that each CTA holds, in whole boxes
    auto share = [](int n) { return (n + kGgBoxN * CG - 1) / (kGgBoxN * CG) * kGgBoxN; };

    if (warp == 8) {
        // ---------------- TMA producer
        GgRing r, c;
        const uint32_t ring_at = smem_u32(ring), sf_at = smem_u32(sfbuf);
        const uint32_t bars = CG == 1 ? smem_u32(sh->full) : cluster_addr(sh->full, 0);
        if (gg_elect()) {
            walk([&](int e, int q0, int n, int m0) -> bool {
                const int rows = share(n);
                for (int k = 0; k < nk; ++k) {
                    if (sf_tma && k % kG4SfStages == 0) {
                        if (!gg_wait(&s4->cempty[c.s], c.ph ^ 1u, &sh->abort)) return false;
                        const uint32_t sf = sf_at + c.s * sf_bytes, bar = smem_u32(&s4->cfull[c.s]);
                        mbar_arrive_expect_tx(&s4->cfull[c.s], (128u + (uint32_t)(rows * CG)) * 64u);
                        gg_load3<1>(sf, &p.tsa, k * 16, m0, e, bar);
                        for (int i = 0; i < rows * CG; i += kGgBoxN)
                            gg_load2<1>(sf + 8192 + i * 64, &p.tsb, k * 16, q0 + i, bar);
                        c.next(2);
                    }
                    if (!gg_wait(&sh->empty[r.s], r.ph ^ 1u, &sh->abort)) return false;
                    const uint32_t st = ring_at + r.s * stage_bytes, bar = bars + r.s * 8u;
                    if (rank == 0) mbar_arrive_expect_tx(&sh->full[r.s], CG * (kG4A + (uint32_t)rows * 128u));
                    gg_load3<CG>(st, &p.ta, k * 128, m0, e, bar);
                    if (rows == 128)
                        gg_load2<CG>(st + kG4A, &p.tb_all, k * 128, q0 + (int)rank * 128, bar);
                    else
                        for (int i = 0; i < rows; i += kGgBoxN)
                            gg_load2<CG>(st + kG4A + i * 128, &p.tb, k * 128, q0 + (int)rank * rows + i, bar);
                    r.next(S);
                }
                return true;
            });
            // teardown: also the copies of scales have landed
            gg_drain<CG>(sh, S, r, rank);
            for (uint32_t u = 0; u < 2 && u < c.uses; ++u) gg_settle(&s4->cfull[u], u < c.s ? c.ph : c.ph ^ 1u);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ---------------- MMA issuer (one thread of the leader)
        GgRing r;
        int buf = 0;
        uint32_t free_ph = 1;
        const uint32_t ring_at = smem_u32(ring);
        if (rank == 0 && gg_elect()) walk([&](int e, int q0, int n, int m0) -> bool {
            const uint32_t idesc = umma_idesc_nvfp4(128 * CG, share(n) * CG);
            if (!gg_wait(&sh->acc_empty[buf], free_ph, &sh->abort)) return false;
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf * Cfg::BN);
            uint32_t acc = 0;
            for (int k = 0; k < nk; ++k) {
                if (!gg_wait(&sh->full[r.s], r.ph, &sh->abort)) return false;
                tc_fence_after();
                const uint32_t st = ring_at + r.s * stage_bytes;
                const uint32_t sfa = tmem + kG4SfCol + r.s * (uint32_t)(Cfg::SFA + Cfg::SFB), sfb = sfa + Cfg::SFA;
                const int left = p.K - k * 256;
                const uint64_t ad = umma_sdesc(st), bd = umma_sdesc(st + kG4A);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk * 64 >= left) break;
                    umma_nvfp4<CG>(tacc, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc,
                                   sfa + kk * (Cfg::SFA / 4), sfb + kk * (Cfg::SFB / 4), acc);
                    acc = 1;
                }
                gg_commit<CG>(&sh->empty[r.s]);
                r.next(S);
            }
            gg_commit<CG>(&sh->acc_full[buf]);
            if (++buf == Cfg::ACC) {
                buf = 0;
                free_ph ^= 1u;
            }
            return true;
        });
        __syncwarp();
        if (rank == 0 && gg_elect()) {
            gg_commit_own<CG>(&sh->mma_done);
            gg_settle(&sh->mma_done, 0u);
        }
        __syncwarp();
    } else if (warp >= 10) {
        // ---------------- scales into this warp's quarter of tensor memory
        GgRing r, c;
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        constexpr int NB = Cfg::BN / 32;
        // one stage's words: rows 32 j + lane of the weights (a) and of the tile (b)
        auto put = [&](const uint4(&a)[4], const uint4(&b)[NB]) -> bool {
            if (!gg_wait_warp(&sh->empty[r.s], r.ph ^ 1u, &sh->abort)) return false;
            tc_fence_after();
            const uint32_t at = tmem + quarter + kG4SfCol + r.s * (uint32_t)(Cfg::SFA + Cfg::SFB);
            const uint32_t wa[16] = {a[0].x, a[1].x, a[2].x, a[3].x, a[0].y, a[1].y, a[2].y, a[3].y,
                                     a[0].z, a[1].z, a[2].z, a[3].z, a[0].w, a[1].w, a[2].w, a[3].w};
            tmem_st16(at, wa);
            uint32_t wb[4 * NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                wb[j] = b[j].x;
                wb[NB + j] = b[j].y;
                wb[2 * NB + j] = b[j].z;
                wb[3 * NB + j] = b[j].w;
            }
#pragma unroll
            for (int j = 0; j < 4 * NB; j += 16)
                tmem_st16(at + Cfg::SFA + j, *reinterpret_cast<const uint32_t(*)[16]>(wb + j));
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 1)
                    mbar_arrive(&sh->full[r.s]);
                else
                    mbar_arrive_cluster(&sh->full[r.s], 0);
            }
            r.next(S);
            return true;
        };
        if (sf_tma) {
            const unsigned char* sf0 = sfbuf + lane * 64;
            walk([&](int e, int q0, int n, int m0) -> bool {
                for (int k = 0; k < nk; ++k) {
                    const int kq = k % kG4SfStages;
                    if (kq == 0 && !gg_wait_warp(&s4->cfull[c.s], c.ph, &sh->abort)) return false;
                    // 64-byte swizzle: 16-byte chunk kq of row r is at chunk kq ^ ((r >> 1) & 3)
                    const unsigned char* sf = sf0 + c.s * sf_bytes + (kq ^ ((lane >> 1) & 3)) * 16;
                    uint4 a[4], b[NB];
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] = *reinterpret_cast<const uint4*>(sf + j * 2048);
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        b[j] = 32 * j < n ? *reinterpret_cast<const uint4*>(sf + 8192 + j * 2048) : make_uint4(0, 0, 0, 0);
                    if (kq == kG4SfStages - 1 || k == nk - 1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s4->cempty[c.s]);
                        c.next(2);
                    }
                    if (!put(a, b)) return false;
                }
                return true;
            });
        } else {
            walk([&](int e, int q0, int n, int m0) -> bool {
                for (int k = 0; k < nk; ++k) {
                    // rows beyond the tile's end take the last one's scales:
                    // what they scale is zero or never stored
                    uint4 a[4], b[NB];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        a[j] = g4_row_scales(p.wbs + ((size_t)e * p.M + min(m0 + 32 * j + lane, p.M - 1)) * nb, k * 16, nb);
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        b[j] = 32 * j < n ? g4_row_scales(p.xbs + (size_t)(q0 + min(32 * j + lane, n - 1)) * nb, k * 16, nb)
                                          : make_uint4(0, 0, 0, 0);
                    if (!put(a, b)) return false;
                }
                return true;
            });
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: lane quarter warp & 3, half of the columns
        int buf = 0;
        uint32_t full_ph = 0;
        constexpr int COLS = Cfg::BN / 2;
        const int c0 = (warp >> 2) * COLS;
        float* xg = s4->xg[warp];  // this warp's columns' scales
        walk([&](int e, int q0, int n, int m0) -> bool {
            const int m = m0 + (warp & 3) * 32 + lane;
            const int mine = min(COLS, n - c0);  // columns of this warp; none below 1
            const float wg = ld_input_f(p.wgs + e);
            float mg[COLS / 32];
#pragma unroll
            for (int i = 0; i < COLS / 32; ++i) mg[i] = 32 * i + lane < mine ? ld_input_f(p.xgs + q0 + c0 + 32 * i + lane) : 0.0f;
            if (!gg_wait_warp(&sh->acc_full[buf], full_ph, &sh->abort)) return false;
#pragma unroll
            for (int i = 0; i < COLS / 32; ++i) xg[32 * i + lane] = mg[i];
            __syncwarp();
            tc_fence_after();
            const uint32_t taddr = tmem + (uint32_t)(buf * Cfg::BN + c0) + ((uint32_t)((warp & 3) * 32) << 16);
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 1)
                        mbar_arrive(&sh->acc_empty[buf]);
                    else
                        mbar_arrive_cluster(&sh->acc_empty[buf], 0);
                }
            };
            auto scaled = [&](uint32_t(&v)[32], int c) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(xg + c + j);
                    v[j] = __float_as_uint(__uint_as_float(v[j]) * x.x * wg);
                    v[j + 1] = __float_as_uint(__uint_as_float(v[j + 1]) * x.y * wg);
                    v[j + 2] = __float_as_uint(__uint_as_float(v[j + 2]) * x.z * wg);
                    v[j + 3] = __float_as_uint(__uint_as_float(v[j + 3]) * x.w * wg);
                }
            };
            if (mine <= 0) {
                release();
            } else if (p.out_f32 || mine < COLS) {
#pragma unroll 1
                for (int c = 0; c < mine; c += 32) {
                    uint32_t v[32];
                    gg_ld32(taddr + c, v);
                    gg_ld_wait(v);
                    if (c + 32 >= mine) release();
                    scaled(v, c);
                    gg_store32(v, p.out, p.out_f32, (size_t)q0 + c0 + c, min(32, mine - c), m, p.M);
                }
            } else {
                // everything into registers, all but the last 32 columns as
                // bf16; then the release, then the stores
                uint32_t h[COLS / 32 - 1][16], v[32];
#pragma unroll
                for (int i = 0; i < COLS / 32 - 1; ++i) {
                    gg_ld32(taddr + 32 * i, v);
                    gg_ld_wait(v);
                    scaled(v, 32 * i);
#pragma unroll
                    for (int j = 0; j < 16; ++j) h[i][j] = gg_pack(v[2 * j], v[2 * j + 1]);
                }
                gg_ld32(taddr + COLS - 32, v);
                gg_ld_wait(v);
                release();
                const int odd = m & 1;
                const uint32_t sel = gg_pair_select(odd);
                const bool live = m < p.M;
                uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                          ((size_t)q0 + c0 + odd) * (size_t)p.M + (m - odd));
#pragma unroll
                for (int j = 0; j < COLS / 2 - 16; ++j, o += p.M) {
                    const uint32_t w = gg_pair(h[j / 16][j % 16], sel);
                    if (live) *o = w;
                }
                scaled(v, COLS - 32);
                gg_store32(v, p.out, 0, (size_t)q0 + c0 + COLS - 32, 32, m, p.M);
            }
            if (++buf == Cfg::ACC) {
                buf = 0;
                full_ph ^= 1u;
            }
            return true;
        });
    }
    __syncthreads();
    if (*(volatile int*)&sh->abort && threadIdx.x == 0) set_status(p.status, MOE_DEV_TIMEOUT);
    if (CG == 2) cluster_sync();
    if (warp == 9) {
        tc_fence_after();
        gg_tmem_dealloc<CG>(tmem, kGgTmemCols);
    }
}

// ------------------------------------------------------- a few rows at once
// The NVFP4 product for a handful of rows, a warp per weight row as in
// gg_gemv_kernel: 32 elements (16 bytes of codes, two block scales) a lane at
// a time.  A block's products are summed in f16 pairs without rounding: eight
// products of E2M1 values a lane half, multiples of 1/4 up to 288; the scales'
// product is exact in fp32.
constexpr int kG4vRows = 2;  // weight rows a warp: a decoded piece of x serves them all

__device__ __forceinline__ __half2 g4_half2(uint32_t codes, int byte) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((codes >> (8 * byte)) & 0xffu), __NV_E2M1);
    return *reinterpret_cast<const __half2*>(&h);
}

// sum over a block: 16 codes of w, x decoded
__device__ __forceinline__ float g4_block(uint32_t w0, uint32_t w1, const __half2* x) {
    __half2 s = __hmul2(g4_half2(w0, 0), x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = __hfma2(g4_half2(w0, i), x[i], s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __hfma2(g4_half2(w1, i), x[4 + i], s);
    const float2 f = __half22float2(s);
    return f.x + f.y;
}

template <int J>
__global__ void __launch_bounds__(256) g4_gemv_kernel(const uint8_t* xq, const uint8_t* xbs,
                                                      const float* xgs, const uint8_t* wq,
                                                      const uint8_t* wbs, const float* wgs,
                                                      const int32_t* offsets, int R, int N, int K, int E,
                                                      void* y, int out_f32, int32_t* status) {
    constexpr int RW = kG4vRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    const int r = blockIdx.y;
    int p0, p1;
    const int e = gg_row_segment(offsets, E, R, r, p0, p1, status);
    if (e < 0 || (r - p0) % kGgvTok) return;
    const int nt = min(kGgvTok, p1 - r);
    const int n = (blockIdx.x * 8 + warp) * RW;  // N is a multiple of RW
    if (n >= N) return;
    const int chunks = K / 32;  // 16 bytes of codes, 2 bytes of scales each
    const size_t wrow = ((size_t)e * N + n) * chunks, xrow = (size_t)r * chunks;
    float acc[kGgvTok][RW] = {};
    for (int c0 = 0; c0 < chunks; c0 += 32 * J) {
        uint4 wv[J][RW];
        uint32_t ws[J][RW];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = c0 + j * 32 + lane;
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const size_t at = wrow + (size_t)i * chunks + c;
                wv[j][i] = c < chunks ? ld_stream_v4(wq + at * 16) : make_uint4(0, 0, 0, 0);
                ws[j][i] = c < chunks ? reinterpret_cast<const uint16_t*>(wbs)[at] : 0;
            }
        }
#pragma unroll
        for (int t = 0; t < kGgvTok; ++t) {
            if (t >= nt) break;
            uint4 xv[J];
            uint32_t xs[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = c0 + j * 32 + lane;
                const size_t at = xrow + (size_t)t * chunks + c;
                xv[j] = c < chunks ? *reinterpret_cast<const uint4*>(xq + at * 16) : make_uint4(0, 0, 0, 0);
                xs[j] = c < chunks ? reinterpret_cast<const uint16_t*>(xbs)[at] : 0;
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                __half2 h[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = g4_half2(xv[j].x, i);
                    h[4 + i] = g4_half2(xv[j].y, i);
                    h[8 + i] = g4_half2(xv[j].z, i);
                    h[12 + i] = g4_half2(xv[j].w, i);
                }
                // the scales as unsigned E4M3, like the tensor cores
                const float2 sx = f8x2_to_f2(xs[j] & 0x7f7fu);
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const float2 sw = f8x2_to_f2(ws[j][i] & 0x7f7fu);
                    acc[t][i] = fmaf(g4_block(wv[j][i].x, wv[j][i].y, h), sw.x * sx.x, acc[t][i]);
                    acc[t][i] = fmaf(g4_block(wv[j][i].z, wv[j][i].w, h + 8), sw.y * sx.y, acc[t][i]);
                }
            }
        }
    }
    const float wg = wgs[e];
#pragma unroll
    for (int t = 0; t < kGgvTok; ++t) {
        if (t >= nt) break;
        const float xg = xgs[r + t];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const float v = warp_sum(acc[t][i]) * xg * wg;
            if (lane == 0) {
                const size_t at = (size_t)(r + t) * N + n + i;
                if (out_f32)
                    static_cast<float*>(y)[at] = v;
                else
                    static_cast<uint16_t*>(y)[at] = f2bf_bits(v);
            }
        }
    }
}

}  // namespace moe
