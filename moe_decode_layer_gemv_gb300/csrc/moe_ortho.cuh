// moe_ortho.cuh -- orthogonalising matrices by Newton-Schulz products: the
// norm and the conversion ahead of them (the products: gg_kernel with the
// kGgSym, kGgAxpy and kGgResult epilogues, moe_grouped.cuh).
//
//   X = G / (|G|_F + eps);  A = X X^T;  X <- a X + (b A + c A A) X
//
// on the shorter side: a tall G is transposed as it is converted, and the last
// product stores its transpose.  What the products read is held in fp16, with
// |X|_2 near 1, so that nothing overflows (bf16 operands would be off by 8
// times as much).  X itself is carried in two fp16 values, 22 bits, from step
// to step: whatever is rounded off it in directions that G does not have grows
// by a factor of a in each step, the last one included, and a gradient of few
// tokens has few directions (256 x 256 of rank 24: 3.1e-2 of the result with X
// in fp16 alone, 1.5e-3 so; 1.6e-3 with the high half alone in the last step,
// and 1.9e-3 instead of 1.7e-3 for 130 x 500 of rank 1).  In the last two steps
// A' = A - 1/2 takes A's place,
//   a + b A + c A A = (a + b/2 + c/4) + (b + c) A' + c A' A',
// since most eigenvalues of A are near 1 by then and b A + c A A several times
// as large as what is left of it, and its roundings too (random 300 x 900
// matrices: 1.7e-3 without, 1.0e-3 so).  In the directions that G lacks it
// costs some of the low half's good: B is 1.9 there instead of 0, more than half of a,
// and multiplies X's high half alone; in earlier steps it would undo the above.  The bf16 result's own rounding is 1.7e-3, which adds to
// all of these in squares.  Short sides average over few
// roundings (20 x 300: 2.2e-3), and cost little: up to 96 rows A and B too are
// held in two values, and the products that contract over them, A A and B X,
// take three terms (high high + high low + low high) and no shift.  20 x 300
// then end 3.8e-4 off, 16 x 16 1.1e-3, of X's rounding in X X^T alone.  X
// carries a factor of 2^8, which keeps the entries of the largest matrices
// (2^-14 on average at 16384 x 16384) out of fp16's subnormals; a single entry
// of 1 is still far from 65504.
//
// 64 matrices of 2048 x 768 in bf16, five steps: 1525 us.  Norm 53 and
// conversion 136 (HBM), then a step: X X^T 76 and A A 40 (384 tiles on 76 pairs
// of CTAs: six rounds for five), B X 155 (1 GB of HBM traffic; the last 136).
// Groups of 6 to 38 matrices, whose X stays in L2, take longer (3465 to 1908 us
// when all took 1732): their products do not fill the GPU and cost 3 to 5 us
// each to start.
#pragma once

#include <math_constants.h>

#include "moe_common.cuh"
#include "moe_grouped.cuh"
#include "moe_ptx.cuh"

namespace moe {

constexpr int kNsScaleLog2 = 8;
constexpr float kNsShift = 0.5f;
constexpr int kNsShifted = 2;  // last steps with the shift
constexpr int kNsSplitRows = 96;
constexpr int kNsParts = 64;  // blocks that sum one matrix's squares, at most

__device__ __forceinline__ float ns_value(const void* g, bool f32, size_t i) {
    return f32 ? __ldcg(static_cast<const float*>(g) + i)
               : __uint_as_float((uint32_t)__ldcg(static_cast<const unsigned short*>(g) + i) << 16);
}

// Sums of squares that neither overflow nor underflow (Blue 1978): values
// beyond 2^48 are summed times 2^-80, those below 2^-48 times 2^80.
// parts [E, gridDim.x, 3].  A thread adds up 32 squares at a time and carries
// what the addition of such a sum to the others rounds off (Knuth's two-sum):
// 16384 one after the other, as many as there are in the largest matrices, would be off by
// up to 2^-12 where the values are alike, 2.4e-4.  45 additions at most remain
// (32, five within a warp and eight across the block), 2^-19 of the norm.
struct NsSum {
    float s[3] = {0.0f, 0.0f, 0.0f}, run[3] = {0.0f, 0.0f, 0.0f}, left[3] = {0.0f, 0.0f, 0.0f};
    __device__ __forceinline__ void add(float x) {
        const float a = fabsf(x);
        const float big = a > 0x1p48f ? x * 0x1p-80f : 0.0f, tiny = a < 0x1p-48f ? x * 0x1p80f : 0.0f;
        const float mid = a > 0x1p48f || a < 0x1p-48f ? 0.0f : x;  // (a NaN goes here)
        run[0] = fmaf(big, big, run[0]);
        run[1] = fmaf(mid, mid, run[1]);
        run[2] = fmaf(tiny, tiny, run[2]);
    }
    __device__ __forceinline__ void put_aside() {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const float t = s[j] + run[j], b = t - s[j];
            left[j] += (s[j] - (t - b)) + (run[j] - b);
            s[j] = t;
            run[j] = 0.0f;
        }
    }
    // (an infinite sum leaves no number behind, and stands for itself)
    __device__ __forceinline__ float total(int j) const { return isfinite(s[j]) ? s[j] + left[j] : s[j]; }
};

__global__ void __launch_bounds__(256) ns_norm_kernel(const void* g, int f32, size_t n, float* parts) {
    __shared__ float s_sum[3][8];
    grid_dep_launch();
    grid_dep_wait();
    const size_t base = blockIdx.y * n;
    NsSum sum;
    const size_t step = (size_t)gridDim.x * 256, first = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (n % 8 == 0) {
        const size_t pieces = f32 ? n / 4 : n / 8;  // of 16 bytes, four in flight a thread
        const unsigned char* from = static_cast<const unsigned char*>(g) + base * (f32 ? 4 : 2);
        for (size_t i = first; i < pieces; i += 4 * step) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = i + k * step < pieces ? ld_input_v4(from + 16 * (i + k * step)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (f32) {
                        sum.add(__uint_as_float(u[j]));
                    } else {
                        const float2 f = bf16x2_to_f2(u[j]);
                        sum.add(f.x);
                        sum.add(f.y);
                    }
                }
            }
            sum.put_aside();
        }
    } else {
        for (size_t i = first; i < n; i += 32 * step) {
#pragma unroll 4
            for (int k = 0; k < 32; ++k)
                if (i + k * step < n) sum.add(ns_value(g, f32, base + i + k * step));
            sum.put_aside();
        }
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const float s = warp_sum(sum.total(j));
        if ((threadIdx.x & 31) == 0) s_sum[j][threadIdx.x >> 5] = s;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += s_sum[threadIdx.x][w];
        parts[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 3 + threadIdx.x] = t;
    }
}

// X [E, rows, cols] = 2^8 G / (|G|_F + eps), or its transpose, in fp16, and in
// `low` what that leaves; zeros beyond G's N x K.  A block takes 64 rows of G
// and `strip` columns, 64 at a time, a thread eight values of two rows; a tall G's
// tiles are transposed through shared memory, two rows' values a word (an odd
// pitch: two lanes a bank).  A matrix with a NaN or an infinity becomes NaN
// throughout.
__global__ void __launch_bounds__(256) ns_convert_kernel(const void* g, int f32, int N, int K, const float* parts, int nparts,
                                                         float eps, int trans, uint16_t* x, uint16_t* low, int rows,
                                                         int cols, int strip) {
    __shared__ uint32_t tile[2][64][33];
    __shared__ float s_scale[2];
    grid_dep_launch();
    grid_dep_wait();
    const int e = blockIdx.z, r0 = blockIdx.y * 64, tid = threadIdx.x;
    if (tid < 32) {
        double s[3] = {0.0, 0.0, 0.0};
        for (int i = tid; i < nparts; i += 32)
            for (int j = 0; j < 3; ++j) s[j] += (double)__ldcg(parts + ((size_t)e * nparts + i) * 3 + j);
#pragma unroll
        for (int j = 0; j < 3; ++j)
            for (int o = 16; o > 0; o >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
        if (tid == 0) {
            const double sum = s[0] * 0x1p160 + s[1] + s[2] * 0x1p-160;
            const double scale = ldexp(1.0, kNsScaleLog2) / (sqrt(sum) + (double)eps);
            // in two factors, since the whole may lie outside fp32's range
            int ex = 0;
            const double f = frexp(scale, &ex);
            const bool ok = isfinite(sum) && isfinite(scale);
            s_scale[0] = ok ? ldexpf(1.0f, ex / 2) : CUDART_NAN_F;
            s_scale[1] = ok ? (float)ldexp(f, ex - ex / 2) : CUDART_NAN_F;
        }
    }
    __syncthreads();
    const float s0 = s_scale[0], s1 = s_scale[1];
    const bool whole = K % 8 == 0;
    for (int c0 = blockIdx.x * strip; c0 < (blockIdx.x + 1) * strip && c0 < (trans ? rows : cols); c0 += 64) {
        const int c = c0 + (tid & 7) * 8;
        uint32_t hi[2][4], lo[2][4];  // two rows' eight values, in pairs
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + (tid >> 3) * 2 + k;
            const size_t at = ((size_t)e * N + r) * K + c;
            float v[8];
            if (r < N && whole && c < K) {
                if (f32) {
                    const uint4 a = ld_input_v4(static_cast<const float*>(g) + at);
                    const uint4 b = ld_input_v4(static_cast<const float*>(g) + at + 4);
                    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(u[j]);
                } else {
                    const uint4 a = ld_input_v4(static_cast<const uint16_t*>(g) + at);
                    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = bf16x2_to_f2(u[j]);
                        v[2 * j] = f.x;
                        v[2 * j + 1] = f.y;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r < N && c + j < K ? ns_value(g, f32, at + j) : 0.0f;  // (all in flight)
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = v[2 * j] * s0 * s1, b = v[2 * j + 1] * s0 * s1;
                hi[k][j] = gg_pack_f16(a, b);
                const float2 h = f16x2_to_f2(hi[k][j]);
                lo[k][j] = gg_pack_f16(a - h.x, b - h.y);
            }
            if (!trans && r < rows && c < cols) {  // (cols is a multiple of 64)
                const size_t to = ((size_t)e * rows + r) * cols + c;
                *reinterpret_cast<uint4*>(x + to) = make_uint4(hi[k][0], hi[k][1], hi[k][2], hi[k][3]);
                *reinterpret_cast<uint4*>(low + to) = make_uint4(lo[k][0], lo[k][1], lo[k][2], lo[k][3]);
            }
        }
        if (!trans) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t* to = &tile[0][(tid & 7) * 8 + 2 * j][tid >> 3];
            to[0] = __byte_perm(hi[0][j], hi[1][j], 0x5410);
            to[33] = __byte_perm(hi[0][j], hi[1][j], 0x7632);
            to += 64 * 33;
            to[0] = __byte_perm(lo[0][j], lo[1][j], 0x5410);
            to[33] = __byte_perm(lo[0][j], lo[1][j], 0x7632);
        }
        __syncthreads();
#pragma unroll
        for (int k = tid >> 5; k < 64; k += 8) {  // X's row c0 + k, a warp a row
            const int lane = tid & 31;
            if (c0 + k >= rows || r0 + 2 * lane >= cols) continue;
            const size_t to = ((size_t)e * rows + c0 + k) * cols + r0 + 2 * lane;
            *reinterpret_cast<uint32_t*>(x + to) = tile[0][k][lane];
            *reinterpret_cast<uint32_t*>(low + to) = tile[1][k][lane];
        }
        __syncthreads();
    }
}

}  // namespace moe
