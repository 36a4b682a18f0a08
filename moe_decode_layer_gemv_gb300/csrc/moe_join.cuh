// moe_join.cuh -- what joins a routed (or dense) block to the residual stream:
// the weighted sum of a token's rows, a norm behind the block, the residual
// add with its scale and the norm before the next block, in one kernel, and
// the gradients of all of it in another.
//
//   z[t] = sum_j w[t, j] o[pos[t, j]]           b = rms(z) z post, or z
//   y[t] = x[t] + scale b                       n = rms(y) y pre
//   rms(v) = 1 / sqrt(mean(v^2) + eps)
#pragma once

#include "moe_common.cuh"
#include "moe_grouped.cuh"
#include "moe_ptx.cuh"

namespace moe {

struct JoinParams {
    const void *x, *o;      // x: y in the backward pass
    const int32_t* pos;     // [T, k], or nullptr: row t k + j
    const float *w, *post, *scale, *pre;
    void *y, *n;            // y: dx in the backward pass
    int x_f32, n_f32;
    int T, H, R, k;
    float scale_all, eps;
    // backward
    const void *dy, *dn;
    void* d_o;
    float* dw;
    float* parts;           // [gridDim.x][sums][H] column sums: of those wanted, dpost, dscale, dpre
    int sums;
    int32_t* status;
};

// ---------------------------------------------------------------- eight values
// Inputs may come from the kernel ahead on the stream: coherent loads, past L1
// where a value is read once.
struct Raw8 {
    uint4 a, b;
};
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
// elements 8 v .. 8 v + 7 of row `row` of a [.., H] tensor
__device__ __forceinline__ Raw8 raw8(const void* p, bool f32, size_t row, int H, int v) {
    Raw8 r;
    const size_t at = row * (size_t)H + 8 * (size_t)v;
    if (f32) {
        r.a = ld_once_v4(static_cast<const float*>(p) + at);
        r.b = ld_once_v4(static_cast<const float*>(p) + at + 4);
    } else {
        r.a = ld_once_v4(static_cast<const uint16_t*>(p) + at);
        r.b = make_uint4(0, 0, 0, 0);
    }
    return r;
}
__device__ __forceinline__ void values8(const Raw8& r, bool f32, float (&v)[8]) {
    const uint32_t a[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (f32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f2(a[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
__device__ __forceinline__ void put8(void* p, bool f32, size_t row, int H, int v, const float (&f)[8]) {
    const size_t at = row * (size_t)H + 8 * (size_t)v;
    if (f32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        o[0] = make_float4(f[0], f[1], f[2], f[3]);
        o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = gg_pack(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}
__device__ __forceinline__ void vector8(const float* p, int v, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p + 8 * v), b = *reinterpret_cast<const float4*>(p + 8 * v + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Eight columns' sums in shared memory, owned by one thread: the first and the
// last four of each vector in two arrays, so that a warp's accesses are dense.
__device__ __forceinline__ void add8(float* sums, int nvec, int v, const float (&f)[8]) {
    float4* s = reinterpret_cast<float4*>(sums);
    float4 a = s[v], b = s[nvec + v];
    s[v] = make_float4(a.x + f[0], a.y + f[1], a.z + f[2], a.w + f[3]);
    s[nvec + v] = make_float4(b.x + f[4], b.y + f[5], b.z + f[6], b.w + f[7]);
}

// ---------------------------------------------------------------- reductions
// Eight values' sums over a warp: lanes take over half of the values at each of
// three steps, so that nine shuffles do instead of forty; lane 4 v + .. ends
// with value v's sum.
__device__ __forceinline__ float warp_sum8(const float (&v)[8], int lane) {
    float a[4], b[2], c;
    const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = (h16 ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, h16 ? v[i] : v[i + 4], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = (h8 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, h8 ? a[i] : a[i + 2], 8);
    c = (h4 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, h4 ? b[0] : b[1], 4);
    c += __shfl_xor_sync(0xffffffffu, c, 2);
    return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// The sum over a block (whole warps, every thread takes part).  `buf`: 32
// floats, free again after the next barrier of the block.
__device__ __forceinline__ float block_sum(float v, float* buf) {
    v = warp_sum(v);
    if (blockDim.x == 32) return v;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? buf[lane] : 0.0f);
}

// 1 / sqrt of a mean square with eps, and 0 where that is nothing (eps = 0 and
// a row of zeros, a token's without rows for instance): the norm of zeros is
// zeros, and so is its gradient.
__device__ __forceinline__ float norm_factor(float v) { return v == 0.0f ? 0.0f : 1.0f / sqrtf(v); }

// The rows and weights of a token's routes; a row of -1 is none.
__device__ __forceinline__ void token_routes(const JoinParams& p, int t, int (&row)[MOE_MAX_TOPK],
                                             float (&w)[MOE_MAX_TOPK]) {
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
        row[j] = -1;
        w[j] = 0.0f;
        if (j < p.k && p.o) {
            const size_t at = (size_t)t * p.k + j;
            row[j] = p.pos ? p.pos[at] : (int)at;
            w[j] = p.w ? p.w[at] : 1.0f;
            if (row[j] < -1 || row[j] >= p.R) {
                set_status(p.status, MOE_DEV_BAD_ROUTE);
                row[j] = -1;
            }
        }
    }
}

// z of eight columns, G rows on their way at a time
template <bool OF32, int G>
__device__ __forceinline__ void gather8(const JoinParams& p, const int (&row)[MOE_MAX_TOPK], const float (&w)[MOE_MAX_TOPK],
                                        int v, float (&z)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = 0.0f;
#pragma unroll
    for (int g = 0; g < MOE_MAX_TOPK; g += G) {
        Raw8 r[G];
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (row[g + j] >= 0) r[j] = raw8(p.o, OF32, row[g + j], p.H, v);
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (row[g + j] >= 0) {
                float f[8];
                values8(r[j], OF32, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = fmaf(w[g + j], f[i], z[i]);
            }
    }
}

// ---------------------------------------------------------------- forward
// A token a block of up to MT threads; a thread holds the columns of NV vectors
// of eight.  Bound by HBM: 8192 tokens, top-8, 2048 columns, an fp32 stream: 78
// us, 0.81 of the copy bandwidth.
template <bool OF32, int NV, int MT>
__global__ void __launch_bounds__(MT) join_kernel(JoinParams p) {
    __shared__ float buf[2][32];
    grid_dep_wait();
    const int t = blockIdx.x, nvec = p.H / 8;
    int row[MOE_MAX_TOPK];
    float w[MOE_MAX_TOPK], s = 0.0f, b[NV][8];
    Raw8 rx;  // (NV = 1: the stream's columns are on their way with the rows)
    if (NV == 1 && (int)threadIdx.x < nvec) rx = raw8(p.x, p.x_f32, t, p.H, threadIdx.x);
    token_routes(p, t, row, w);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        gather8<OF32, 8>(p, row, w, v, b[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) s = fmaf(b[i][c], b[i][c], s);
    }
    float r = 1.0f;
    if (p.post) {
        r = norm_factor(block_sum(s, buf[0]) / (float)p.H + p.eps);
    }
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float f[8], x[8];
        if (p.post) {
            vector8(p.post, v, f);
#pragma unroll
            for (int c = 0; c < 8; ++c) b[i][c] *= r * f[c];
        }
        values8(NV == 1 ? rx : raw8(p.x, p.x_f32, t, p.H, v), p.x_f32, x);
        if (p.scale) {
            vector8(p.scale, v, f);
#pragma unroll
            for (int c = 0; c < 8; ++c) b[i][c] = fmaf(f[c], b[i][c], x[c]);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) b[i][c] = fmaf(p.scale_all, b[i][c], x[c]);
        }
        if (p.y) put8(p.y, p.x_f32, t, p.H, v, b[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) s = fmaf(b[i][c], b[i][c], s);
    }
    if (!p.pre) return;
    r = norm_factor(block_sum(s, buf[1]) / (float)p.H + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float f[8];
        vector8(p.pre, v, f);
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] *= b[i][c] * r;
        put8(p.n, p.n_f32, t, p.H, v, f);
    }
}

// ---------------------------------------------------------------- backward
// With d the gradient of y (a = dn pre):
//   d  = dy + rms(y) a - (y rms(y)) rms(y) (rms(y) mean(a y))        dx = d
//   g  = scale d (the gradient of b);  with a norm behind the block, c = g post:
//   dz = rms(z) c - (z rms(z)) rms(z) (rms(z) mean(c z)), else g
//   do[pos_j] = w_j dz,  dw_j = <dz, o[pos_j]>
//   dpre = sum_t dn y rms(y),  dscale = sum_t d b,  dpost = sum_t g z rms(z)
// With f = scale post, the sums of c z come from those of dy f z, a f z and y f z:
// all that depends on a whole row is summed in one pass over it, with one
// barrier of the block a token, and the token's dw is written behind the next
// token's barrier.
// A block walks tokens and keeps the column sums in shared memory, each column
// by the thread that owns it; the blocks' sums are joined in a fixed order.
// After kJoinRun tokens they are added to the block's part of the workspace: n
// additions one after the other are off by up to n / 2 2^-24 of a sum of one
// sign, and the most tokens are 27594 a block (4 to 9e-5 at 6900).
//
// Bound by HBM and, with 16 warps an SM, by the latency between a token's loads
// and its stores.  With NV = 1 a thread keeps what it read of a token (its rows
// of o, two of the stream, dn) in registers to the token's end, all loads in
// flight at once, and the next token's inputs are brought into L2 meanwhile.
// Wider rows are read again, from L2.  8192 tokens, top-8, 2048 columns, norm
// and scale behind the block: 161 us, 0.70 of the copy bandwidth (178 without
// the prefetch, 169 with one of two tokens; 222 with the rows read again and
// three blocks an SM; 206 with a ring of bulk copies feeding two groups of 256
// threads from shared memory, whose 52 KB a token leave it three or four deep).
// fp32 rows, eight of eight columns a thread, do not fit in the 128 registers
// beside the rest (140 bytes of a thread are spilled): 281 us, 0.69 of it.
constexpr int kJoinRun = 256;

template <bool OF32, int NV, int MT>
__global__ void __launch_bounds__(MT) join_back_kernel(JoinParams p) {
    extern __shared__ __align__(16) float cols[];  // [sums][H]
    __shared__ float buf[2][16][8];                // by the token's parity: the warps' sums ...
    __shared__ float dbuf[2][16][MOE_MAX_TOPK];    // ... and dw
    constexpr bool HOLD = NV == 1;
    const int nvec = p.H / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int i = threadIdx.x; i < p.sums * p.H; i += blockDim.x) cols[i] = 0.0f;
    float* at = cols;
    float* c_post = p.post ? at : nullptr;
    at += p.post ? p.H : 0;
    float* c_scale = p.scale ? at : nullptr;
    at += p.scale ? p.H : 0;
    float* c_pre = at;
    grid_dep_wait();
    __syncthreads();
    // the routes of a token, lane j the j-th
    int r_next = -1;
    float w_next = 0.0f;
    auto routes = [&](int t) {
        r_next = -1;
        w_next = 0.0f;
        if (p.o && lane < p.k && t < p.T) {
            const size_t i = (size_t)t * p.k + lane;
            r_next = p.pos ? p.pos[i] : (int)i;
            w_next = p.w ? p.w[i] : 1.0f;
        }
    };
    auto write_dw = [&](int t, int parity) {
        if (!p.dw || (int)threadIdx.x >= p.k) return;
        float sum = 0.0f;
        for (int i = 0; i < warps; ++i) sum += dbuf[parity][i][threadIdx.x];
        p.dw[(size_t)t * p.k + threadIdx.x] = sum;
    };
    // The block's column sums into its part of the workspace, or added to what is there: each column by the thread
    // that owns it.
    bool first = true;
    auto put_aside = [&]() {
        float4* out = reinterpret_cast<float4*>(p.parts + (size_t)blockIdx.x * p.sums * p.H);
        float4* in = reinterpret_cast<float4*>(cols);
        for (int s = 0; s < p.sums; ++s)
            for (int v = threadIdx.x; v < nvec; v += blockDim.x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 &sum = in[2 * s * nvec + h * nvec + v], &to = out[2 * (s * nvec + v) + h];
                    float4 a = sum;
                    if (!first) a = make_float4(a.x + to.x, a.y + to.y, a.z + to.z, a.w + to.w);
                    to = a;
                    sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
        first = false;
    };
    routes(blockIdx.x);
    int parity = 0, t = blockIdx.x, run = 0;
    for (; t < p.T; t += gridDim.x, parity ^= 1) {
        if (++run > kJoinRun) {
            put_aside();
            run = 1;
        }
        if (r_next < -1 || r_next >= p.R) {
            set_status(p.status, MOE_DEV_BAD_ROUTE);
            r_next = -1;
        }
        int row[MOE_MAX_TOPK];
        float w[MOE_MAX_TOPK], s[8] = {}, z[NV][8];
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j) {
            row[j] = __shfl_sync(0xffffffffu, r_next, j);
            w[j] = __shfl_sync(0xffffffffu, w_next, j);
        }
        Raw8 ro[HOLD ? MOE_MAX_TOPK : 1], ry, rn, rd;
        const bool mine = (int)threadIdx.x < nvec;
        if (HOLD && mine) {
            if (p.pre) {
                ry = raw8(p.x, p.x_f32, t, p.H, threadIdx.x);
                rn = raw8(p.dn, p.n_f32, t, p.H, threadIdx.x);
            }
            if (p.dy) rd = raw8(p.dy, p.x_f32, t, p.H, threadIdx.x);
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
                if (row[j] >= 0) ro[HOLD ? j : 0] = raw8(p.o, OF32, row[j], p.H, threadIdx.x);
        }
        routes(t + gridDim.x);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= nvec) continue;
            if (HOLD) {
#pragma unroll
                for (int c = 0; c < 8; ++c) z[i][c] = 0.0f;
#pragma unroll
                for (int j = 0; j < MOE_MAX_TOPK; ++j)
                    if (row[j] >= 0) {
                        float f[8];
                        values8(ro[HOLD ? j : 0], OF32, f);
#pragma unroll
                        for (int c = 0; c < 8; ++c) z[i][c] = fmaf(w[j], f[c], z[i][c]);
                    }
            } else if (p.o) {
                gather8<OF32, OF32 ? 2 : 4>(p, row, w, v, z[i]);
            }
            float fz[8];  // f z
            if (p.post) {
                float f[8];
                vector8(p.post, v, fz);
                if (p.scale) vector8(p.scale, v, f);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    s[2] = fmaf(z[i][c], z[i][c], s[2]);
                    fz[c] *= (p.scale ? f[c] : p.scale_all) * z[i][c];
                }
                if (p.dy) {
                    values8(HOLD ? rd : raw8(p.dy, p.x_f32, t, p.H, v), p.x_f32, f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) s[3] = fmaf(f[c], fz[c], s[3]);
                }
            }
            if (p.pre) {
                float y[8], a[8], f[8];
                values8(HOLD ? ry : raw8(p.x, p.x_f32, t, p.H, v), p.x_f32, y);
                values8(HOLD ? rn : raw8(p.dn, p.n_f32, t, p.H, v), p.n_f32, a);
                vector8(p.pre, v, f);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    a[c] *= f[c];
                    s[0] = fmaf(y[c], y[c], s[0]);
                    s[1] = fmaf(a[c], y[c], s[1]);
                }
                if (p.post) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        s[4] = fmaf(a[c], fz[c], s[4]);
                        s[5] = fmaf(y[c], fz[c], s[5]);
                    }
                }
            }
        }
        // every thread's totals: lane 4 v + k adds a quarter of the warps' sums of value v
        {
            const float one = warp_sum8(s, lane);
            if ((lane & 3) == 0) buf[parity][warp][lane >> 2] = one;
            __syncthreads();
            float sum = 0.0f;
            for (int i = lane & 3; i < warps; i += 4) sum += buf[parity][i][lane >> 2];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int j = 0; j < 6; ++j) s[j] = __shfl_sync(0xffffffffu, sum, 4 * j);
        }
        // the next token's inputs on their way into L2 meanwhile, a lane a row
        if (warp == 0 && t + (int)gridDim.x < p.T) {
            const size_t sx = (size_t)p.H * (p.x_f32 ? 4 : 2), sn = (size_t)p.H * (p.n_f32 ? 4 : 2), so = (size_t)p.H * (OF32 ? 4 : 2);
            const size_t next = (size_t)t + gridDim.x;
            if (r_next >= 0 && r_next < p.R)
                bulk_prefetch_l2(static_cast<const unsigned char*>(p.o) + r_next * so, (uint32_t)so);
            if (lane == 29 && p.pre) bulk_prefetch_l2(static_cast<const unsigned char*>(p.x) + next * sx, (uint32_t)sx);
            if (lane == 30 && p.pre) bulk_prefetch_l2(static_cast<const unsigned char*>(p.dn) + next * sn, (uint32_t)sn);
            if (lane == 31 && p.dy) bulk_prefetch_l2(static_cast<const unsigned char*>(p.dy) + next * sx, (uint32_t)sx);
        }
        if (t != (int)blockIdx.x) write_dw(t - gridDim.x, parity ^ 1);
        // (factors in the order that keeps them within fp32's range wherever the rows and their squares' sums are)
        const float n = 1.0f / (float)p.H;
        const float ny = norm_factor(s[0] * n + p.eps), my = ny * (ny * (s[1] * n));
        const float nz = norm_factor(s[2] * n + p.eps);
        const float mz = nz * (nz * ((s[3] + (p.pre ? ny * (s[4] - my * s[5]) : 0.0f)) * n));
        float dots[MOE_MAX_TOPK] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= nvec) continue;
            float d[8], f[8];
            if (p.dy) {
                values8(HOLD ? rd : raw8(p.dy, p.x_f32, t, p.H, v), p.x_f32, d);
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c) d[c] = 0.0f;
            }
            if (p.pre) {
                float y[8], a[8];
                values8(HOLD ? ry : raw8(p.x, p.x_f32, t, p.H, v), p.x_f32, y);
                values8(HOLD ? rn : raw8(p.dn, p.n_f32, t, p.H, v), p.n_f32, a);
                vector8(p.pre, v, f);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    y[c] *= ny;
                    d[c] += ny * (a[c] * f[c]) - y[c] * my;
                    f[c] = a[c] * y[c];
                }
                add8(c_pre, nvec, v, f);
            }
            put8(p.y, p.x_f32, t, p.H, v, d);
            if (!p.o) continue;
            float q[8];
            if (p.post) vector8(p.post, v, q);
            if (c_scale) {
#pragma unroll
                for (int c = 0; c < 8; ++c) f[c] = d[c] * (p.post ? z[i][c] * nz * q[c] : z[i][c]);
                add8(c_scale, nvec, v, f);
            }
            if (p.scale) {
                vector8(p.scale, v, f);
#pragma unroll
                for (int c = 0; c < 8; ++c) d[c] *= f[c];
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c) d[c] *= p.scale_all;
            }
            if (p.post) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float hat = z[i][c] * nz;
                    f[c] = d[c] * hat;
                    d[c] = nz * (d[c] * q[c]) - hat * mz;
                }
                add8(c_post, nvec, v, f);
            }
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
                if (row[j] >= 0) {
                    if (p.dw) {
                        values8(HOLD ? ro[HOLD ? j : 0] : raw8(p.o, OF32, row[j], p.H, v), OF32, f);
#pragma unroll
                        for (int c = 0; c < 8; ++c) dots[j] = fmaf(d[c], f[c], dots[j]);
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) f[c] = w[j] * d[c];
                    put8(p.d_o, OF32, row[j], p.H, v, f);
                }
        }
        if (p.dw) {
            const float one = warp_sum8(dots, lane);
            if ((lane & 3) == 0) dbuf[parity][warp][lane >> 2] = one;
        }
    }
    __syncthreads();
    write_dw(t - gridDim.x, parity ^ 1);
    put_aside();
}

// The blocks' column sums in a fixed order: a block takes 32 columns, its
// eight warps every eighth part.
static __global__ void __launch_bounds__(256) join_sums_kernel(const float* parts, int grid, int n, int H, float* a, float* b,
                                                               float* c) {
    __shared__ float s_sum[8][32];
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (i < n) {
#pragma unroll 8
        for (int k = warp; k < grid; k += 8) s += __ldcg(parts + (size_t)k * n + i);
    }
    s_sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < n) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += s_sum[k][lane];
        float* const to[3] = {a, b, c};
        to[i / H][i % H] = s;
    }
}

}  // namespace moe
