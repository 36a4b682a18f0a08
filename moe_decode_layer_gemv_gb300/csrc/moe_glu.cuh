// moe_glu.cuh -- the experts' gated unit for a handful of rows (tiles:
// gg_kernel with the kGgGlu epilogue, moe_grouped.cuh).
#pragma once

#include "moe_grouped.cuh"

namespace moe {

// h[r, i] = act(g) u for up to 32 rows: a warp per output i streams the gate
// and the up row of its expert, J chunks of 256 elements of each in flight,
// for up to kGgvTok rows of one segment at a time.  Block (b, r) takes the
// outputs 8b .. 8b + 7 of the rows r .. of a segment when r starts a group of
// kGgvTok there.  Bound by the weights' bytes and the latency of one chain
// offsets -> weights: two rows of 1536 x 2048 on two experts take 10 us a call,
// most of it on the host.
template <int J>
__global__ void __launch_bounds__(256) glu_gemv_kernel(const uint16_t* x, const uint16_t* gate_up, const int32_t* offsets,
                                                       int R, int I, int H, int E, void* h, int h_f32, uint16_t* gu,
                                                       float c0, float c1, int32_t* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    const int r = blockIdx.y;
    int p0, p1;
    const int e = gg_row_segment(offsets, E, R, r, p0, p1, status);
    if (e < 0 || (r - p0) % kGgvTok) return;
    const int nt = min(kGgvTok, p1 - r);
    const int i = blockIdx.x * 8 + warp;
    if (i >= I) return;
    const uint16_t* wg = gate_up + ((size_t)e * 2 * I + i) * H;
    const uint16_t* wu = wg + (size_t)I * H;
    const uint16_t* xr = x + (size_t)r * H;
    float g[kGgvTok] = {}, u[kGgvTok] = {};
    const int chunks = H / 8;
    for (int b = 0; b < chunks; b += 32 * J) {
        const int nj = min(J, (chunks - b + 31) / 32);
        uint4 gv[J], uv[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (j >= nj) break;
            const int c = b + j * 32 + lane;
            gv[j] = c < chunks ? ld_stream_v4(wg + (size_t)c * 8) : make_uint4(0, 0, 0, 0);
            uv[j] = c < chunks ? ld_stream_v4(wu + (size_t)c * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < kGgvTok; ++t) {
            if (t >= nt) break;
            uint4 xv[J];  // the first row's are on their way with the weights
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j >= nj) break;
                const int c = b + j * 32 + lane;
                xv[j] = c < chunks ? ld_input_v4(xr + (size_t)t * H + (size_t)c * 8) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j >= nj) break;
                const uint32_t gs[4] = {gv[j].x, gv[j].y, gv[j].z, gv[j].w};
                const uint32_t us[4] = {uv[j].x, uv[j].y, uv[j].z, uv[j].w};
                const uint32_t xs[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 a = bf16x2_to_f2(gs[q]), b2 = bf16x2_to_f2(us[q]), f = bf16x2_to_f2(xs[q]);
                    g[t] = fmaf(a.y, f.y, fmaf(a.x, f.x, g[t]));
                    u[t] = fmaf(b2.y, f.y, fmaf(b2.x, f.x, u[t]));
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kGgvTok; ++t) {
        if (t >= nt) break;
        const float gs = warp_sum(g[t]), us = warp_sum(u[t]);
        if (lane == 0) {
            const size_t row = (size_t)(r + t);
            float grad;
            const float v = glu_act(gs, c0, c1, grad) * us;
            if (h_f32)
                static_cast<float*>(h)[row * I + i] = v;
            else
                static_cast<uint16_t*>(h)[row * I + i] = f2bf_bits(v);
            if (gu) {
                gu[row * 2 * I + i] = f2bf_bits(gs);
                gu[row * 2 * I + I + i] = f2bf_bits(us);
            }
        }
    }
}

}  // namespace moe
