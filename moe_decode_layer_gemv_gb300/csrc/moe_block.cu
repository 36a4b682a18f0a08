// moe_block.cu -- the C ABI of the operators around the grouped products
// (declared in include/moe.h): the experts' gated unit and its gradient,
// what joins a block to the residual stream and its gradients, and the
// orthogonalised update.  Argument checks, the choice of a kernel, its launch.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "moe.h"
#include "moe_glu.cuh"
#include "moe_grouped.cuh"
#include "moe_host.cuh"
#include "moe_join.cuh"
#include "moe_launch.cuh"
#include "moe_ortho.cuh"

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
    return gg_pairs(R, 2 * I, E, F32 ? kGgPairRowsGluF32 : kGgPairRowsGlu)
               ? launch_persistent<2>(gg_kernel<kGgFwd, 2, F32, kGgGlu>, p, GgCfg<kGgFwd, 2, F32>::kThreads, sms, st)
               : launch_persistent<1>(gg_kernel<kGgFwd, 1, F32, kGgGlu>, p, GgCfg<kGgFwd, 1, F32>::kThreads, sms, st);
}

// What a token's row of `out` covers may be read for another token, unless `in` lies at the same place in the same type.
static bool clash(const void* out, int out_dtype, const void* in, int in_dtype, size_t n) {
    if (out == in && out_dtype == in_dtype) return false;
    return overlap(out, n * (out_dtype == MOE_DT_F32 ? 4 : 2), in, n * (in_dtype == MOE_DT_F32 ? 4 : 2));
}

static int check_join(int T, int H, int R, int k, bool o, bool pre, int x_dtype, int o_dtype, int n_dtype, float eps) {
    if (T < 0 || T > MOE_MAX_ROWS || H < 8 || H > MOE_MAX_DIM || (H & 7)) return MOE_ERR_INVALID_ARG;
    if (!o && !pre) return MOE_ERR_INVALID_ARG;
    if (o && (R < 0 || R > MOE_MAX_ROWS || k < 1 || k > MOE_MAX_TOPK)) return MOE_ERR_INVALID_ARG;
    for (const int dt : {x_dtype, o_dtype, n_dtype})
        if (dt != MOE_DT_F32 && dt != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    if (!(eps >= 0.0f && eps <= 1.0f)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Vectors of eight columns that a thread holds, given the threads a token may take.
static int join_vectors(int H, int threads) {
    int nv = 1;
    while (H / 8 > nv * threads) nv *= 2;
    return nv;
}
static unsigned join_threads(int H, int nv) { return (unsigned)ceil_div(ceil_div(H / 8, nv), 32) * 32; }

template <bool OF32, int MT>
static int run_join(const JoinParams& p, cudaStream_t st) {
    const int nv = join_vectors(p.H, MT);
    const unsigned block = join_threads(p.H, nv), grid = (unsigned)p.T;
    switch (nv) {
        case 1: return launch_pdl(join_kernel<OF32, 1, MT>, grid, block, 0, st, p);
        case 2: return launch_pdl(join_kernel<OF32, 2, MT>, grid, block, 0, st, p);
        case 4: return launch_pdl(join_kernel<OF32, 4, MT>, grid, block, 0, st, p);
        default: return launch_pdl(join_kernel<OF32, MOE_MAX_DIM / 8 / MT, MT>, grid, block, 0, st, p);
    }
}

// A block a token, of up to 512 threads while there are few, else of 256: top-8, 4096 columns, by 512 and 256, 64
// tokens 10.7 and 10.7 us, 152 10.7 and 12.8, 304 16.8 and 12.7, 2432 74 and 50 (up to 2048 columns both are the
// same).  Several tokens a block gain next to nothing where rows are short and cost up to a tenth else: 65536 tokens,
// top-2, 64 to 1024 columns, one and eight: 56 and 58 us, 58 and 58, 60 and 62, 123 and 134, 248 and 261 (16384 of 64
// columns: 21 and 19).
template <bool OF32>
static int run_join(const JoinParams& p, int sms, cudaStream_t st) {
    return p.T < 2 * sms ? run_join<OF32, 512>(p, st) : run_join<OF32, 256>(p, st);
}

// The backward pass: up to 512 threads a token of one vector each, beyond of
// several; as many blocks an SM as its registers (128 a thread) and shared
// memory hold.
static int join_back_vectors(int H) { return join_vectors(H, 512); }
static int join_back_grid(int T, int H, int sums, int sms) {
    const int threads = (int)join_threads(H, join_back_vectors(H));
    int per = 512 / threads;
    const int fit = (int)((200 * 1024) / ((size_t)sums * H * 4 + 4096));
    if (per > fit) per = fit;
    per = per < 1 ? 1 : per > 16 ? 16 : per;
    return T < per * sms ? T : per * sms;
}

template <bool OF32, int NV>
static int launch_join_back(const JoinParams& p, int grid, cudaStream_t st) {
    // (with the kernel's static part 48 KB are passed earlier)
    const size_t smem = (size_t)p.sums * p.H * 4;
    const int rc = smem > 32 * 1024 ? allow_smem(join_back_kernel<OF32, NV, 512>, 3 * MOE_MAX_DIM * 4) : MOE_OK;
    return rc ? rc : launch_pdl(join_back_kernel<OF32, NV, 512>, (unsigned)grid, join_threads(p.H, NV), smem, st, p);
}

template <bool OF32>
static int run_join_back(const JoinParams& p, int grid, cudaStream_t st) {
    switch (join_back_vectors(p.H)) {
        case 1: return launch_join_back<OF32, 1>(p, grid, st);
        case 2: return launch_join_back<OF32, 2>(p, grid, st);
        default: return launch_join_back<OF32, 4>(p, grid, st);
    }
}

// ---------------------------------------------------------- orthogonalisation
struct NsPlan {
    int m, n;        // rows and columns of X, padded
    int parts;       // blocks that sum a matrix's squares
    bool pairs;      // tiles of CTA pairs
    int narrow;      // tiles of 32 columns, 2: and split products
    size_t x, a, p;  // bytes of X, of A, of the sums
    size_t bytes;
};

static int ns_plan(int E, int N, int K, int sms, NsPlan* q) {
    if (E < 1 || E > MOE_MAX_E || N < 1 || N > MOE_MAX_DIM || K < 1 || K > MOE_MAX_DIM) return MOE_ERR_INVALID_ARG;
    q->m = ceil_div(N < K ? N : K, 16) * 16;
    q->n = ceil_div(N < K ? K : N, 64) * 64;
    // pairs of CTAs where their larger tiles still give every pair work
    const int t = ceil_div(q->m, 256);
    const int tri = t * (t + 1) / 2;
    q->pairs = (int64_t)E * tri >= sms / 2;
    // narrow tiles while they leave no SM a second one of the symmetric products.  Measured, a product of the
    // chain with tiles of 128 and of 32 columns: one matrix of 390 x 515 6.7 and 4.6 us, 512 x 2048 8.8 and 7.3,
    // 768 x 2048 9.8 and 9.2, 1024 x 1024 8.9 and 10.2; four of 390 x 515 6.8 and 6.6, eight 7.8 and 9.5
    // Up to kNsSplitRows rows the products whose contraction that is are split (moe_ortho.cuh).
    q->narrow = q->m <= kNsSplitRows ? 2 : (int64_t)E * ceil_div(q->m, 32) * ceil_div(q->m, 128) <= sms;
    q->parts = ceil_div(8 * sms, E);
    const int most = (int)(((size_t)N * K + 2047) / 2048);
    if (q->parts > most) q->parts = most;
    if (q->parts > kNsParts) q->parts = kNsParts;
    q->x = align_up(sizeof(uint16_t) * (size_t)E * q->m * q->n, 256);
    q->a = align_up(sizeof(uint16_t) * (size_t)E * q->m * q->m, 256);
    q->p = align_up(sizeof(float) * 3 * (size_t)E * q->parts, 256);
    q->bytes = (q->narrow == 2 ? 4 * q->x + 4 * q->a : 3 * q->x + 2 * q->a) + q->p + 256;  // (the parts are aligned to 256)
    return MOE_OK;
}

// Every product's parameters, with the tensor maps encoded once: X X^T and B X
// from either copy of X, A A, and the last B X.
struct NsProducts {
    GgParams xx[2], aa, bx[2], last[2];
};

// A value in two fp16 buffers; low is nullptr where it is held in one.
struct NsHalves {
    uint16_t *high, *low;
};

// in: what the epilogue reads beside the product; split: into the product of both operands' halves.
static bool ns_params(const NsPlan& q, int E, NsHalves w, NsHalves x, int cols, NsHalves in, NsHalves out, bool split, bool sym,
                      GgParams* p) {
    memset(p, 0, sizeof *p);
    p->rows = q.m;
    p->low = out.low;
    p->halves = split;
    p->out = out.high;
    const uint64_t R = (uint64_t)E * q.m;
    bool ok;
    if (sym) {  // x [E m, cols] times its own rows
        p->M = q.m;
        p->C = cols;
        ok = encode_map(&p->ta, w.high, 2, cols, q.m, E, 128) && (!split || encode_map(&p->ta_lo, w.low, 2, cols, q.m, E, 128));
    } else {  // x = B [E m, m], w = X [E, m, n]
        p->M = q.n;
        p->C = q.m;
        p->a_blocked = 1;
        ok = encode_blocked(&p->ta, w.high, q.n, q.m, E) && (!split || encode_blocked(&p->ta_lo, w.low, q.n, q.m, E));
    }
    ok = ok && encode_map(&p->tb, x.high, 2, p->C, R, 0, kGgBoxN) && encode_map(&p->tb_all, x.high, 2, p->C, R, 0, 128) &&
         (!split || encode_map(&p->tb_lo, x.low, 2, p->C, R, 0, kGgBoxN));
    if (in.high) {
        constexpr int rows = GgIn<kGgSym>::kRows;  // (the other products' as well)
        ok = ok && encode_input(&p->tin[0], in.high, p->M, R, rows) && (!in.low || encode_input(&p->tin[1], in.low, p->M, R, rows));
        p->planes = in.low ? 2 : 1;
    }
    return ok;
}

template <int CG, int NARROW>
static int ns_allow() {
    int rc = allow_smem(gg_kernel<kGgFwd, CG, false, kGgSym, NARROW>, kGgSmem);
    if (!rc) rc = allow_smem(gg_kernel<kGgDx, CG, false, kGgAxpy, NARROW>, kGgSmem);
    return rc ? rc : allow_smem(gg_kernel<kGgDx, CG, false, kGgResult, NARROW>, kGgSmem);
}

// One product of E matrices, on no more SMs than it has tiles.
template <int EP, int CG, int NARROW>
static int run_ns(GgParams& p, int E, float alpha, float beta, float shift, int sms, cudaStream_t st) {
    constexpr int MODE = EP == kGgSym ? kGgFwd : kGgDx;
    p.E = E;
    p.R = E * p.rows;
    p.alpha = alpha;
    p.beta = beta;
    p.shift = shift;
    const int64_t t = ceil_div(p.rows, NARROW ? 32 : 128 * CG);
    const int64_t tiles = E * (EP == kGgSym && !NARROW ? t * (t + 1) / 2 : t * ceil_div(p.M, 128 * CG));
    return launch_clusters<CG>(gg_kernel<MODE, CG, false, EP, NARROW>, p, GgRole<MODE, CG, false, EP, NARROW>::kThreads,
                               tiles * CG < sms ? (int)tiles * CG : sms, st);
}

template <int CG, int NARROW>
static int run_ns_steps(NsProducts& s, int E, int steps, float a, float b, float c, int sms, cudaStream_t st) {
    const float up = (float)(1 << kNsScaleLog2), down = 1.0f / up;
    for (int i = 0; i < steps; ++i) {
        // a + b A + c A A of A = S + A': one + lin A' + c A' A'
        const float S = NARROW < 2 && steps - i <= kNsShifted ? kNsShift : 0.0f, lin = b + 2.0f * c * S, one = a + b * S + c * S * S;
        int rc = run_ns<kGgSym, CG, NARROW>(s.xx[i & 1], E, down * down, 0.0f, S, sms, st);
        if (!rc) rc = run_ns<kGgSym, CG, NARROW>(s.aa, E, c, lin, 0.0f, sms, st);
        if (!rc)
            rc = i + 1 < steps ? run_ns<kGgAxpy, CG, NARROW>(s.bx[i & 1], E, 1.0f, one, 0.0f, sms, st)
                               : run_ns<kGgResult, CG, NARROW>(s.last[i & 1], E, down, one * down, 0.0f, sms, st);
        if (rc) return rc;
    }
    return MOE_OK;
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
    const size_t rows = 2 * (size_t)R, hn = rows * I * (h_dtype == MOE_DT_F32 ? 2 : 1), gun = 2 * rows * I;
    if (overlap(h, hn, gu, gun) || overlap(h, hn, x, rows * H) || overlap(gu, gun, x, rows * H)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 2) return MOE_ERR_CUDA;
    const int f32 = h_dtype == MOE_DT_F32;
    // a few rows.  Measured, by rows and by tiles, of 1536 x 2048 on experts of their own: 2 rows 10.8 and 14.8 us, 8
    // 16.9 and 18.9, 12 21 and 23, 32 41 and 39; on one expert 2 rows 10.8 and 14.8, 12 14.8 and 14.8, 16 18.9 and
    // 14.8; of 512 x 1024 on one expert 8 rows 10.8 and 12.8, 32 12.8 and 12.8
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
    // (gu and dy are read ahead of what is written)
    const size_t rows = 2 * (size_t)R, hn = rows * I, gun = 2 * hn;
    if (overlap(dgu, gun, gu, gun) || overlap(dgu, gun, dy, rows * H) || overlap(h, hn, gu, gun) ||
        overlap(h, hn, dy, rows * H) || overlap(h, hn, dgu, gun))
        return MOE_ERR_INVALID_ARG;
    MOE_OPT(dev_status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 2) return MOE_ERR_CUDA;
    p.a_blocked = I % 64 == 0;
    if (!(p.a_blocked ? encode_blocked(&p.ta, down, I, H, E) : encode_map(&p.ta, down, 2, I, H, E, 64)) ||
        !encode_map(&p.tb, dy, 2, H, R, 0, kGgBoxN) || !encode_map(&p.tb_all, dy, 2, H, R, 0, 128) ||
        !encode_input(&p.tin[0], gu, 2 * I, R, GgIn<kGgGluBack>::kRows))
        return MOE_ERR_UNSUPPORTED;
    p.tin[1] = p.tin[0];
    p.planes = 2;
    p.tin_at[1] = I;
    p.offsets = offsets;
    p.E = E;
    p.R = R;
    p.M = I;
    p.C = H;
    p.out = dgu;
    p.out2 = h;
    p.status = dev_status;
    return gg_pairs(R, I, E, kGgPairRowsGluBack)
               ? launch_persistent<2>(gg_kernel<kGgDx, 2, false, kGgGluBack>, p, GgRole<kGgDx, 2, false, kGgGluBack>::kThreads, sms, st)
               : launch_persistent<1>(gg_kernel<kGgDx, 1, false, kGgGluBack>, p, GgRole<kGgDx, 1, false, kGgGluBack>::kThreads, sms, st);
}

int moe_combine_norm(const void* x, int x_dtype, const void* o, int o_dtype, const int32_t* pos, const float* w, int T, int H,
                     int R, int k, const float* post, const float* scale, float scale_all, const float* pre, float eps,
                     void* y, void* n, int n_dtype, int32_t* dev_status, void* stream) {
    const int rc = check_join(T, H, R, k, o != nullptr, pre != nullptr, x_dtype, o_dtype, n_dtype, eps);
    if (rc) return rc;
    if (o && !pos && (int64_t)T * k > R) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    JoinParams p;
    memset(&p, 0, sizeof p);
    MOE_REQ(x);
    MOE_OPT(o);
    MOE_OPT(pos);
    MOE_OPT(w);
    MOE_OPT(post);
    MOE_OPT(scale);
    MOE_OPT(pre);
    if (o) MOE_REQ(y);
    if (pre) MOE_REQ(n);
    MOE_OPT(dev_status);
    p.y = o ? y : nullptr;
    p.n = pre ? n : nullptr;
    const size_t th = (size_t)T * H, xn = th * (x_dtype == MOE_DT_F32 ? 4 : 2), nn = th * (n_dtype == MOE_DT_F32 ? 4 : 2);
    const size_t on = (size_t)R * H * (o_dtype == MOE_DT_F32 ? 4 : 2);
    if (clash(p.y, x_dtype, x, x_dtype, th) || clash(p.n, n_dtype, x, x_dtype, th) || overlap(p.y, xn, p.n, nn))
        return MOE_ERR_INVALID_ARG;
    const bool own = !pos && k == 1;  // (a token reads the row of its own place alone)
    if ((!(own && p.y == o && x_dtype == o_dtype) && overlap(p.y, xn, o, on)) ||
        (!(own && p.n == o && n_dtype == o_dtype) && overlap(p.n, nn, o, on)))
        return MOE_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms < 1) return MOE_ERR_CUDA;
    p.x = x;
    p.o = o;
    p.pos = pos;
    p.w = w;
    p.post = o ? post : nullptr;
    p.scale = o ? scale : nullptr;
    p.pre = pre;
    p.x_f32 = x_dtype == MOE_DT_F32;
    p.n_f32 = n_dtype == MOE_DT_F32;
    p.T = T;
    p.H = H;
    p.R = R;
    p.k = o ? k : 0;
    p.scale_all = o ? scale_all : 1.0f;
    p.eps = eps;
    p.status = dev_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return o_dtype == MOE_DT_F32 ? run_join<true>(p, sms, st) : run_join<false>(p, sms, st);
}

int moe_combine_norm_backward_workspace_bytes(int T, int H, int sums, size_t* bytes) {
    if (T < 0 || T > MOE_MAX_ROWS || H < 8 || H > MOE_MAX_DIM || (H & 7) || sums < 0 || sums > 3 || !bytes)
        return MOE_ERR_INVALID_ARG;
    const int sms = sm_count();
    *bytes = sizeof(float) * (size_t)join_back_grid(T, H, sums, sms > 0 ? sms : kMaxSms) * sums * H;
    return MOE_OK;
}

int moe_combine_norm_backward(const void* dy, const void* dn, int n_dtype, const void* y, int y_dtype, const void* o,
                              int o_dtype, const int32_t* pos, const float* w, int T, int H, int R, int k, const float* post,
                              const float* scale, float scale_all, const float* pre, float eps, void* dx, void* d_o, float* dw,
                              float* dpost, float* dscale, float* dpre, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream) {
    const int rc = check_join(T, H, R, k, o != nullptr, pre != nullptr, y_dtype, o_dtype, n_dtype, eps);
    if (rc) return rc;
    if (o && !pos && (int64_t)T * k > R) return MOE_ERR_INVALID_ARG;
    if (!o) post = scale = nullptr;
    MOE_OPT(post);
    MOE_OPT(scale);
    MOE_OPT(pre);
    if (post) MOE_REQ(dpost);
    if (scale) MOE_REQ(dscale);
    if (pre) MOE_REQ(dpre);
    MOE_OPT(dev_status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sums = (post != nullptr) + (scale != nullptr) + (pre != nullptr);
    float* to[3];
    int i = 0;
    if (post) to[i++] = dpost;
    if (scale) to[i++] = dscale;
    if (pre) to[i++] = dpre;
    while (i < 3) to[i++] = nullptr;
    if (T == 0) {
        int bad = MOE_OK;
        for (i = 0; i < sums && !bad; ++i) bad = to_status(cudaMemsetAsync(to[i], 0, sizeof(float) * (size_t)H, st));
        return bad;
    }
    MOE_OPT(dy);
    if (pre) MOE_REQ(dn);
    if (pre) MOE_REQ(y);
    MOE_REQ(dx);
    MOE_OPT(o);
    if (o) MOE_REQ(d_o);
    const size_t th = (size_t)T * H, xn = th * (y_dtype == MOE_DT_F32 ? 4 : 2), nn = th * (n_dtype == MOE_DT_F32 ? 4 : 2);
    const size_t on = (size_t)R * H * (o_dtype == MOE_DT_F32 ? 4 : 2);
    if (overlap(d_o, on, o, on)) return MOE_ERR_INVALID_ARG;  // (wide rows are read again behind the first writes)
    MOE_OPT(pos);
    MOE_OPT(w);
    MOE_OPT(dw);
    const int sms = sm_count();
    const int grid = join_back_grid(T, H, sums, sms > 0 ? sms : kMaxSms);
    if (sums) {
        if (!workspace || workspace_bytes < sizeof(float) * (size_t)grid * sums * H) return MOE_ERR_WORKSPACE;
        MOE_REQ(workspace);
    }
    const void* const yr = pre ? y : nullptr;  // (what is read)
    if (clash(dx, y_dtype, dy, y_dtype, th) || clash(dx, y_dtype, pre ? dn : nullptr, n_dtype, th) ||
        clash(dx, y_dtype, yr, y_dtype, th) || overlap(dx, xn, o, on))
        return MOE_ERR_INVALID_ARG;
    if (o && (overlap(d_o, on, dy, xn) || overlap(d_o, on, pre ? dn : nullptr, nn) || overlap(d_o, on, yr, xn) ||
              overlap(d_o, on, dx, xn)))
        return MOE_ERR_INVALID_ARG;
    JoinParams p;
    memset(&p, 0, sizeof p);
    p.x = y;
    p.o = o;
    p.pos = pos;
    p.w = w;
    p.post = post;
    p.scale = scale;
    p.pre = pre;
    p.y = dx;
    p.x_f32 = y_dtype == MOE_DT_F32;
    p.n_f32 = n_dtype == MOE_DT_F32;
    p.T = T;
    p.H = H;
    p.R = R;
    p.k = o ? k : 0;
    p.scale_all = scale_all;
    p.eps = eps;
    p.dy = dy;
    p.dn = dn;
    p.d_o = d_o;
    p.dw = w && o ? dw : nullptr;
    p.parts = static_cast<float*>(workspace);
    p.sums = sums;
    p.status = dev_status;
    const int bad = o_dtype == MOE_DT_F32 ? run_join_back<true>(p, grid, st) : run_join_back<false>(p, grid, st);
    if (bad || !sums) return bad;
    const int n = sums * H;
    return launch_pdl(join_sums_kernel, (unsigned)ceil_div(n, 32), 256, 0, st, (const float*)workspace, grid, n, H, to[0],
                      to[1], to[2]);
}

int moe_orthogonalize_workspace_bytes(int E, int N, int K, size_t* bytes) {
    NsPlan q;
    const int sms = sm_count();
    const int rc = ns_plan(E, N, K, sms > 1 ? sms : kMaxSms, &q);
    if (rc) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = q.bytes;
    return MOE_OK;
}

int moe_orthogonalize(const void* g, int g_dtype, int E, int N, int K, int steps, float a, float b, float c, float eps,
                      uint16_t* out, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    NsPlan q;
    const int sms = sm_count();
    int rc = ns_plan(E, N, K, sms > 1 ? sms : kMaxSms, &q);
    if (rc) return rc;
    if (g_dtype != MOE_DT_F32 && g_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    if (steps < 1 || steps > MOE_MAX_NS_STEPS || !(eps >= 0.0f && eps <= 1.0f)) return MOE_ERR_INVALID_ARG;
    for (const float v : {a, b, c})
        if (!(v >= -16.0f && v <= 16.0f)) return MOE_ERR_INVALID_ARG;
    MOE_REQ(g);
    MOE_REQ(out);
    MOE_OPT(dev_status);
    if (!workspace || workspace_bytes < q.bytes) return MOE_ERR_WORKSPACE;
    MOE_REQ(workspace);
    if (sms < 2) return MOE_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* ws = reinterpret_cast<unsigned char*>(align_up(reinterpret_cast<uintptr_t>(workspace), 256));
    auto take = [&](size_t bytes) {
        void* p = ws;
        ws += bytes;
        return p;
    };
    auto halves = [&](size_t bytes, bool both) {
        NsHalves h;
        h.high = static_cast<uint16_t*>(take(bytes));
        h.low = both ? static_cast<uint16_t*>(take(bytes)) : nullptr;
        return h;
    };
    // X's low half is read where it is written, but for split products, which read it all over
    const bool split = q.narrow == 2;
    NsHalves x[2] = {halves(q.x, true), halves(q.x, split)};
    if (!split) x[1].low = x[0].low;
    const NsHalves A = halves(q.a, split), B = halves(q.a, split), none = {nullptr, nullptr};
    float* parts = static_cast<float*>(take(q.p));
    const int f32 = g_dtype == MOE_DT_F32, trans = N > K;
    NsProducts s;
    bool ok = ns_params(q, E, A, A, q.m, A, B, split, true, &s.aa);
    for (int i = 0; i < 2 && ok; ++i) {
        ok = ns_params(q, E, x[i], x[i], q.n, none, A, false, true, &s.xx[i]) &&
             ns_params(q, E, x[i], B, 0, x[i], x[i ^ 1], split, false, &s.bx[i]);
        s.xx[i].status = s.bx[i].status = dev_status;
        s.last[i] = s.bx[i];
        s.last[i].res_rows = N;
        s.last[i].res_cols = K;
        s.last[i].res_trans = trans;
        s.last[i].res_sectors = K % 16 == 0 && aligned32(out);
    }
    if (!ok) return MOE_ERR_UNSUPPORTED;
    s.aa.status = dev_status;
    rc = q.narrow == 2 ? ns_allow<1, 2>() : q.narrow ? ns_allow<1, 1>() : q.pairs ? ns_allow<2, 0>() : ns_allow<1, 0>();
    if (rc) return rc;
    rc = launch_pdl(ns_norm_kernel, dim3((unsigned)q.parts, (unsigned)E), 256, 0, st, g, f32, (size_t)N * K, parts);
    if (rc) return rc;
    // (the blocks cover the padded X: its rows are G's columns where G is tall)
    const int rows = trans ? q.n : q.m, cols = trans ? q.m : q.n;
    // A block finds the norm first: with many blocks one serves four tiles.  Calls of one step, bf16 matrices of 2048 x
    // 768, one tile a block and four: one matrix (384 tiles) 46 and 48 us, two 52 and 58, four 64 and 62, six 76 and
    // 70, 16 158 and 142, 64 498 and 439
    const int64_t tiles = (int64_t)E * ceil_div(cols, 64) * ceil_div(rows, 64);
    const int strip = tiles >= 12 * sms ? 256 : 64;
    rc = launch_pdl(ns_convert_kernel, dim3((unsigned)ceil_div(cols, strip), (unsigned)ceil_div(rows, 64), (unsigned)E), 256, 0,
                    st, g, f32, N, K, (const float*)parts, q.parts, eps, trans, x[0].high, x[0].low, q.m, q.n, strip);
    if (rc) return rc;
    s.last[(steps - 1) & 1].out = out;
    return q.narrow == 2 ? run_ns_steps<1, 2>(s, E, steps, a, b, c, sms, st)
           : q.narrow    ? run_ns_steps<1, 1>(s, E, steps, a, b, c, sms, st)
           : q.pairs     ? run_ns_steps<2, 0>(s, E, steps, a, b, c, sms, st)
                         : run_ns_steps<1, 0>(s, E, steps, a, b, c, sms, st);
}

}  // extern "C"
