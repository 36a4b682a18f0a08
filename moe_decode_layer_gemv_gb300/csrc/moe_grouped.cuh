// moe_grouped.cuh -- matrix products grouped by expert with ragged segments,
// bf16 operands, fp32 accumulation (tcgen05, TMA, tensor memory).
//
// Segment e holds the rows offsets[e] .. offsets[e+1]-1 of x [R, K] and
// dy [R, N]; w is [E, N, K].  Three products share one kernel:
//   forward  y[r, n]     = sum_k w[e, n, k] x[r, k]
//   dx       dx[r, k]    = sum_n w[e, n, k] dy[r, n]
//   dw       dw[e, n, k] = sum_r dy[r, n] x[r, k]   (r over the segment)
// Each is computed as tiles D[m, n] whose m (the tensor-memory lanes) is the
// output's contiguous dimension, so that a warp's stores are contiguous, and
// whose n is the segment's rows (forward, dx) or the weight's rows (dw):
//   forward  A = w   (m = n-index of w; contraction k contiguous: K-major)
//            B = x   (K-major)
//   dx       A = w   (m = k; contraction over w's rows: MN-major), B = dy (K-major)
//   dw       A = x   (m = k; contraction over rows: MN-major), B = dy (MN-major)
// The segments are read on the device: no launch depends on their sizes.
//
// The same kernel, with other epilogues, makes the experts' gated unit, its
// gradient and the products of orthogonalisation (enum below).
//
// Measured (L2 flushed): 65536 rows over 64 experts of 1536 x 2048, paired
// tiles: forward 249 us (1655 TFLOP/s, tensor pipe 78 % busy, 12 TB/s from L2),
// dx 254, dw 254 (call after call without a pause, at the power limit: 289,
// 288, 287); 19 even segments of 4096 rows: 1830 to 1865 TFLOP/s, the ragged
// ends and the last round cost the rest.  With few rows the weights' (dw: the
// gradients') bytes bound it: 512 rows over 256 experts 206 us, the copy
// bandwidth.
#pragma once

#include "moe_common.cuh"
#include "moe_ptx.cuh"
#include "moe_umma.cuh"

namespace moe {

enum { kGgFwd = 0, kGgDx = 1, kGgDw = 2 };

// What the epilogue makes of a tile: the product itself; a gated unit of a
// forward product's gate and up rows; the gated unit's gradient of a dx
// product; and, with fp16 operands and segments of one length, the products of
// orthogonalisation (moe_ortho.cuh): a symmetric one, of which half the tiles
// are computed and stored twice, a general one, and one into the bf16 result.
enum { kGgStore = 0, kGgGlu = 1, kGgGluBack = 2, kGgSym = 3, kGgAxpy = 4, kGgResult = 5 };

constexpr int kGgMaxStages = 12;
constexpr int kGgBoxN = 32;          // rows per TMA box of a K-major B operand
constexpr int kGgTile = 128 * 128;   // bytes of one 128 x 64 bf16 operand tile
constexpr int kGgSmem = 227 * 1024;
constexpr uint32_t kGgWaitNs = 20000;     // a wait sleeps this long at a time ...
constexpr uint32_t kGgWaitLimit = 1u << 17;  // ... and gives up after so many times
constexpr uint32_t kGgTmemCols = 512;
// The tensor cores add to an accumulator with truncation, which makes a sum
// smaller with every addition: sums of one sign by 1.0e-6 in 64 MMAs (16 deep),
// by 7.4e-5 in 1024 and by 1.5e-3 in 16384, most of half a bf16 step.  So an
// accumulator takes at most so many 64-wide steps, 64 MMAs, whatever the
// result's type; the parts are added in fp32, rounded to nearest.
constexpr int kGgPartSteps = 16;

struct GgParams {
    CUtensorMap ta, tb;
    CUtensorMap tb_all;  // forward, dx: tb with boxes of 128 rows
    const int32_t* offsets;  // [E + 1]
    int E, R;
    int M;     // extent of the output's contiguous dimension
    int C;     // contraction length (forward, dx)
    int NW;    // dw: rows of a weight matrix
    int split; // dw: parts that each segment's rows are cut into, part p's result at out + p E NW M
    void* out;
    int a_blocked, b_blocked;  // MN-major operands: the map has a 64-column block dimension
    // gated units
    void* out2;      // forward: gu [R, 2 M] bf16, or nullptr; backward: h [R, M] bf16
    float c0, c1;    // the activation's coefficients
    // inputs of the epilogue, maps of GgIn's rows x 128 columns of [R, ..] (kGgGluBack: g and u, of one tensor;
    // orthogonalisation: in and what fp16 left of it), how many, the columns at which their m = 0 lies
    CUtensorMap tin[2];
    int planes, tin_at[2];
    // orthogonalisation: out = alpha product + beta in - shift 1
    float alpha, beta, shift;
    void* low;       // receives what fp16 leaves of out (but of a symmetric product that is not split)
    CUtensorMap ta_lo, tb_lo;  // split products: what fp16 left of the operands
    int halves;      // high high + high low + low high, three products in one sum
    int rows;        // of every segment (offsets is then not read)
    int res_rows, res_cols, res_trans;  // the result's matrices: [E, res_rows, res_cols], transposed or not
    int res_sectors;  // every sixteenth column of it lies on 32 bytes
    CUtensorMap zero[4];  // dw: boxes of 64 columns x 8, 4, 2 and 1 rows, for rows of zeros from behind x's end
    int32_t* status;
};

// CG CTAs (a cluster) work on one tile: with CG = 2 each holds 128 of the
// tile's 256 m and half of its n, and one tcgen05.mma.cta_group::2 reads both
// CTAs' shared memory.  KSUB 64-wide contraction steps fill one stage.
// Pairs halve what each SM reads of the shared operand: with 128 x 128 tiles
// the training batch is bound by the copies from L2 (340 us).
// Warps: EPI epilogue warps (lane quarter w & 3, share of the columns w >> 2),
// the TMA producer, the MMA issuer and for dw one that clears rows behind a
// segment.  Eight epilogue warps, since the parts of a sum are added in their
// registers (added in the output, by four, fp32 results of 65536 rows cost
// 330 us instead of 270), and since the weight gradient of few rows is all
// epilogue (0.4 GB in bf16: 126 us with four, 88 with eight, 72 by now).
template <int MODE, int CG, bool F32>
struct GgCfg {
    static constexpr int EPI = 8;
    static constexpr int kThreads = 32 * (EPI + (MODE == kGgDw ? 3 : 2));
    static constexpr int COLS = 128 * CG / (EPI / 4);  // columns an epilogue warp takes
    static constexpr int BM = 128 * CG;
    static constexpr int BN = 128 * CG;
    static constexpr int KSUB = (CG == 1 && MODE != kGgDw) ? 2 : 1;
};

// The epilogues that read inputs (kGgGluBack and later ones) get them by
// copies, a few rows of both planes for each part of the columns at a time, so
// many of them ahead.  (Loads into registers ahead of their use, beside 128
// registers of sums, were spilled as they arrived: 683 us for the training
// batch's backward pass.)  They read their tile out of tensor memory as they
// go, from one accumulator for the whole sum: a loop of few registers and
// little code.  Its truncated additions (kGgPartSteps) cost a sum of one sign
// up to 7.4e-5 of 16384 terms, 2 % of half a step of the bf16 or 15 % of
// one of the fp16 results.
constexpr int kGgInMax = 4;  // parts of the columns, and slots each, at most

// The inputs' geometry: parts of a tile's columns (with four epilogue warps
// each), rows a slot, slots a part.  What they take is lost to the ring of the
// operands: the gated unit's gradient of 65536 rows takes 205 us with 24 KB of
// them, 188 with 32 and 48, 205 with 64, 225 with 96; eight or sixteen
// epilogue warps make no difference there, as it waits for L2 by then.
template <int EP, int NARROW = 0>
struct GgIn {
    static constexpr bool kOn = EP >= kGgGluBack;
    static constexpr int kParts = EP == kGgGluBack || NARROW ? 2 : 4, kRows = 16, kSlots = EP == kGgGluBack ? 3 : 2;
    static constexpr int kPlane = kRows * 256, kSlot = kPlane * (EP == kGgSym && NARROW != 2 ? 1 : 2);  // bytes
    static constexpr int kBytes = kOn ? kParts * kSlots * kSlot : 0;
};

// Roles and limits by epilogue, over GgCfg's.  NARROW tiles of 32 columns are
// for products too small to fill the GPU: an SM takes in some 100 GB/s of
// operands, so that it is the number of SMs that counts (orthogonalisation);
// with NARROW = 2 operands and results may be in two fp16 values.
template <int MODE, int CG, bool F32, int EP, int NARROW = 0>
struct GgRole {
    static constexpr bool kIn = GgIn<EP, NARROW>::kOn;
    static constexpr int kInBytes = GgIn<EP, NARROW>::kBytes;
    static constexpr int EPI = kIn ? 4 * GgIn<EP, NARROW>::kParts : GgCfg<MODE, CG, F32>::EPI;  // epilogue warps
    static constexpr int BN = NARROW ? 32 : GgCfg<MODE, CG, F32>::BN;
    static constexpr int COLS = BN / (EPI / 4);
    static constexpr int kThreads = kIn ? 32 * (EPI + 3) : GgCfg<MODE, CG, F32>::kThreads;
    // steps an accumulator takes; fewer for a gated unit in fp32, which is a product of two sums and is to lose no
    // more of sums of one sign than one product does (1.0e-6): 1.9e-6 of the result with parts of 1024 terms, 6.5e-7
    // with 384, 4.5e-7 with 256; 65536 rows over 64 experts of 1536 x 2048: 269, 368 and 384 us
    static constexpr int kPart = kIn ? 1 << 30 : EP == kGgGlu && F32 ? 6 : kGgPartSteps;
    // (beside the inputs two steps a stage would leave room for two stages)
    static constexpr int KSUB = kIn ? 1 : GgCfg<MODE, CG, F32>::KSUB;
};

struct GgShared {
    uint64_t in_full[kGgInMax][kGgInMax], in_empty[kGgInMax][kGgInMax];
    uint64_t full[kGgMaxStages];    // leader: a stage's tiles landed (in both CTAs)
    uint64_t tfull[kGgMaxStages];   // dw: the stage that a segment ends in landed in this CTA ...
    uint64_t clear[kGgMaxStages];   // ... leader: and its rows behind the segment are zero (in both CTAs)
    uint64_t empty[kGgMaxStages];   // the MMAs have read a stage
    uint64_t acc_full[2];           // an accumulator's MMAs are complete
    uint64_t acc_empty[2];          // leader: the epilogue warps (of both CTAs) have read an accumulator
    uint64_t mma_done;
    uint32_t tmem_slot;
    int abort;                      // a bounded wait ran out
    int nmax;                       // rows of the largest segment
    int p0[MOE_MAX_E], cnt[MOE_MAX_E];
    int start[MOE_MAX_E + 1];       // tiles of rows before each segment (forward, dx)
};
static_assert(sizeof(GgShared) <= 4096, "control block");

// ------------------------------------------------------------ PTX wrappers
// Tiled loads of a stage, from and to 32-bit shared-memory addresses.  Of a
// pair (CG = 2) each CTA loads its own tiles, and `bar` is the leader's
// barrier (an address of the cluster's shared memory): one barrier then says
// that both CTAs' tiles landed.
template <int CG>
__device__ __forceinline__ void gg_load2(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void gg_load3(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void gg_load4(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                         uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void gg_load5(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                         uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
            : "memory");
}

// 64 rows x 128 columns of an MN-major operand: two 64-column blocks, one
// copy where the tensor's rows are whole blocks (the map then has a block
// dimension), else a copy each.
template <int CG>
__device__ __forceinline__ void gg_load_mn(uint32_t dst, const CUtensorMap* map, bool blocked, int col, int row,
                                           uint32_t bar) {
    if (blocked) {
        gg_load3<CG>(dst, map, 0, row, col >> 6, bar);
    } else {
        gg_load2<CG>(dst, map, col, row, bar);
        gg_load2<CG>(dst + 8192, map, col + 64, row, bar);
    }
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One lane of a converged warp.  Through elect.sync the compiler knows that a
// single thread issues what follows; behind lane == 0 each MMA's and copy's
// operands cost it some 200 cycles more.
__device__ __forceinline__ bool gg_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// The address in CTA `rank` of the cluster of what is at p here.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

// Arrive on the barrier at the same place in CTA `rank` of the cluster, for
// tensor memory that has been read or written: tcgen05.wait has completed the
// accesses, no memory that a cache may hold is handed over, and the default
// scope is enough (a cluster-scope release waits for every outstanding store:
// it doubled the time of the NVFP4 product).  What one CTA of a pair puts into
// shared memory for the leader's MMAs comes by copies that count on the
// leader's barrier, never by stores.
__device__ __forceinline__ void mbar_arrive_cluster(uint64_t* bar, uint32_t rank) {
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t"
        "mapa.shared::cluster.u32 ra, %0, %1;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}" ::"r"(smem_u32(bar)),
        "r"(rank)
        : "memory");
}

// MN-major operand, 128-byte swizzle: 64 elements (128 bytes) of the M or N
// dimension per contraction row, 8-row groups 1024 bytes apart (stride byte
// offset), 64-element blocks of M or N `lbo` bytes apart (leading byte offset).
__device__ __forceinline__ uint64_t umma_sdesc_mn(uint32_t saddr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(lbo >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

template <int CG>
__device__ __forceinline__ void gg_mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    if (CG == 1)
        umma_bf16(tmem_d, adesc, bdesc, idesc, accumulate);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Arrive on `bar` (with CG = 2: at that place in both CTAs) when every MMA
// issued so far is complete.
template <int CG>
__device__ __forceinline__ void gg_commit(uint64_t* bar) {
    if (CG == 1)
        umma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}

// Arrive on this CTA's `bar` alone.
template <int CG>
__device__ __forceinline__ void gg_commit_own(uint64_t* bar) {
    if (CG == 1)
        umma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
}

template <int CG>
__device__ __forceinline__ void gg_tmem_alloc(uint32_t* slot, uint32_t ncols) {
    if (CG == 1) {
        tmem_alloc(slot, ncols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void gg_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    if (CG == 1)
        tmem_dealloc(taddr, ncols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Bounded wait that also gives up once another role of the CTA has raised
// the abort flag.  The thread sleeps in hardware: warps that poll take the
// issue slots of the one that issues the MMAs (measured: a stage of the NVFP4
// product took twice the time).
__device__ __forceinline__ bool gg_wait(uint64_t* bar, uint32_t parity, int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < kGgWaitLimit; ++i) {
        if (mbar_try_wait_sleep(bar, parity, kGgWaitNs)) return true;
        if (*(volatile int*)abort) return false;
    }
    *(volatile int*)abort = 1;
    return false;
}

// The same for a whole warp, with one answer for its lanes.
__device__ __forceinline__ bool gg_wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
    return __all_sync(0xffffffffu, gg_wait(bar, parity, abort));
}

// A place in a ring of S stages and the parity of its current use: waits and
// addresses without a division in the single-thread issue loops, whose time a
// stage would otherwise be bound by.
struct GgRing {
    uint32_t s = 0, ph = 0, uses = 0;
    __device__ __forceinline__ void next(uint32_t S) {
        ++uses;
        if (++s == S) {
            s = 0;
            ph ^= 1u;
        }
    }
};

// Tiles unit, unit + units, ... as (outer, inner) with inner < n, without a
// division a tile.
struct GgWalk {
    int outer, inner, d_outer, d_inner, n;
    __device__ __forceinline__ GgWalk(int unit, int units, int n_) : n(n_) {
        outer = unit / n;
        inner = unit - outer * n;
        d_outer = units / n;
        d_inner = units - d_outer * n;
    }
    __device__ __forceinline__ void next() {
        outer += d_outer;
        inner += d_inner;
        if (inner >= n) {
            inner -= n;
            ++outer;
        }
    }
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// The segment of row tile `it`, which is not before segment e.
__device__ __forceinline__ int gg_seek(const int* start, int E, int it, int e) {
    if (it < start[e + 1]) return e;
    int lo = e + 1, hi = E - 1;  // the last segment with start <= it
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= it)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Bounded wait for what is certainly under way, abort or not.
__device__ __forceinline__ void gg_settle(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < kGgWaitLimit; ++i)
        if (mbar_try_wait_sleep(bar, parity, kGgWaitNs)) return;
}

// The producer's teardown: no copy, and no release of a stage by the
// leader's MMAs, may be on its way when the CTA exits.  (After an abort some
// copies cannot be waited for here, those of a pair's other CTA and of a
// segment's end: they are given the time to land.)
template <int CG>
__device__ __forceinline__ void gg_drain(GgShared* sh, uint32_t S, const GgRing& r, uint32_t rank) {
    for (uint32_t s = 0; s < S && s < r.uses; ++s) {
        const uint32_t ph = s < r.s ? r.ph : r.ph ^ 1u;  // the parity of the stage's last use
        if (rank == 0) gg_settle(&sh->full[s], ph);
        if (CG == 2) gg_wait(&sh->empty[s], ph, &sh->abort);
    }
    if (*(volatile int*)&sh->abort)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// Whether a 64-row step with `left` rows to the segment's end needs clearing.
__device__ __forceinline__ bool gg_ragged(int left) { return left < 64 && (left & 15); }

// ---------------------------------------------------------------- loads
// Every input may come from the kernel ahead on the stream, which may still
// run when this one is launched (grid_dep_wait): none is read-only for this
// kernel's whole life, so none is read through the non-coherent path (no
// ld.global.nc, no __restrict__).  Volatile, so that a few rows' products
// issue them with the weights' loads (4.3 us for 5.2).
__device__ __forceinline__ uint4 ld_input_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ float ld_input_f(const float* p) {
    float r;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(r) : "l"(p));
    return r;
}
// What is read once:
__device__ __forceinline__ uint4 ld_stream_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// ------------------------------------------------------------- segments
// The segments into shared memory.  Offsets outside [0, R] or descending
// leave their segment out (and set MOE_DEV_BAD_OFFSETS): nothing is read or
// written outside the tensors.  start[e] = tiles of bn rows before segment e.
__device__ __forceinline__ void gg_segments(GgShared* sh, const int32_t* offsets, int rows, int E, int R, int bn,
                                            int32_t* status) {
    const int tid = threadIdx.x;
    if (tid == 0) sh->nmax = 0;
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) {
        const int a = rows ? e * rows : offsets[e], b = rows ? a + rows : offsets[e + 1];
        const bool ok = a >= 0 && b >= a && b <= R;
        if (!ok && blockIdx.x == 0) set_status(status, MOE_DEV_BAD_OFFSETS);
        sh->p0[e] = ok ? a : 0;
        sh->cnt[e] = ok ? b - a : 0;
        if (ok && b > a) atomicMax(&sh->nmax, b - a);
    }
    __syncthreads();
    if (tid < 32) {  // exclusive scan, 8 segments a lane
        int c[MOE_MAX_E / 32], sum = 0;
#pragma unroll
        for (int j = 0; j < MOE_MAX_E / 32; ++j) {
            const int e = tid * (MOE_MAX_E / 32) + j;
            c[j] = sum;
            sum += e < E ? (sh->cnt[e] + bn - 1) / bn : 0;
        }
        int run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o);
            if (tid >= o) run += v;
        }
#pragma unroll
        for (int j = 0; j < MOE_MAX_E / 32; ++j) {
            const int e = tid * (MOE_MAX_E / 32) + j;
            if (e < E) sh->start[e] = run - sum + c[j];
        }
        if (tid == 31) sh->start[E] = run;
    }
    __syncthreads();
}

// ------------------------------------------------------------- epilogue
// 32 consecutive fp32 columns of this warp's 32 TMEM lanes; the registers are
// valid after gg_ld_wait (which names them, so that no use moves above it).
__device__ __forceinline__ void gg_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void gg_ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// This lane's two neighbouring m of one row, in bf16, from two rows' values
// in lanes 2i and 2i + 1: the even lane takes the first row, the odd the second.
__device__ __forceinline__ uint32_t gg_pack(uint32_t first, uint32_t second) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(first), __uint_as_float(second));
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t gg_pair(uint32_t packed, uint32_t select) {
    return __byte_perm(packed, __shfl_xor_sync(0xffffffffu, packed, 1), select);
}
__device__ __forceinline__ uint32_t gg_pair_select(int odd) { return odd ? 0x3276u : 0x5410u; }

// Store 32 columns (output rows row0 .. row0 + nc - 1) of this lane's m:
// fp32 as they are, a warp writing 128 contiguous bytes a row; bf16 after
// lanes 2i and 2i + 1 have exchanged a value per pair of rows, so that each
// lane writes two neighbouring m (4 bytes) of one row.
__device__ __forceinline__ void gg_store32(const uint32_t (&r)[32], void* out, int out_f32, size_t row0, int nc, int m,
                                           int M) {
    const bool whole = nc >= 32;
    if (out_f32) {
        uint32_t* o = static_cast<uint32_t*>(out) + row0 * (size_t)M + m;
        if (m >= M) return;
        if (whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j, o += M) *o = r[j];
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j, o += M)
                if (j < nc) *o = r[j];
        }
        return;
    }
    const int odd = m & 1;
    const uint32_t sel = gg_pair_select(odd);
    uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + (row0 + odd) * (size_t)M + (m - odd));
    const int last = m < M ? nc - odd : 0;  // rows row0 + odd + j, j < last
    if (__all_sync(0xffffffffu, whole && m < M)) {
#pragma unroll
        for (int j = 0; j < 32; j += 2, o += M) *o = gg_pair(gg_pack(r[j], r[j + 1]), sel);
    } else {
#pragma unroll
        for (int j = 0; j < 32; j += 2, o += M) {
            const uint32_t v = gg_pair(gg_pack(r[j], r[j + 1]), sel);
            if (j < last) *o = v;
        }
    }
}

// An accumulator's COLS columns into `sum` (the first part), or added to it.
template <int COLS>
__device__ __forceinline__ void gg_gather(uint32_t taddr, uint32_t (&sum)[COLS / 32][32], int n, bool first) {
    if (first) {
#pragma unroll
        for (int i = 0; i < COLS / 32; ++i)
            if (32 * i < n) gg_ld32(taddr + 32 * i, sum[i]);
#pragma unroll
        for (int i = 0; i < COLS / 32; ++i) gg_ld_wait(sum[i]);
    } else {
#pragma unroll
        for (int i = 0; i < COLS / 16; ++i) {
            if (16 * i >= n) break;
            float v[16];
            tmem_ld16(taddr + 16 * i, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                uint32_t& t = sum[i / 2][i % 2 * 16 + j];
                t = __float_as_uint(__uint_as_float(t) + v[j]);
            }
        }
    }
}

// ------------------------------------------------------------- gated units
// act(g) = g s(q), s the logistic function and q = g (c0 + c1 g^2): SiLU with
// c0 = 1, c1 = 0, GELU's tanh form with c0 = 2 sqrt(2 / pi), c1 = 0.044715 c0
// (g (1 + tanh(q / 2)) / 2 = g s(q)).
//   act'(g) = s + g s (1 - s) q',   q' = c0 + 3 c1 g^2
// g^2 is kept finite, so that c1 = 0 and s = 0 or 1 count for what they are.
__device__ __forceinline__ float glu_act(float g, float c0, float c1, float& grad) {
    const float gg = fminf(g * g, 1e30f);
    const float s = __fdividef(1.0f, 1.0f + expf(-g * fmaf(c1, gg, c0)));
    const float a = g * s;
    grad = fmaf(a * (1.0f - s), fmaf(3.0f * c1, gg, c0), s);
    return a;
}

// The gated unit of a forward tile.  A CTA's 128 rows are gate rows and up
// rows in alternating groups of eight (one five-dimensional copy brings them
// so), which leaves g and u of one output eight lanes apart: each lane of the
// pair gives the other one of two rows' values and makes one row's result.  i0:
// the first of this warp's 16 outputs.  (Gate and up rows in halves of the
// tile, exchanged through shared memory, would need barriers between warps;
// two accumulators with g and u in one lane 5/4 of the copies from L2.)
// 65536 rows over 64 experts of 1536 x 2048, L2 flushed: 256 us, the product
// alone 252; 288 with gu, 200 MB, stored as well.
template <int COLS, bool F32, typename P>
__device__ __forceinline__ void glu_store(const P& p, uint32_t (&sum)[COLS / 32][32], size_t row0, int mine, int i0,
                                          int lane) {
    const int up = (lane >> 3) & 1, i = i0 + ((lane >> 4) << 3) + (lane & 7), I = p.M;
    const int col = i < I ? i + (up ? I : 0) : 2 * I;
#pragma unroll
    for (int k = 0; k < COLS / 32; ++k) {
        const int nc = mine - 32 * k;
        if (nc <= 0) break;
        uint32_t(&r)[32] = sum[k];
        if (p.out2) gg_store32(r, p.out2, 0, row0 + 32 * k, min(32, nc), col, 2 * I);
        // bf16: lanes 2 l and 2 l + 1 swap once more, so that each writes two neighbouring outputs (4 bytes) of one row
        const int odd = i & 1;
        const size_t at = (row0 + 32 * k + up + (F32 ? 0 : 2 * odd)) * (size_t)I + (F32 ? i : i - odd);
        const int last = i < I ? nc - up - (F32 ? 0 : 2 * odd) : 0;
        float before = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? r[j] : r[j + 1], 8);
            const float g = __uint_as_float(up ? got : r[j]), u = __uint_as_float(up ? r[j + 1] : got);
            float grad;
            const float h = glu_act(g, p.c0, p.c1, grad) * u;
            if (F32) {
                if (j < last) static_cast<float*>(p.out)[at + (size_t)j * I] = h;
            } else if (j % 4 == 0) {
                before = h;
            } else {
                const uint32_t v = gg_pair(gg_pack(__float_as_uint(before), __float_as_uint(h)), gg_pair_select(odd));
                if (j - 2 < last) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at + (size_t)(j - 2) * I) = v;
            }
        }
    }
}

// A place in the ring of a part's epilogue inputs.
template <int SLOTS>
struct GgInRing {
    uint32_t s = 0, ph = 0, uses = 0;
    __device__ __forceinline__ void next() {
        ++uses;
        if (++s == SLOTS) {
            s = 0;
            ph ^= 1u;
        }
    }
};

__device__ __forceinline__ float in_f16(const uint16_t* at, int row) {
    return __half2float(*reinterpret_cast<const __half*>(at + row * 128));
}
__device__ __forceinline__ uint32_t in_pair(const uint16_t* at, int row) {
    return *reinterpret_cast<const uint32_t*>(at + row * 128);
}

// Two rows' sums of this lane's m (d0, d1) into two neighbouring m, m - odd and
// m - odd + 1, of row `odd` of the two: the lanes of a pair swap one each, and
// what is read and written beside them then comes in 4-byte pieces as it lies
// in memory.
__device__ __forceinline__ float2 gg_swap(float d0, float d1, int odd) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? d0 : d1, 1);
    return odd ? make_float2(got, d1) : make_float2(d0, got);
}

// Two rows' values of this lane's m, packed, the same way into 4 bytes of `to`.
__device__ __forceinline__ void gg_put(uint16_t* to, uint32_t packed, uint32_t sel, bool there) {
    const uint32_t v = gg_pair(packed, sel);
    if (there) *reinterpret_cast<uint32_t*>(to) = v;
}

// The gated unit's gradient of ROWS rows of a dx tile (dh, d), this lane's m:
//   dg = dh u act'(g),  du = dh act(g),  h = act(g) u
// row: the first of them; n: how many are there; ins: the inputs at m = 0 of this warp's 32.
// 65536 rows over 64 experts of 2048 x 768, L2 flushed: 191 us, 0.75 of what
// its 0.97 GB take at the copy bandwidth; what crosses from and to L2, 2.2 GB,
// takes about as long as that.
template <int ROWS, typename P>
__device__ __forceinline__ void glu_back_rows(const P& p, const float* d, const uint16_t* ins, size_t row, int n, int m,
                                              int lane) {
    const int I = p.M, odd = lane & 1;
    const int last = m < I ? n - odd : 0;  // rows row + odd + j, j < last
    const uint16_t *g = ins + (lane - odd) + odd * 128, *u = g + ROWS * 128;
    uint16_t* dg = static_cast<uint16_t*>(p.out) + (row + odd) * 2 * (size_t)I + (m - odd);
    uint16_t* hp = static_cast<uint16_t*>(p.out2) + (row + odd) * (size_t)I + (m - odd);
#pragma unroll
    for (int j = 0; j < ROWS; j += 2, dg += 4 * (size_t)I, hp += 2 * (size_t)I) {
        const float2 dh = gg_swap(d[j], d[j + 1], odd), gf = bf16x2_to_f2(in_pair(g, j)), uf = bf16x2_to_f2(in_pair(u, j));
        float e0, e1;
        const float a0 = glu_act(gf.x, p.c0, p.c1, e0), a1 = glu_act(gf.y, p.c0, p.c1, e1);
        auto pack = [](float v0, float v1) { return gg_pack(__float_as_uint(v0), __float_as_uint(v1)); };
        if (j < last) {
            *reinterpret_cast<uint32_t*>(dg) = pack(dh.x * uf.x * e0, dh.y * uf.y * e1);
            *reinterpret_cast<uint32_t*>(dg + I) = pack(dh.x * a0, dh.y * a1);
            *reinterpret_cast<uint32_t*>(hp) = pack(a0 * uf.x, a1 * uf.y);
        }
    }
}

// ------------------------------------------------------- orthogonalisation
__device__ __forceinline__ uint32_t gg_pack_f16(float first, float second) {
    const __half2 h = __floats2half2_rn(first, second);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 bytes, a whole sector, in one store (32-byte aligned)
__device__ __forceinline__ void st_v8(void* to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ float2 f16x2_to_f2(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

// out = alpha product + beta in for ROWS rows of this lane's m, from row r of
// segment e on, n of them there; in and out in two fp16 values each.
template <int ROWS, typename P>
__device__ __forceinline__ void ns_axpy_rows(const P& p, const float* d, const uint16_t* ins, int e, int r, int n, int m,
                                             int lane) {
    const int M = p.M, odd = lane & 1;
    const int last = m < M ? n - odd : 0;  // rows r + odd + j, j < last
    const uint16_t *in = ins + (lane - odd) + odd * 128, *lo = in + ROWS * 128;
    const size_t pair = ((size_t)e * p.rows + r + odd) * M + (m - odd);
    uint16_t *to = static_cast<uint16_t*>(p.out) + pair, *tl = static_cast<uint16_t*>(p.low) + pair;
#pragma unroll
    for (int j = 0; j < ROWS; j += 2, to += 2 * (size_t)M, tl += 2 * (size_t)M) {
        const float2 v = gg_swap(d[j], d[j + 1], odd), f = f16x2_to_f2(in_pair(in, j)), l = f16x2_to_f2(in_pair(lo, j));
        const float v0 = fmaf(p.beta, f.x + l.x, p.alpha * v.x), v1 = fmaf(p.beta, f.y + l.y, p.alpha * v.y);
        const uint32_t w = gg_pack_f16(v0, v1);
        const float2 t = f16x2_to_f2(w);
        const uint32_t x = gg_pack_f16(v0 - t.x, v1 - t.y);
        if (j < last) {
            *reinterpret_cast<uint32_t*>(to) = w;
            *reinterpret_cast<uint32_t*>(tl) = x;
        }
    }
}

// The same without (unless SPLIT) the low parts, of a symmetric product less shift on the
// diagonal, into rows of p.M fp16 values (a multiple of 16, as are the rows);
// of a tile below the diagonal also into its mirror image, where a lane's
// values lie side by side, 32 bytes.
template <int ROWS, bool SPLIT, typename P>
__device__ __forceinline__ void ns_sym_rows(const P& p, const float* d, const uint16_t* ins, int e, int r, int m, int lane,
                                            bool mirror) {
    const int M = p.M, odd = lane & 1;
    const uint32_t sel = gg_pair_select(odd);
    const bool there = m < M;
    uint16_t* out = static_cast<uint16_t*>(p.out);
    uint16_t* to = out + ((size_t)e * p.rows + r + odd) * M + (m - odd);
    uint16_t* tl = SPLIT ? static_cast<uint16_t*>(p.low) + (to - out) : nullptr;
    uint32_t w[ROWS / 2];  // rows j and j + 1 of this lane's m
#pragma unroll
    for (int j = 0; j < ROWS; j += 2, to += 2 * (size_t)M) {
        float v0 = p.alpha * d[j], v1 = p.alpha * d[j + 1];
        if (p.planes) {
            float f0 = in_f16(ins + lane, j), f1 = in_f16(ins + lane, j + 1);
            if (SPLIT) f0 += in_f16(ins + ROWS * 128 + lane, j), f1 += in_f16(ins + ROWS * 128 + lane, j + 1);
            v0 = fmaf(p.beta, f0, v0);
            v1 = fmaf(p.beta, f1, v1);
        }
        if (!mirror) {
            v0 -= r + j == m ? p.shift : 0.0f;
            v1 -= r + j + 1 == m ? p.shift : 0.0f;
        }
        w[j / 2] = gg_pack_f16(v0, v1);
        gg_put(to, w[j / 2], sel, there);
        if (SPLIT) {
            const float2 t = f16x2_to_f2(w[j / 2]);
            gg_put(tl, gg_pack_f16(v0 - t.x, v1 - t.y), sel, there);
            tl += 2 * (size_t)M;
        }
    }
    if (mirror && there) {
        static_assert(ROWS == 16, "a sector");
        st_v8(out + ((size_t)e * p.rows + m) * M + r, w);
    }
}

// The last product: bf16 into matrices of any size, as they are or transposed.
template <int ROWS, typename P>
__device__ __forceinline__ void ns_result_rows(const P& p, const float* d, const uint16_t* ins, int e, int r, int n, int m,
                                               int lane) {
    const int odd = lane & 1;
    const uint32_t sel = gg_pair_select(odd);
    const uint16_t *in = ins + lane, *lo = in + ROWS * 128;
    uint16_t* out = static_cast<uint16_t*>(p.out);
    uint32_t w[ROWS / 2];  // rows j and j + 1 of this lane's m
#pragma unroll
    for (int j = 0; j < ROWS; j += 2) {
        const float v0 = fmaf(p.beta, in_f16(in, j) + in_f16(lo, j), p.alpha * d[j]);
        const float v1 = fmaf(p.beta, in_f16(in, j + 1) + in_f16(lo, j + 1), p.alpha * d[j + 1]);
        w[j / 2] = gg_pack(__float_as_uint(v0), __float_as_uint(v1));
    }
    if (p.res_trans) {
        if (m >= p.res_rows) return;
        uint16_t* to = out + ((size_t)e * p.res_rows + m) * p.res_cols + r;
        const int k = min(n, p.res_cols - r);
        static_assert(ROWS == 16, "a sector");
        if (k == ROWS && p.res_sectors) {
            st_v8(to, w);
            return;
        }
#pragma unroll
        for (int j = 0; j < ROWS; j += 8) {
            if (j + 8 <= k && p.res_cols % 8 == 0) {
                *reinterpret_cast<uint4*>(to + j) = make_uint4(w[j / 2], w[j / 2 + 1], w[j / 2 + 2], w[j / 2 + 3]);
            } else {
                const bool even = p.res_cols % 2 == 0;  // (pairs then lie on 4 bytes, and k is even)
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    if (j + i >= k) break;
                    if (even) {
                        *reinterpret_cast<uint32_t*>(to + j + i) = w[(j + i) / 2];
                    } else {
                        to[j + i] = (uint16_t)w[(j + i) / 2];
                        if (j + i + 1 < k) to[j + i + 1] = (uint16_t)(w[(j + i) / 2] >> 16);
                    }
                }
            }
        }
    } else {
        const int rows = min(n, p.res_rows - r);
        uint16_t* to = out + ((size_t)e * p.res_rows + r) * p.res_cols + m;
        const bool even = p.res_cols % 2 == 0;
#pragma unroll
        for (int j = 0; j < ROWS; j += 2, to += 2 * (size_t)p.res_cols) {
            const uint32_t v = gg_pair(w[j / 2], sel);
            if (m >= p.res_cols) continue;
            if (even) {
                if (j + odd < rows) *reinterpret_cast<uint32_t*>(to + (size_t)odd * p.res_cols - odd) = v;
            } else {
                if (j < rows) to[0] = (uint16_t)w[j / 2];
                if (j + 1 < rows) to[p.res_cols] = (uint16_t)(w[j / 2] >> 16);
            }
        }
    }
}

// ------------------------------------------------------------- the kernel
// Persistent: one CTA per SM (or one pair of CTAs per SM pair) walks the
// tiles.  Three roles run through the same tile sequence, each at its own
// pace: the producer fills the ring, the MMA issuer accumulates tile d into
// tensor-memory buffer d mod 2, the epilogue warps read the other buffer out.
template <int MODE, int CG, bool F32, int EP = kGgStore, int NARROW = 0>
__global__ void __launch_bounds__((GgRole<MODE, CG, F32, EP, NARROW>::kThreads), 1) gg_kernel(const __grid_constant__ GgParams p) {
    using Cfg = GgCfg<MODE, CG, F32>;
    extern __shared__ __align__(1024) unsigned char gg_smem_raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(gg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    GgShared* sh = reinterpret_cast<GgShared*>(base);
    using Role = GgRole<MODE, CG, F32, EP, NARROW>;
    using In = GgIn<EP, NARROW>;
    constexpr bool kMirror = EP == kGgSym && !NARROW;  // half the tiles, stored twice
    unsigned char* ins = base + 4096;
    unsigned char* ring = ins + Role::kInBytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const int unit = (int)blockIdx.x / CG, units = (int)gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int s = 0; Role::kIn && s < kGgInMax * kGgInMax; ++s) {
            mbar_init(&sh->in_full[0][s], 1);
            mbar_init(&sh->in_empty[0][s], 4);
        }
        for (int s = 0; s < kGgMaxStages; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->tfull[s], 1);
            mbar_init(&sh->clear[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], Role::EPI * CG);
        }
        mbar_init(&sh->mma_done, 1);
        sh->abort = 0;
        fence_mbar_init();
        prefetch_map(&p.ta);
        prefetch_map(&p.tb);
        if (MODE != kGgDw) prefetch_map(&p.tb_all);
    }
    if (warp == Role::EPI + 1) gg_tmem_alloc<CG>(&sh->tmem_slot, kGgTmemCols);
    if (EP == kGgSym || EP == kGgAxpy) grid_dep_launch();  // (what follows touches nothing before its grid_dep_wait)
    if (EP < kGgSym) grid_dep_wait();
    constexpr int MW = EP == kGgGlu ? 64 : 128, BMW = MW * CG;  // outputs that a CTA's 128 rows and a tile give
    const int mtiles = (p.M + BMW - 1) / BMW;
    gg_segments(sh, p.offsets, EP >= kGgSym ? p.rows : 0, p.E, p.R, Role::BN, p.status);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_slot;
    if (EP >= kGgSym) grid_dep_wait();  // (the segments came from no memory)

    // Ring geometry.  A stage holds Role::KSUB A tiles and Role::KSUB B tiles; where the
    // B operand is the segment's rows, its tiles are as high as the largest
    // segment needs, so that few rows leave more bytes of weights in flight.
    uint32_t b_tile = kGgTile;
    if (MODE != kGgDw && CG == 1)
        b_tile = (uint32_t)min(Role::BN, max(kGgBoxN, (sh->nmax + kGgBoxN - 1) / kGgBoxN * kGgBoxN)) * 128u;
    const uint32_t stage_bytes = Role::KSUB * (kGgTile + b_tile);
    const uint32_t b_off = Role::KSUB * kGgTile;
    const uint32_t S = min((uint32_t)kGgMaxStages, ((uint32_t)kGgSmem - 1023u - 4096u - Role::kInBytes) / stage_bytes);

    const int ntiles_w = (p.NW + Role::BN - 1) / Role::BN;  // dw
    const int tri = kMirror ? mtiles * (mtiles + 1) / 2 : 0;  // tiles on and below the diagonal
    const int outers = kMirror ? p.E : MODE == kGgDw ? p.split * p.E : sh->start[p.E];

    // f(e, q0, n, n0, m0, len): segment e; first row q0 (forward, dx: of the
    // tile; dw: of the segment's part); n valid columns from n0 on; m from m0
    // on; contraction length.  (dw: e counts part after part, part * E + e)
    auto walk = [&](auto f) {
        int e = 0;
        for (GgWalk w(unit, units, kMirror ? tri : MODE == kGgDw ? mtiles * ntiles_w : mtiles); w.outer < outers; w.next()) {
            int q0, n, n0, m0, len;
            if (kMirror) {
                e = w.outer;
                int i = 0, j = w.inner;  // row i of the triangle holds i + 1 tiles
                while (j > i) j -= ++i;
                m0 = j * BMW;
                n0 = i * Role::BN;
                n = min(Role::BN, p.rows - n0);
                q0 = e * p.rows + n0;
                len = p.C;
            } else if (MODE == kGgDw) {
                e = w.outer;
                const int tn = w.inner / mtiles;
                m0 = (w.inner - tn * mtiles) * BMW;
                n0 = tn * Role::BN;
                n = min(Role::BN, p.NW - n0);
                const int seg = p.split == 1 ? e : e % p.E, cnt = sh->cnt[seg];
                int part = cnt, at = 0;
                if (p.split > 1) {
                    part = ((cnt + p.split - 1) / p.split + 63) / 64 * 64;
                    at = min(cnt, e / p.E * part);
                }
                q0 = sh->p0[seg] + at;
                len = min(part, cnt - at);
            } else {
                e = gg_seek(sh->start, p.E, w.outer, e);
                m0 = w.inner * BMW;
                n0 = (w.outer - sh->start[e]) * Role::BN;
                n = min(Role::BN, sh->cnt[e] - n0);
                q0 = sh->p0[e] + n0;
                len = p.C;
            }
            if (!f(e, q0, n, n0, m0, len)) break;
        }
    };
    if (warp == Role::EPI) {
        // ---------------- TMA producer
        GgRing r;
        const uint32_t ring_at = smem_u32(ring);
        const uint32_t bars = CG == 1 ? smem_u32(sh->full) : cluster_addr(sh->full, 0);
        if (gg_elect()) {
            walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
                const int nk = (len + 63) / 64, nks = NARROW == 2 && p.halves ? 3 * nk : nk;
                // rows of B that this CTA holds (forward, dx), in whole boxes
                const int rows = MODE == kGgDw ? 128 : (n + kGgBoxN * CG - 1) / (kGgBoxN * CG) * kGgBoxN;
                const uint32_t bytes = CG * (kGgTile + (uint32_t)rows * 128u);
                const int am = m0 + (int)rank * MW, bn = (MODE == kGgDw ? n0 : q0) + (int)rank * rows;
                for (int k0 = 0; k0 < nks; k0 += Role::KSUB) {
                    if (!gg_wait(&sh->empty[r.s], r.ph ^ 1u, &sh->abort)) return false;
                    const uint32_t st = ring_at + r.s * stage_bytes, bar = bars + r.s * 8u;
                    const int ke = min(Role::KSUB, nks - k0);
                    // dw: the stage that a segment ends in, if not with a whole MMA, lands on
                    // each CTA's own barrier and is cleared there before it counts as full
                    const bool tail = MODE == kGgDw && gg_ragged(len - k0 * 64);
                    const uint32_t tbar = smem_u32(&sh->tfull[r.s]);
                    if (tail) mbar_arrive_expect_tx(&sh->tfull[r.s], kGgTile + (uint32_t)rows * 128u);
                    if (rank == 0) {
                        if (tail)
                            mbar_arrive(&sh->full[r.s]);
                        else
                            mbar_arrive_expect_tx(&sh->full[r.s], (uint32_t)ke * bytes);
                    }
#pragma unroll
                    for (int u = 0; u < Role::KSUB; ++u) {
                        if (u >= ke) break;
                        const uint32_t sa = st + u * kGgTile, sb = st + b_off + u * b_tile;
                        const int part = NARROW == 2 ? (k0 + u) / nk : 0;  // of a split product
                        const int c = (k0 + u - part * nk) * 64;
                        const CUtensorMap* const ta = part == 2 ? &p.ta_lo : &p.ta;
                        const CUtensorMap* const tb = part == 1 ? &p.tb_lo : &p.tb;
                        if (EP == kGgGlu) {
                            gg_load5<CG>(sa, &p.ta, c, 0, 0, am >> 3, e, bar);
                        } else if (MODE == kGgFwd) {
                            gg_load3<CG>(sa, ta, c, am, e, bar);
                        } else if (MODE == kGgDx) {
                            if (p.a_blocked) {
                                gg_load4<CG>(sa, ta, 0, c, am >> 6, e, bar);
                            } else {
                                gg_load3<CG>(sa, &p.ta, am, c, e, bar);
                                gg_load3<CG>(sa + 8192, &p.ta, am + 64, c, e, bar);
                            }
                        } else if (tail) {
                            gg_load_mn<1>(sa, &p.ta, p.a_blocked, am, q0 + c, tbar);
                            gg_load_mn<1>(sb, &p.tb, p.b_blocked, bn, q0 + c, tbar);
                        } else {
                            gg_load_mn<CG>(sa, &p.ta, p.a_blocked, am, q0 + c, bar);
                            gg_load_mn<CG>(sb, &p.tb, p.b_blocked, bn, q0 + c, bar);
                        }
                        if (MODE == kGgDw) {
                        } else if (rows == 128) {
                            gg_load2<CG>(sb, &p.tb_all, c, bn, bar);
                        } else {
                            for (int i = 0; i < rows; i += kGgBoxN) gg_load2<CG>(sb + i * 128, tb, c, bn + i, bar);
                        }
                    }
                    r.next(S);
                }
                return true;
            });
            gg_drain<CG>(sh, S, r, rank);
        }
        __syncwarp();
    } else if (warp == Role::EPI + 1) {
        // ---------------- MMA issuer (one thread of the leader)
        GgRing r;
        int buf = 0;
        uint32_t free_ph = 1;  // parity of acc_empty to wait for (at first: nothing)
        uint32_t tails = 0;    // parity of each stage's next use as a segment's end
        const uint32_t ring_at = smem_u32(ring);
        if (rank == 0 && gg_elect()) walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
            const int nk = ((len + 63) / 64) * (NARROW == 2 && p.halves ? 3 : 1);
            const int npad = MODE == kGgDw ? Role::BN : (n + kGgBoxN * CG - 1) / (kGgBoxN * CG) * (kGgBoxN * CG);
            const uint32_t idesc = (EP >= kGgSym ? umma_idesc_f16(Cfg::BM, npad) : umma_idesc_bf16(Cfg::BM, npad)) | (MODE != kGgFwd ? 1u << 15 : 0u) |
                                   (MODE == kGgDw ? 1u << 16 : 0u);
            uint32_t acc = 0, tacc = 0;
            int room = 0;  // steps that the accumulator still takes
            for (int k0 = 0; k0 < nk; k0 += Role::KSUB) {
                if (room == 0) {
                    if (!gg_wait(&sh->acc_empty[buf], free_ph, &sh->abort)) return false;
                    tacc = tmem + (uint32_t)(buf * Role::BN);
                    acc = 0;
                    room = Role::kPart;
                }
                if (!gg_wait(&sh->full[r.s], r.ph, &sh->abort)) return false;
                const uint32_t sta = ring_at + r.s * stage_bytes;
                int steps = 4;  // MMAs (16 deep) of a 64-wide step
                if (MODE == kGgDw) {
                    const int valid = len - k0 * 64;
                    if (valid < 64) steps = (valid + 15) / 16;
                    if (gg_ragged(valid)) {
                        if (!gg_wait(&sh->clear[r.s], (tails >> r.s) & 1u, &sh->abort)) return false;
                        tails ^= 1u << r.s;
                    }
                }
                room -= Role::KSUB;  // (a whole number of stages)
                const bool last = room == 0 || k0 + Role::KSUB >= nk;
                tc_fence_after();
                const int ke = min(Role::KSUB, nk - k0);
#pragma unroll
                for (int u = 0; u < Role::KSUB; ++u) {
                    if (u >= ke) break;
                    // the 16-deep steps of a tile: 32 bytes of a K-major row, 16 rows of an MN-major tile
                    const uint32_t aa = sta + u * kGgTile, ba = sta + b_off + u * b_tile;
                    const uint64_t ad = MODE == kGgFwd ? umma_sdesc(aa) : umma_sdesc_mn(aa, 8192);
                    const uint64_t bd = MODE == kGgDw ? umma_sdesc_mn(ba, 8192) : umma_sdesc(ba);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (MODE == kGgDw && kk >= steps) break;
                        gg_mma<CG>(tacc, ad + (uint64_t)(kk * (MODE == kGgFwd ? 32 : 2048) / 16),
                                   bd + (uint64_t)(kk * (MODE == kGgDw ? 2048 : 32) / 16), idesc,
                                   u == 0 && kk == 0 ? acc : 1u);
                    }
                }
                gg_commit<CG>(&sh->empty[r.s]);
                if (last) gg_commit<CG>(&sh->acc_full[buf]);
                acc = 1;
                if (last) {
                    room = 0;
                    buf ^= 1;
                    if (buf == 0) free_ph ^= 1u;
                }
                r.next(S);
            }
            return true;
        });
        __syncwarp();
        if (rank == 0 && gg_elect()) {
            gg_commit_own<CG>(&sh->mma_done);
            gg_settle(&sh->mma_done, 0u);
        }
        __syncwarp();
    } else if (Role::kIn && warp == Role::EPI + 2) {
        // ---------------- inputs of the epilogue
        GgInRing<In::kSlots> r[In::kParts];
        if (p.planes && gg_elect()) {
            walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
                const int m = m0 + (int)rank * MW;
                for (int c = 0; c < Role::COLS; c += In::kRows)
#pragma unroll
                    for (int h = 0; h < In::kParts; ++h) {
                        const int row = h * Role::COLS + c;
                        if (row >= n) break;
                        if (!gg_wait(&sh->in_empty[h][r[h].s], r[h].ph ^ 1u, &sh->abort)) return false;
                        uint64_t* bar = &sh->in_full[h][r[h].s];
                        const uint32_t to = smem_u32(ins) + (h * In::kSlots + r[h].s) * In::kSlot;
                        mbar_arrive_expect_tx(bar, p.planes * In::kPlane);
                        for (int i = 0; i < p.planes; ++i)
                            gg_load2<1>(to + i * In::kPlane, &p.tin[i], p.tin_at[i] + m, q0 + row, smem_u32(bar));
                        r[h].next();
                    }
                return true;
            });
            // no copy may be on its way when the CTA exits
#pragma unroll
            for (int h = 0; h < In::kParts; ++h)
                for (uint32_t s = 0; s < In::kSlots && s < r[h].uses; ++s)
                    gg_settle(&sh->in_full[h][s], s < r[h].s ? r[h].ph : r[h].ph ^ 1u);
        }
        __syncwarp();
    } else if (MODE == kGgDw && warp == Role::EPI + 2) {
        // ---------------- dw: the segment's end.  Rows behind it belong to
        // the next segment (or to no one), so both operands' rows up to the
        // last MMA's end are zeroed -- zeroing one would leave 0 x infinity or
        // 0 x NaN.  A warp of its own does it in each CTA as soon as the rows
        // landed, with copies of rows behind the tensor's end, which read as
        // zeros and count on the leader's barrier as the tiles do: nothing
        // written by a thread passes from one CTA to the other's MMAs.
        // (Stores of zeros handed over by a release at cluster scope take the
        // training batch from 254 to 280 us, loading a segment's last rows
        // piecemeal instead 258.)
        GgRing r;
        uint32_t tails = 0;
        walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
            const int nk = (len + 63) / 64, left = len - (nk - 1) * 64;
            for (int k = 0; k + 1 < nk; ++k) r.next(S);
            if (nk > 0) {
                if (gg_ragged(left)) {
                    if (!gg_wait_warp(&sh->tfull[r.s], (tails >> r.s) & 1u, &sh->abort)) return false;
                    tails ^= 1u << r.s;
                    if (gg_elect()) {
                        // (two boxes of the largest height that fits, overlapping)
                        const int rows = 16 - (left & 15), i = rows >= 8 ? 0 : rows >= 4 ? 1 : rows >= 2 ? 2 : 3, h = 8 >> i;
                        const uint32_t at = smem_u32(ring) + r.s * stage_bytes + left * 128;
                        const uint32_t bar = CG == 1 ? smem_u32(&sh->clear[r.s]) : cluster_addr(&sh->clear[r.s], 0);
                        if (rank == 0) mbar_arrive_expect_tx(&sh->clear[r.s], CG * (rows > h ? 2 : 1) * h * 512u);
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            const uint32_t to = at + (o >> 1) * b_off + (o & 1) * 8192;
                            gg_load2<CG>(to, &p.zero[i], 0, p.R, bar);
                            if (rows > h) gg_load2<CG>(to + (rows - h) * 128, &p.zero[i], 0, p.R, bar);
                        }
                    }
                    __syncwarp();
                }
                r.next(S);
            }
            return true;
        });
        __syncwarp();
    } else {
        int buf = 0;
        uint32_t full_ph = 0;
        const int c0 = (warp >> 2) * Role::COLS;
        GgInRing<In::kSlots> in;
        walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
            const int nk = (len + 63) / 64;
            const int m = m0 + (int)rank * 128 + (warp & 3) * 32 + lane;
            const int mine = min(Role::COLS, n - c0);  // columns of this warp; none below 1
            const size_t row0 = (MODE == kGgDw ? (size_t)e * p.NW + n0 : (size_t)q0) + c0;
            if (MODE == kGgDw && nk == 0) {  // no rows: zeros
                uint32_t z[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) z[j] = 0;
                for (int c = 0; c < mine; c += 32) gg_store32(z, p.out, F32, row0 + c, min(32, mine - c), m, p.M);
                return true;
            }
            if constexpr (Role::kIn) {
                const uint32_t taddr = tmem + (uint32_t)(buf * Role::BN + c0) + ((uint32_t)((warp & 3) * 32) << 16);
                const int h = warp >> 2;
                if (!gg_wait_warp(&sh->acc_full[buf], full_ph, &sh->abort)) return false;
                tc_fence_after();
                static_assert(In::kRows == 16, "one load of tensor memory a slot");
                for (int c = 0; c < mine; c += In::kRows) {
                    float d[In::kRows];
                    tmem_ld16(taddr + c, d);
                    if (p.planes && !gg_wait_warp(&sh->in_full[h][in.s], in.ph, &sh->abort)) return false;
                    const uint16_t* at =
                        reinterpret_cast<const uint16_t*>(ins + (h * In::kSlots + in.s) * In::kSlot) + (warp & 3) * 32;
                    const int r = n0 + c0 + c, rows = min(In::kRows, mine - c);
                    if constexpr (EP == kGgGluBack) glu_back_rows<In::kRows>(p, d, at, row0 + c, rows, m, lane);
                    if constexpr (EP == kGgSym) ns_sym_rows<In::kRows, NARROW == 2>(p, d, at, e, r, m, lane, kMirror && n0 > m0);
                    if constexpr (EP == kGgAxpy) ns_axpy_rows<In::kRows>(p, d, at, e, r, rows, m, lane);
                    if constexpr (EP == kGgResult) ns_result_rows<In::kRows>(p, d, at, e, r, rows, m, lane);
                    if (p.planes) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh->in_empty[h][in.s]);
                        in.next();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 1)
                        mbar_arrive(&sh->acc_empty[buf]);
                    else
                        mbar_arrive_cluster(&sh->acc_empty[buf], 0);
                }
                buf ^= 1;
                if (buf == 0) full_ph ^= 1u;
                return true;
            } else {
                uint32_t sum[Role::COLS / 32][32];  // the parts' sum
                for (int k = 0; k < nk; k += Role::kPart) {
                    if (!gg_wait_warp(&sh->acc_full[buf], full_ph, &sh->abort)) return false;
                    tc_fence_after();
                    const uint32_t taddr = tmem + (uint32_t)(buf * Role::BN + c0) + ((uint32_t)((warp & 3) * 32) << 16);
                    if (mine > 0) gg_gather<Role::COLS>(taddr, sum, mine, k == 0);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 1)
                            mbar_arrive(&sh->acc_empty[buf]);
                        else
                            mbar_arrive_cluster(&sh->acc_empty[buf], 0);
                    }
                    buf ^= 1;
                    if (buf == 0) full_ph ^= 1u;
                }
                if constexpr (EP == kGgGlu) {
                    glu_store<Role::COLS, F32>(p, sum, row0, mine, m0 + (int)rank * MW + (warp & 3) * 16, lane);
                } else {
#pragma unroll
                    for (int i = 0; i < Role::COLS / 32; ++i)
                        if (32 * i < mine) gg_store32(sum[i], p.out, F32, row0 + 32 * i, min(32, mine - 32 * i), m, p.M);
                }
                return true;
            }
        });
    }
    __syncthreads();
    if (*(volatile int*)&sh->abort && threadIdx.x == 0) set_status(p.status, MOE_DEV_TIMEOUT);
    if (CG == 2) cluster_sync();
    if (warp == Role::EPI + 1) {
        tc_fence_after();
        gg_tmem_dealloc<CG>(tmem, kGgTmemCols);
    }
}

// dw of a split launch: the parts' sums in a fixed order.  A block takes 32
// pieces of four values; its eight warps sum every eighth part, and the first
// adds their sums.
static __global__ void __launch_bounds__(256) gg_join_kernel(const float4* parts, size_t n4, int split, void* out,
                                                      int out_f32) {
    __shared__ float4 s_sum[8][32];
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto add = [](float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); };
    for (size_t i0 = (size_t)blockIdx.x * 32; i0 < n4; i0 += (size_t)gridDim.x * 32) {
        const size_t i = i0 + lane;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < n4) {
#pragma unroll 4
            for (int k = warp; k < split; k += 8) a = add(a, __ldcg(parts + (size_t)k * n4 + i));
        }
        s_sum[warp][lane] = a;
        __syncthreads();
        if (warp == 0 && i < n4) {
#pragma unroll
            for (int w = 1; w < 8; ++w) a = add(a, s_sum[w][lane]);
            if (out_f32)
                static_cast<float4*>(out)[i] = a;
            else
                static_cast<uint2*>(out)[i] = make_uint2(gg_pack(__float_as_uint(a.x), __float_as_uint(a.y)),
                                                         gg_pack(__float_as_uint(a.z), __float_as_uint(a.w)));
        }
        __syncthreads();
    }
}

// ------------------------------------------------------- a few rows at once
// Forward product for a handful of rows: a warp per weight row (256 J elements
// of it in flight at a time), up to kGgvTok rows of one segment at a time.
// Two rows of 1536 x 2048, weights from HBM: 4.3 us, the tiles above 9.8.  Block (i, r) takes 8 weight rows
// for the rows r .. of a segment when r starts a group of kGgvTok there.
constexpr int kGgvTok = 4;

// The segment of row r, found by the whole block (a thread per segment:
// E <= blockDim.x), and its rows p0 .. p1 - 1; -1 where no segment holds r.
__device__ __forceinline__ int gg_row_segment(const int32_t* offsets, int E, int R, int r, int& p0, int& p1,
                                              int32_t* status) {
    __shared__ int s_e, s_p0, s_p1;
    bool mine = false, bad = false;
    int a = 0, b = 0;
    if ((int)threadIdx.x < E) {
        a = offsets[threadIdx.x];
        b = offsets[threadIdx.x + 1];
        bad = a < 0 || b < a || b > R;
        mine = !bad && a <= r && r < b;
    }
    if (threadIdx.x == 0) s_e = -1;
    __syncthreads();
    if (bad && blockIdx.x == 0 && r == 0) set_status(status, MOE_DEV_BAD_OFFSETS);
    if (mine) {
        s_e = threadIdx.x;
        s_p0 = a;
        s_p1 = b;
    }
    __syncthreads();
    p0 = s_p0;
    p1 = s_p1;
    return s_e;
}

template <int J>
__global__ void __launch_bounds__(256) gg_gemv_kernel(const uint16_t* x, const uint16_t* w, const int32_t* offsets, int R, int N, int K, int E,
                                                      void* y, int out_f32, int32_t* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    const int r = blockIdx.y;
    int p0, p1;
    const int e = gg_row_segment(offsets, E, R, r, p0, p1, status);
    if (e < 0 || (r - p0) % kGgvTok) return;
    const int nt = min(kGgvTok, p1 - r);
    const int n = blockIdx.x * 8 + warp;
    if (n >= N) return;
    const uint16_t* wr = w + ((size_t)e * N + n) * K;
    const uint16_t* xr = x + (size_t)r * K;
    float acc[kGgvTok] = {};
    const int chunks = K / 8;
    for (int c0 = 0; c0 < chunks; c0 += 32 * J) {
        const int nj = min(J, (chunks - c0 + 31) / 32);
        uint4 wv[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (j >= nj) break;
            const int c = c0 + j * 32 + lane;
            wv[j] = c < chunks ? ld_stream_v4(wr + (size_t)c * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < kGgvTok; ++t) {
            if (t >= nt) break;
            uint4 xv[J];  // the first row's are on their way with the weights
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j >= nj) break;
                const int c = c0 + j * 32 + lane;
                xv[j] = c < chunks ? ld_input_v4(xr + (size_t)t * K + (size_t)c * 8)
                                   : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j >= nj) break;
                const uint32_t ws[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w}, xs[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 wf = bf16x2_to_f2(ws[i]), xf = bf16x2_to_f2(xs[i]);
                    acc[t] = fmaf(wf.x, xf.x, acc[t]);
                    acc[t] = fmaf(wf.y, xf.y, acc[t]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kGgvTok; ++t) {
        if (t >= nt) break;
        const float v = warp_sum(acc[t]);
        if (lane == 0) {
            const size_t at = (size_t)(r + t) * N + n;
            if (out_f32)
                static_cast<float*>(y)[at] = v;
            else
                static_cast<uint16_t*>(y)[at] = f2bf_bits(v);
        }
    }
}

}  // namespace moe
