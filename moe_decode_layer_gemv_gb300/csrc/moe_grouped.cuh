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

struct GgShared {
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
__device__ __forceinline__ void gg_segments(GgShared* sh, const int32_t* offsets, int E, int R, int bn,
                                            int32_t* status) {
    const int tid = threadIdx.x;
    if (tid == 0) sh->nmax = 0;
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) {
        const int a = offsets[e], b = offsets[e + 1];
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

// ------------------------------------------------------------- the kernel
// Persistent: one CTA per SM (or one pair of CTAs per SM pair) walks the
// tiles.  Three roles run through the same tile sequence, each at its own
// pace: the producer fills the ring, the MMA issuer accumulates tile d into
// tensor-memory buffer d mod 2, the epilogue warps read the other buffer out.
template <int MODE, int CG, bool F32>
__global__ void __launch_bounds__((GgCfg<MODE, CG, F32>::kThreads), 1) gg_kernel(const __grid_constant__ GgParams p) {
    using Cfg = GgCfg<MODE, CG, F32>;
    extern __shared__ __align__(1024) unsigned char gg_smem_raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(gg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    GgShared* sh = reinterpret_cast<GgShared*>(base);
    unsigned char* ring = base + 4096;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const int unit = (int)blockIdx.x / CG, units = (int)gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kGgMaxStages; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->tfull[s], 1);
            mbar_init(&sh->clear[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], Cfg::EPI * CG);
        }
        mbar_init(&sh->mma_done, 1);
        sh->abort = 0;
        fence_mbar_init();
        prefetch_map(&p.ta);
        prefetch_map(&p.tb);
        if (MODE != kGgDw) prefetch_map(&p.tb_all);
    }
    if (warp == Cfg::EPI + 1) gg_tmem_alloc<CG>(&sh->tmem_slot, kGgTmemCols);
    grid_dep_wait();
    const int mtiles = (p.M + Cfg::BM - 1) / Cfg::BM;
    gg_segments(sh, p.offsets, p.E, p.R, Cfg::BN, p.status);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_slot;

    // Ring geometry.  A stage holds KSUB A tiles and KSUB B tiles; where the
    // B operand is the segment's rows, its tiles are as high as the largest
    // segment needs, so that few rows leave more bytes of weights in flight.
    uint32_t b_tile = kGgTile;
    if (MODE != kGgDw && CG == 1)
        b_tile = (uint32_t)min(Cfg::BN, max(kGgBoxN, (sh->nmax + kGgBoxN - 1) / kGgBoxN * kGgBoxN)) * 128u;
    const uint32_t stage_bytes = Cfg::KSUB * (kGgTile + b_tile);
    const uint32_t b_off = Cfg::KSUB * kGgTile;
    const uint32_t S = min((uint32_t)kGgMaxStages, ((uint32_t)kGgSmem - 1023u - 4096u) / stage_bytes);

    const int ntiles_w = (p.NW + Cfg::BN - 1) / Cfg::BN;  // dw
    const int outers = MODE == kGgDw ? p.split * p.E : sh->start[p.E];

    // f(e, q0, n, n0, m0, len): segment e; first row q0 (forward, dx: of the
    // tile; dw: of the segment's part); n valid columns from n0 on; m from m0
    // on; contraction length.  (dw: e counts part after part, part * E + e)
    auto walk = [&](auto f) {
        int e = 0;
        for (GgWalk w(unit, units, MODE == kGgDw ? mtiles * ntiles_w : mtiles); w.outer < outers; w.next()) {
            int q0, n, n0, m0, len;
            if (MODE == kGgDw) {
                e = w.outer;
                const int tn = w.inner / mtiles;
                m0 = (w.inner - tn * mtiles) * Cfg::BM;
                n0 = tn * Cfg::BN;
                n = min(Cfg::BN, p.NW - n0);
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
                m0 = w.inner * Cfg::BM;
                n0 = (w.outer - sh->start[e]) * Cfg::BN;
                n = min(Cfg::BN, sh->cnt[e] - n0);
                q0 = sh->p0[e] + n0;
                len = p.C;
            }
            if (!f(e, q0, n, n0, m0, len)) break;
        }
    };
    if (warp == Cfg::EPI) {
        // ---------------- TMA producer
        GgRing r;
        const uint32_t ring_at = smem_u32(ring);
        const uint32_t bars = CG == 1 ? smem_u32(sh->full) : cluster_addr(sh->full, 0);
        if (gg_elect()) {
            walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
                const int nk = (len + 63) / 64;
                // rows of B that this CTA holds (forward, dx), in whole boxes
                const int rows = MODE == kGgDw ? 128 : (n + kGgBoxN * CG - 1) / (kGgBoxN * CG) * kGgBoxN;
                const uint32_t bytes = CG * (kGgTile + (uint32_t)rows * 128u);
                const int am = m0 + (int)rank * 128, bn = (MODE == kGgDw ? n0 : q0) + (int)rank * rows;
                for (int k0 = 0; k0 < nk; k0 += Cfg::KSUB) {
                    if (!gg_wait(&sh->empty[r.s], r.ph ^ 1u, &sh->abort)) return false;
                    const uint32_t st = ring_at + r.s * stage_bytes, bar = bars + r.s * 8u;
                    const int ke = min(Cfg::KSUB, nk - k0);
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
                    for (int u = 0; u < Cfg::KSUB; ++u) {
                        if (u >= ke) break;
                        const uint32_t sa = st + u * kGgTile, sb = st + b_off + u * b_tile;
                        const int c = (k0 + u) * 64;
                        if (MODE == kGgFwd) {
                            gg_load3<CG>(sa, &p.ta, c, am, e, bar);
                        } else if (MODE == kGgDx) {
                            if (p.a_blocked) {
                                gg_load4<CG>(sa, &p.ta, 0, c, am >> 6, e, bar);
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
                            for (int i = 0; i < rows; i += kGgBoxN) gg_load2<CG>(sb + i * 128, &p.tb, c, bn + i, bar);
                        }
                    }
                    r.next(S);
                }
                return true;
            });
            gg_drain<CG>(sh, S, r, rank);
        }
        __syncwarp();
    } else if (warp == Cfg::EPI + 1) {
        // ---------------- MMA issuer (one thread of the leader)
        GgRing r;
        int buf = 0;
        uint32_t free_ph = 1;  // parity of acc_empty to wait for (at first: nothing)
        uint32_t tails = 0;    // parity of each stage's next use as a segment's end
        const uint32_t ring_at = smem_u32(ring);
        if (rank == 0 && gg_elect()) walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
            const int nk = (len + 63) / 64;
            const int npad = MODE == kGgDw ? Cfg::BN : (n + kGgBoxN * CG - 1) / (kGgBoxN * CG) * (kGgBoxN * CG);
            const uint32_t idesc = umma_idesc_bf16(Cfg::BM, npad) | (MODE != kGgFwd ? 1u << 15 : 0u) |
                                   (MODE == kGgDw ? 1u << 16 : 0u);
            uint32_t acc = 0, tacc = 0;
            int room = 0;  // steps that the accumulator still takes
            for (int k0 = 0; k0 < nk; k0 += Cfg::KSUB) {
                if (room == 0) {
                    if (!gg_wait(&sh->acc_empty[buf], free_ph, &sh->abort)) return false;
                    tacc = tmem + (uint32_t)(buf * Cfg::BN);
                    acc = 0;
                    room = kGgPartSteps;
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
                room -= Cfg::KSUB;  // (a whole number of stages)
                const bool last = room == 0 || k0 + Cfg::KSUB >= nk;
                tc_fence_after();
                const int ke = min(Cfg::KSUB, nk - k0);
#pragma unroll
                for (int u = 0; u < Cfg::KSUB; ++u) {
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
    } else if (warp == Cfg::EPI + 2) {
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
        const int c0 = (warp >> 2) * Cfg::COLS;
        walk([&](int e, int q0, int n, int n0, int m0, int len) -> bool {
            const int nk = (len + 63) / 64;
            const int m = m0 + (int)rank * 128 + (warp & 3) * 32 + lane;
            const int mine = min(Cfg::COLS, n - c0);  // columns of this warp; none below 1
            const size_t row0 = (MODE == kGgDw ? (size_t)e * p.NW + n0 : (size_t)q0) + c0;
            if (MODE == kGgDw && nk == 0) {  // no rows: zeros
                uint32_t z[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) z[j] = 0;
                for (int c = 0; c < mine; c += 32) gg_store32(z, p.out, F32, row0 + c, min(32, mine - c), m, p.M);
                return true;
            }
            uint32_t sum[Cfg::COLS / 32][32];  // the parts' sum
            for (int k = 0; k < nk; k += kGgPartSteps) {
                if (!gg_wait_warp(&sh->acc_full[buf], full_ph, &sh->abort)) return false;
                tc_fence_after();
                const uint32_t taddr = tmem + (uint32_t)(buf * Cfg::BN + c0) + ((uint32_t)((warp & 3) * 32) << 16);
                if (mine > 0) gg_gather<Cfg::COLS>(taddr, sum, mine, k == 0);
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
#pragma unroll
            for (int i = 0; i < Cfg::COLS / 32; ++i)
                if (32 * i < mine) gg_store32(sum[i], p.out, F32, row0 + 32 * i, min(32, mine - 32 * i), m, p.M);
            return true;
        });
    }
    __syncthreads();
    if (*(volatile int*)&sh->abort && threadIdx.x == 0) set_status(p.status, MOE_DEV_TIMEOUT);
    if (CG == 2) cluster_sync();
    if (warp == Cfg::EPI + 1) {
        tc_fence_after();
        gg_tmem_dealloc<CG>(tmem, kGgTmemCols);
    }
}

// dw of a split launch: the parts' sums in a fixed order.  A block takes 32
// pieces of four values; its eight warps sum every eighth part, and the first
// adds their sums.
__global__ void __launch_bounds__(256) gg_join_kernel(const float4* parts, size_t n4, int split, void* out,
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
