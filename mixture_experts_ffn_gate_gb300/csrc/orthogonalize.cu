// orthogonalize.cu -- Newton-Schulz orthogonalisation of a batch of updates
// on the tensor cores.
//
// With X [m, n], m <= n (a tall matrix is transposed on its way in and out),
// X = G / (||G||_F + eps), a step is
//   gram     A  = X X^T                    [m, m]
//   poly     Bm = b A + c A A              [m, m]
//   apply    X  = a X + Bm X               [m, n]
// A and Bm are symmetric: only the tiles on and above the diagonal are
// computed and stored, and what lies below it is read from its mirror image
// (as an MN-major operand instead of a K-major one), which takes a step from
// 4 m^2 n + 2 m^3 operations to 3 m^2 n + m^3 (and the diagonal tiles' other
// halves).
//
// Numbers.  BF16 operands lose too much here (a polynomial whose slope at
// zero is 3.4 raises the rounding noise of the small singular values with
// them: 1e-2 after five steps, up to 0.2 for a matrix of low rank plus
// noise).  FP16 has three more bits at the same rate, and its range is
// enough because every singular value is at most about 1.2: the stored X is
// 2^10 X, A 2^14 A, Bm 2^11 Bm.  X between steps is a pair of FP16 values,
// hi and lo = 2^12 (X - hi), so that a X, the part that carries the singular
// directions from step to step, has about 22 bits; the products read hi.  In
// 64-bit simulations of these roundings the result, before its rounding to
// BF16, is within 2e-4 (rank one, as an expert's gradient from one token) to
// 2e-3 (Gaussian matrices of side 64) of the exact one; measured with that
// rounding, 2.9e-3 at most from side 64 on, 3.8e-3 from 16, 5.9e-3 from 8 and
// 1.6e-2 below, where a rounding has few others to average with.  A single FP16 X is 2e-2
// off for a matrix of low rank, and a lo part of 8 bits (E4M3) 3.5e-3 to
// 2e-2 for one of rank one.
//
// The products.  A pair of CTAs (a cluster of two) computes a 256 x BN tile,
// BN = 256 or, where the pairs outnumber a product's tiles of 128, 128,
// with tcgen05.mma.cta_group::2: each CTA loads its 128 rows of the left and
// its BN / 2 rows of the right operand, so a byte of shared memory feeds
// twice the work of a single CTA's tile.  Warp 0 of each CTA loads a ring of
// 64-deep K stages by TMA (both CTAs' copies complete on the first CTA's
// barrier), warp 1 of the first CTA issues the MMAs for both into one of two
// TMEM accumulators, warps 2-9 of each CTA drain the other one.  The right
// operand of `apply`, X read down its columns, is taken as MN-major tiles.
// The epilogue moves its operands and results through shared memory by TMA
// (32 x 64 blocks).
//
// One launch.  All steps are one cooperative launch of one pair per two SMs:
// the tiles of all products form a list (step by step, gram, poly, apply,
// matrix by matrix), pair p takes tiles p, p + pairs, ...  A matrix's tiles
// of one product need all of its tiles of the one before: each CTA adds one
// to the matrix's counter when its half of a tile has been written (the last
// of its epilogue warps does, so that a tile costs one fence to the GPU's
// scope; one per warp cost more than the products), and the loads of a later
// tile wait for the count.  A waiting tile
// only needs tiles that come before it in the list, and every pair is
// resident, so the list moves on; with several matrices the tail of one
// product is filled by the next one's first tiles, where a launch per
// product left pairs idle (16 matrices of 1536 x 2048: 4.4 and 10.1 waves
// rounded up to 5 and 11).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace moe {

__device__ uint32_t g_ortho_fault_word = 0;

cudaError_t read_ortho_fault_word(uint32_t *flags, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_ortho_fault_word, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_ortho_fault_word, &zero, sizeof(uint32_t));
}

namespace {

// the powers of two that X, A, Bm and X's lo part (beside X's own) are stored with
constexpr int kXBits = 10, kABits = 14, kBBits = 11;
constexpr float kLoScale = 4096.0f, kLoInv = 1.0f / 4096.0f;

constexpr int BK = 64;                    // K per stage: 128 bytes of FP16, the swizzle's width
constexpr int A_BYTES = 128 * BK * 2;     // one CTA's left operand of a stage
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int BLOCK = 32 * 64 * 2;        // one staged 32 x 64 FP16 block
// The producer says of a tile that its operands are complete on one of kSlots
// barriers.  It can be ahead of the epilogue by the tiles in the ring (one per
// stage where K is a single step) and the two accumulators; a barrier must not
// come round again before the epilogue has waited for it.
constexpr int kSlots = 16;
constexpr uint64_t kWaitNs = 2000000000ull;

enum : int { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };  // kLast: the last step's apply, into the output

// BN of the symmetric products and of apply.
template <int BS, int BX>
struct Cfg {
    static constexpr int BN = BS > BX ? BS : BX;
    static constexpr int B_BYTES = BN / 2 * BK * 2;  // one CTA's right operand of a stage, at most
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 5 : 6;
    static constexpr int STAGING = kEpiWarps * 2 * BLOCK;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + STAGING + 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(STAGES + 2 < kSlots, "a ready barrier would come round too soon");
};

// The tensor maps over X (two hi buffers, used in turn, and lo), A and Bm:
// left operands (K-major, box 64 x 128 rows), right ones (K-major, box 64 x
// BS / 2 rows), MN-major ones (box 64 x 64 rows) and the epilogue's blocks
// (64 x 32 rows).
struct OrthoMaps {
    CUtensorMap x_left[2], x_right[2], x_cols[2], x_blk[2], lo_blk, a_left, a_right, a_cols, a_blk, b_left, b_cols,
        b_blk;
};

struct OrthoArgs {
    int m, n, batch, steps;  // X is [batch][m][n]
    int row_tiles, sym_cols, x_cols;  // tiles of 256 rows, of BS columns of A and BX of X
    int sym_tiles, x_tiles;  // per matrix: of a symmetric product (on and above the diagonal), of apply
    // the factors of the epilogues, powers of two folded in: gram A = g acc;
    // poly Bm = pb A + pc acc; apply X = xa X + xc acc; last: times out_scale
    float g, pb, pc, xa, xc, out_scale;
    __nv_bfloat16 *out;
    int out_cols;            // the caller's N
    int transposed;          // out is [n][m]
    uint32_t *done;          // [batch] the counters, zero before the launch
};

// A tile of the list.
struct Tile {
    int b, step, kind, r0, c0;  // matrix, step, product, first row and column
    uint32_t need;              // the matrix's count that it waits for
};

// ------------------------------------------------------------ cluster and pair forms
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

// The cluster address of this shared-memory address in CTA `rank`.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// An arrival on a barrier of either CTA that passes on TMEM alone (ordered by
// the tcgen05 fences): a release at the cluster's scope would wait for all of
// the thread's stores, 1.2 us per tile.
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Whether the phase is complete, without a wait (try_wait may suspend the
// thread for a microsecond or more before it says no).
__device__ __forceinline__ bool test_wait(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(ptx::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// ptx::mbar_wait_bounded, the first try with the suspend-time hint too: the
// waits here are short, and reading the clock after a failed try cost 5% of
// the large batches' time.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const volatile int *abort)
{
    if (ptx::mbar_try_wait_sleep(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (;;) {
        if (ptx::mbar_try_wait_sleep(bar, parity)) return true;
        if (*abort) return false;
        if (ptx::globaltimer_ns() - t0 > kWaitNs) return false;
    }
}

// A TMA load into this CTA's shared memory that completes on a barrier of
// either CTA of the pair.
__device__ __forceinline__ void pair_load_3d(void *dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                                             uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(add)
        : "memory");
}

// Arrives once on the barrier at this address of both CTAs when the MMAs
// issued before it have completed.
__device__ __forceinline__ void pair_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void pair_tmem_alloc(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(dst)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Instruction descriptor, kind::f16: D = F32, A = B = F16, shape 256 x N, A
// and B MN-major or not.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t N, bool a_mn, bool b_mn)
{
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((256u >> 4) << 24);
}

__device__ __forceinline__ void raise(uint32_t bit) { atomicOr(&g_ortho_fault_word, bit); }

__device__ __forceinline__ uint32_t half_pair(float lo, float hi)
{
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ float2 half_unpair(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Waits (bounded) until a matrix's count has reached `need`; what was counted
// may then be read by TMA.
__device__ __forceinline__ bool wait_count(const uint32_t *done, uint32_t need, const volatile int *abort)
{
    if (need == 0) return true;
    if (ld_acquire(done) < need) {
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ld_acquire(done) < need) {
            const uint64_t t = ptx::globaltimer_ns() - t0;
            if (*abort || t > kWaitNs) return false;
            if (t > 5000) __nanosleep(200);
        }
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    return true;
}

template <int BS, int BX>
__device__ __forceinline__ Tile decode_tile(int i, const OrthoArgs &a)
{
    const int per_step = 2 * a.sym_tiles + a.x_tiles;  // of one matrix
    Tile t;
    t.step = i / (per_step * a.batch);
    i -= t.step * per_step * a.batch;
    const int sym = a.sym_tiles * a.batch;
    t.kind = i < sym ? kGram : i < 2 * sym ? kPoly : t.step + 1 < a.steps ? kApply : kLast;
    i -= t.kind == kGram ? 0 : t.kind == kPoly ? sym : 2 * sym;
    const int tiles = t.kind <= kPoly ? a.sym_tiles : a.x_tiles;
    t.b = i / tiles;
    i -= t.b * tiles;
    t.need = 2u * (uint32_t)(t.step * per_step + (t.kind == kGram   ? 0
                                                             : t.kind == kPoly ? a.sym_tiles
                                                                               : 2 * a.sym_tiles));
    if (t.kind <= kPoly) {
        // row tile rt has the column tiles from the one that holds its first
        // row's diagonal on
        int rt = 0;
        for (;; ++rt) {
            const int from = rt * 256 / BS, here = a.sym_cols - from;
            if (i < here) {
                i += from;
                break;
            }
            i -= here;
        }
        t.r0 = rt * 256;
        t.c0 = i * BS;
    } else {
        // down the rows first: neighbouring pairs share the right operand
        const int ct = i / a.row_tiles;
        t.r0 = (i - ct * a.row_tiles) * 256;
        t.c0 = ct * BX;
    }
    return t;
}

// Which K steps of a tile's operands are read as MN-major tiles: those before
// left_mn, right_mn.  A and Bm hold their 256 x 256 tiles on and above the
// diagonal, so columns before the row tile's diagonal come from the mirror
// image; X's columns are MN-major all the way.
struct Sides {
    int left_mn, right_mn;
};

__device__ __forceinline__ Sides sides_of(const Tile &t)
{
    return {t.kind == kGram ? 0 : t.r0 / BK, t.kind == kGram ? 0 : t.kind == kPoly ? (t.c0 & ~255) / BK : 1 << 30};
}

// What an epilogue warp carries along.
struct Epilogue {
    uint8_t *st, *st_lo;   // its staging blocks
    uint64_t *bar;         // of the blocks' loads
    uint32_t load_phase;
    int q, half, lane;
    uint32_t rank;
    uint32_t *stored;      // [kSlots] in shared memory: warps whose part of a tile is written
    uint32_t *pending;     // lane 0: the counter of a tile that it has not reported yet,
    int pending_slot;      // and its slot

    // Reports this warp's part of its last tile once its stores are
    // complete; the last of the CTA's warps counts the CTA's half.  Lane 0.
    __device__ __forceinline__ void flush()
    {
        if (!pending) return;
        ptx::bulk_wait_all();
        __threadfence_block();
        if (atomicAdd(stored + pending_slot, 1u) == kEpiWarps - 1) {
            stored[pending_slot] = 0;
            ptx::fence_acq_rel_gpu();
            asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(pending), "r"(1u) : "memory");
        }
        pending = nullptr;
    }
};

// One tile's epilogue for one warp: lane quarter q (rows r0 + 128 rank + 32 q
// ..), columns half * BN / 2 ... in blocks of 64.  Lane l holds row l of a
// block; its 16-byte piece j is at (j ^ (l % 8)) * 16 of the row's 128 bytes
// in the staging buffer (the tensor maps' swizzle).  The warp reports its previous
// tile while this tile's first loads are on their way; before any wait that
// may need that tile it reports first.  Returns false when a wait gave up.
template <int KIND, int BN>
__device__ __forceinline__ bool epilogue(const Tile &t, const OrthoMaps &maps, const OrthoArgs &args, Epilogue &ep,
                                         uint64_t *ready, uint32_t ready_phase, uint64_t *tfull, uint32_t tfull_phase,
                                         uint32_t acc_tmem, volatile int *abort_flag)
{
    constexpr bool SYM = KIND == kGram || KIND == kPoly;
    constexpr bool PAIR_IN = KIND == kApply || KIND == kLast;
    const int lane = ep.lane, x = t.step & 1;
    const int rows = args.m, cols = SYM ? args.m : args.n;
    const int row0 = t.r0 + 128 * (int)ep.rank + 32 * ep.q, row = row0 + lane;
    uint8_t *const st = ep.st, *const st_lo = ep.st_lo;
    bool failed = false;
#pragma unroll 1
    for (int blk = 0; blk < BN / 128; ++blk) {
        const int cb = ep.half * (BN / 2) + 64 * blk, col0 = t.c0 + cb;
        const bool in = row0 < rows && col0 < cols;
        if (lane == 0) {
            // the block's own operands, while the products run
            if (KIND != kGram) {
                if (blk == 0 && !test_wait(ready, ready_phase)) {
                    ep.flush();
                    failed = !wait_bar(ready, ready_phase, abort_flag);
                }
                if (in && !failed) {
                    ptx::bulk_wait_group_read<0>();  // the buffers' last stores have read them
                    ptx::mbar_arrive_expect_tx(ep.bar, (PAIR_IN ? 2 : 1) * BLOCK);
                    ptx::tma_load_3d(st, PAIR_IN ? &maps.x_blk[x] : &maps.a_blk, col0, row0, t.b, ep.bar);
                    if (PAIR_IN) ptx::tma_load_3d(st_lo, &maps.lo_blk, col0, row0, t.b, ep.bar);
                }
            }
            ep.flush();
        }
        failed = __any_sync(0xffffffffu, failed);
        if (blk == 0) {
            failed = failed || *abort_flag || !wait_bar(tfull, tfull_phase, abort_flag);
            failed = __any_sync(0xffffffffu, failed);
            ptx::tc_fence_after();
        }
        if (in && KIND != kGram) {
            const int keep = 0;
            const bool got = failed || wait_bar(ep.bar, ep.load_phase, &keep);
            ep.load_phase ^= 1;
            failed = __any_sync(0xffffffffu, failed || !got);
        }
        if (failed) return false;
        if (!in) continue;
        if (KIND == kGram) {
            if (lane == 0) ptx::bulk_wait_group_read<0>();
            __syncwarp();
        }
        const uint32_t taddr = acc_tmem + ((uint32_t)(32 * ep.q) << 16) + cb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            ptx::tmem_ld32(taddr + 32 * h, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = lane * 128 + (((4 * h + j) ^ (lane & 7)) << 4);
                uint4 *p = reinterpret_cast<uint4 *>(st + at), *p_lo = reinterpret_cast<uint4 *>(st_lo + at);
                uint32_t in_w[4] = {0, 0, 0, 0}, lo_w[4] = {0, 0, 0, 0}, o[4], o_lo[4];
                float last[8];
                if (KIND != kGram) {
                    const uint4 w = *p;
                    in_w[0] = w.x, in_w[1] = w.y, in_w[2] = w.z, in_w[3] = w.w;
                }
                if (PAIR_IN) {
                    const uint4 w = *p_lo;
                    lo_w[0] = w.x, lo_w[1] = w.y, lo_w[2] = w.z, lo_w[3] = w.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 8 * j + 2 * e;
                    const float a0 = __uint_as_float(r[c]), a1 = __uint_as_float(r[c + 1]);
                    float v0, v1;
                    if (KIND == kGram) {
                        v0 = a0 * args.g, v1 = a1 * args.g;
                    } else if (KIND == kPoly) {
                        const float2 y = half_unpair(in_w[e]);
                        v0 = fmaf(args.pc, a0, args.pb * y.x), v1 = fmaf(args.pc, a1, args.pb * y.y);
                    } else {
                        const float2 y = half_unpair(in_w[e]), z = half_unpair(lo_w[e]);
                        v0 = fmaf(args.xc, a0, args.xa * fmaf(z.x, kLoInv, y.x));
                        v1 = fmaf(args.xc, a1, args.xa * fmaf(z.y, kLoInv, y.y));
                    }
                    if (KIND == kLast) {
                        last[2 * e] = v0 *= args.out_scale, last[2 * e + 1] = v1 *= args.out_scale;
                        const __nv_bfloat162 z = __floats2bfloat162_rn(v0, v1);
                        o[e] = *reinterpret_cast<const uint32_t *>(&z);
                    } else {
                        o[e] = half_pair(v0, v1);
                    }
                    if (KIND == kApply) {
                        const float2 hi = half_unpair(o[e]);
                        o_lo[e] = half_pair((v0 - hi.x) * kLoScale, (v1 - hi.y) * kLoScale);
                    }
                }
                *p = make_uint4(o[0], o[1], o[2], o[3]);
                if (KIND == kApply) *p_lo = make_uint4(o_lo[0], o_lo[1], o_lo[2], o_lo[3]);
                if (KIND == kLast && args.transposed && row < rows) {
                    const int c = col0 + 32 * h + 8 * j;
                    __nv_bfloat16 *dst = args.out + (int64_t)t.b * rows * cols + row;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < cols) dst[(int64_t)(c + e) * args.out_cols] = __float2bfloat16_rn(last[e]);
                }
            }
        }
        if (KIND == kLast) {
            // the caller's rows have any pitch: from the staging buffer, a
            // row's 64 elements at a time, two per lane
            __syncwarp();
            if (!args.transposed) {
                const int c = col0 + 2 * lane;
                __nv_bfloat16 *dst = args.out + (int64_t)t.b * rows * cols + c;
                for (int rr = 0; rr < 32 && row0 + rr < rows; ++rr) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(
                        st + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4);
                    __nv_bfloat16 *d = dst + (int64_t)(row0 + rr) * args.out_cols;
                    const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&w);
                    if (args.out_cols % 2 == 0) {
                        if (c < cols) *reinterpret_cast<__nv_bfloat162 *>(d) = z;
                    } else {
                        if (c < cols) d[0] = z.x;
                        if (c + 1 < cols) d[1] = z.y;
                    }
                }
            }
            // the next block's TMA load overwrites what the warp has read
            ptx::fence_proxy_async_smem();
            __syncwarp();
        } else {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                // rows and columns past the matrix are not written by the stores
                ptx::tma_store_3d(KIND == kGram   ? &maps.a_blk
                                  : KIND == kPoly ? &maps.b_blk
                                                  : &maps.x_blk[x ^ 1],
                                  st, col0, row0, t.b);
                if (KIND == kApply) ptx::tma_store_3d(&maps.lo_blk, st_lo, col0, row0, t.b);
                ptx::bulk_commit_group();
            }
        }
    }
    return true;
}

template <int BS, int BX>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ortho_kernel(const __grid_constant__ OrthoMaps maps, const __grid_constant__ OrthoArgs args)
{
    using C = Cfg<BS, BX>;
    constexpr int BN = C::BN;  // TMEM columns per accumulator
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *staging = smem + C::STAGES * C::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + C::STAGING);
    uint64_t *empty = full + C::STAGES;
    uint64_t *tfull = empty + C::STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint64_t *loaded = drain + 1;           // [kEpiWarps]: an epilogue warp's operand blocks
    uint64_t *ready = loaded + kEpiWarps;   // [kSlots]: the tile's operands are complete
    uint32_t *stored = reinterpret_cast<uint32_t *>(ready + kSlots);  // [kSlots]
    uint32_t *tmem_slot = stored + kSlots;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(full + s, 1);
            ptx::mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(tfull + b, 1);
            ptx::mbar_init(tempty + b, 2 * kEpiWarps);
        }
        ptx::mbar_init(drain, 1);
        for (int w = 0; w < kEpiWarps; ++w) ptx::mbar_init(loaded + w, 1);
        for (int w = 0; w < kSlots; ++w) {
            ptx::mbar_init(ready + w, 1);
            stored[w] = 0;
        }
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    __syncwarp();
    if (warp == 1) pair_tmem_alloc(tmem_slot, 2 * BN);
    ptx::tc_fence_before();
    cluster_sync();  // barriers initialised and TMEM allocated in both CTAs
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int pairs = gridDim.x / 2, first = blockIdx.x / 2;
    const int total = args.batch * args.steps * (2 * args.sym_tiles + args.x_tiles);

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int li = 0;
            for (int i = first; i < total && !*abort_flag; i += pairs, ++li) {
                const Tile t = decode_tile<BS, BX>(i, args);
                const int x = t.step & 1;
                const int ksteps = ((t.kind == kGram ? args.n : args.m) + BK - 1) / BK;
                const int bn = t.kind <= kPoly ? BS : BX;
                const int row = t.r0 + 128 * (int)rank, col = t.c0 + bn / 2 * (int)rank;
                const uint32_t bytes = 2 * (A_BYTES + bn / 2 * BK * 2);  // of both CTAs
                const Sides sides = sides_of(t);
                const CUtensorMap *left = t.kind == kGram   ? &maps.x_left[x]
                                          : t.kind == kPoly ? &maps.a_left
                                                            : &maps.b_left;
                const CUtensorMap *left_mn = t.kind == kPoly ? &maps.a_cols : &maps.b_cols;
                const CUtensorMap *right = t.kind == kGram ? &maps.x_right[x] : &maps.a_right;
                const CUtensorMap *right_mn = t.kind == kPoly ? &maps.a_cols : &maps.x_cols[x];
                if (!wait_count(args.done + t.b, t.need, abort_flag)) {
                    if (!*abort_flag) raise(FAULT_GEMM_PRODUCER);
                    *abort_flag = 1;
                    break;
                }
                ptx::mbar_arrive(ready + li % kSlots);
                for (int ks = 0; ks < ksteps; ++ks) {
                    if (!wait_bar(empty + stage, phase ^ 1, abort_flag)) {
                        if (!*abort_flag) raise(FAULT_GEMM_PRODUCER);
                        *abort_flag = 1;
                        break;
                    }
                    // both CTAs' bytes complete on the first CTA's barrier
                    const uint32_t bar = map_to(ptx::smem_u32(full + stage), 0);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(full + stage, bytes);
                    uint8_t *l = smem + stage * C::STAGE_BYTES;
                    uint8_t *r = l + A_BYTES;
                    if (ks < sides.left_mn) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            pair_load_3d(l + h * (64 * BK * 2), left_mn, row + 64 * h, ks * BK, t.b, bar);
                    } else {
                        pair_load_3d(l, left, ks * BK, row, t.b, bar);
                    }
                    if (ks < sides.right_mn) {
                        for (int h = 0; h < bn / 128; ++h)
                            pair_load_3d(r + h * (64 * BK * 2), right_mn, col + 64 * h, ks * BK, t.b, bar);
                    } else {
                        pair_load_3d(r, right, ks * BK, col, t.b, bar);
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (*abort_flag) {  // copies in flight land within microseconds
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 1000000ull) {
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer, for both CTAs
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int li = 0;
            for (int i = first; i < total && !*abort_flag; i += pairs, ++li) {
                const Tile t = decode_tile<BS, BX>(i, args);
                const int ksteps = ((t.kind == kGram ? args.n : args.m) + BK - 1) / BK;
                const Sides sides = sides_of(t);
                const int acc = li & 1;
                if (!wait_bar(tempty + acc, ((li >> 1) & 1) ^ 1, abort_flag)) {
                    if (!*abort_flag) raise(FAULT_GEMM_MMA);
                    *abort_flag = 1;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d = tmem + acc * BN;
                bool ok = true;
                for (int ks = 0; ks < ksteps; ++ks) {
                    if (!wait_bar(full + stage, phase, abort_flag)) {
                        if (!*abort_flag) raise(FAULT_GEMM_MMA);
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t l = ptx::smem_u32(smem + stage * C::STAGE_BYTES);
                    const uint32_t r = l + A_BYTES;
                    // K-major: a K step of 16 is 32 bytes along the rows; MN-major:
                    // 16 rows of 128 bytes, the next 64 of M or N a box on
                    const bool l_mn = ks < sides.left_mn, r_mn = ks < sides.right_mn;
                    const uint32_t idesc = idesc_f16(t.kind <= kPoly ? BS : BX, l_mn, r_mn);
                    uint64_t ld = l_mn ? ptx::sw128_desc_mn(l, 64 * BK * 2) : ptx::sw128_desc(l);
                    uint64_t rd = r_mn ? ptx::sw128_desc_mn(r, 64 * BK * 2) : ptx::sw128_desc(r);
                    const uint64_t l_step = l_mn ? 2048 >> 4 : 32 >> 4, r_step = r_mn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) pair_mma(d, ld + k * l_step, rd + k * r_step, idesc, (ks | k) != 0);
                    pair_commit(empty + stage);
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                pair_commit(tfull + acc);
            }
            // the drain barrier of both CTAs; this CTA's says that all is done
            pair_commit(drain);
            wait_bar(drain, 0, abort_flag);
        }
    } else {
        // ---------------------------------------------------- epilogue
        Epilogue ep;
        ep.st = staging + (warp - 2) * 2 * BLOCK;
        ep.st_lo = ep.st + BLOCK;
        ep.bar = loaded + (warp - 2);
        ep.load_phase = 0;
        ep.q = warp & 3;
        ep.half = (warp - 2) >> 2;
        ep.lane = lane;
        ep.rank = rank;
        ep.stored = stored;
        ep.pending = nullptr;
        int li = 0;
        for (int i = first; i < total; i += pairs, ++li) {
            const Tile t = decode_tile<BS, BX>(i, args);
            const int acc = li & 1;
            const uint32_t ph = (li >> 1) & 1, at = tmem + acc * BN;
            uint64_t *rd = ready + li % kSlots;
            const uint32_t rph = (li / kSlots) & 1;
            bool ok;
            if (t.kind == kGram)
                ok = epilogue<kGram, BS>(t, maps, args, ep, rd, rph, tfull + acc, ph, at, abort_flag);
            else if (t.kind == kPoly)
                ok = epilogue<kPoly, BS>(t, maps, args, ep, rd, rph, tfull + acc, ph, at, abort_flag);
            else if (t.kind == kApply)
                ok = epilogue<kApply, BX>(t, maps, args, ep, rd, rph, tfull + acc, ph, at, abort_flag);
            else
                ok = epilogue<kLast, BX>(t, maps, args, ep, rd, rph, tfull + acc, ph, at, abort_flag);
            if (!ok) {
                if (lane == 0) {
                    if (!*abort_flag) raise(FAULT_GEMM_EPILOGUE);
                    *abort_flag = 1;
                }
                break;
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                arrive_cluster(map_to(ptx::smem_u32(tempty + acc), 0));
                ep.pending = args.done + t.b;
                ep.pending_slot = li % kSlots;
            }
        }
        if (lane == 0) ep.flush();
        if (lane == 0) ptx::bulk_wait_all();
        __syncwarp();
    }

    __syncwarp();
    ptx::tc_fence_before();
    cluster_sync();  // neither CTA uses TMEM or signals the other any more
    ptx::tc_fence_after();
    if (warp == 1) pair_tmem_dealloc(tmem, 2 * BN);
    cluster_sync();
}

// ---------------------------------------------------------------- the input
constexpr int kMaxParts = 64;
// G is read twice, for its norm and to be scaled, both bound by memory (16
// matrices of 1536 x 2048 in FP32: 34 and 66 us).  Taking the matrices in
// turns that fit L2 costs more in short launches than it saves (128 us).

// 8 consecutive elements, 16-byte aligned (BF16) or 32 (FP32)
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    unpack8(__ldg(reinterpret_cast<const uint4 *>(p)), v);
}

// Squares of FP32 values leave FP32's range, so there are two sums: of the
// values times 2^30, which says the norm from 2^-93 times one element (1e-28)
// up to 2^34, and of the values times 2^-80, for what is larger (an element
// that matters there is at least 2^19: 2^30 elements at most).  The factors
// are powers of two, so the norm has the bits of a plain sum in range.
struct Squares {
    float near, far;
    __device__ __forceinline__ void add(float v)
    {
        const float a = v * 0x1p30f, b = v * 0x1p-80f;
        near = fmaf(a, a, near);
        far = fmaf(b, b, far);
    }
    __device__ __forceinline__ void add(const Squares &o)
    {
        near += o.near;
        far += o.far;
    }
    // 2^kXBits / (norm + eps); NaN where the norm is no finite FP32 number
    __device__ __forceinline__ float factor(float eps) const
    {
        const float norm = near < INFINITY ? sqrtf(near) * 0x1p-30f : sqrtf(far) * 0x1p80f;
        return (float)(1 << kXBits) / (norm + eps) + (norm - norm);
    }
};

__device__ __forceinline__ Squares warp_sum(const Squares &s)
{
    float v[2] = {s.near, s.far};
    warp_sum_n(v);
    return Squares{v[0], v[1]};
}

// partial[b][p]: the sums of squares of a slice of matrix b.
template <typename T>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const T *__restrict__ g, int64_t count,
                                                         Squares *__restrict__ partial, uint32_t *__restrict__ done)
{
    __shared__ Squares sums[8];
    const int b = blockIdx.y;
    const T *p = g + (int64_t)b * count;
    Squares s[8] = {};
    const int64_t stride = (int64_t)gridDim.x * 256, start = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (count % 8 == 0) {
        const int64_t n = count / 8;
        auto add = [&](const float(&v)[8]) {
#pragma unroll
            for (int q = 0; q < 8; ++q) s[q].add(v[q]);
        };
        int64_t i = start;
        for (; i + 3 * stride < n; i += 4 * stride) {  // four loads in flight
            float v[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) load8(p + 8 * (i + u * stride), v[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) add(v[u]);
        }
        for (; i < n; i += stride) {
            float v[8];
            load8(p + 8 * i, v);
            add(v);
        }
    } else {
        for (int64_t i = start; i < count; i += stride) s[0].add((float)p[i]);
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2)
#pragma unroll
        for (int q = 0; q < 8; q += 2 * d) s[q].add(s[q + d]);
    const Squares t = warp_sum(s[0]);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        Squares v{};
#pragma unroll
        for (int q = 0; q < 8; ++q) v.add(sums[q]);
        partial[b * kMaxParts + blockIdx.x] = v;
        if (blockIdx.x == 0) done[b] = 0;  // for the products that follow
    }
}

// 2^kXBits / (||G|| + eps) of a matrix from its partial sums.  Whole warp.
__device__ __forceinline__ float input_factor(const Squares *partial, int parts, float eps)
{
    const int lane = threadIdx.x & 31;
    Squares s{};
    if (lane < parts) s.add(partial[lane]);
    if (lane + 32 < parts) s.add(partial[lane + 32]);
    static_assert(kMaxParts == 64, "two partial sums per lane");
    return warp_sum(s).factor(eps);
}

__device__ __forceinline__ void split8(const float (&v)[8], __half *hi, __half *lo)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        h[q] = half_pair(v[2 * q], v[2 * q + 1]);
        const float2 f = half_unpair(h[q]);
        l[q] = half_pair((v[2 * q] - f.x) * kLoScale, (v[2 * q + 1] - f.y) * kLoScale);
    }
    *reinterpret_cast<uint4 *>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}

// X hi and lo [b][m][pitch] from g [b][M][N]: M and N multiples of 8.  WIDE:
// the rows of X are those of g.  Else a block transposes 64 x 64 elements
// through shared memory.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) ortho_split8_kernel(const T *__restrict__ g, int M, int N,
                                                           const Squares *__restrict__ partial, int parts, float eps,
                                                           __half *__restrict__ hi, __half *__restrict__ lo)
{
    const int b = blockIdx.z;
    const float f = input_factor(partial + b * kMaxParts, parts, eps);
    const int64_t base = (int64_t)b * M * N;
    if constexpr (WIDE) {
        const int64_t n = (int64_t)M * N / 8, stride = (int64_t)gridDim.x * 256;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
            float v[8];
            load8(g + base + 8 * i, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= f;
            split8(v, hi + base + 8 * i, lo + base + 8 * i);
        }
    } else {
        __shared__ float tile[64][65];
        const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;  // in g
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int e = threadIdx.x + 256 * u, y = e >> 3, c = (e & 7) * 8;
            if (r0 + y < M && c0 + c < N) {
                float v[8];
                load8(g + base + (int64_t)(r0 + y) * N + c0 + c, v);
#pragma unroll
                for (int q = 0; q < 8; ++q) tile[y][c + q] = v[q] * f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int e = threadIdx.x + 256 * u, y = e >> 3, c = (e & 7) * 8;  // row c0 + y of X
            if (c0 + y < N && r0 + c < M) {
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = tile[c + q][y];
                const int64_t at = base + (int64_t)(c0 + y) * M + r0 + c;
                split8(v, hi + at, lo + at);
            }
        }
    }
}

// The same for any M and N, in 32 x 32 tiles (X's rows have `pitch` elements).
template <typename T>
__global__ void __launch_bounds__(256) ortho_split_kernel(const T *__restrict__ g, int M, int N,
                                                          const Squares *__restrict__ partial, int parts, float eps,
                                                          bool tall, int64_t pitch, __half *__restrict__ hi,
                                                          __half *__restrict__ lo)
{
    __shared__ float tile[32][33];
    const int b = blockIdx.z, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const float f = input_factor(partial + b * kMaxParts, parts, eps);
    const int m = tall ? N : M;
    const T *src = g + (int64_t)b * M * N;
    const int64_t base = (int64_t)b * m * pitch;
    const int r0 = blockIdx.y * 32, c0 = blockIdx.x * 32;  // in g
    auto put = [&](int r, int c, float v) {
        const __half h = __float2half_rn(v);
        hi[base + r * pitch + c] = h;
        lo[base + r * pitch + c] = __float2half_rn((v - __half2float(h)) * kLoScale);
    };
    for (int y = ty; y < 32; y += 8) {
        const int r = r0 + y, c = c0 + tx;
        float v = 0.0f;
        if (r < M && c < N) v = (float)src[(int64_t)r * N + c] * f;
        if (!tall) {
            if (r < M && c < N) put(r, c, v);
        } else {
            tile[y][tx] = v;
        }
    }
    if (!tall) return;
    __syncthreads();
    for (int y = ty; y < 32; y += 8) {
        const int r = c0 + y, c = r0 + tx;  // in X
        if (r < N && c < M) put(r, c, tile[tx][y]);
    }
}

// ---------------------------------------------------------------- small matrices
// m, n <= 256: one pair of CTAs keeps a matrix in shared memory through all
// its steps, one launch, no workspace.  CTA r holds rows 128 r .. of X
// (K-major, the left and, as its half of N, the right operand of gram) and of
// A, then Bm in its place (left and right operand of poly, left of apply; A is
// symmetric), and columns 128 r .. of X (MN-major, the right operand of
// apply), of which the other CTA writes its rows' share through the cluster.
// lo stays in registers: thread (row, a quarter of its columns) in the epilogue of
// every product.  Rows and columns past the matrix are zeros.  The general
// kernel's tiles go through L2 between products, 4.4 us each; here a product
// takes 3.4 us (1.3 us of MMAs, 0.9 to 2.2 us of epilogue, the rest signals).
// Measured, us there and here: 8 x 256 x 256 86, 65; 76 x 256 x 256 120, 67;
// 300 x 256 x 256 328, 266; 1 x 72 x 71 68, 52; 300 x 128 x 128 212, 191
// (600 x 64 x 64, the one that is slower here, 271, 324).
constexpr int kSmall = 256;
constexpr int kSmallWarps = 16;                 // of the epilogue (eight took 1.3 to 4 us for a product's)
constexpr int kSmallThreads = 32 * (kSmallWarps + 1);  // and the MMA issuer
constexpr int kTile = 128 * BK * 2;             // 128 rows of 64 FP16
constexpr int kRows = 4 * kTile;                // 128 rows of 256
constexpr int kSmallSmem = 1024 + 3 * kRows + 256;
static_assert(kSmallSmem <= 227 * 1024, "shared memory");

struct SmallArgs {
    const void *g;
    int M, N, steps;
    float eps, gram, pb, pc, xa, xc, out_scale;  // as in OrthoArgs
    __nv_bfloat16 *out;
};

__device__ __forceinline__ void st_cluster(uint32_t addr, const uint4 &v)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kSmallThreads, 1) ortho_small_kernel(const SmallArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const xr = smem, *const ar = xr + kRows, *const xc = ar + kRows;
    uint64_t *go = reinterpret_cast<uint64_t *>(xc + kRows);  // operands of the next product written, by 32 warps
    uint64_t *done = go + 1;                                  // a product's MMAs have completed
    Squares *sums = reinterpret_cast<Squares *>(done + 1);    // a warp's sums of squares; then, first, the CTA's
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sums + kSmallWarps + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int b = blockIdx.x / 2;
    const bool tall = args.M > args.N;
    const int m = tall ? args.N : args.M, n = tall ? args.M : args.N;
    const T *g = (const T *)args.g + (int64_t)b * args.M * args.N;
    if (threadIdx.x == 0) {
        ptx::mbar_init(go, 2 * kSmallWarps);
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    __syncwarp();
    if (warp == kSmallWarps) pair_tmem_alloc(tmem_slot, kSmall);
    // the sum of squares, half of the elements per CTA
    {
        const int count = args.M * args.N;
        Squares s{};
        const int first = (int)rank * kSmallThreads + threadIdx.x;
        if (count % 8 == 0) {  // the matrix starts on 16 bytes: all of a thread's loads at once
#pragma unroll
            for (int i = 0; i < kSmall * kSmall / 8; i += 2 * kSmallThreads) {
                if (i + first >= count / 8) continue;
                float v[8];
                load8(g + 8 * (i + first), v);
#pragma unroll
                for (int e = 0; e < 8; ++e) s.add(v[e]);
            }
        } else {
            for (int i = first; i < count; i += 2 * kSmallThreads) s.add((float)g[i]);
        }
        s = warp_sum(s);
        if (lane == 0) sums[warp] = s;
    }
    ptx::tc_fence_before();
    __syncthreads();
    Squares mine{};
    for (int w = 0; w <= kSmallWarps; ++w) mine.add(sums[w]);
    __syncthreads();
    if (threadIdx.x == 0) sums[0] = mine;
    cluster_sync();  // barriers initialised, TMEM allocated, both sums written
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Squares all;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(all.near), "=f"(all.far)
                 : "r"(map_to(ptx::smem_u32(sums), rank ^ 1)));
    all.add(mine);
    const float f = all.factor(args.eps);

    const int products = 3 * args.steps;
    if (warp == kSmallWarps) {
        // ---------------------------------------------------- MMA issuer, for both CTAs
        if (lane == 0 && rank == 0) {
            const uint32_t xr_a = ptx::smem_u32(xr), ar_a = ptx::smem_u32(ar), xc_a = ptx::smem_u32(xc);
            for (int p = 0; p < products; ++p) {
                const int kind = p % 3;
                uint32_t ok = 0;
                const uint64_t t0 = ptx::globaltimer_ns();
                do {  // the other CTA's stores to its shared memory are read by the MMAs
                    asm volatile(
                        "{\n\t.reg .pred q;\n\t"
                        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 q, [%1], %2, %3;\n\t"
                        "selp.u32 %0, 1, 0, q;\n\t}"
                        : "=r"(ok)
                        : "r"(ptx::smem_u32(go)), "r"((uint32_t)(p & 1)), "n"(ptx::kSuspendNs)
                        : "memory");
                } while (!ok && !*abort_flag && ptx::globaltimer_ns() - t0 < kWaitNs);
                if (!ok) {
                    if (!*abort_flag) raise(FAULT_GEMM_MMA);
                    *abort_flag = 1;
                    break;
                }
                ptx::tc_fence_after();
                const int blocks = ((kind == kGram ? n : m) + BK - 1) / BK;
                const uint32_t idesc = idesc_f16(kSmall, false, kind == 2);
                const uint32_t left = kind == kGram ? xr_a : ar_a;
                for (int kb = 0; kb < blocks; ++kb) {
                    const uint64_t ld = ptx::sw128_desc(left + kb * kTile);
                    const uint64_t rd = kind == 2 ? ptx::sw128_desc_mn(xc_a + kb * 64 * 128, kRows / 2)
                                                  : ptx::sw128_desc(left + kb * kTile);
                    const uint64_t r_step = kind == 2 ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) pair_mma(tmem, ld + k * (32 >> 4), rd + k * r_step, idesc, (kb | k) != 0);
                }
                pair_commit(done);
            }
            // (the epilogues wait for every product's MMAs)
        }
    } else {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3, part = warp >> 2;
        const int r = 32 * q + lane, row = 128 * (int)rank + r;  // this thread's row, in the CTA and the matrix
        // this thread's 16-byte piece of columns c .. c + 7 (c a multiple of 8)
        // in 128 rows of 256, and of X's columns for CTA c / 128
        auto piece = [&](uint8_t *rows, int c) {
            return reinterpret_cast<uint4 *>(rows + (c / 64) * kTile + r * 128 + (((c / 8 % 8) ^ (r & 7)) << 4));
        };
        const bool own = (uint32_t)(part >> 1) == rank;  // this thread's columns are this CTA's
        const uint32_t xc_other = map_to(ptx::smem_u32(xc), rank ^ 1);
        auto put_x = [&](int c, const uint4 &v) {
            *piece(xr, c) = v;
            const uint32_t at = (part & 1) * (kRows / 2) + row * 128 + (((c / 8 % 8) ^ (row & 7)) << 4);
            if (own)
                *reinterpret_cast<uint4 *>(xc + at) = v;
            else
                st_cluster(xc_other + at, v);
        };
        auto publish = [&] {
            ptx::tc_fence_before();
            asm volatile("fence.proxy.async;" ::: "memory");  // this thread's stores, the other CTA's memory too
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                 map_to(ptx::smem_u32(go), 0))
                             : "memory");
        };
        uint32_t lo[2][16];  // 64 columns' low parts
        // X = f G: this row's columns 64 part ..
#pragma unroll
        for (int c4 = 0; c4 < 2; ++c4)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 64 * part + 32 * c4 + 8 * j;
                float v[8];
                if (!tall && args.N % 8 == 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
                    if (row < m && c < n) load8(g + (int64_t)row * n + c, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = row < m && c + e < n ? (float)(tall ? g[(int64_t)(c + e) * m + row]
                                                                  : g[(int64_t)row * n + c + e])
                                                    : 0.0f;
                }
                uint32_t hi[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v0 = v[2 * e] * f, v1 = v[2 * e + 1] * f;
                    hi[e] = half_pair(v0, v1);
                    const float2 h = half_unpair(hi[e]);
                    lo[c4][4 * j + e] = half_pair((v0 - h.x) * kLoScale, (v1 - h.y) * kLoScale);
                }
                put_x(c, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                *piece(ar, c) = make_uint4(0, 0, 0, 0);  // what gram leaves out past m
            }
        publish();
        for (int p = 0; p < products; ++p) {
            const int kind = p % 3;
            bool ok = wait_bar(done, p & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0) {
                    if (!*abort_flag) raise(FAULT_GEMM_EPILOGUE);
                    *abort_flag = 1;
                }
                break;
            }
            ptx::tc_fence_after();
            const bool last = p + 1 == products;
#pragma unroll
            for (int c4 = 0; c4 < 2; ++c4) {
                const int c0 = 64 * part + 32 * c4;
                if (c0 >= (kind == 2 ? n : m)) continue;  // zeros, as they were
                uint32_t acc[32];
                ptx::tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + c0, acc);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = c0 + 8 * j;
                    uint32_t o[4];
                    if (kind == kGram) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = half_pair(__uint_as_float(acc[8 * j + 2 * e]) * args.gram,
                                             __uint_as_float(acc[8 * j + 2 * e + 1]) * args.gram);
                        *piece(ar, c) = make_uint4(o[0], o[1], o[2], o[3]);
                    } else if (kind == kPoly) {
                        const uint4 a = *piece(ar, c);
                        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = half_unpair(w[e]);
                            o[e] = half_pair(fmaf(args.pc, __uint_as_float(acc[8 * j + 2 * e]), args.pb * y.x),
                                             fmaf(args.pc, __uint_as_float(acc[8 * j + 2 * e + 1]), args.pb * y.y));
                        }
                        *piece(ar, c) = make_uint4(o[0], o[1], o[2], o[3]);
                    } else {
                        const uint4 a = *piece(xr, c);
                        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = half_unpair(w[e]), z = half_unpair(lo[c4][4 * j + e]);
                            v[2 * e] = fmaf(args.xc, __uint_as_float(acc[8 * j + 2 * e]), args.xa * fmaf(z.x, kLoInv, y.x));
                            v[2 * e + 1] =
                                fmaf(args.xc, __uint_as_float(acc[8 * j + 2 * e + 1]), args.xa * fmaf(z.y, kLoInv, y.y));
                        }
                        if (!last) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[e] = half_pair(v[2 * e], v[2 * e + 1]);
                                const float2 h = half_unpair(o[e]);
                                lo[c4][4 * j + e] = half_pair((v[2 * e] - h.x) * kLoScale, (v[2 * e + 1] - h.y) * kLoScale);
                            }
                            put_x(c, make_uint4(o[0], o[1], o[2], o[3]));
                        } else if (row < m) {
                            __nv_bfloat16 *out = args.out + (int64_t)b * m * n;
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] *= args.out_scale;
                            if (!tall && n % 8 == 0) {
                                if (c < n) {
                                    uint32_t z[4];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                                        z[e] = *reinterpret_cast<const uint32_t *>(&t);
                                    }
                                    *reinterpret_cast<uint4 *>(out + (int64_t)row * n + c) =
                                        make_uint4(z[0], z[1], z[2], z[3]);
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (c + e < n)
                                        out[tall ? (int64_t)(c + e) * m + row : (int64_t)row * n + c + e] =
                                            __float2bfloat16_rn(v[e]);
                            }
                        }
                    }
                }
            }
            if (!last) publish();
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    cluster_sync();  // neither CTA uses TMEM, or the other's memory, any more
    ptx::tc_fence_after();
    if (warp == kSmallWarps) pair_tmem_dealloc(tmem, kSmall);
    cluster_sync();
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// [batch][rows][cols] FP16 with `pitch` elements per row, boxes of 64
// columns (128 bytes, 128-byte swizzle) x box_rows rows
cudaError_t make_map(CUtensorMap *map, const __half *base, int64_t batch, int64_t rows, int64_t cols, int64_t pitch,
                     int box_rows)
{
    EncodeFn enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)(pitch * rows) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Region {
    size_t partial, done, hi[2], lo, a, bm, total;
    int64_t m, n, x_pitch, a_pitch;
};

Region layout(int64_t B, int64_t M, int64_t N)
{
    Region L{};
    L.m = M < N ? M : N;
    L.n = M < N ? N : M;
    L.x_pitch = round_up(L.n, 8);  // rows start on 16 bytes
    L.a_pitch = round_up(L.m, 8);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) & ~size_t(255);
        return at;
    };
    L.partial = take((size_t)B * kMaxParts * sizeof(Squares));
    L.done = take((size_t)B * 4);
    const size_t x = (size_t)(B * L.m * L.x_pitch) * 2, a = (size_t)(B * L.m * L.a_pitch) * 2;
    L.hi[0] = take(x);
    L.hi[1] = take(x);
    L.lo = take(x);
    L.a = take(a);
    L.bm = take(a);
    L.total = o;
    return L;
}

int sym_tiles(int64_t m, int bn)
{
    const int cols = (int)ceil_div(m, bn);
    int n = 0;
    for (int rt = 0; rt < ceil_div(m, 256); ++rt) n += cols - rt * 256 / bn;
    return n;
}

template <int BS, int BX>
cudaError_t run_steps(const OrthoCall &c, char *ws, const Region &L, int pairs, cudaStream_t s)
{
    auto *A = (__half *)(ws + L.a), *Bm = (__half *)(ws + L.bm);
    __half *hi[2] = {(__half *)(ws + L.hi[0]), (__half *)(ws + L.hi[1])};
    OrthoMaps t;
    cudaError_t e = cudaSuccess;
    auto map = [&](CUtensorMap *m, const __half *p, int64_t cols, int64_t pitch, int box_rows) {
        if (e == cudaSuccess) e = make_map(m, p, c.B, L.m, cols, pitch, box_rows);
    };
    for (int i = 0; i < 2; ++i) {
        map(&t.x_left[i], hi[i], L.n, L.x_pitch, 128);
        map(&t.x_right[i], hi[i], L.n, L.x_pitch, BS / 2);
        map(&t.x_cols[i], hi[i], L.n, L.x_pitch, 64);
        map(&t.x_blk[i], hi[i], L.n, L.x_pitch, 32);
    }
    map(&t.lo_blk, (const __half *)(ws + L.lo), L.n, L.x_pitch, 32);
    map(&t.a_left, A, L.m, L.a_pitch, 128);
    map(&t.a_right, A, L.m, L.a_pitch, BS / 2);
    map(&t.a_cols, A, L.m, L.a_pitch, 64);
    map(&t.a_blk, A, L.m, L.a_pitch, 32);
    map(&t.b_left, Bm, L.m, L.a_pitch, 128);
    map(&t.b_cols, Bm, L.m, L.a_pitch, 64);
    map(&t.b_blk, Bm, L.m, L.a_pitch, 32);
    if (e != cudaSuccess) return e;

    auto pow2 = [](int p) { return ldexpf(1.0f, p); };
    OrthoArgs a{};
    a.m = (int)L.m;
    a.n = (int)L.n;
    a.batch = (int)c.B;
    a.steps = c.steps;
    a.row_tiles = (a.m + 255) / 256;
    a.sym_cols = (a.m + BS - 1) / BS;
    a.x_cols = (a.n + BX - 1) / BX;
    a.sym_tiles = sym_tiles(L.m, BS);
    a.x_tiles = a.row_tiles * a.x_cols;
    a.g = pow2(kABits - 2 * kXBits);
    a.pb = c.b * pow2(kBBits - kABits);
    a.pc = c.c * pow2(kBBits - 2 * kABits);
    a.xa = c.a;
    a.xc = pow2(-kBBits);
    a.out_scale = c.out_scale * pow2(-kXBits);
    a.out = (__nv_bfloat16 *)c.out;
    a.out_cols = (int)c.N;
    a.transposed = c.M > c.N;
    a.done = (uint32_t *)(ws + L.done);
    // the most tiles that can run at once: one product's of the whole batch
    const int64_t at_once = (int64_t)a.batch * (a.x_tiles > a.sym_tiles ? a.x_tiles : a.sym_tiles);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (at_once < pairs ? at_once : pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<BS, BX>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // tiles wait for tiles: every pair has to be resident
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ortho_kernel<BS, BX>, t, a);
}

template <typename T>
cudaError_t launch_input(const OrthoCall &c, const Region &L, Squares *partial, uint32_t *done, __half *hi, __half *lo,
                         cudaStream_t s)
{
    const int64_t count = c.M * c.N;
    const int64_t slices = ceil_div(count, 8192);
    const int parts = (int)(slices < kMaxParts ? slices : kMaxParts);
    const bool tall = c.M > c.N, by8 = c.M % 8 == 0 && c.N % 8 == 0;
    const unsigned B = (unsigned)c.B;
    const T *g = (const T *)c.g;
    const int M = (int)c.M, N = (int)c.N;
    ortho_norm_kernel<<<dim3(parts, B), 256, 0, s>>>(g, count, partial, done);
    if (by8 && !tall)
        ortho_split8_kernel<T, true><<<dim3((unsigned)ceil_div(count, 8 * 256 * 4), 1, B), 256, 0, s>>>(
            g, M, N, partial, parts, c.eps, hi, lo);
    else if (by8)
        ortho_split8_kernel<T, false><<<dim3((unsigned)ceil_div(N, 64), (unsigned)ceil_div(M, 64), B), 256, 0, s>>>(
            g, M, N, partial, parts, c.eps, hi, lo);
    else
        ortho_split_kernel<<<dim3((unsigned)ceil_div(N, 32), (unsigned)ceil_div(M, 32), B), 256, 0, s>>>(
            g, M, N, partial, parts, c.eps, tall, L.x_pitch, hi, lo);
    return cudaPeekAtLastError();
}

}  // namespace

size_t ortho_workspace_bytes(int64_t B, int64_t M, int64_t N) { return layout(B, M, N).total; }

cudaError_t ortho_init_device(int *pairs)
{
    cudaError_t e = cudaFuncSetAttribute(ortho_kernel<256, 256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Cfg<256, 256>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ortho_kernel<128, 256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<128, 256>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ortho_kernel<128, 128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<128, 128>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ortho_small_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ortho_small_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmallSmem);
    if (e != cudaSuccess) return e;
    // the pairs of CTAs that the device can hold at once
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<256, 256>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(pairs, ortho_kernel<256, 256>, &cfg);
}

cudaError_t launch_orthogonalize(const OrthoCall &c, void *workspace, int pairs, cudaStream_t s)
{
    if (c.M <= kSmall && c.N <= kSmall) {
        auto pow2 = [](int p) { return ldexpf(1.0f, p); };
        const SmallArgs a{c.g, (int)c.M, (int)c.N, c.steps, c.eps, pow2(kABits - 2 * kXBits),
                          c.b * pow2(kBBits - kABits), c.c * pow2(kBBits - 2 * kABits), c.a, pow2(-kBBits),
                          c.out_scale * pow2(-kXBits), (__nv_bfloat16 *)c.out};
        if (c.g_f32)
            ortho_small_kernel<float><<<2 * (unsigned)c.B, kSmallThreads, kSmallSmem, s>>>(a);
        else
            ortho_small_kernel<__nv_bfloat16><<<2 * (unsigned)c.B, kSmallThreads, kSmallSmem, s>>>(a);
        return cudaPeekAtLastError();
    }
    const Region L = layout(c.B, c.M, c.N);
    char *ws = (char *)workspace;
    auto *partial = (Squares *)(ws + L.partial);
    auto *hi = (__half *)(ws + L.hi[0]);
    auto *lo = (__half *)(ws + L.lo);
    auto *done = (uint32_t *)(ws + L.done);
    const cudaError_t e = c.g_f32 ? launch_input<float>(c, L, partial, done, hi, lo, s)
                                  : launch_input<__nv_bfloat16>(c, L, partial, done, hi, lo, s);
    if (e != cudaSuccess) return e;
    // 256-wide tiles feed the tensor cores best (a byte of shared memory does a
    // third more work); 128-wide ones are twice as many and take their turn
    // where the pairs outnumber them, or nearly so in a batch, whose matrices
    // fill the last wave.  Measured, us for 256 / 256, 128 / 256, 128 / 128
    // (symmetric products / apply): 1 x 1536 x 2048 220, 197, 225 (42 and 96
    // tiles of 128 for 76 pairs); 1 x 1000 x 1000 204, 176, 156 (20, 32);
    // 2 x 1536 x 2048 249, 253, 277 (84, 192); 6 x 768 x 2048 218, 204, 231
    // (72, 288).  A batch's 13 / 12, without and with it, where it decides:
    // 40 x 256 x 300 126, 112 and 20 x 384 x 1000 197, 183 (80 symmetric
    // tiles); 13 x 256 x 768 104, 98 (78 of apply), 10 x 300 x 500 112, 109 (80)
    auto fit = [&](int64_t tiles) { return c.B == 1 ? tiles <= pairs : 12 * c.B * tiles <= 13 * pairs; };
    const bool sym128 = fit(sym_tiles(L.m, 128));
    const bool x128 = fit(ceil_div(L.m, 256) * ceil_div(L.n, 128));
    if (!sym128) return run_steps<256, 256>(c, ws, L, pairs, s);
    return x128 ? run_steps<128, 128>(c, ws, L, pairs, s) : run_steps<128, 256>(c, ws, L, pairs, s);
}

}  // namespace moe
