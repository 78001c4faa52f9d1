// orthogonalize.cu -- Newton-Schulz orthogonalisation of a batch of updates
// on the tensor cores.
//
// With X [m, n], m <= n (a tall matrix is transposed on its way in and out),
// X = G / (||G||_F + eps), a step is
//   gram     A  = X X^T                    [m, m]
//   poly     Bm = b A + c A A              [m, m]
//   apply    X  = a X + Bm X               [m, n]
// Each is one launch over the whole batch.  A and Bm are symmetric: only the
// tiles on and above the diagonal are computed, the others written as their
// mirror images, which takes a step from 4 m^2 n + 2 m^3 operations to
// 3 m^2 n + m^3 (and the diagonal tiles' other halves).
//
// Numbers.  BF16 operands lose too much here (a polynomial whose slope at
// zero is 3.4 raises the rounding noise of the small singular values with
// them: 1e-2 after five steps, up to 0.2 for a matrix of low rank plus
// noise).  FP16 has three more bits at the same rate, and its range is
// enough because every singular value is at most about 1.2: the stored X is
// 2^10 X, A 2^14 A, Bm 2^11 Bm.  X between steps is a pair hi + lo, so that
// a X, the part that carries the singular directions from step to step, is
// exact to about 22 bits; the products read hi.  In 64-bit simulations of
// these roundings the result is within 8e-4 (low rank, power-law spectra) to
// 2.6e-3 (Gaussian) of the exact one, and a single FP16 X within 2e-2.
//
// The products.  A pair of CTAs (a cluster of two) computes a 256 x BN tile
// with tcgen05.mma.cta_group::2: each CTA loads its 128 rows of the left and
// its BN / 2 rows of the right operand, so a byte of shared memory feeds
// twice the work of a single CTA's tile.  Warp 0 of each CTA loads a ring of
// 64-deep K stages by TMA (both CTAs' copies complete on the first CTA's
// barrier), warp 1 of the first CTA issues the MMAs for both into one of two
// TMEM accumulators, warps 2-9 of each CTA drain the other one.  The right
// operand of `apply`, X read down its columns, is taken as MN-major tiles.
// The epilogue moves its operands and results through shared memory by TMA
// (32 x 64 blocks), the mirror images by plain stores (a warp's 32 lanes are
// 32 consecutive elements of a mirrored row).
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

constexpr int kXBits = 10, kABits = 14, kBBits = 11;  // the powers of two that X, A and Bm are stored with

constexpr int BK = 64;                    // K per stage: 128 bytes of FP16, the swizzle's width
constexpr int A_BYTES = 128 * BK * 2;     // one CTA's left operand of a stage
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int BLOCK = 32 * 64 * 2;        // one staged 32 x 64 FP16 block
constexpr uint64_t kWaitNs = 2000000000ull;

enum : int { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };  // kLast: the last step's apply, into the output

template <int BN>
struct Cfg {
    static constexpr int B_BYTES = BN / 2 * BK * 2;  // one CTA's right operand of a stage
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 5 : 6;
    static constexpr int STAGING = kEpiWarps * 2 * BLOCK;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + STAGING + 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct OrthoArgs {
    int m, n, batch;       // X is [batch][m][n]
    int rows, cols, depth; // of the product: rows x cols, K = depth
    int row_tiles, col_tiles, tiles;  // tiles of one matrix (symmetric: on and above the diagonal)
    float ca, cb, cc;      // the step's coefficients, powers of two folded in
    __half *mirror;        // kGram, kPoly: the output, for the mirror images
    int64_t mirror_pitch, mirror_matrix;  // elements per row, per matrix
    __nv_bfloat16 *out;    // kLast
    int out_cols;          // the caller's N
    int transposed;        // kLast: out is [n][m]
    float out_scale;
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

__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(ptx::smem_u32(bar)), "r"(parity), "n"(ptx::kSuspendNs)
        : "memory");
    return ok != 0;
}

// mbar_wait_bounded for a barrier that the other CTA arrives on.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, const volatile int *abort)
{
    if (try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (;;) {
        if (try_wait_cluster(bar, parity)) return true;
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

// Instruction descriptor, kind::f16: D = F32, A = B = F16, shape 256 x N, B
// MN-major or not.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t N, bool b_mn)
{
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((256u >> 4) << 24);
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

// tmL, tmR: the left (K-major, box 64 x 128 rows) and right operand (K-major,
// box 64 x BN / 2 rows; apply: MN-major, box 64 x 64 rows).  tmIn, tmInLo:
// the epilogue's operands (poly: A; apply: X hi and lo), tmOut, tmOutLo: the
// results (gram: A, poly: Bm, apply: X hi and lo), boxes of 64 x 32 rows.
template <int KIND, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ortho_gemm_kernel(const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmR,
                      const __grid_constant__ CUtensorMap tmIn, const __grid_constant__ CUtensorMap tmInLo,
                      const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmOutLo,
                      const OrthoArgs args)
{
    using C = Cfg<BN>;
    constexpr bool SYM = KIND == kGram || KIND == kPoly;
    constexpr bool PAIR_IN = KIND == kApply || KIND == kLast;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *staging = smem + C::STAGES * C::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + C::STAGING);
    uint64_t *empty = full + C::STAGES;
    uint64_t *tfull = empty + C::STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint64_t *loaded = drain + 1;  // [kEpiWarps]: an epilogue warp's operand blocks
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(loaded + kEpiWarps);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    ptx::griddep_launch_dependents();
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
        *abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&tmL);
        ptx::prefetch_tensormap(&tmR);
        if (KIND != kGram) ptx::prefetch_tensormap(&tmIn);
        if (KIND != kLast) ptx::prefetch_tensormap(&tmOut);
    }
    __syncwarp();
    if (warp == 1) pair_tmem_alloc(tmem_slot, 2 * BN);
    ptx::tc_fence_before();
    cluster_sync();  // barriers initialised and TMEM allocated in both CTAs
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();  // the previous launch's results, its plain stores too
    asm volatile("fence.proxy.async;" ::: "memory");

    const int clusters = gridDim.x / 2, first = blockIdx.x / 2;
    const int total = args.tiles * args.batch;
    const int ksteps = (args.depth + BK - 1) / BK;
    // tile i: its matrix, first row and first column
    auto decode = [&](int i, int &b, int &r0, int &c0) {
        b = i / args.tiles;
        int rem = i - b * args.tiles;
        if (SYM) {
            // row tile rt has the column tiles from the one that holds its
            // first row's diagonal on
            int rt = 0;
            for (;; ++rt) {
                const int from = rt * 256 / BN, here = args.col_tiles - from;
                if (rem < here) {
                    rem += from;
                    break;
                }
                rem -= here;
            }
            r0 = rt * 256;
            c0 = rem * BN;
        } else {
            // down the rows first: neighbouring clusters share the right operand
            const int ct = rem / args.row_tiles;
            r0 = (rem - ct * args.row_tiles) * 256;
            c0 = ct * BN;
        }
    };

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int i = first; i < total && !*abort_flag; i += clusters) {
                int b, r0, c0;
                decode(i, b, r0, c0);
                const int row = r0 + 128 * (int)rank, col = c0 + BN / 2 * (int)rank;
                for (int ks = 0; ks < ksteps; ++ks) {
                    if (!wait_cluster(empty + stage, phase ^ 1, abort_flag)) {
                        if (!*abort_flag) raise(FAULT_GEMM_PRODUCER);
                        *abort_flag = 1;
                        break;
                    }
                    // both CTAs' bytes complete on the first CTA's barrier
                    const uint32_t bar = map_to(ptx::smem_u32(full + stage), 0);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(full + stage, 2 * C::STAGE_BYTES);
                    uint8_t *l = smem + stage * C::STAGE_BYTES;
                    uint8_t *r = l + A_BYTES;
                    pair_load_3d(l, &tmL, ks * BK, row, b, bar);
                    if (PAIR_IN) {
#pragma unroll
                        for (int h = 0; h < BN / 128; ++h)
                            pair_load_3d(r + h * (64 * BK * 2), &tmR, col + 64 * h, ks * BK, b, bar);
                    } else {
                        pair_load_3d(r, &tmR, ks * BK, col, b, bar);
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
            constexpr uint32_t idesc = idesc_f16(BN, PAIR_IN);
            for (int i = first; i < total && !*abort_flag; i += clusters, ++li) {
                const int acc = li & 1;
                if (!wait_cluster(tempty + acc, ((li >> 1) & 1) ^ 1, abort_flag)) {
                    if (!*abort_flag) raise(FAULT_GEMM_MMA);
                    *abort_flag = 1;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d = tmem + acc * BN;
                bool ok = true;
                for (int ks = 0; ks < ksteps; ++ks) {
                    if (!wait_cluster(full + stage, phase, abort_flag)) {
                        if (!*abort_flag) raise(FAULT_GEMM_MMA);
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t l = ptx::smem_u32(smem + stage * C::STAGE_BYTES);
                    const uint32_t r = l + A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        pair_mma(d, ptx::sw128_desc(l + k * 32),
                                 PAIR_IN ? ptx::sw128_desc_mn(r + k * 2048, 64 * BK * 2) : ptx::sw128_desc(r + k * 32),
                                 idesc, (ks | k) != 0);
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
            wait_cluster(drain, 0, abort_flag);
        }
    } else {
        // ---------------------------------------------------- epilogue
        // warps 2..9: TMEM lane quarter warp % 4 (rows r0 + 128 rank + 32 q
        // ..), columns half * BN / 2 ... in blocks of 64.  Lane l holds row l
        // of a block; its 16-byte piece j is at (j ^ (l % 8)) * 16 of the
        // row's 128 bytes in the staging buffer (the tensor maps' swizzle).
        const int q = warp & 3, half = (warp - 2) >> 2;
        uint8_t *st = staging + (warp - 2) * 2 * BLOCK, *st_lo = st + BLOCK;
        uint64_t *bar = loaded + (warp - 2);
        uint32_t load_phase = 0;
        int li = 0;
        for (int i = first; i < total; i += clusters, ++li) {
            int b, r0, c0;
            decode(i, b, r0, c0);
            const int row0 = r0 + 128 * (int)rank + 32 * q, row = row0 + lane;
            const bool mirrored = SYM && r0 + 256 <= c0;  // a tile wholly above the diagonal's tiles
            const int acc = li & 1;
            bool have = false, failed = false;
#pragma unroll 1
            for (int blk = 0; blk < BN / 128; ++blk) {
                const int cb = half * (BN / 2) + 64 * blk, col0 = c0 + cb;
                const bool in = row0 < args.rows && col0 < args.cols;
                // the block's own operands, while the products run
                if (in && KIND != kGram) {
                    if (lane == 0) {
                        ptx::bulk_wait_group_read<0>();  // the buffers' last stores have read them
                        ptx::mbar_arrive_expect_tx(bar, (PAIR_IN ? 2 : 1) * BLOCK);
                        ptx::tma_load_3d(st, &tmIn, col0, row0, b, bar);
                        if (PAIR_IN) ptx::tma_load_3d(st_lo, &tmInLo, col0, row0, b, bar);
                    }
                    __syncwarp();
                }
                if (!have) {
                    have = true;
                    if (*abort_flag || !wait_cluster(tfull + acc, (li >> 1) & 1, abort_flag)) {
                        if (!*abort_flag) raise(FAULT_GEMM_EPILOGUE);
                        *abort_flag = 1;
                        failed = true;
                    }
                    failed = __any_sync(0xffffffffu, failed);
                    ptx::tc_fence_after();
                }
                if (in && KIND != kGram) {
                    const int keep = 0;
                    if (!ptx::mbar_wait_bounded(bar, load_phase, &keep, kWaitNs)) {
                        if (!*abort_flag) raise(FAULT_GEMM_EPILOGUE);
                        *abort_flag = 1;
                        failed = true;
                    }
                    load_phase ^= 1;
                    failed = __any_sync(0xffffffffu, failed);
                }
                if (failed) break;
                if (!in) continue;
                if (KIND == kGram) {
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                }
                const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + acc * BN + cb;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[32];
                    ptx::tmem_ld32(taddr + 32 * h, r);
                    ptx::tmem_wait_ld();
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = lane * 128 + (((4 * h + j) ^ (lane & 7)) << 4);
                        uint4 *p = reinterpret_cast<uint4 *>(st + at), *p_lo = reinterpret_cast<uint4 *>(st_lo + at);
                        uint32_t in_w[4] = {0, 0, 0, 0}, lo_w[4] = {0, 0, 0, 0}, o[4], o_lo[4];
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
                                v0 = a0 * args.cc, v1 = a1 * args.cc;
                            } else if (KIND == kPoly) {
                                const float2 x = half_unpair(in_w[e]);
                                v0 = fmaf(args.cc, a0, args.cb * x.x), v1 = fmaf(args.cc, a1, args.cb * x.y);
                            } else {
                                const float2 x = half_unpair(in_w[e]), y = half_unpair(lo_w[e]);
                                v0 = fmaf(args.cc, a0, args.ca * (x.x + y.x));
                                v1 = fmaf(args.cc, a1, args.ca * (x.y + y.y));
                            }
                            v[c] = v0, v[c + 1] = v1;
                            if (KIND == kLast) {
                                const __nv_bfloat162 z = __floats2bfloat162_rn(v0 * args.out_scale, v1 * args.out_scale);
                                o[e] = *reinterpret_cast<const uint32_t *>(&z);
                            } else {
                                o[e] = half_pair(v0, v1);
                            }
                            if (KIND == kApply) {
                                const float2 hi = half_unpair(o[e]);
                                o_lo[e] = half_pair(v0 - hi.x, v1 - hi.y);
                            }
                        }
                        *p = make_uint4(o[0], o[1], o[2], o[3]);
                        if (KIND == kApply) *p_lo = make_uint4(o_lo[0], o_lo[1], o_lo[2], o_lo[3]);
                    }
                    if (mirrored && row < args.rows) {
                        __half *dst = args.mirror + b * args.mirror_matrix + row;
                        const int c = col0 + 32 * h;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c + e < args.cols) dst[(c + e) * args.mirror_pitch] = __float2half_rn(v[e]);
                    }
                    if (KIND == kLast && args.transposed && row < args.rows) {
                        __nv_bfloat16 *dst = args.out + (int64_t)b * args.rows * args.cols + row;
                        const int c = col0 + 32 * h;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c + e < args.cols)
                                dst[(int64_t)(c + e) * args.out_cols] = __float2bfloat16_rn(v[e] * args.out_scale);
                    }
                }
                if (KIND == kLast) {
                    // the caller's rows have any pitch: from the staging buffer,
                    // a row's 64 elements at a time, two per lane
                    __syncwarp();
                    if (!args.transposed) {
                        const int c = col0 + 2 * lane;
                        __nv_bfloat16 *dst = args.out + (int64_t)b * args.rows * args.cols + c;
                        for (int rr = 0; rr < 32 && row0 + rr < args.rows; ++rr) {
                            const uint32_t w = *reinterpret_cast<const uint32_t *>(
                                st + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4);
                            __nv_bfloat16 *d = dst + (int64_t)(row0 + rr) * args.out_cols;
                            const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&w);
                            if (args.out_cols % 2 == 0) {
                                if (c < args.cols) *reinterpret_cast<__nv_bfloat162 *>(d) = z;
                            } else {
                                if (c < args.cols) d[0] = z.x;
                                if (c + 1 < args.cols) d[1] = z.y;
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
                        ptx::tma_store_3d(&tmOut, st, col0, row0, b);
                        if (KIND == kApply) ptx::tma_store_3d(&tmOutLo, st_lo, col0, row0, b);
                        ptx::bulk_commit_group();
                    }
                }
            }
            if (failed) break;
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(map_to(ptx::smem_u32(tempty + acc), 0));
        }
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

// partial[b][p]: the sum of squares of a slice of matrix b.
template <typename T>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const T *__restrict__ g, int64_t count,
                                                         float *__restrict__ partial)
{
    __shared__ float sums[8];
    const T *p = g + (int64_t)blockIdx.y * count;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const int64_t stride = (int64_t)gridDim.x * 256;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (; i + 3 * stride < count; i += 4 * stride) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v = (float)p[i + q * stride];
            s[q] = fmaf(v, v, s[q]);
        }
    }
    for (; i < count; i += stride) {
        const float v = (float)p[i];
        s[0] = fmaf(v, v, s[0]);
    }
    const float t = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v += sums[q];
        partial[blockIdx.y * kMaxParts + blockIdx.x] = v;
    }
}

// X hi and lo [b][m][pitch] from g [b][M][N], in 32 x 32 tiles (transposed
// through shared memory where the matrix is tall).
template <typename T>
__global__ void __launch_bounds__(256) ortho_split_kernel(const T *__restrict__ g, int M, int N,
                                                          const float *__restrict__ partial, int parts, float eps,
                                                          bool tall, int64_t pitch, __half *__restrict__ hi,
                                                          __half *__restrict__ lo)
{
    __shared__ float tile[32][33];
    const int b = blockIdx.z, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    float ss = 0.0f;
    for (int p = 0; p < parts; ++p) ss += __ldg(partial + b * kMaxParts + p);
    const float f = (float)(1 << kXBits) / (sqrtf(ss) + eps);
    const int m = tall ? N : M;
    const T *src = g + (int64_t)b * M * N;
    const int64_t base = (int64_t)b * m * pitch;
    const int r0 = blockIdx.y * 32, c0 = blockIdx.x * 32;  // in g
    auto put = [&](int r, int c, float v) {
        const __half h = __float2half_rn(v);
        hi[base + r * pitch + c] = h;
        lo[base + r * pitch + c] = __float2half_rn(v - __half2float(h));
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

template <int KIND, int BN>
cudaError_t launch_gemm(const CUtensorMap &l, const CUtensorMap &r, const CUtensorMap &in, const CUtensorMap &in_lo,
                        const CUtensorMap &out, const CUtensorMap &out_lo, OrthoArgs a, int pairs, cudaStream_t s)
{
    a.row_tiles = (a.rows + 255) / 256;
    a.col_tiles = (a.cols + BN - 1) / BN;
    if (KIND == kGram || KIND == kPoly) {
        a.tiles = 0;
        for (int rt = 0; rt < a.row_tiles; ++rt) a.tiles += a.col_tiles - rt * 256 / BN;
    } else {
        a.tiles = a.row_tiles * a.col_tiles;
    }
    const int64_t total = (int64_t)a.tiles * a.batch;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (total < pairs ? total : pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<BN>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ortho_gemm_kernel<KIND, BN>, l, r, in, in_lo, out, out_lo, a);
}

template <int KIND, int BN>
cudaError_t set_smem()
{
    return cudaFuncSetAttribute(ortho_gemm_kernel<KIND, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<BN>::SMEM);
}

struct Region {
    size_t partial, hi[2], lo, a, bm, total;
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
    L.partial = take((size_t)B * kMaxParts * 4);
    const size_t x = (size_t)(B * L.m * L.x_pitch) * 2, a = (size_t)(B * L.m * L.a_pitch) * 2;
    L.hi[0] = take(x);
    L.hi[1] = take(x);
    L.lo = take(x);
    L.a = take(a);
    L.bm = take(a);
    L.total = o;
    return L;
}

template <int BN>
cudaError_t run_steps(const OrthoCall &c, char *ws, const Region &L, int pairs, cudaStream_t s)
{
    auto *lo = (__half *)(ws + L.lo), *A = (__half *)(ws + L.a), *Bm = (__half *)(ws + L.bm);
    __half *hi[2] = {(__half *)(ws + L.hi[0]), (__half *)(ws + L.hi[1])};
    const int64_t B = c.B;
    CUtensorMap x_left[2], x_right[2], x_cols[2], x_blk[2], lo_blk, a_left, a_right, a_blk, b_left, b_blk;
    cudaError_t e = cudaSuccess;
    auto map = [&](CUtensorMap *t, const __half *p, int64_t cols, int64_t pitch, int box_rows) {
        if (e == cudaSuccess) e = make_map(t, p, B, L.m, cols, pitch, box_rows);
    };
    for (int i = 0; i < 2; ++i) {
        map(&x_left[i], hi[i], L.n, L.x_pitch, 128);
        map(&x_right[i], hi[i], L.n, L.x_pitch, BN / 2);
        map(&x_cols[i], hi[i], L.n, L.x_pitch, 64);
        map(&x_blk[i], hi[i], L.n, L.x_pitch, 32);
    }
    map(&lo_blk, lo, L.n, L.x_pitch, 32);
    map(&a_left, A, L.m, L.a_pitch, 128);
    map(&a_right, A, L.m, L.a_pitch, BN / 2);
    map(&a_blk, A, L.m, L.a_pitch, 32);
    map(&b_left, Bm, L.m, L.a_pitch, 128);
    map(&b_blk, Bm, L.m, L.a_pitch, 32);
    if (e != cudaSuccess) return e;

    OrthoArgs base{};
    base.m = (int)L.m;
    base.n = (int)L.n;
    base.batch = (int)B;
    auto pow2 = [](int p) { return ldexpf(1.0f, p); };
    for (int i = 0; i < c.steps; ++i) {
        const int x = i & 1, y = x ^ 1;
        OrthoArgs a = base;
        a.rows = a.cols = (int)L.m;
        a.depth = (int)L.n;
        a.cc = pow2(kABits - 2 * kXBits);
        a.mirror = A;
        a.mirror_pitch = L.a_pitch;
        a.mirror_matrix = L.m * L.a_pitch;
        e = launch_gemm<kGram, BN>(x_left[x], x_right[x], a_blk, a_blk, a_blk, a_blk, a, pairs, s);
        if (e != cudaSuccess) return e;
        a.depth = (int)L.m;
        a.cb = c.b * pow2(kBBits - kABits);
        a.cc = c.c * pow2(kBBits - 2 * kABits);
        a.mirror = Bm;
        e = launch_gemm<kPoly, BN>(a_left, a_right, a_blk, a_blk, b_blk, b_blk, a, pairs, s);
        if (e != cudaSuccess) return e;
        a = base;
        a.rows = (int)L.m;
        a.cols = (int)L.n;
        a.depth = (int)L.m;
        a.ca = c.a;
        a.cc = pow2(-kBBits);
        if (i + 1 < c.steps) {
            e = launch_gemm<kApply, BN>(b_left, x_cols[x], x_blk[x], lo_blk, x_blk[y], lo_blk, a, pairs, s);
        } else {
            a.out = (__nv_bfloat16 *)c.out;
            a.out_cols = (int)c.N;
            a.transposed = c.M > c.N;
            a.out_scale = c.out_scale * pow2(-kXBits);
            e = launch_gemm<kLast, BN>(b_left, x_cols[x], x_blk[x], lo_blk, x_blk[y], lo_blk, a, pairs, s);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t ortho_workspace_bytes(int64_t B, int64_t M, int64_t N) { return layout(B, M, N).total; }

cudaError_t ortho_init_device(int *pairs)
{
    cudaError_t e = set_smem<kGram, 256>();
    if (e == cudaSuccess) e = set_smem<kPoly, 256>();
    if (e == cudaSuccess) e = set_smem<kApply, 256>();
    if (e == cudaSuccess) e = set_smem<kLast, 256>();
    if (e == cudaSuccess) e = set_smem<kGram, 128>();
    if (e == cudaSuccess) e = set_smem<kPoly, 128>();
    if (e == cudaSuccess) e = set_smem<kApply, 128>();
    if (e == cudaSuccess) e = set_smem<kLast, 128>();
    if (e != cudaSuccess) return e;
    // the pairs of CTAs that the device can hold at once
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<256>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(pairs, ortho_gemm_kernel<kApply, 256>, &cfg);
}

cudaError_t launch_orthogonalize(const OrthoCall &c, void *workspace, int pairs, cudaStream_t s)
{
    const Region L = layout(c.B, c.M, c.N);
    char *ws = (char *)workspace;
    auto *partial = (float *)(ws + L.partial);
    auto *hi = (__half *)(ws + L.hi[0]), *lo = (__half *)(ws + L.lo);
    const int64_t count = c.M * c.N;
    const int64_t slices = ceil_div(count, 4096);
    const int parts = (int)(slices < kMaxParts ? slices : kMaxParts);
    const dim3 tiles((unsigned)ceil_div(c.N, 32), (unsigned)ceil_div(c.M, 32), (unsigned)c.B);
    const bool tall = c.M > c.N;
    if (c.g_f32) {
        ortho_norm_kernel<<<dim3(parts, (unsigned)c.B), 256, 0, s>>>((const float *)c.g, count, partial);
        ortho_split_kernel<<<tiles, 256, 0, s>>>((const float *)c.g, (int)c.M, (int)c.N, partial, parts, c.eps, tall,
                                                 L.x_pitch, hi, lo);
    } else {
        ortho_norm_kernel<<<dim3(parts, (unsigned)c.B), 256, 0, s>>>((const __nv_bfloat16 *)c.g, count, partial);
        ortho_split_kernel<<<tiles, 256, 0, s>>>((const __nv_bfloat16 *)c.g, (int)c.M, (int)c.N, partial, parts, c.eps,
                                                 tall, L.x_pitch, hi, lo);
    }
    cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess) return e;
    // 256-wide tiles feed the tensor cores best; where they leave pairs of
    // CTAs without one, 128-wide tiles are twice as many
    const int64_t rt = ceil_div(L.m, 256);
    const bool wide = c.B * (rt * (rt + 1) / 2) >= pairs;
    return wide ? run_steps<256>(c, ws, L, pairs, s) : run_steps<128>(c, ws, L, pairs, s);
}

}  // namespace moe
