// balance.cu -- the gate's load-balance loss with the experts' counts and
// mean probabilities, and its gradient.
//
//   s = softmax(l), or sigmoid(l) / sum sigmoid(l); sequence i has n_i rows,
//   N = sum n_i, c_ie of them chose e, P_ie = mean of s_te over them
//   balance = sum_i n_i / N * E * sum_e c_ie / (k n_i) P_ie
//   z = sum_t lse_t^2 / N;  loss = coef balance + z_coef z
//   dl_te from balance: with a_e = coef E c_ie / (k n_i N),
//     softmax s_e (a_e - sum a s), sigmoid (a_e - sum a s) q_e (1 - q_e) / sum q
//   and from z: 2 z_coef / N lse_t softmax(l)_e
//
// A row lives in `lpr` lanes of a warp (32, fewer for up to 64 experts, whose
// rows share a warp), PER logits to a lane.  A block has a run of rows and
// goes through the sequences that meet it.  Per sequence its lanes add the
// probabilities in registers, its warps meet in shared memory, and the sums
// go to the slot (block + sequence): along the rows either the block or the
// sequence grows, so no two pairs share a slot, and there are blocks +
// sequences of them.  A second, small kernel adds the slots in order.  No
// sum depends on the order in which blocks run.
//
// DRAM bounds a large call's first kernel (131072 x 256, 37 sequences: 26 us,
// floor at the copy rate 20.4) and latency the second (6 us: the slots, their
// sum, the release to the block that ends last): 32 us in all.  Without the
// hardware's exponentials the first kernel's instructions took longer than its
// bytes; with the slots counted before the rows instead of between them it
// waited for them (40 us).  8191 x 128 with z: 9.8 us, of which the second
// kernel about 5.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kMostChunks = 512;   // blocks of the first kernel
constexpr int kLeastRows = 64;     // and their rows, where there are several
constexpr int kCached = 1024;      // offsets that a block keeps in shared memory
// A call whose rows take one block's warps up to so many turns, in up to so
// many sequences, runs as one block, which ends it by itself.  One block and
// two kernels, us: 256 x 128 6.7 and 7.0, 512 x 128 10.5 and 7.4; 128 x 256 5.7
// and 7.6, 256 x 256 8.4 and 7.6; 32 x 1000 6.4 and 8.3, 64 x 1000 9.6 and 9.8;
// 256 x 16 4.6 and 7.4, 1024 x 16 8.6 and 7.6; 64 x 16 in two sequences 6.9 and
// 9.6, in four 10.5 and 10.7, in eight 17 and 13.  One launch less on the host.
constexpr int kOneBlockTurns = 4, kOneBlockRows = 512, kOneBlockSequences = 3;

// Warps per block and rows of a warp in flight, by what the registers hold
// with two blocks on an SM.  Few large blocks: every one adds a slot that the
// second kernel reads (131072 x 256: 34.4 us with four blocks of 8 warps).
// Softmax, us, as it is, with fewer warps, with more: 256 experts 30.6, 33.7 (8
// warps), 31.0 (12); 512 30.4, 33.1 (8), 32.6 (16); 1000 29.8, 34.6 (4), 46.8 (12).
// Half the rows in flight: 128 experts 38.8 (35.0), 256 35.2 (30.6), but 64 29.9
// (33.3); twice as many: 256 49, 512 40, 1000 53.
constexpr int kPerSm = 2;

template <int PER>
struct RowShape {
    static constexpr int WARPS = PER <= 8 ? 16 : PER <= 16 ? 12 : 8, THREADS = 32 * WARPS;
    static constexpr int ROWS = PER <= 4 ? 4 : PER <= 8 ? 2 : 1;
};

// Blocks and warps of the second kernel that an SM holds (10 KB of shared memory
// a block, 64 registers a thread).
constexpr int kSumBlocksPerSm = 20, kSumWarpsPerSm = 32;

// The gradient's blocks add nothing up and are smaller; a warp has fewer rows
// in flight, for each brings the incoming gradient along.  Blocks per SM, one
// less and one more (softmax, us, the logits' bytes alike): 256 experts 65, 63.6
// and 72; 384 65.8, 65.5 and 67; 768 59.4, 66 and 70; 1000 63, 66 and 84; sigmoid at
// 512 66.1, 78 and 67.
constexpr int kGradWarps = 8;

template <int PER>
struct GradShape {
    static constexpr int PER_SM = PER <= 8 ? 5 : PER <= 16 ? 3 : 2;
    static constexpr int ROWS = PER <= 4 ? 2 : 1;
};

// Instances by what a row needs: one set of exponentials or two.
enum Kind { kSoftmax, kSigmoid, kSigmoidAndZ };

struct BalanceArgs {
    const float *logits;
    const int32_t *idx, *offsets;  // offsets nullable: one sequence of all rows
    int T, S, E, k, kp, lpr, chunk;  // kp: k as a power of two; chunk: rows per block
    float coef, z_coef;
    float *loss, *prob;
    int32_t *counts;
    // per slot: [E] sums, [E] counts, one sum of lse^2
    float *sums, *zs;
    int32_t *cnts;
    float2 *parts;  // [blocks of the second kernel]: the loss's two sums
    unsigned *ticket;
};

struct BalanceGradArgs {
    const float *logits, *dloss, *base;  // dloss, base nullable
    const int32_t *counts, *offsets;
    int T, S, E, k, lpr, chunk;
    float coef, z_coef;
    float *out;  // may be base
};

__device__ __forceinline__ int clamp_row(int v, int T) { return min(max(v, 0), T); }

// The offsets where the block's lanes read them: its shared memory if they
// fit.  Ends with a barrier.
__device__ __forceinline__ const int32_t *cache_offsets(const int32_t *offsets, int S, int T, int32_t *kept)
{
    if (!offsets) {
        if (threadIdx.x == 0) kept[0] = 0, kept[1] = T;
    } else if (S < kCached) {
        for (int i = threadIdx.x; i <= S; i += blockDim.x) kept[i] = offsets[i];
    }
    __syncthreads();
    return offsets && S >= kCached ? offsets : kept;
}

// How many of off[1..S] are at most `row`: the sequence of that row where it
// has one.  A warp halves the range 32-fold per step.
__device__ __forceinline__ int find_sequence(const int32_t *off, int S, int row)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = S;
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int at = min((lane + 1) * step, len);
        const int c = __popc(__ballot_sync(0xffffffffu, off[lo + at] <= row)) * step;
        lo += min(c, len);
        len = max(min(step, len - c) - 1, 0);
    }
    return lo;
}

// 1 / x by the hardware's approximation, within a unit in the last place;
// results below 2^-126 are zero.
__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(x), x <= 88: 2^y by the hardware (two units in the last place, zero below
// 2^-126), y = x log2 e rounded down, times 1 + c for what the rounding took: c =
// x - y ln 2 is in [0, 1e-5], exact but for y times the rounding of ln 2, 2e-9.
// In all within three units and |x| / 40 of one, where without c it is |x|; a NaN
// of a NaN.  Saturation makes c of an infinity, which is none, zero.
// 131072 x 256: sigmoid 30.7 us, softmax 30.9, sigmoid and z 43.8; without c 30.4,
// 30.1 and 39.6; with ln 2 in two parts and a clamp of x instead 31.6, 32.1, 47.9.
__device__ __forceinline__ float exp_to_88(float x)
{
    constexpr float log2e = 1.4426950408889634f, ln2 = 0.6931471805599453f;
    const float y = __fmul_rd(x, log2e);
    float e, c;
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(c) : "f"(-y), "f"(ln2), "f"(x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    return fmaf(e, c, e);
}

// Whether softmax's terms of a row of -inf, or a sigmoid row's, have a sum to
// divide by.
__device__ __forceinline__ float inverse_of(float total) { return total < 1.17549435e-38f ? 0.0f : reciprocal(total); }

// The lane's logits of a row, -inf past the last expert and without a row.
// VEC (E % 4 == 0): 16 bytes at a time, neighbouring lanes side by side.
template <int PER, bool VEC>
__device__ __forceinline__ int expert_of(int i, int sub, int lpr)
{
    return VEC ? (i / 4) * 4 * lpr + 4 * sub + i % 4 : i * lpr + sub;
}

template <int PER, bool VEC>
__device__ __forceinline__ void load_row(const float *row, bool valid, int E, int sub, int lpr, float fill,
                                         float (&l)[PER])
{
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int e = expert_of<PER, VEC>(i, sub, lpr);
            float4 v = make_float4(fill, fill, fill, fill);
            if (valid && e < E) v = *reinterpret_cast<const float4 *>(row + e);
            l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_of<PER, VEC>(i, sub, lpr);
            l[i] = valid && e < E ? row[e] : fill;
        }
    }
}

template <int PER, bool VEC>
__device__ __forceinline__ void store_row(float *row, int E, int sub, int lpr, const float (&l)[PER])
{
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int e = expert_of<PER, VEC>(i, sub, lpr);
            if (e < E) *reinterpret_cast<float4 *>(row + e) = make_float4(l[i], l[i + 1], l[i + 2], l[i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_of<PER, VEC>(i, sub, lpr);
            if (e < E) row[e] = l[i];
        }
    }
}

// Sums (maxima) over the lanes of a row, for ROWS rows at once.
template <int ROWS>
__device__ __forceinline__ void row_sum(float (&v)[ROWS], int lpr)
{
    for (int o = lpr >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < ROWS; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
}

template <int ROWS>
__device__ __forceinline__ void row_max(float (&v)[ROWS], int lpr)
{
    for (int o = lpr >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < ROWS; ++u) v[u] = fmaxf(v[u], __shfl_xor_sync(0xffffffffu, v[u], o));
}

// exp(l - max l) of each row, with the sums and maxima.  A row of -inf gets
// zeros; a NaN or +inf makes its row's sum NaN.
template <int PER, int ROWS>
__device__ __forceinline__ void exponentials(const float (&l)[ROWS][PER], int lpr, float (&e)[ROWS][PER],
                                             float (&top)[ROWS], float (&total)[ROWS])
{
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        top[u] = l[u][0];
#pragma unroll
        for (int i = 1; i < PER; ++i) top[u] = fmaxf(top[u], l[u][i]);
    }
    row_max(top, lpr);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        if (top[u] == -INFINITY) top[u] = 0.0f;
        total[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            e[u][i] = exp_to_88(l[u][i] - top[u]);
            total[u] += e[u][i];
        }
    }
    row_sum(total, lpr);
}

// 1 / (1 + exp(-l)) with the sums.
template <int PER, int ROWS>
__device__ __forceinline__ void sigmoids(const float (&l)[ROWS][PER], int lpr, float (&q)[ROWS][PER],
                                         float (&total)[ROWS])
{
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        total[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float x = -l[u][i];
            asm("min.NaN.f32 %0, %0, 0f42B00000;" : "+f"(x));  // 88: there q is zero
            q[u][i] = reciprocal(1.0f + exp_to_88(x));
            total[u] += q[u][i];
        }
    }
    row_sum(total, lpr);
}

template <int PER, int ROWS>
__device__ __forceinline__ void copy_rows(const float (&from)[ROWS][PER], float (&to)[ROWS][PER])
{
#pragma unroll
    for (int u = 0; u < ROWS; ++u)
#pragma unroll
        for (int i = 0; i < PER; ++i) to[u][i] = from[u][i];
}

// log of the sum of exponentials; 0 for a row of -inf, which has none.
__device__ __forceinline__ float lse_of(float top, float total) { return total == 0.0f ? 0.0f : top + logf(total); }

// A lane's slot among those of the rows [at, end): kp slots (k, as a power
// of two) to a row.  -1 where there is none.
__device__ __forceinline__ int load_slot(const int32_t *idx, int at, int end, int lane, int k, int kp)
{
    const int t = at + lane / kp, j = lane & (kp - 1);
    return t < end && j < k ? idx[(int64_t)t * k + j] : -1;
}

// Adds the slots of a warp's rows to the counts, a row's equal ones once.
__device__ __forceinline__ void count_slots(int e, int E, int lane, int kp, int32_t *hist)
{
    const bool valid = e >= 0 && e < E;
    // equal keys: the same expert in the same row
    const unsigned same = __match_any_sync(0xffffffffu, valid ? (lane / kp) * 1024 + e : -1);
    if (valid && (same & ((1u << lane) - 1u)) == 0) atomicAdd(hist + e, 1);
}

// A sum over the block, the same for every thread, in an order fixed by the
// threads alone.  `part`: a word per warp.
__device__ __forceinline__ float sum_of_block(float v, float *part, int warps)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += part[w];
    return s;
}

template <int PER, bool VEC, Kind KIND>
__global__ void __launch_bounds__(RowShape<PER>::THREADS, kPerSm) balance_kernel(const BalanceArgs a)
{
    constexpr int ROWS = RowShape<PER>::ROWS, WARPS = RowShape<PER>::WARPS, THREADS = 32 * WARPS;
    __shared__ float warp_sums[WARPS][32 * PER];
    __shared__ int32_t hist[32 * PER];
    __shared__ int32_t kept[kCached];
    __shared__ float part[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, T = a.T, S = a.S;
    const int lpr = PER > 4 ? 32 : a.lpr;
    const int sub = lane & (lpr - 1), group = lane / lpr, rows_per_warp = PER > 4 ? 1 : 32 / lpr;
    const bool alone = gridDim.x == 1;
    ptx::griddep_wait();
    if (!alone && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    const int32_t *off = cache_offsets(a.offsets, S, T, kept);
    float balance = 0.0f, z_total = 0.0f;  // alone: this thread's part of the two sums
    if (alone) {
        for (int i = threadIdx.x; i < S * E; i += THREADS) a.prob[i] = 0.0f, a.counts[i] = 0;
        __syncthreads();
    }
    int row = blockIdx.x * a.chunk;
    const int end = (int)min((int64_t)T, (int64_t)row + a.chunk);
    while (row < end) {
        const int i = find_sequence(off, S, row);
        if (i >= S) break;  // rows behind the last sequence
        const int lo = max(row, clamp_row(off[i], T)), hi = min(end, clamp_row(off[i + 1], T));
        row = max(row + 1, hi);
        if (lo >= hi) continue;
        // a warp takes `own` rows at a time, its next ones (and their first
        // slots) on their way while it works
        const int own = ROWS * rows_per_warp, step = WARPS * own;
        int at = lo + warp * own;
        auto fetch = [&](int at, float (&l)[ROWS][PER]) {
            const float *row = a.logits + (int64_t)(at + group) * E;
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                load_row<PER, VEC>(row + (int64_t)(u * rows_per_warp) * E, at + u * rows_per_warp + group < hi, E, sub,
                                   lpr, -INFINITY, l[u]);
        };
        float l[ROWS][PER], next[ROWS][PER];
        fetch(at, l);
        int slot = load_slot(a.idx, at, min(at + own, hi), lane, a.k, a.kp), next_slot;
        for (int e = threadIdx.x; e < E; e += THREADS) hist[e] = 0;
        __syncthreads();
        float sum[PER], z = 0.0f;
#pragma unroll
        for (int q = 0; q < PER; ++q) sum[q] = 0.0f;
        for (; at < hi; at += step) {
            float top[ROWS], total[ROWS];
            fetch(at + step, next);
            next_slot = load_slot(a.idx, at + step, min(at + step + own, hi), lane, a.k, a.kp);
            count_slots(slot, E, lane, a.kp, hist);
            // more rows than a warp has lanes for their slots
            const int at_once = 32 / a.kp;
            for (int r = at_once; r < own; r += 4 * at_once) {
                int more[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    more[u] = load_slot(a.idx, at + r + u * at_once, min(at + own, hi), lane, a.k, a.kp);
#pragma unroll
                for (int u = 0; u < 4; ++u) count_slots(more[u], E, lane, a.kp, hist);
            }
            slot = next_slot;
            if constexpr (KIND != kSigmoid) {
                float e[ROWS][PER];
                exponentials<PER, ROWS>(l, lpr, e, top, total);
                if (KIND == kSigmoidAndZ || a.z_coef != 0.0f) {
#pragma unroll
                    for (int u = 0; u < ROWS; ++u) {
                        const float lse = lse_of(top[u], total[u]);
                        if (sub == 0) z = fmaf(lse, lse, z);
                    }
                }
                if constexpr (KIND == kSoftmax) copy_rows(e, l);
            }
            if constexpr (KIND != kSoftmax) sigmoids<PER, ROWS>(l, lpr, l, total);
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const float inv = inverse_of(total[u]);
#pragma unroll
                for (int q = 0; q < PER; ++q) sum[q] = fmaf(l[u][q], inv, sum[q]);
            }
            copy_rows(next, l);
        }
        for (int o = lpr; o < 32; o <<= 1)
#pragma unroll
            for (int q = 0; q < PER; ++q) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], o);
        if (group == 0) {
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const int e = expert_of<PER, VEC>(q, sub, lpr);
                if (e < E) warp_sums[warp][e] = sum[q];
            }
        }
        if (a.z_coef != 0.0f) {
            z = warp_sum(z);
            if (lane == 0) part[warp] = z;
        }
        __syncthreads();
        const int64_t place = (int64_t)blockIdx.x + i;
        const float inv_n = 1.0f / (float)(hi - lo);
        for (int e = threadIdx.x; e < E; e += THREADS) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += warp_sums[w][e];
            if (alone) {
                s *= inv_n;
                a.prob[i * E + e] = s;
                a.counts[i * E + e] = hist[e];
                balance = fmaf((float)hist[e], s, balance);
            } else {
                a.sums[place * E + e] = s;
                a.cnts[place * E + e] = hist[e];
            }
        }
        if (a.z_coef != 0.0f && warp == 0) {
            z = warp_sum(lane < WARPS ? part[lane] : 0.0f);
            if (alone)
                z_total += z;
            else if (lane == 0)
                a.zs[place] = z;
        }
        __syncthreads();  // the sums and counts are read before the next sequence's
    }
    if (alone) {
        balance = sum_of_block(balance, part, WARPS);
        if (threadIdx.x == 0) {
            const int n = max(clamp_row(off[S], T) - clamp_row(off[0], T), 0);
            balance = n ? balance * (float)E / ((float)a.k * (float)n) : 0.0f;
            z_total = n ? z_total / (float)n : 0.0f;
            a.loss[0] = a.coef * balance + a.z_coef * z_total;
            a.loss[1] = balance;
            a.loss[2] = z_total;
        }
    }
}

__device__ __forceinline__ unsigned add_acq_rel(unsigned *at, unsigned v)
{
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(at), "r"(v) : "memory");
    return old;
}

// A sum that keeps what its additions round off (Kahan, Commun. ACM 8, 1965), so
// that its error does not grow with their number.
struct Sum {
    float sum = 0.0f, lost = 0.0f;

    __device__ __forceinline__ void add(float v)
    {
        const float y = v - lost, t = sum + y;
        lost = isinf(t) ? 0.0f : (t - sum) - y;
        sum = t;
    }
};

// The slots' sums: a block of 32 experts by depth warps for one sequence after
// another, whose parts of the loss it adds up; the block that ends last adds the
// blocks' parts, in their order.  The blocks are at most as many as the device
// holds at once, so no lane's sum there grows with the sequences (8191 x 256 in
// 4096 of them: 150 us with a block for each and every part in one warp's sums,
// 74 so).  All of a warp's slots are loaded at once, which takes 64 registers:
// with the 32 that two blocks of 1024 threads would leave, 0.5 to 1.4 us more.
__global__ void __launch_bounds__(1024, 1) balance_sum_kernel(const BalanceArgs a)
{
    constexpr int FLIGHT = 10;
    __shared__ float sums[32][33], part[32], terms[32];
    __shared__ int32_t cnts[32][33];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, depth = blockDim.x >> 5;
    const int T = a.T, S = a.S, E = a.E, e = blockIdx.x * 32 + lane;
    ptx::griddep_wait();
    auto offset = [&](int i) { return a.offsets ? clamp_row(a.offsets[i], T) : i ? T : 0; };
    const float rows = (float)max(offset(S) - offset(0), 0);
    Sum my_balance, my_z;  // thread 0's: the block's parts
    for (int i = blockIdx.y; i < S; i += gridDim.y) {
        const int lo = offset(i), hi = offset(i + 1), n = max(hi - lo, 0);
        float s = 0.0f, z = 0.0f;
        int32_t c = 0;
        if (n > 0) {
            const int first = lo / a.chunk, end = (hi - 1) / a.chunk;
            if (blockIdx.x == 0 && a.z_coef != 0.0f)
                for (int b = first + (int)threadIdx.x; b <= end; b += blockDim.x) z += a.zs[(int64_t)b + i];
            if (e < E)
                for (int b = first + y; b <= end; b += depth * FLIGHT) {
                    float v[FLIGHT];
                    int32_t many[FLIGHT];
#pragma unroll
                    for (int u = 0; u < FLIGHT; ++u) {
                        const int64_t slot = (int64_t)b + u * depth + i;
                        const bool in = b + u * depth <= end;
                        v[u] = in ? a.sums[slot * E + e] : 0.0f;
                        many[u] = in ? a.cnts[slot * E + e] : 0;
                    }
#pragma unroll
                    for (int u = 0; u < FLIGHT; ++u) s += v[u], c += many[u];
                }
        }
        sums[y][lane] = s;
        cnts[y][lane] = c;
        z = warp_sum(z);
        if (lane == 0) part[y] = z;
        __syncthreads();
        if (y == 0) {
            s = 0.0f;
            c = 0;
#pragma unroll 8
            for (int w = 0; w < depth; ++w) s += sums[w][lane], c += cnts[w][lane];
            s = n > 0 ? s / (float)n : 0.0f;
            if (e < E) {
                a.prob[(int64_t)i * E + e] = s;
                a.counts[(int64_t)i * E + e] = c;
            }
            const float term = warp_sum((float)c * s);
            z = warp_sum(lane < depth ? part[lane] : 0.0f);
            my_balance.add(term);
            my_z.add(z);
        }
        __syncthreads();
    }
    const int blocks = gridDim.x * gridDim.y;
    if (threadIdx.x == 0) a.parts[blockIdx.y * gridDim.x + blockIdx.x] = make_float2(my_balance.sum, my_z.sum);
    // thread 0 wrote the block's parts, and its addition to the ticket releases
    // them to the block whose addition is the last
    if (threadIdx.x == 0) last = add_acq_rel(a.ticket, 1u) == (unsigned)blocks - 1;
    __syncthreads();
    if (!last) return;
    float b4[4] = {}, z4[4] = {};
    for (int j = threadIdx.x; j < blocks; j += 4 * blockDim.x)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int at = j + u * blockDim.x;
            const float2 v = at < blocks ? __ldcg(a.parts + at) : make_float2(0.0f, 0.0f);
            b4[u] += v.x;
            z4[u] += v.y;
        }
    float balance = warp_sum((b4[0] + b4[1]) + (b4[2] + b4[3])), z = warp_sum((z4[0] + z4[1]) + (z4[2] + z4[3]));
    if (lane == 0) terms[y] = balance, part[y] = z;
    __syncthreads();
    if (y == 0) {
        balance = warp_sum(lane < depth ? terms[lane] : 0.0f);
        z = warp_sum(lane < depth ? part[lane] : 0.0f);
    }
    if (threadIdx.x == 0) {
        balance = rows > 0.0f ? balance * (float)E / ((float)a.k * rows) : 0.0f;
        z = rows > 0.0f ? z / rows : 0.0f;
        a.loss[0] = a.coef * balance + a.z_coef * z;
        a.loss[1] = balance;
        a.loss[2] = z;
    }
}

// ---------------------------------------------------------------- gradient
// The scores are computed again from the logits.  Rows of no sequence take
// the gradient that comes in, or zero, whatever their logits hold.  Bound by
// DRAM: 131072 x 256 with 37 sequences and an incoming gradient 62.5 us (floor
// at the copy rate 59.3), without one 44.7 (39.5); 100000 x 128, softmax and
// z, 25.7 (22.6).  One row of a warp in flight from 129 experts on, two below:
// two of 256 logits 73.7 where one takes 62.4, one of 128 54.8 (50.0).  Sigmoid
// and z, three exponentials and reciprocals a logit, is bound by instructions:
// 200000 x 128 60 (45), 32768 x 1000 75 (58).
//
// Wide rows fill the registers, and the compiler then loads them bit by bit as
// it works.  The warp's barrier after the loads keeps them together (32768 x
// 1000, softmax: 70.8 to 62.9).  For sigmoids, whose work on one logit waits for
// no other, it did not; there the incoming gradient is loaded at the end, from
// L2, where its row is fetched to meanwhile (40000 x 768: 86 to 60.5).  With z the
// next row's logits are fetched there (67.5 to 61.3).
template <int PER, bool VEC, Kind KIND>
__global__ void __launch_bounds__(32 * kGradWarps, GradShape<PER>::PER_SM) balance_grad_kernel(const BalanceGradArgs a)
{
    constexpr int ROWS = GradShape<PER>::ROWS, WARPS = kGradWarps;
    constexpr bool LATE = PER > 8 && KIND == kSigmoid;  // the incoming gradient is loaded at the end
    __shared__ int32_t kept[kCached];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, T = a.T, S = a.S;
    const int lpr = PER > 4 ? 32 : a.lpr;
    const int sub = lane & (lpr - 1), group = lane / lpr, rows_per_warp = 32 / lpr;
    ptx::griddep_wait();
    const int32_t *off = cache_offsets(a.offsets, S, T, kept);
    const float up = a.dloss ? *a.dloss : 1.0f;
    const float per_row = 1.0f / (float)max(clamp_row(off[S], T) - clamp_row(off[0], T), 1);
    const float scale = up * a.coef * (float)E / (float)a.k * per_row;
    const float z_scale = 2.0f * up * a.z_coef * per_row;
    auto pass = [&](int from, int to) {  // rows of no sequence
        for (int at = from + warp * rows_per_warp; at < to; at += WARPS * rows_per_warp) {
            const int t = at + group;
            if (t >= to) continue;
            float v[PER];
            load_row<PER, VEC>(a.base + (int64_t)t * E, a.base != nullptr, E, sub, lpr, 0.0f, v);
            store_row<PER, VEC>(a.out + (int64_t)t * E, E, sub, lpr, v);
        }
    };
    auto fetch = [&](const float *row) {  // of a warp's row, to L2: a lane for each 128 bytes
        if (lane * 32 < E) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + lane * 32));
    };
    int row = blockIdx.x * a.chunk;
    const int end = (int)min((int64_t)T, (int64_t)row + a.chunk);
    while (row < end) {
        const int i = find_sequence(off, S, row);
        const int lo = i < S ? min(end, max(row, clamp_row(off[i], T))) : end;
        const int hi = i < S ? max(lo, min(end, clamp_row(off[i + 1], T))) : end;
        if (row < lo) pass(row, lo);
        row = max(row + 1, hi);
        if (lo >= hi) continue;
        float share[PER];  // a_e of the sequence
        const float inv_n = scale / (float)(clamp_row(off[i + 1], T) - clamp_row(off[i], T));
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int e = expert_of<PER, VEC>(q, sub, lpr);
            share[q] = e < E ? (float)a.counts[(int64_t)i * E + e] * inv_n : 0.0f;
        }
        for (int at = lo + warp * rows_per_warp; at < hi; at += WARPS * rows_per_warp * ROWS) {
            float l[ROWS][PER], p[ROWS][PER], top[ROWS], total[ROWS], mean[ROWS], lse[ROWS], base[ROWS][PER];
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const int t = at + u * WARPS * rows_per_warp + group;
                load_row<PER, VEC>(a.logits + (int64_t)t * E, t < hi, E, sub, lpr, -INFINITY, l[u]);
                if (!LATE)
                    load_row<PER, VEC>(a.base + (int64_t)t * E, a.base != nullptr && t < hi, E, sub, lpr, 0.0f, base[u]);
                lse[u] = 0.0f;
            }
            if (PER > 8 && KIND == kSigmoidAndZ && at + WARPS < hi) fetch(a.logits + (int64_t)(at + WARPS) * E);
            if (LATE && a.base != nullptr) fetch(a.base + (int64_t)at * E);
            __syncwarp();
            float d[ROWS][PER];
            if constexpr (KIND != kSigmoid) {
                exponentials<PER, ROWS>(l, lpr, p, top, total);
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    const float inv = inverse_of(total[u]);
                    if (a.z_coef != 0.0f) lse[u] = z_scale * lse_of(top[u], total[u]);
#pragma unroll
                    for (int q = 0; q < PER; ++q) {
                        p[u][q] *= inv;
                        // with the sigmoids still to come the incoming gradient joins here
                        d[u][q] = KIND == kSigmoidAndZ ? fmaf(lse[u], p[u][q], base[u][q]) : lse[u] * p[u][q];
                    }
                }
            }
            if constexpr (KIND != kSoftmax) {
                // p: q (1 - q), of x = exp(-|l|), which is q / (1 - q) or its
                // inverse.  A difference of q from one would lose it for large
                // logits (17% of it at 15, all of it from 17 on).
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    mean[u] = total[u] = 0.0f;
#pragma unroll
                    for (int q = 0; q < PER; ++q) {
                        const float x = exp_to_88(-fabsf(l[u][q])), r = reciprocal(1.0f + x), xr = x * r;
                        const float s = l[u][q] < 0.0f ? xr : r;
                        total[u] += s;
                        mean[u] = fmaf(share[q], s, mean[u]);
                        p[u][q] = xr * r;
                    }
                }
                row_sum(total, lpr);
                row_sum(mean, lpr);
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    const float inv = inverse_of(total[u]);
                    mean[u] *= inv;
#pragma unroll
                    for (int q = 0; q < PER; ++q) {
                        const float g = (share[q] - mean[u]) * inv * p[u][q];
                        d[u][q] = KIND == kSigmoidAndZ ? d[u][q] + g : g;
                    }
                }
            } else {
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    mean[u] = 0.0f;
#pragma unroll
                    for (int q = 0; q < PER; ++q) mean[u] = fmaf(share[q], p[u][q], mean[u]);
                }
                row_sum(mean, lpr);
#pragma unroll
                for (int u = 0; u < ROWS; ++u)
#pragma unroll
                    for (int q = 0; q < PER; ++q) d[u][q] = fmaf(p[u][q], share[q] - mean[u], d[u][q]);
            }
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const int t = at + u * WARPS * rows_per_warp + group;
                if (t >= hi) continue;
                if (LATE) load_row<PER, VEC>(a.base + (int64_t)t * E, a.base != nullptr, E, sub, lpr, 0.0f, base[u]);
#pragma unroll
                for (int q = 0; q < PER; ++q)
                    if (KIND != kSigmoidAndZ) d[u][q] += base[u][q];
                store_row<PER, VEC>(a.out + (int64_t)t * E, E, sub, lpr, d[u]);
            }
        }
    }
}

// Logits per lane and lanes per row.
int lanes_per_row(int E)
{
    int lpr = 1;
    while (lpr < 32 && 4 * lpr < E) lpr <<= 1;
    return lpr;
}

// f(PER, VEC, KIND) for E experts.
template <bool VEC, Kind KIND, typename F>
cudaError_t with_per(int E, F f)
{
    std::integral_constant<bool, VEC> vec;
    std::integral_constant<Kind, KIND> kind;
    const int per = (E + 31) / 32;
    if (per <= 4) return f(std::integral_constant<int, 4>(), vec, kind);
    if (per <= 8) return f(std::integral_constant<int, 8>(), vec, kind);
    if (per <= 12) return f(std::integral_constant<int, 12>(), vec, kind);
    if (per <= 16) return f(std::integral_constant<int, 16>(), vec, kind);
    if (per <= 24) return f(std::integral_constant<int, 24>(), vec, kind);
    return f(std::integral_constant<int, 32>(), vec, kind);
}

template <Kind KIND, typename F>
cudaError_t with_vec(int E, F f)
{
    return E % 4 == 0 ? with_per<true, KIND>(E, f) : with_per<false, KIND>(E, f);
}

template <typename F>
cudaError_t with_row(int E, bool sigmoid, bool z, F f)
{
    return !sigmoid ? with_vec<kSoftmax>(E, f) : z ? with_vec<kSigmoidAndZ>(E, f) : with_vec<kSigmoid>(E, f);
}

// Blocks of the first kernel: of kLeastRows rows, or as many as there are
// sequences (a block goes through the sequences of its rows one by one).
int most_chunks(int64_t T, int64_t S)
{
    int64_t c = ceil_div(T, kLeastRows);
    if (c < S) c = S < T ? S : T;
    return (int)(c < 1 ? 1 : c < kMostChunks ? c : kMostChunks);
}

// The workspace's parts, each on 256 bytes.
struct Places {
    size_t sums, cnts, zs, parts, bytes;
};

Places places(int64_t T, int64_t S, int64_t E)
{
    const int64_t slots = most_chunks(T, S) + S;
    Places p;
    p.sums = 256;  // the ticket before them
    p.cnts = p.sums + round_up(slots * E * 4, 256);
    p.zs = p.cnts + round_up(slots * E * 4, 256);
    p.parts = p.zs + round_up(slots * 4, 256);
    p.bytes = p.parts + round_up(S * ceil_div(E, 32) * 8, 256);
    return p;
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int64_t S, int64_t E) { return places(T, S, E).bytes; }

cudaError_t launch_balance(const BalanceCall &c, void *workspace, int n_sm, cudaStream_t s)
{
    const Places p = places(c.T, c.S, c.E);
    char *ws = (char *)workspace;
    BalanceArgs a{c.logits, c.idx, c.offsets, (int)c.T, c.S, c.E, c.k, pow2_ceil(c.k), lanes_per_row(c.E), 0,
                  c.coef, c.z_coef, c.loss, c.prob, c.counts, (float *)(ws + p.sums), (float *)(ws + p.zs),
                  (int32_t *)(ws + p.cnts), (float2 *)(ws + p.parts), (unsigned *)ws};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    bool alone = false;
    int blocks = 1;
    cudaError_t e = with_row(c.E, c.sigmoid, c.z_coef != 0.0f, [&](auto per, auto vec, auto kind) {
        constexpr int PER = decltype(per)::value;
        constexpr bool VEC = decltype(vec)::value;
        const int turn = RowShape<PER>::WARPS * RowShape<PER>::ROWS * (PER > 4 ? 1 : 32 / a.lpr);
        alone = c.S <= kOneBlockSequences && c.T <= kOneBlockRows && c.T <= (int64_t)turn * kOneBlockTurns;
        if (!alone) {
            blocks = most_chunks(c.T, c.S);
            if (blocks > n_sm * kPerSm) blocks = n_sm * kPerSm;
            if (blocks < 2) blocks = 2;  // one is the block that ends the call by itself
        }
        a.chunk = (int)ceil_div(c.T, blocks);
        if (a.chunk < 1) a.chunk = 1;
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(RowShape<PER>::THREADS);
        return cudaLaunchKernelEx(&cfg, balance_kernel<PER, VEC, decltype(kind)::value>, (const BalanceArgs)a);
    });
    if (e != cudaSuccess || alone) return e;
    // a warp takes a few of a sequence's slots, all at once
    int depth = 1;
    while (depth < 32 && 4 * depth * c.S < blocks + c.S) depth <<= 1;
    const int64_t tiles = ceil_div(c.E, 32), per_sm = kSumWarpsPerSm / depth;
    const int64_t resident = n_sm * (per_sm < kSumBlocksPerSm ? per_sm : kSumBlocksPerSm);
    const int64_t most = resident > tiles ? resident / tiles : 1;
    cfg.gridDim = dim3((unsigned)tiles, (unsigned)(c.S < most ? c.S : most));
    cfg.blockDim = dim3(32 * depth);
    return cudaLaunchKernelEx(&cfg, balance_sum_kernel, (const BalanceArgs)a);
}

cudaError_t launch_balance_grad(const BalanceGradCall &c, int n_sm, cudaStream_t s)
{
    BalanceGradArgs a{c.logits, c.dloss, c.base, c.counts, c.offsets, (int)c.T, c.S, c.E, c.k, lanes_per_row(c.E), 0,
                      c.coef, c.z_coef, c.out};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return with_row(c.E, c.sigmoid, c.z_coef != 0.0f, [&](auto per, auto vec, auto kind) {
        constexpr int PER = decltype(per)::value;
        constexpr bool VEC = decltype(vec)::value;
        const int64_t rows = kGradWarps * (PER > 4 ? 1 : 32 / a.lpr), fit = ceil_div(c.T, rows);
        const int64_t most = (int64_t)n_sm * GradShape<PER>::PER_SM, blocks = fit < most ? fit : most;
        a.chunk = (int)ceil_div(c.T, blocks);
        cfg.blockDim = dim3(32 * kGradWarps);
        cfg.gridDim = dim3((unsigned)blocks);
        return cudaLaunchKernelEx(&cfg, balance_grad_kernel<PER, VEC, decltype(kind)::value>, (const BalanceGradArgs)a);
    });
}

}  // namespace moe
