// gate.cu -- the gate: expert scores, the choice of k experts with a balance
// bias and expert groups, their weights and the experts' loads; and the
// logits' gradient.
//
//   s = softmax(l) or 1 / (1 + exp(-l));  c = l, or s + bias
//   the experts of the topk_groups best groups stay (rank: the largest c, or
//   with a bias the sum of the two largest), of them the k largest c
//   w_j = scale s_j (/ sum of the chosen s)
//
// One warp per token.  Lane q owns the PER consecutive experts q PER ..., as
// 32-bit keys in the order of c, and sorts its (at most) 8 largest once (a
// sorting network on key and index); the list waits in shared memory, its
// head in registers.  A round of the selection is one warp maximum of the
// heads (redux); on equal keys the lowest lane that has it holds the lowest
// index, so the 32-bit keys decide (the router of the expert layer, whose
// lanes own experts 32 apart, compares 64 bits), and that lane pops its list.
//
// The bytes (4 E per token in, 8 k out) would take 2.6 us for 16384 tokens of
// 256 experts at the copy rate; the instructions bound it (the scores' exp
// and division, the sort, k rounds).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "route_block.cuh"

namespace moe {

namespace {

constexpr int kGateWarps = 8;
// up to this many tokens run as one block, which owns the counts (no zeroing
// before it, no atomics to global memory)
constexpr int kGateOneBlock = kGateWarps;
constexpr int kList = 8;  // sorted keys per lane

struct GateArgs {
    const float *logits, *bias;
    int64_t T;
    int E, k, groups, group_size, topk_groups;
    bool sigmoid, renorm;
    float scale;
    int32_t *idx;
    float *w;
    int32_t *counts;
};

// logit_key in three instructions: adding +0 turns -0 into +0 and every NaN
// into the one positive NaN that the GPU's FP32 additions give.
__device__ __forceinline__ uint32_t gate_key(float f)
{
    const int b = __float_as_int(__fadd_rn(f, 0.0f));
    return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}

// The 8 largest of two descending lists, into `list`: the larger of each
// list[q], x[7 - q] pair form a bitonic sequence, sorted by half-cleaners.
__device__ __forceinline__ void merge8_desc(unsigned long long (&list)[8], const unsigned long long (&x)[8])
{
#pragma unroll
    for (int q = 0; q < 8; ++q) list[q] = list[q] > x[7 - q] ? list[q] : x[7 - q];
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (!(q & d)) key_order(list[q], list[q + d]);
}

__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }

// exp(l - top), zero for a logit of -inf (also where top is -inf)
__device__ __forceinline__ float exp_below(float l, float top)
{
    return l == -INFINITY ? 0.0f : expf(l - top);
}

// The lane's logits of one token, -inf past the last expert.
template <int PER>
__device__ __forceinline__ void load_logits(const float *row, int E, float (&l)[PER])
{
    const int e0 = (threadIdx.x & 31) * PER;
    if constexpr (PER % 4 == 0) {
        if (E % 4 == 0) {  // every row starts on 16 bytes
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (e0 + i < E) v = ld_nc_f4(row + e0 + i);
                l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = e0 + i < E ? __ldg(row + e0 + i) : -INFINITY;
}

// Its counterpart: the lane's gradients of one token.
template <int PER>
__device__ __forceinline__ void store_logits(float *row, int E, const float (&l)[PER])
{
    const int e0 = (threadIdx.x & 31) * PER;
    if constexpr (PER % 4 == 0) {
        if (E % 4 == 0) {
#pragma unroll
            for (int i = 0; i < PER; i += 4)
                if (e0 + i < E)
                    *reinterpret_cast<float4 *>(row + e0 + i) = make_float4(l[i], l[i + 1], l[i + 2], l[i + 3]);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (e0 + i < E) row[e0 + i] = l[i];
}

// m1 >= m2: the two largest of {m1, m2, a, b} with a >= b
__device__ __forceinline__ void top2_merge(uint32_t &m1, uint32_t &m2, uint32_t a, uint32_t b)
{
    const uint32_t lo = min(m1, a);
    m1 = max(m1, a);
    m2 = max(lo, max(m2, b));
}

template <int PER>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const GateArgs a)
{
    constexpr bool AHEAD = PER <= 12;  // the next token's logits are loaded before this one's are used
    extern __shared__ int32_t hist[];  // [E], with counts
    __shared__ unsigned long long lists[kGateWarps][kList][32];
    __shared__ unsigned long long chosen[kGateWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, k = a.k, e0 = lane * PER;
    if (a.counts) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
    float l[PER];
    if (AHEAD && t < a.T) load_logits<PER>(a.logits + t * E, E, l);
    for (; t < a.T; t += stride) {
        float ln[PER];
        if (AHEAD) {
            if (t + stride < a.T) load_logits<PER>(a.logits + (t + stride) * E, E, ln);
        } else {
            load_logits<PER>(a.logits + t * E, E, l);
        }
        // the row's maximum and sum, where the scores themselves are needed
        float top = 0.0f, total = 1.0f;
        if (!a.sigmoid && (a.bias || !a.renorm)) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) m = max(m, gate_key(l[i]));
            top = key_logit(__reduce_max_sync(0xffffffffu, m));
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) total += exp_below(l[i], top);
            total = warp_sum(total);
        }
        uint32_t key[PER];
        if (!a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) key[i] = e0 + i < E ? gate_key(l[i]) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                float s;
                if (a.sigmoid)
                    s = sigmoid_of(l[i]);
                else
                    s = total > 0.0f ? exp_below(l[i], top) / total : 0.0f;
                key[i] = e0 + i < E ? gate_key(s + __ldg(a.bias + e0 + i)) : 0u;
            }
        }
        // groups that are a power of two of neighbouring lanes are ranked
        // from the lanes' lists, others from the keys
        const int size = a.group_size, lanes = size / PER;
        const bool whole = lanes * PER == size && (lanes & (lanes - 1)) == 0;
        uint32_t kept = 0;
        auto keep_best = [&](uint32_t rank) {  // lane g holds the rank of group g
            for (int r = 0; r < a.topk_groups; ++r) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, lane < a.groups ? rank : 0u);
                const int g = __ffs(__ballot_sync(0xffffffffu, rank == m && lane < a.groups)) - 1;
                kept |= 1u << g;
                if (lane == g) rank = 0;
            }
        };
        auto rank_of = [&](uint32_t m1, uint32_t m2) {
            return a.bias && size > 1 ? gate_key(key_logit(m1) + key_logit(m2)) : m1;
        };
        if (a.groups > 1 && !whole) {
            uint32_t rank = 0;
            for (int g = 0; g < a.groups; ++g) {
                uint32_t m1 = 0, m2 = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (e0 + i >= g * size && e0 + i < (g + 1) * size) top2_merge(m1, m2, key[i], 0u);
                const uint32_t g1 = __reduce_max_sync(0xffffffffu, m1);
                const int owner = __ffs(__ballot_sync(0xffffffffu, m1 == g1)) - 1;
                const uint32_t g2 = __reduce_max_sync(0xffffffffu, lane == owner ? m2 : m1);
                if (lane == g) rank = rank_of(g1, g2);
            }
            keep_best(rank);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (e0 + i < E && !(kept >> ((unsigned)(e0 + i) / (unsigned)size) & 1)) key[i] = 0;
        }
        // the lane's list: (key, ~index), so that the lower index is the larger
        unsigned long long list[kList];
#pragma unroll
        for (int c = 0; c < (PER + 7) / 8; ++c) {
            unsigned long long x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int i = 8 * c + q;
                x[q] = i < PER && key[i < PER ? i : 0]
                           ? ((unsigned long long)key[i < PER ? i : 0] << 32) | (uint32_t)~(uint32_t)(e0 + i)
                           : 0ull;
            }
            if (PER == 2)
                key_order(x[0], x[1]);
            else if (PER > 2)
                sort8_desc(x);
            if (c == 0) {
#pragma unroll
                for (int q = 0; q < 8; ++q) list[q] = x[q];
            } else {
                merge8_desc(list, x);
            }
        }
        unsigned long long head = list[0];
        if (a.groups > 1 && whole) {
            uint32_t m1 = (uint32_t)(list[0] >> 32), m2 = (uint32_t)(list[1] >> 32);
            for (int o = 1; o < lanes; o <<= 1)
                top2_merge(m1, m2, __shfl_xor_sync(0xffffffffu, m1, o), __shfl_xor_sync(0xffffffffu, m2, o));
            keep_best(__shfl_sync(0xffffffffu, rank_of(m1, m2), (lane * lanes) & 31));
            if (!(kept >> (lane / lanes) & 1)) head = 0;
        }
#pragma unroll
        for (int q = 1; q < (PER < kList ? PER : kList); ++q) lists[warp][q][lane] = list[q];
        // k rounds (the experts that stay are at least k, so no round comes to
        // a head of 0)
        int next = 1;
        for (int r = 0; r < k; ++r) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32));
            const int owner = __ffs(__ballot_sync(0xffffffffu, (uint32_t)(head >> 32) == m)) - 1;
            if (lane == owner) {
                chosen[warp][r] = head;
                if (next < (PER < kList ? PER : kList)) {
                    head = lists[warp][next++][lane];
                } else {
                    // the list is used up: the largest key below the last one
                    const unsigned long long last = head;
                    head = 0;
                    if (PER > kList)
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const unsigned long long x =
                                ((unsigned long long)key[i] << 32) | (uint32_t)~(uint32_t)(e0 + i);
                            if (key[i] && x < last && x > head) head = x;
                        }
                }
            }
        }
        __syncwarp();
        float s = 0.0f;
        int sel = 0;
        if (lane < k) {
            const unsigned long long mine = chosen[warp][lane];
            sel = (int)~(uint32_t)mine;
            // without a bias the key is the logit's
            const float lj = a.bias ? __ldg(a.logits + t * E + sel) : key_logit((uint32_t)(mine >> 32));
            if (a.sigmoid)
                s = sigmoid_of(lj);
            else if (a.renorm)
                s = exp_below(lj, a.bias ? top : key_logit((uint32_t)(chosen[warp][0] >> 32)));
            else
                s = total > 0.0f || total != total ? exp_below(lj, top) / total : 0.0f;
        }
        __syncwarp();  // the lists and choices are read before the next token's
        if (a.renorm) {
            const float sum = warp_sum(s);
            s = sum == 0.0f ? 0.0f : s / sum;
        }
        if (lane < k) {
            a.idx[t * k + lane] = sel;
            a.w[t * k + lane] = s * a.scale;
            if (a.counts) atomicAdd(hist + sel, 1);
        }
        if (AHEAD)
#pragma unroll
            for (int i = 0; i < PER; ++i) l[i] = ln[i];
    }
    if (a.counts) {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            if (gridDim.x == 1)
                a.counts[e] = hist[e];
            else if (hist[e])
                atomicAdd(a.counts + e, hist[e]);
        }
    }
}

// ---------------------------------------------------------------- gradient
// One warp per token; lane j owns slot j.  Only softmax weights that are not
// renormalised give every logit a gradient and need the whole row; the other
// forms gather the k chosen logits.  Every row of dlogits is written whole
// before the slots' lanes put theirs in.
template <int PER>
__global__ void __launch_bounds__(32 * kGateWarps) gate_grad_kernel(const float *__restrict__ logits,
                                                                    const int32_t *__restrict__ idx,
                                                                    const float *__restrict__ dw, int64_t T, int E,
                                                                    int k, bool sigmoid, bool renorm, float scale,
                                                                    float *__restrict__ dlogits)
{
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * kGateWarps;
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5); t < T; t += stride) {
        const float *row = logits + t * E;
        float *out = dlogits + t * E;
        int e = -1;
        float d = 0.0f;
        if (lane < k) {
            e = __ldg(idx + t * k + lane);
            d = scale * __ldg(dw + t * k + lane);
        }
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const bool used = e >= 0 && e < E && (same & ((1u << lane) - 1u)) == 0;
        const float l = used ? __ldg(row + e) : -INFINITY;
        if (!used) d = 0.0f;
        const bool dense = !sigmoid && !renorm;
        float p, mine = 0.0f, common = 0.0f;
        float v[PER];
        if (dense) {
            load_logits<PER>(row, E, v);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) m = max(m, gate_key(v[i]));
            const float top = key_logit(__reduce_max_sync(0xffffffffu, m));
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                v[i] = exp_below(v[i], top);
                total += v[i];
            }
            total = warp_sum(total);
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] *= inv;
            p = used ? exp_below(l, top) * inv : 0.0f;
            common = warp_sum(used ? d * p : 0.0f);
            mine = p * (d - common);
        } else {
            if (sigmoid) {
                p = used ? sigmoid_of(l) : 0.0f;
            } else {
                const float top = key_logit(__reduce_max_sync(0xffffffffu, used ? gate_key(l) : 0u));
                p = used ? exp_below(l, top) : 0.0f;
            }
            float ds = d;
            if (renorm) {
                const float total = warp_sum(p);
                // one chosen expert has the share 1 exactly and no gradient
                const float share = total == 0.0f ? 0.0f : p / total;
                const float mean = warp_sum(used ? d * share : 0.0f);
                ds = total == 0.0f ? 0.0f : (d - mean) / total;
            }
            // softmax: the factor p_j of the scores' gradient, sums cancelled
            mine = sigmoid ? ds * p * (1.0f - p) : ds * p;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = dense ? -v[i] * common : 0.0f;
        store_logits<PER>(out, E, v);
        __syncwarp();
        if (used) out[e] = mine;
    }
}

// Experts per lane: the smallest of these that covers E.
template <typename F>
cudaError_t with_per(int E, F f)
{
    const int per = (E + 31) / 32;
    if (per <= 1) return f(std::integral_constant<int, 1>());
    if (per <= 2) return f(std::integral_constant<int, 2>());
    if (per <= 4) return f(std::integral_constant<int, 4>());
    if (per <= 8) return f(std::integral_constant<int, 8>());
    if (per <= 12) return f(std::integral_constant<int, 12>());
    if (per <= 16) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace

cudaError_t launch_gate(const GateCall &c, int n_sm, cudaStream_t s)
{
    const GateArgs a{c.logits, c.bias,        c.T,         c.E,         c.k,       c.groups, c.E / c.groups,
                     c.topk_groups, c.sigmoid, c.renorm, c.scale, c.idx, c.w, c.counts};
    int grid = 1, warps = (int)c.T;
    if (c.T > kGateOneBlock) {
        warps = kGateWarps;
        const int64_t blocks = ceil_div(c.T, kGateWarps);
        grid = (int)(blocks < (int64_t)n_sm * 4 ? blocks : (int64_t)n_sm * 4);
        if (c.counts) {
            cudaError_t e = cudaMemsetAsync(c.counts, 0, (size_t)c.E * 4, s);
            if (e != cudaSuccess) return e;
        }
    }
    const size_t smem = c.counts ? (size_t)c.E * 4 : 0;
    return with_per(c.E, [&](auto per) {
        gate_kernel<decltype(per)::value><<<grid, 32 * warps, smem, s>>>(a);
        return cudaPeekAtLastError();
    });
}

cudaError_t launch_gate_grad(const float *logits, const int32_t *idx, const float *dw, int64_t T, int E, int k,
                             bool sigmoid, bool renorm, float scale, float *dlogits, int n_sm, cudaStream_t s)
{
    const int64_t blocks = ceil_div(T, kGateWarps);
    const int grid = (int)(blocks < (int64_t)n_sm * 8 ? blocks : (int64_t)n_sm * 8);
    return with_per(E, [&](auto per) {
        gate_grad_kernel<decltype(per)::value>
            <<<grid, 32 * kGateWarps, 0, s>>>(logits, idx, dw, T, E, k, sigmoid, renorm, scale, dlogits);
        return cudaPeekAtLastError();
    });
}

}  // namespace moe
