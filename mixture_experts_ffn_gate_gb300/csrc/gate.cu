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
// sorting network of minima and maxima on the keys alone); the list waits in
// shared memory, its head in a register.  A round of the selection is one
// warp maximum of the heads (redux); on equal keys the lowest lane that has
// it holds the lowest index, and that lane moves on in its list.  Which
// expert a chosen key belongs to is looked up afterwards, by lane j for round
// j, among the owner's keys in shared memory: carrying the index through the
// sort took twice its instructions.
//
// The bytes (4 E per token in, 8 k out) would take 2.6 us for 16384 tokens of
// 256 experts at the copy rate; the instructions bound it (the scores' exp
// and reciprocal, the sort, k rounds).  Measured there with sigmoid scores, a
// bias, 4 of 8 groups and k = 8: 18.4 us (15.1 without the counts); softmax
// scores without a bias: 11.7 (9.6).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "route_block.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kGradWarps = 8;
// up to this many tokens run as one block, which owns the counts (no zeroing
// before it, no atomics to global memory)
constexpr int kGateOneBlock = 8;

// Warps per block and blocks per SM: what the registers of a lane's PER
// experts let an SM hold, in few blocks, because each adds its counts to the
// same E words at the end (16384 tokens, 256 experts: 2.5 us less with 2
// blocks of 16 warps than with 4 of 8).
template <int PER>
struct GateShape {
    static constexpr int WARPS = PER <= 8 ? 16 : 8, BLOCKS = PER <= 8 || PER > 16 ? 2 : 3;
};
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

// a >= b afterwards
__device__ __forceinline__ void order_desc(uint32_t &a, uint32_t &b)
{
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// 8 keys in descending order: 19 comparators, depth 6
__device__ __forceinline__ void sort8_desc(uint32_t (&x)[8])
{
    constexpr int pairs[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6}, {3, 7}, {0, 1}, {2, 3},
                                  {4, 5}, {6, 7}, {2, 4}, {3, 5}, {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) order_desc(x[pairs[i][0]], x[pairs[i][1]]);
}

// The 8 largest of two descending lists, into `list`: the larger of each
// list[q], x[7 - q] pair form a bitonic sequence, sorted by half-cleaners.
__device__ __forceinline__ void merge8_desc(uint32_t (&list)[8], const uint32_t (&x)[8])
{
#pragma unroll
    for (int q = 0; q < 8; ++q) list[q] = max(list[q], x[7 - q]);
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (!(q & d)) order_desc(list[q], list[q + d]);
}

// N words to and from shared memory (16 bytes at a time where N allows)
template <int N>
__device__ __forceinline__ void put_words(uint32_t *dst, const uint32_t *v)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) dst[i] = v[i];
    }
}

template <int N>
__device__ __forceinline__ void get_words(uint32_t *v, const uint32_t *src)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 w = *reinterpret_cast<const uint4 *>(src + i);
            v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = src[i];
    }
}

__device__ __forceinline__ float sigmoid_of(float l) { return __frcp_rn(1.0f + expf(-l)); }

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
                if (e0 + i < E) v = *reinterpret_cast<const float4 *>(row + e0 + i);
                l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = e0 + i < E ? row[e0 + i] : -INFINITY;
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
__global__ void __launch_bounds__(32 * GateShape<PER>::WARPS, GateShape<PER>::BLOCKS) gate_kernel(const GateArgs a)
{
    constexpr int WARPS = GateShape<PER>::WARPS;
    constexpr bool KEEP_BIAS = PER <= 12;  // the lane's biases stay in registers
    constexpr int LIST = PER < kList ? PER : kList;
    // words per lane: rows of 16-byte pieces start in different banks (of 8
    // and 32 keys some meet, which leaves room for the warps)
    constexpr int KEYS = PER == 16 ? PER + 4 : PER, ROW = 12;
    static_assert(4 * 32 * WARPS * (KEYS + ROW) + 4 * 32 * PER <= 48 * 1024, "shared memory");
    extern __shared__ int32_t hist[];  // [E], with counts
    __shared__ __align__(16) uint32_t keys[WARPS][32 * KEYS];  // by expert
    __shared__ __align__(16) uint32_t lists[WARPS][32 * ROW];  // sorted, then a 0
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, k = a.k, e0 = lane * PER;
    const unsigned lower = (1u << lane) - 1u;
    uint32_t *const my_list = lists[warp] + lane * ROW, *const my_keys = keys[warp] + lane * KEYS;
    my_list[LIST] = 0;
    // what the kernel before this one wrote is there from here on (plain loads
    // below: read-only ones may be moved before this)
    ptx::griddep_wait();
    if (a.counts) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    float bias[PER];
    if (KEEP_BIAS)
#pragma unroll
        for (int i = 0; i < PER; ++i) bias[i] = a.bias && e0 + i < E ? a.bias[e0 + i] : 0.0f;
    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp; t < a.T; t += stride) {
        float l[PER];
        load_logits<PER>(a.logits + t * E, E, l);
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
            for (int i = 0; i < PER; ++i) key[i] = gate_key(l[i]);
        } else {
            float c[PER];
            if (a.sigmoid) {
#pragma unroll
                for (int i = 0; i < PER; ++i) c[i] = sigmoid_of(l[i]);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) c[i] = total == 0.0f ? 0.0f : exp_below(l[i], top) / total;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                key[i] = gate_key(c[i] + (KEEP_BIAS ? bias[i] : e0 + i < E ? a.bias[e0 + i] : 0.0f));
        }
        if (E < 32 * PER) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (e0 + i >= E) key[i] = 0;
        }
        // groups that are a power of two of neighbouring lanes are ranked
        // from the lanes' lists, others from the keys
        const int size = a.group_size, lanes = size / PER;
        const bool whole = lanes * PER == size && (lanes & (lanes - 1)) == 0;
        uint32_t kept = 0;
        auto keep_best = [&](uint32_t rank) {  // lane g holds the rank of group g
            bool in = false;
            rank = lane < a.groups ? rank : 0u;
            for (int r = 0; r < a.topk_groups; ++r) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, rank);
                const unsigned b = __ballot_sync(0xffffffffu, rank == m);
                if (rank == m && (b & lower) == 0) in = true, rank = 0;
            }
            kept = __ballot_sync(0xffffffffu, in);
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
        put_words<PER>(my_keys, key);
        uint32_t list[kList];
#pragma unroll
        for (int c = 0; c < (PER + 7) / 8; ++c) {
            uint32_t x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = 8 * c + q < PER ? key[8 * c + q < PER ? 8 * c + q : 0] : 0u;
            if (PER == 2)
                order_desc(x[0], x[1]);
            else if (PER > 2)
                sort8_desc(x);
            if (c == 0) {
#pragma unroll
                for (int q = 0; q < 8; ++q) list[q] = x[q];
            } else {
                merge8_desc(list, x);
            }
        }
        put_words<LIST>(my_list, list);
        uint32_t head = list[0];
        if (a.groups > 1 && whole) {
            uint32_t m1 = list[0], m2 = list[1];
            for (int o = 1; o < lanes; o <<= 1)
                top2_merge(m1, m2, __shfl_xor_sync(0xffffffffu, m1, o), __shfl_xor_sync(0xffffffffu, m2, o));
            keep_best(__shfl_sync(0xffffffffu, rank_of(m1, m2), (lane * lanes) & 31));
            if (!(kept >> (lane / lanes) & 1)) head = 0;
        }
        // k rounds (the experts that stay are at least k, so no round comes to
        // a head of 0); lane r keeps round r's key and the lanes that had it
        uint32_t won = 0, who = 1;
        int at = 0;
        for (int r = 0; r < k; ++r) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, head);
            const unsigned b = __ballot_sync(0xffffffffu, head == m);
            if (lane == r) won = m, who = b;
            if (head == m && (b & lower) == 0) {
                ++at;
                if (PER <= kList || at < LIST) {
                    head = my_list[at];
                } else {
                    // the list is used up: the key again if there are more of
                    // it than the lane has given, else the largest below it
                    int n = 0;
                    uint32_t next = 0;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        n += key[i] >= head;
                        if (key[i] < head) next = max(next, key[i]);
                    }
                    if (n <= at) head = next;
                }
            }
        }
        // the expert of lane j's key: the owner's first one that has it, or,
        // where the rounds before gave equal keys of the same owner (they
        // follow one another), the one after theirs
        const int owner = __ffs(who) - 1;
        const uint32_t won_before = __shfl_up_sync(0xffffffffu, won, 1);
        const int owner_before = __shfl_up_sync(0xffffffffu, owner, 1);
        const bool again = lane > 0 && lane < k && won_before == won && owner_before == owner;
        const unsigned repeats = __ballot_sync(0xffffffffu, again);
        const float first = key_logit(__shfl_sync(0xffffffffu, won, 0));
        __syncwarp();
        float s = 0.0f;
        int sel = 0;
        if (lane < k) {
            const uint32_t *row = keys[warp] + owner * KEYS;
            uint32_t v[PER];
            get_words<PER>(v, row);
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (v[i] == won) sel = i;
            if (again) {
                int skip = lane - (31 - __clz(~repeats & ((2u << lane) - 1u)));
                for (int i = 0; i < PER; ++i)
                    if (row[i] == won && skip-- == 0) sel = i;
            }
            sel += owner * PER;
            // without a bias the key is the logit's
            const float lj = a.bias ? a.logits[t * E + sel] : key_logit(won);
            if (a.sigmoid)
                s = sigmoid_of(lj);
            else if (a.renorm)
                s = total != total ? total : exp_below(lj, a.bias ? top : first);
            else
                s = total == 0.0f ? 0.0f : exp_below(lj, top) / total;
        }
        __syncwarp();  // the keys are read before the next token's are written
        if (a.renorm) {
            const float sum = warp_sum(s);
            s = sum == 0.0f ? 0.0f : s / sum;
        }
        if (lane < k) {
            a.idx[t * k + lane] = sel;
            a.w[t * k + lane] = s * a.scale;
            if (a.counts) atomicAdd(hist + sel, 1);
        }
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

// The counts before a launch of several blocks.  Both launches are scheduled
// while the work before them drains (a memset in this one's place put 4 us
// before the gate, this about 2).
__global__ void __launch_bounds__(256) zero_counts_kernel(int32_t *counts, int E)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    for (int e = threadIdx.x; e < E; e += 256) counts[e] = 0;
}

// ---------------------------------------------------------------- gradient
// One warp per token; lane j owns slot j.  Only softmax weights that are not
// renormalised give every logit a gradient and need the whole row; the other
// forms gather the k chosen logits.  Every row of dlogits is written whole
// before the slots' lanes put theirs in.
//
// Bound by latency and DRAM: the slots, their logits and the row follow one
// another, so the next token's slots are on their way while this one's are
// used, and the grid is what an SM holds, each warp going on to its next
// tokens.  Measured (floor at the copy rate): 131072 tokens, 256 experts, all
// logits 53.5 us (41.4; 76 without the two), chosen ones only 43.8 (21.6; 61);
// 8191 x 384, all: 8.4 (3.8).  The next row's loads ahead as well cost more
// registers than they brought (56.5).
template <int PER>
constexpr int kGradBlocks = PER <= 2 ? 8 : PER <= 8 ? 6 : PER <= 16 ? 4 : 2;

template <int PER>
__global__ void __launch_bounds__(32 * kGradWarps, kGradBlocks<PER>) gate_grad_kernel(const float *__restrict__ logits,
                                                                    const int32_t *__restrict__ idx,
                                                                    const float *__restrict__ dw, int64_t T, int E,
                                                                    int k, bool sigmoid, bool renorm, float scale,
                                                                    float *__restrict__ dlogits)
{
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * kGradWarps;
    const bool dense = !sigmoid && !renorm;
    int64_t t = (int64_t)blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    // the next token's slots are loaded before this one's are used, its row first of all
    int e = -1, e_next = -1;
    float d = 0.0f, d_next = 0.0f;
    auto load_slots = [&](int64_t at) {
        e_next = -1;
        if (at < T && lane < k) {
            e_next = __ldg(idx + at * k + lane);
            d_next = scale * __ldg(dw + at * k + lane);
        }
    };
    load_slots(t);
    for (; t < T; t += stride) {
        const float *row = logits + t * E;
        float *out = dlogits + t * E;
        float v[PER];
        if (dense) {
            load_logits<PER>(row, E, v);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = 0.0f;
            store_logits<PER>(out, E, v);
        }
        e = e_next;
        d = d_next;
        load_slots(t + stride);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const bool used = e >= 0 && e < E && (same & ((1u << lane) - 1u)) == 0;
        const float l = used ? __ldg(row + e) : -INFINITY;
        if (!used) d = 0.0f;
        float p, mine = 0.0f;
        if (dense) {
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
            const float common = warp_sum(used ? d * p : 0.0f);
            mine = p * (d - common);
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = -v[i] * common;
            store_logits<PER>(out, E, v);
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
    const bool several = c.T > kGateOneBlock, zero = several && c.counts;
    const GateArgs a{c.logits, c.bias,        c.T,         c.E,         c.k,       c.groups, c.E / c.groups,
                     c.topk_groups, c.sigmoid, c.renorm, c.scale, c.idx, c.w, c.counts};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (zero) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(256);
        cudaError_t e = cudaLaunchKernelEx(&cfg, zero_counts_kernel, c.counts, c.E);
        if (e != cudaSuccess) return e;
    }
    cfg.dynamicSmemBytes = c.counts ? (size_t)c.E * 4 : 0;
    return with_per(c.E, [&](auto per) {
        constexpr int PER = decltype(per)::value;
        using G = GateShape<PER>;
        const int64_t blocks = ceil_div(c.T, G::WARPS), most = (int64_t)n_sm * G::BLOCKS;
        cfg.gridDim = dim3(several ? (unsigned)(blocks < most ? blocks : most) : 1);
        cfg.blockDim = dim3(32 * (several ? (unsigned)G::WARPS : (unsigned)c.T));
        return cudaLaunchKernelEx(&cfg, gate_kernel<PER>, a);
    });
}

cudaError_t launch_gate_grad(const float *logits, const int32_t *idx, const float *dw, int64_t T, int E, int k,
                             bool sigmoid, bool renorm, float scale, float *dlogits, int n_sm, cudaStream_t s)
{
    const int64_t blocks = ceil_div(T, kGradWarps);
    return with_per(E, [&](auto per) {
        constexpr int PER = decltype(per)::value;
        // as many blocks as the registers let an SM hold: each goes on to its next tokens
        const int64_t most = (int64_t)n_sm * kGradBlocks<PER>;
        gate_grad_kernel<PER><<<(unsigned)(blocks < most ? blocks : most), 32 * kGradWarps, 0, s>>>(
            logits, idx, dw, T, E, k, sigmoid, renorm, scale, dlogits);
        return cudaPeekAtLastError();
    });
}

}  // namespace moe
