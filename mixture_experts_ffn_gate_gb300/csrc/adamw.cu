// adamw.cu -- the norm of many gradients with the factor that clips it, and
// an AdamW step of many tensors with states in FP32 or in 8 bits.
//
//   norm = sqrt(sum g^2), factor = min(1, max / norm)
//   g' = factor g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   w = w - (lr wd w + lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// The tensors' addresses and sizes travel in the kernel's parameters, up to
// 256 (512) of them per launch, so a call copies nothing to the device first and
// may be captured.  A block takes one chunk of one tensor, found by bisection
// in the chunks' running count.  Both kernels read every byte once and write
// every byte once, and DRAM bounds them (us, and the floor at the copy rate):
// the norm of 1.5e8 FP32 gradients 88.7 (88.9); the step of as many BF16
// weights with FP32 masters and gradients, FP32 states 645 (667); with BF16
// gradients and 8-bit states 353 (357).  Where a step with 8-bit states moves
// few bytes, its instructions come near (BF16 weights and gradients without
// masters 279, 223): 64 an element at first, of which the block maxima by
// shuffles, a full division and the chunks' bounds are gone.  Many small
// tensors leave chunks part empty (192 of 501 to 261522 elements: 53, 45).
//
// 8-bit states: E4M3 codes of m / scale and sqrt(v) / scale, with one FP32
// scale per 256 elements, the largest magnitude times the rounded 1 / 448.  A
// floating code keeps small elements to 2^-4 of their size next to large ones.
// The scale is FP32 and not a power of two because it then follows the largest
// element, whose code stays 448, to a rounding: a block without gradients decays
// by the factor b1 or b2 through it, where a rounded scale would hold it.
// sqrt(v) needs half of v's range, and one that is not zero takes at least
// the lowest code, so that no m is divided by eps alone.  Codes are rounded to
// nearest, or at random where the betas are so close to 1 that a step changes a
// moment by less than half of its code's spacing and nearest would hold it where
// it is.  The numbers drawn cost instructions: BF16 weights with masters and BF16
// gradients 411 us (355 to nearest), without masters 381 (280), all FP32 424 (370).
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kSmallBatch = 16;   // tensors of a launch, in calls of few
constexpr int kStepBatch = 256;   // and in others: 21 KB of parameters
constexpr int kNormBatch = 512;   // 14 KB
constexpr int kThreads = 256;
constexpr int kBlock8 = 256;        // elements that share a scale: eight to a lane
constexpr int kChunk = 4096;        // elements of a block of the step
constexpr int kStepPerSm = 4;       // its blocks that an SM holds
constexpr int kNormChunk = 8192;    // elements that a block of the norm takes at a time
constexpr int kNormPerSm = 3;       // its blocks that an SM holds
constexpr int kNormBlocks = 512;    // its partial sums per launch, at most
constexpr float kTop = 448.0f;      // the largest E4M3 value
constexpr float kLowest = 0.001953125f;  // the smallest, 2^-9
constexpr float kNormal = 0.015625f;     // the smallest with a full mantissa, 2^-6
constexpr float kShrink = 5.421010862427522e-20f;  // 2^-64

// The tensors of one launch; first[i] is the chunks before tensor i.
template <typename Tensor, int CAP>
struct Batch {
    Tensor t[CAP];
    uint32_t first[CAP + 1];
    int count;
};

// Which tensor a chunk belongs to.
template <typename B>
__device__ __forceinline__ int find_tensor(const B &b, uint32_t chunk)
{
    int lo = 0, hi = b.count;  // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (b.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------- elements
// N consecutive elements from `e` on as they are kept, FP32 or BF16, zero
// from n on; FULL: there are N.
template <typename T, int N>
struct Raw;

template <int N>
struct Raw<float, N> {
    float4 q[N / 4];

    template <bool FULL>
    __device__ __forceinline__ void load(const float *p, int e, int n)
    {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            if (FULL || e + N <= n) {
                q[i] = *reinterpret_cast<const float4 *>(p + e + 4 * i);
            } else {
                const int at = e + 4 * i;
                q[i].x = at < n ? p[at] : 0.0f;
                q[i].y = at + 1 < n ? p[at + 1] : 0.0f;
                q[i].z = at + 2 < n ? p[at + 2] : 0.0f;
                q[i].w = at + 3 < n ? p[at + 3] : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[N]) const
    {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) v[4 * i] = q[i].x, v[4 * i + 1] = q[i].y, v[4 * i + 2] = q[i].z, v[4 * i + 3] = q[i].w;
    }
};

template <int N>
struct Raw<__nv_bfloat16, N> {
    uint32_t q[N / 2];

    template <bool FULL>
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int e, int n)
    {
        if (FULL || e + N <= n) {
            if constexpr (N == 8) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p + e);
                q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(p + e);
                q[0] = x.x, q[1] = x.y;
            }
        } else {
            const uint16_t *const bits = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const int at = e + 2 * i;
                q[i] = (at < n ? bits[at] : 0u) | (at + 1 < n ? (uint32_t)bits[at + 1] << 16 : 0u);
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[N]) const
    {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) v[2 * i] = bf16lo(q[i]), v[2 * i + 1] = bf16hi(q[i]);
    }
};

template <int N, bool FULL>
__device__ __forceinline__ void store_n(float *p, int e, int n, const float (&v)[N])
{
    if (FULL || e + N <= n) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4 *>(p + e + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e + i < n) p[e + i] = v[i];
    }
}

template <int N, bool FULL>
__device__ __forceinline__ void store_n(__nv_bfloat16 *p, int e, int n, const float (&v)[N])
{
    if (FULL || e + N <= n) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&q);
        }
        if constexpr (N == 8)
            *reinterpret_cast<uint4 *>(p + e) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(p + e) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e + i < n) p[e + i] = __float2bfloat16_rn(v[i]);
    }
}

// Eight E4M3 codes from `e` on, and their values without a scale.
template <bool FULL>
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int e, int n)
{
    uint2 w = make_uint2(0u, 0u);
    if (FULL || e + 8 <= n) {
        w = *reinterpret_cast<const uint2 *>(p + e);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < n) (i < 4 ? w.x : w.y) |= (uint32_t)p[e + i] << (8 * (i & 3));
    }
    return w;
}

__device__ __forceinline__ void unpack_codes(const uint2 &w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = ((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xffffu;
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t *p, int e, int n, const float (&v)[8])
{
    uint2 w = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        (i < 2 ? w.x : w.y) |= two << (16 * (i & 1));
    }
    if (FULL || e + 8 <= n) {
        *reinterpret_cast<uint2 *>(p + e) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < n) p[e + i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
}

// ---------------------------------------------------------------- norm
using NormBatch = Batch<TensorRef, kNormBatch>;
using NormBatchSmall = Batch<TensorRef, kSmallBatch>;

// A block's sums of squares of its chunks: of the elements and of the
// elements times 2^-64, which holds where the first one is beyond FP32.  Few
// blocks with eight 16-byte loads of a thread in flight: six blocks per SM with
// four took 8.3 us for 1.6e6 elements (5.2) and 21 for 1.8e7 (16.6).
template <typename B>
__global__ void __launch_bounds__(kThreads, kNormPerSm) grad_norm_kernel(const __grid_constant__ B b, float2 *partial)
{
    __shared__ float2 part[kThreads / 32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    float s[4] = {}, r[4] = {};
    auto add = [&](const float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = fmaf(v[i], v[i], s[i]);
            const float small = v[i] * kShrink;
            r[i] = fmaf(small, small, r[i]);
        }
    };
    auto pass = [&](auto *p, int n, auto full) {
        constexpr bool FULL = decltype(full)::value;
        constexpr int FLIGHT = kNormChunk / (kThreads * 4);
        Raw<std::remove_const_t<std::remove_pointer_t<decltype(p)>>, 4> raw[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) raw[u].template load<FULL>(p, (u * kThreads + threadIdx.x) * 4, n);
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            float v[4];
            raw[u].get(v);
            add(v);
        }
    };
    auto run = [&](const auto *p, int64_t left) {
        if (left >= kNormChunk)
            pass(p, kNormChunk, std::true_type());
        else
            pass(p, (int)left, std::false_type());
    };
    const uint32_t chunks = b.first[b.count];
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int k = find_tensor(b, c);
        const int64_t at = (int64_t)(c - b.first[k]) * kNormChunk, left = b.t[k].n - at;
        if (b.t[k].f32)
            run((const float *)b.t[k].data + at, left);
        else
            run((const __nv_bfloat16 *)b.t[k].data + at, left);
    }
    const float x = warp_sum((s[0] + s[1]) + (s[2] + s[3])), y = warp_sum((r[0] + r[1]) + (r[2] + r[3]));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = make_float2(x, y);
    __syncthreads();
    if (warp == 0) {
        const float2 v = lane < kThreads / 32 ? part[lane] : make_float2(0.0f, 0.0f);
        const float2 sums = make_float2(warp_sum(v.x), warp_sum(v.y));
        if (lane == 0) partial[blockIdx.x] = sums;
    }
}

__device__ __forceinline__ double warp_sum64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__global__ void __launch_bounds__(kThreads) norm_factor_kernel(const float2 *partial, int n, float max_norm,
                                                               float *out)
{
    __shared__ double2 part[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::griddep_wait();
    double x = 0.0, y = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) x += (double)partial[i].x, y += (double)partial[i].y;
    x = warp_sum64(x), y = warp_sum64(y);
    if (lane == 0) part[warp] = make_double2(x, y);
    __syncthreads();
    if (warp > 0) return;
    x = warp_sum64(lane < kThreads / 32 ? part[lane].x : 0.0);
    y = warp_sum64(lane < kThreads / 32 ? part[lane].y : 0.0);
    if (lane == 0) {
        const float norm = (float)(isinf(x) ? sqrt(y) * 18446744073709551616.0 : sqrt(x));
        out[0] = norm;
        out[1] = !isfinite(norm) ? NAN : norm > max_norm ? max_norm / norm : 1.0f;
    }
}

// ---------------------------------------------------------------- the step
using StepBatch = Batch<AdamWTensor, kStepBatch>;
using StepBatchSmall = Batch<AdamWTensor, kSmallBatch>;

__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What an element's update takes.
struct Element {
    float b1, a1, b2, a2;  // the betas and 1 - them
    float g_scale, minus_decay, minus_step, root, eps;

    // m, v and w after the step; returns sqrt(v).  The moments' products and
    // sums are rounded one by one: an 8-bit code next to a tie goes by their
    // last bit, which then is the formula's in FP32 and not a contraction's.
    // The reciprocal's unit in the last place is small against w's (it is zero
    // where sqrt(v) is beyond 2^126, which takes gradients whose square is
    // infinite; below 2^-126, where it would be infinite, no denominator comes:
    // sqrt(v) is zero or above 2^-75, and eps is scaled).  The decay is subtracted with the step, and w rounded once: a
    // factor 1 - lr wd would be rounded to 2^-24, which is a tenth of an lr wd
    // of 1e-6.
    __device__ __forceinline__ float operator()(float g, float &m, float &v, float &w) const
    {
        g = __fmul_rn(g, g_scale);
        m = __fadd_rn(__fmul_rn(b1, m), __fmul_rn(a1, g));
        v = __fadd_rn(__fmul_rn(b2, v), __fmul_rn(__fmul_rn(a2, g), g));
        const float r = __fsqrt_rn(v);
        w += fmaf(minus_decay, w, minus_step * (m * reciprocal(fmaf(r, root, eps))));
        return r;
    }
};

// A chunk of a tensor: n elements from each address on.
template <typename W, typename G>
struct Chunk {
    W *w;
    float *master;
    const G *grad;
    void *m, *v;
    float *m_scale, *v_scale;
    int n;
};

template <bool MASTER, typename W, typename G>
__device__ __forceinline__ const auto *source(const Chunk<W, G> &c)
{
    if constexpr (MASTER)
        return (const float *)c.master;
    else
        return (const W *)c.w;
}

// FP32 states: four elements per thread at a time, two such pieces in flight
// (with one 671 us where this takes 645, with four 659).
template <bool MASTER, bool FULL, typename W, typename G>
__device__ __forceinline__ void step_chunk(const Chunk<W, G> &c, const Element &el)
{
    constexpr int FLIGHT = 2;
    float *const ms = (float *)c.m, *const vs = (float *)c.v;
    const int n = FULL ? kChunk : c.n;
    for (int e = threadIdx.x * 4; e < n; e += kThreads * 4 * FLIGHT) {
        Raw<G, 4> rg[FLIGHT];
        Raw<std::remove_const_t<std::remove_pointer_t<decltype(source<MASTER>(c))>>, 4> rw[FLIGHT];
        Raw<float, 4> rm[FLIGHT], rv[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int i = e + u * kThreads * 4;
            rg[u].template load<FULL>(c.grad, i, n);
            rm[u].template load<FULL>(ms, i, n);
            rv[u].template load<FULL>(vs, i, n);
            rw[u].template load<FULL>(source<MASTER>(c), i, n);
        }
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int i = e + u * kThreads * 4;
            float g[4], m[4], v[4], w[4];
            rg[u].get(g), rm[u].get(m), rv[u].get(v), rw[u].get(w);
#pragma unroll
            for (int q = 0; q < 4; ++q) el(g[q], m[q], v[q], w[q]);
            store_n<4, FULL>(ms, i, n, m);
            store_n<4, FULL>(vs, i, n, v);
            if (MASTER) store_n<4, FULL>(c.master, i, n, w);
            store_n<4, FULL>(c.w, i, n, w);
        }
    }
}

// Numbers drawn for a lane's elements, from the step, the tensor and the
// element's place alone: a hash of those (multiplications by odd fractions of
// square roots and the golden ratio, with shifts), then one linear congruential
// step (Knuth, The Art of Computer Programming 2, 3.3.4) per number, whose upper
// 20 bits are taken.
struct Draws {
    uint32_t x;

    static __device__ __forceinline__ uint32_t mix(uint32_t h)
    {
        h = (h ^ (h >> 16)) * 0x9e3779b9u;
        h = (h ^ (h >> 15)) * 0xbb67ae85u;
        return h ^ (h >> 16);
    }
    __device__ __forceinline__ Draws(uint32_t key, int64_t block, int lane)
        : x(mix(mix(key ^ (uint32_t)(block >> 32) * 0x6a09e667u) + (uint32_t)block * 32u + lane))
    {
    }
    __device__ __forceinline__ uint32_t next() { return (x = x * 1664525u + 1013904223u) >> 12; }
};

// x, at most 448 and a rounding, as one of the two E4M3 numbers next to it, the
// nearer one the likelier, so that its mean is x.  Their distance is 2^20 units of
// x's last place, or 2^-9 below 2^-6; r: 20 bits.
__device__ __forceinline__ float round_at_random(float x, uint32_t r)
{
    const float a = fabsf(x), up = a < kNormal ? kNormal : 0.0f, t = a + up;
    const float q = __uint_as_float((__float_as_uint(t) + r) & 0xfff00000u) - up;
    return copysignf(t <= kTop ? q : a, x);  // a NaN stays one
}

// The scale of a warp's 256 values and what they are over it, rounded once:
// with the rounded reciprocal y of the scale, q = x y, r = x - q scale (exact)
// and q + r y is the rounded quotient (Markstein's division by a multiply and
// a correction, IBM J. Res. Dev. 34, 1990).  x y alone is off by a unit now
// and then, and takes other codes next to ties.
__device__ __forceinline__ float scale_block(float (&x)[8], bool up)
{
    float top = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) top = fmaxf(top, fabsf(x[q]));
    // numbers from zero on are ordered as their bits are
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    const float scale = fmaxf(__fmul_rn(top, 1.0f / kTop), 1.17549435e-38f), inv = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = x[i] * inv, r = fmaf(-q, scale, x[i]);
        x[i] = up && x[i] > 0.0f ? fmaxf(fmaf(r, inv, q), kLowest) : fmaf(r, inv, q);
    }
    return scale;
}

// 8-bit states: a warp takes 256 elements, a scale's block, eight to a lane.
// The loads of its two blocks of a chunk come before the first one's work: with
// one block at a time and bounds on every access 519 us where this takes 353.
// Four blocks per SM leave 64 registers, which cost spills where weights and
// gradients are FP32 (371 us; with three blocks 356) and bring more elsewhere
// (353; 366).  RANDOM: codes are rounded at random, by the key and the place of
// the chunk's first block.
template <bool MASTER, bool FULL, bool RANDOM, typename W, typename G>
__device__ __forceinline__ void step_chunk_8bit(const Chunk<W, G> &c, const Element &el, uint32_t key, int64_t place)
{
    const int lane = threadIdx.x & 31, n = FULL ? kChunk : c.n;
    uint8_t *const ms = (uint8_t *)c.m, *const vs = (uint8_t *)c.v;
    constexpr int WARPS = kThreads / 32, FLIGHT = kChunk / kBlock8 / WARPS;
    // all that the warp reads of the chunk, as it is kept
    Raw<G, 8> rg[FLIGHT];
    Raw<std::remove_const_t<std::remove_pointer_t<decltype(source<MASTER>(c))>>, 8> rw[FLIGHT];
    uint2 rm[FLIGHT], rv[FLIGHT];
    float m_scales[FLIGHT], v_scales[FLIGHT];
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
        const int s = (threadIdx.x >> 5) + u * WARPS, e = s * kBlock8 + lane * 8;
        rg[u].template load<FULL>(c.grad, e, n);
        rm[u] = load_codes<FULL>(ms, e, n);
        rv[u] = load_codes<FULL>(vs, e, n);
        rw[u].template load<FULL>(source<MASTER>(c), e, n);
        const bool in = FULL || s * kBlock8 < n;
        m_scales[u] = in ? c.m_scale[s] : 0.0f;
        v_scales[u] = in ? c.v_scale[s] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
        const int s = (threadIdx.x >> 5) + u * WARPS, e = s * kBlock8 + lane * 8;
        if (!FULL && s * kBlock8 >= n) break;
        float g[8], m[8], v[8], w[8];
        rg[u].get(g);
        rw[u].get(w);
        unpack_codes(rm[u], m);
        unpack_codes(rv[u], v);
        const float m_scale = m_scales[u], v_scale = v_scales[u];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            m[q] *= m_scale;
            v[q] *= v_scale;
            v[q] *= v[q];
            v[q] = el(g[q], m[q], v[q], w[q]);
        }
        if (MASTER) store_n<8, FULL>(c.master, e, n, w);
        store_n<8, FULL>(c.w, e, n, w);
        // elements past the tensor's end are zero and stay so: they raise no scale
        const float m_new = scale_block(m, false), v_new = scale_block(v, !RANDOM);
        if constexpr (RANDOM) {
            Draws draws(key, place + s, lane);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                m[q] = round_at_random(m[q], draws.next());
                const float code = round_at_random(v[q], draws.next());
                v[q] = v[q] > 0.0f ? fmaxf(code, kLowest) : code;
            }
        }
        store_codes<FULL>(ms, e, n, m);
        store_codes<FULL>(vs, e, n, v);
        if (lane == 0) c.m_scale[s] = m_new, c.v_scale[s] = v_new;
    }
}

template <bool RANDOM, bool MASTER, typename W, typename G>
__device__ __forceinline__ void step_any(const AdamWTensor &t, int64_t at, const Element &el, uint32_t key)
{
    const int64_t left = t.n - at;
    Chunk<W, G> c{(W *)t.w + at, MASTER ? t.master + at : nullptr, (const G *)t.grad + at, nullptr, nullptr, nullptr, nullptr,
                  (int)(left < kChunk ? left : kChunk)};
    if (t.bits8) {
        c.m = (uint8_t *)t.m + at, c.v = (uint8_t *)t.v + at;
        c.m_scale = t.m_scale + at / kBlock8, c.v_scale = t.v_scale + at / kBlock8;
        c.n == kChunk ? step_chunk_8bit<MASTER, true, RANDOM>(c, el, key, at / kBlock8)
                      : step_chunk_8bit<MASTER, false, RANDOM>(c, el, key, at / kBlock8);
    } else {
        c.m = (float *)t.m + at, c.v = (float *)t.v + at;
        c.n == kChunk ? step_chunk<MASTER, true>(c, el) : step_chunk<MASTER, false>(c, el);
    }
}

template <bool RANDOM, bool MASTER, typename W>
__device__ __forceinline__ void step_grad(const AdamWTensor &t, int64_t at, const Element &el, uint32_t key)
{
    t.grad_f32 ? step_any<RANDOM, MASTER, W, float>(t, at, el, key)
               : step_any<RANDOM, MASTER, W, __nv_bfloat16>(t, at, el, key);
}

// A factor that is no number leaves everything as it is.
template <typename B, bool RANDOM>
__global__ void __launch_bounds__(kThreads, kStepPerSm) adamw_kernel(const __grid_constant__ B b, const AdamWScalars sc)
{
    ptx::griddep_wait();
    const uint32_t chunk = blockIdx.x;
    const float factor = sc.grad_scale ? *sc.grad_scale : 1.0f;
    if (!isfinite(factor)) return;
    const float2 corrections = sc.corrections ? *sc.corrections : sc.host;
    const int k = find_tensor(b, chunk);
    const AdamWTensor &t = b.t[k];
    const int64_t at = (int64_t)(chunk - b.first[k]) * kChunk;
    const float lr = (sc.lr_at ? *sc.lr_at : sc.lr) * t.lr_factor;
    const Element el{sc.beta1, sc.one_minus1, sc.beta2, sc.one_minus2, factor, -lr * t.weight_decay,
                     -lr * corrections.x * sc.den_scale, corrections.y * sc.den_scale, sc.eps};
    uint32_t key = 0;
    if constexpr (RANDOM) key = Draws::mix(Draws::mix(sc.step_at ? (uint32_t)*sc.step_at : sc.step) + t.index);
    if (t.master)
        t.w_f32 ? step_grad<RANDOM, true, float>(t, at, el, key) : step_grad<RANDOM, true, __nv_bfloat16>(t, at, el, key);
    else
        t.w_f32 ? step_grad<RANDOM, false, float>(t, at, el, key)
                : step_grad<RANDOM, false, __nv_bfloat16>(t, at, el, key);
}

// The step's number from device memory: one more than it says, unless the
// step is left out; with it the corrections 1 / (1 - b1^t) and
// 1 / sqrt(1 - b2^t).
__global__ void adamw_count_kernel(int32_t *step, const float *grad_scale, double beta1, double beta2, float2 *out)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if (grad_scale && !isfinite(*grad_scale)) return;
    const int32_t t = *step + 1;
    *step = t;
    *out = make_float2((float)(1.0 / (1.0 - pow(beta1, (double)t))), (float)(1.0 / sqrt(1.0 - pow(beta2, (double)t))));
}

// Calls f with batches of the tensors that have elements, in their order.
template <typename B, typename Tensor, typename F>
cudaError_t in_batches(const Tensor *tensors, int count, int cap, int64_t chunk_size, F f)
{
    B b;
    b.count = 0;
    b.first[0] = 0;
    for (int i = 0; i < count; ++i) {
        const int64_t chunks = ceil_div(tensors[i].n, chunk_size);
        if (chunks == 0) continue;
        if (b.count == cap) {
            const cudaError_t e = f(b);
            if (e != cudaSuccess) return e;
            b.count = 0;
        }
        b.t[b.count] = tensors[i];
        b.first[b.count + 1] = b.first[b.count] + (uint32_t)chunks;
        ++b.count;
    }
    return b.count ? f(b) : cudaSuccess;
}

cudaLaunchConfig_t early(cudaLaunchAttribute *attr, cudaStream_t s)
{
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.blockDim = dim3(kThreads);
    return cfg;
}

}  // namespace

// kNormBlocks sums for each launch of kNormBatch tensors.
size_t grad_norm_workspace_bytes(int64_t count)
{
    const int64_t launches = count < 1 ? 1 : ceil_div(count, (int64_t)kNormBatch);
    return (size_t)(launches * kNormBlocks) * sizeof(float2);
}

cudaError_t launch_grad_norm(const TensorRef *grads, int count, float max_norm, float *out, void *workspace, int n_sm,
                             cudaStream_t s)
{
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = early(&attr, s);
    float2 *const partial = (float2 *)workspace;
    int used = 0;
    auto launch = [&](const auto &b) {
        using B = std::remove_cv_t<std::remove_reference_t<decltype(b)>>;
        const uint32_t chunks = b.first[b.count], most = (uint32_t)(n_sm * kNormPerSm < kNormBlocks ? n_sm * kNormPerSm : kNormBlocks);
        cfg.gridDim = dim3(chunks < most ? chunks : most);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, grad_norm_kernel<B>, b, partial + used);
        used += (int)cfg.gridDim.x;
        return e;
    };
    const cudaError_t e = count <= kSmallBatch
                              ? in_batches<NormBatchSmall>(grads, count, kSmallBatch, kNormChunk, launch)
                              : in_batches<NormBatch>(grads, count, kNormBatch, kNormChunk, launch);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(1);
    return cudaLaunchKernelEx(&cfg, norm_factor_kernel, (const float2 *)partial, used, max_norm, out);
}

cudaError_t launch_adamw(const AdamWTensor *tensors, int count, AdamWScalars sc, double beta1, double beta2,
                         int32_t *step, bool random, void *workspace, cudaStream_t s)
{
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = early(&attr, s);
    if (step) {
        cfg.gridDim = cfg.blockDim = dim3(1);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, adamw_count_kernel, step, sc.grad_scale, beta1, beta2,
                                                 (float2 *)workspace);
        if (e != cudaSuccess) return e;
        cfg.blockDim = dim3(kThreads);
        sc.corrections = (const float2 *)workspace;
        sc.step_at = step;
    }
    auto launch = [&](const auto &b) {
        using B = std::remove_cv_t<std::remove_reference_t<decltype(b)>>;
        cfg.gridDim = dim3(b.first[b.count]);
        return cudaLaunchKernelEx(&cfg, random ? adamw_kernel<B, true> : adamw_kernel<B, false>, b, (const AdamWScalars)sc);
    };
    return count <= kSmallBatch ? in_batches<StepBatchSmall>(tensors, count, kSmallBatch, kChunk, launch)
                                : in_batches<StepBatch>(tensors, count, kStepBatch, kChunk, launch);
}

}  // namespace moe
