// rms_norm.cu -- residual addition with root-mean-square norm, in BF16 and
// MXFP8, and its gradients.
//
//   forward   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//   backward  n = h r,  g = dy w,  dh = r (g - n mean(g n)) + dres,
//             dw = sum over the rows of dy n
//
// Both are bound by memory: every input and output element moves once.  A
// block holds one row in registers between its sum and its outputs, so the
// row is read once; the weight is read once per block and kept in registers
// over the rows the block walks.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

// Elements per thread (of single ones, norm_ept).  VEC consecutive ones are one access: 8 (16 bytes of
// BF16) where H is a multiple of 8, so that every row starts on 16 bytes, 4
// where it is one of 4; other H take single elements, coalesced over the block.
constexpr int kEpt = 16;
constexpr int kNormMaxH = 16384;  // 1024 threads of kEpt elements
static_assert(kNormMaxH == 1024 * kEpt, "one row per block");

template <int VEC>
__device__ __forceinline__ void load_row(const float *p, float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        const float4 a = ld_nc_f4(p), b = ld_nc_f4(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (VEC == 4) {
        const float4 a = ld_nc_f4(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
        v[0] = __ldg(p);
    }
}

template <int VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        unpack8(ld_nc16(p), v);
    } else if constexpr (VEC == 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
        v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
    } else {
        v[0] = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(p)) << 16);
    }
}

// The same through plain loads: for rows that the call may also write (an
// output in the place of its input).
template <int VEC>
__device__ __forceinline__ void load_row_rw(const float *p, float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (VEC == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
        v[0] = *p;
    }
}

template <int VEC>
__device__ __forceinline__ void load_row_rw(const __nv_bfloat16 *p, float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        unpack8(*reinterpret_cast<const uint4 *>(p), v);
    } else if constexpr (VEC == 4) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
    } else {
        v[0] = __bfloat162float(*p);
    }
}

template <int VEC>
__device__ __forceinline__ void store_row(float *p, const float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *p = v[0];
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

template <int VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&v)[VEC])
{
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                                   bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    else if constexpr (VEC == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    else
        *p = __float2bfloat16_rn(v[0]);
}

// Block sums of N values; every thread gets them, the order depends only on
// the block's size.  `part` [2][N][32]: the two halves are used in turn, so
// one barrier per call is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*part)[32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    warp_sum_n(v);
    if (warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? part[i][lane] : 0.0f;
    warp_sum_n(v);
}

struct NormArgs {
    const void *x, *residual;
    const float *weight;
    float eps, inv_h;
    int64_t T;
    int H;
    void *h_out;
    __nv_bfloat16 *y;
    uint8_t *codes, *scales;
    int scale_stride;
};

// Forward.  XT, RT: types of x and of the residual (RT void: none).
template <typename XT, typename RT, int VEC, bool MX, int EPT = kEpt>
__global__ void __launch_bounds__(1024, EPT == 4 ? 2 : 1) norm_kernel(const NormArgs a)
{
    constexpr int NV = EPT / VEC;
    __shared__ float part[2][1][32];
    const int H = a.H;
    float w[NV][VEC];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int i = (c * (int)blockDim.x + (int)threadIdx.x) * VEC;
        if (i < H) load_row<VEC>(a.weight + i, w[c]);
    }
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const int64_t row = t * H;
        float h[NV][VEC];
        float sq[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int i = (c * (int)blockDim.x + (int)threadIdx.x) * VEC;
            if (i < H) {
                load_row<VEC>((const XT *)a.x + row + i, h[c]);
                if constexpr (!std::is_void_v<RT>) {
                    float r[VEC];
                    load_row_rw<VEC>((const RT *)a.residual + row + i, r);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) h[c][q] += r[q];
                }
#pragma unroll
                for (int q = 0; q < VEC; ++q) sq[0] = fmaf(h[c][q], h[c][q], sq[0]);
            }
        }
        // after the row's loads, which the compiler may not move past a store
        // that could be to the residual (4097 columns: 453 us with the stores
        // between them, 277 so)
        if constexpr (!std::is_void_v<RT>)
            if (a.h_out)
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    const int i = (c * (int)blockDim.x + (int)threadIdx.x) * VEC;
                    if (i < H) store_row<VEC>((RT *)a.h_out + row + i, h[c]);
                }
        block_sum(sq, part[turn]);
        // r, and what its roundings leave, r (1 - v r^2) / 2: one error for all
        // of a row's elements turns 422 8-bit codes of 10 x 8192 x 7168 away
        // from the exact ones, with the rest 338 (the other roundings alone 322,
        // at 5% more time); no difference in time
        const float v = fmaf(sq[0], a.inv_h, a.eps), r = 1.0f / sqrtf(v), r2 = r * r;
        const float rest = 0.5f * r * (fmaf(-v, r2, 1.0f) - v * fmaf(r, r, -r2));
        const float r_lo = rest - rest == 0.0f ? rest : 0.0f;  // for v of 0, an infinity or a NaN
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int i = (c * (int)blockDim.x + (int)threadIdx.x) * VEC;
            float y[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) y[q] = i < H ? fmaf(h[c][q], r, h[c][q] * r_lo) * w[c][q] : 0.0f;
            if (a.y && i < H) store_row<VEC>(a.y + row + i, y);
            if constexpr (MX) {
                // a block of 32 elements is four neighbouring lanes, all inside
                // the row or all past it; the largest magnitude as an integer,
                // which orders NaN above infinity
                uint32_t top = 0;
#pragma unroll
                for (int q = 0; q < VEC; ++q) top = max(top, __float_as_uint(y[q]) & 0x7fffffffu);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // floor(log2 top) - 8, biased by 127
                const int e = (int)(top >> 23);
                const uint32_t s = top == 0 ? 127u : e == 255 ? 255u : (uint32_t)max(1, e - 8);
                if (i < H) {
                    const float f = __uint_as_float((254u - min(s, 253u)) << 23);  // 2^(127 - s)
                    uint32_t code[2];
#pragma unroll
                    for (int q = 0; q < VEC; q += 4) {
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[q] * f, y[q + 1] * f),
                                                                     __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[q + 2] * f, y[q + 3] * f),
                                                                     __NV_SATFINITE, __NV_E4M3);
                        code[q / 4] = lo | (hi << 16);
                    }
                    *reinterpret_cast<uint2 *>(a.codes + row + i) = make_uint2(code[0], code[1]);
                    if ((threadIdx.x & 3) == 0) a.scales[t * a.scale_stride + i / 32] = (uint8_t)s;
                }
            }
        }
        if constexpr (MX) {
            const int pad = H / 32 + (int)threadIdx.x;
            if (pad < a.scale_stride) a.scales[t * a.scale_stride + pad] = 0;
        }
    }
}

struct NormGradArgs {
    const void *h, *dy, *dres;
    const float *weight;
    float eps, inv_h;
    int64_t T;
    int H;
    void *dh;
    float *partial;  // [gridDim.x][H]
};

// A piece of a row as it was loaded, VEC elements: half the registers for
// BF16 while it waits.
template <typename T, int VEC>
struct Raw {
    static_assert(VEC == 8 || VEC == 4);
    static constexpr int kWords = VEC * (int)sizeof(T) / 4;
    uint32_t v[kWords];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) v[i] = 0;
    }
    template <bool NC>
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (VEC == 8) {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const void *at = reinterpret_cast<const uint32_t *>(p) + i;
                const uint4 w = NC ? ld_nc16(at) : *reinterpret_cast<const uint4 *>(at);
                v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
            }
        } else if constexpr (sizeof(T) == 4) {
            const uint4 w = NC ? ld_nc16(p) : *reinterpret_cast<const uint4 *>(p);
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            v[0] = w.x, v[1] = w.y;
        }
    }
    __device__ __forceinline__ float get(int q) const
    {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(v[q]);
        else
            return q & 1 ? bf16hi(v[q / 2]) : bf16lo(v[q / 2]);
    }
};

// Backward.  A block walks rows blockIdx.x, blockIdx.x + gridDim.x, ... and
// keeps its columns' sums of dy n in registers; AHEAD loads the next row
// before it reduces this one, so a block of up to 512 threads always has a
// whole row (48 KB at H = 6144) on its way.
template <typename HT, typename GT, int VEC, bool AHEAD>
__global__ void __launch_bounds__(AHEAD ? 512 : 1024, 1) norm_grad_kernel(const NormGradArgs a)
{
    constexpr int NV = kEpt / VEC;
    __shared__ float part[2][2][32];
    const int H = a.H;
    struct Row {
        Raw<HT, VEC> h[NV], dres[NV];
        Raw<GT, VEC> dy[NV];
    };
    float w[NV][VEC], dw[NV][VEC];
    auto column = [&](int c) { return (c * (int)blockDim.x + (int)threadIdx.x) * VEC; };
    auto fetch = [&](int64_t t, Row &r) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int i = column(c);
            r.h[c].zero(), r.dy[c].zero(), r.dres[c].zero();
            if (i < H && t < a.T) {
                r.h[c].template load<true>((const HT *)a.h + t * H + i);
                r.dy[c].template load<true>((const GT *)a.dy + t * H + i);
                // dh may take the place of dres: plain loads
                if (a.dres) r.dres[c].template load<false>((const HT *)a.dres + t * H + i);
            }
        }
    };
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int i = column(c);
#pragma unroll
        for (int q = 0; q < VEC; ++q) w[c][q] = dw[c][q] = 0.0f;
        if (i < H) load_row<VEC>(a.weight + i, w[c]);
    }
    Row r;
    if (AHEAD) fetch(blockIdx.x, r);
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        Row next;
        fetch(AHEAD ? t + gridDim.x : t, AHEAD ? next : r);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float h = r.h[c].get(q);
                s[0] = fmaf(h, h, s[0]);
                s[1] = fmaf(r.dy[c].get(q) * w[c][q], h, s[1]);
            }
        block_sum(s, part[turn]);
        const float inv = 1.0f / sqrtf(fmaf(s[0], a.inv_h, a.eps));
        const float m = s[1] * a.inv_h * inv * inv;  // n mean(g n) = h m
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int i = column(c);
            float o[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float h = r.h[c].get(q), dy = r.dy[c].get(q);
                dw[c][q] = fmaf(dy, h * inv, dw[c][q]);
                o[q] = fmaf(inv, dy * w[c][q] - h * m, r.dres[c].get(q));
            }
            if (i < H) store_row<VEC>((HT *)a.dh + t * H + i, o);
        }
        if (AHEAD) r = next;
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int i = column(c);
        if (i < H) store_row<VEC>(a.partial + (int64_t)blockIdx.x * H + i, dw[c]);
    }
}

// The same for any H, an element at a time.  Kept in registers a row would
// spill (its 16-bit elements take a register each), so it is read again, from
// L1, for the outputs.
template <typename HT, typename GT, int EPT>
__global__ void __launch_bounds__(1024, EPT == 4 ? 2 : 1) norm_grad_any_kernel(const NormGradArgs a)
{
    __shared__ float part[2][2][32];
    const int H = a.H;
    const HT *h = (const HT *)a.h, *dres = (const HT *)a.dres;
    const GT *dy = (const GT *)a.dy;
    float w[EPT], dw[EPT];
#pragma unroll
    for (int c = 0; c < EPT; ++c) {
        const int i = c * (int)blockDim.x + (int)threadIdx.x;
        w[c] = i < H ? __ldg(a.weight + i) : 0.0f;
        dw[c] = 0.0f;
    }
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const int64_t row = t * H;
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < EPT; ++c) {
            const int i = c * (int)blockDim.x + (int)threadIdx.x;
            if (i < H) {
                float hv[1], g[1];
                load_row<1>(h + row + i, hv);
                load_row<1>(dy + row + i, g);
                s[0] = fmaf(hv[0], hv[0], s[0]);
                s[1] = fmaf(g[0] * w[c], hv[0], s[1]);
            }
        }
        block_sum(s, part[turn]);
        const float inv = 1.0f / sqrtf(fmaf(s[0], a.inv_h, a.eps));
        const float m = s[1] * a.inv_h * inv * inv;
#pragma unroll
        for (int c = 0; c < EPT; ++c) {
            const int i = c * (int)blockDim.x + (int)threadIdx.x;
            if (i < H) {
                float hv[1], g[1], o[1] = {0.0f};
                load_row<1>(h + row + i, hv);
                load_row<1>(dy + row + i, g);
                if (dres) load_row_rw<1>(dres + row + i, o);
                dw[c] = fmaf(g[0], hv[0] * inv, dw[c]);
                o[0] = fmaf(inv, g[0] * w[c] - hv[0] * m, o[0]);
                store_row<1>((HT *)a.dh + row + i, o);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < EPT; ++c) {
        const int i = c * (int)blockDim.x + (int)threadIdx.x;
        if (i < H) a.partial[(int64_t)blockIdx.x * H + i] = dw[c];
    }
}

// dweight[c] = sum over the blocks' partial rows.  A block takes 32 columns;
// its 32 warps take the rows in turn, then one warp adds the 32 sums in
// order.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float *__restrict__ partial, int parts, int H,
                                                            float *__restrict__ dweight)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (i < H)
        for (int p = warp; p < parts; p += 32) s += __ldg(partial + (int64_t)p * H + i);
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < H) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < 32; ++q) v += sums[q][lane];
        dweight[i] = v;
    }
}

// Single elements: as few per thread as a block of 1024 can hold the row with
// (more threads, and more loads in flight), 8 only where their block fills an
// SM (6.7e7 elements in rows of 1001, 3001, 4097 and 8191 with 4 / 8 / 16:
// forward 156 / 158 / 203, 189 / 231 / 215, - / 276 / 277, - / 183 / 217 us;
// gradient as chosen 233, 296, 437, about 400).
int norm_ept(int H)
{
    return H % 4 == 0 ? kEpt : H <= 4096 ? 4 : H > 6144 && H <= 8192 ? 8 : 16;
}

int norm_threads(int H)
{
    const int per = norm_ept(H), n = (H + per - 1) / per;
    return (n + 31) / 32 * 32;
}

template <typename XT, typename RT>
cudaError_t norm_launch(const NormArgs &a, bool mx, int grid, int threads, cudaStream_t s)
{
    if (mx)
        norm_kernel<XT, RT, 8, true><<<grid, threads, 0, s>>>(a);
    else if (a.H % 8 == 0)
        norm_kernel<XT, RT, 8, false><<<grid, threads, 0, s>>>(a);
    else if (a.H % 4 == 0)
        norm_kernel<XT, RT, 4, false><<<grid, threads, 0, s>>>(a);
    else if (norm_ept(a.H) == 4)
        norm_kernel<XT, RT, 1, false, 4><<<grid, threads, 0, s>>>(a);
    else if (norm_ept(a.H) == 8)
        norm_kernel<XT, RT, 1, false, 8><<<grid, threads, 0, s>>>(a);
    else
        norm_kernel<XT, RT, 1, false><<<grid, threads, 0, s>>>(a);
    return cudaPeekAtLastError();
}

template <typename HT, typename GT>
cudaError_t norm_grad_launch(const NormGradArgs &a, int grid, int threads, cudaStream_t s)
{
    if (a.H % 8 == 0) {
        if (threads <= 512)
            norm_grad_kernel<HT, GT, 8, true><<<grid, threads, 0, s>>>(a);
        else
            norm_grad_kernel<HT, GT, 8, false><<<grid, threads, 0, s>>>(a);
    } else if (a.H % 4 == 0) {
        if (threads <= 512)
            norm_grad_kernel<HT, GT, 4, true><<<grid, threads, 0, s>>>(a);
        else
            norm_grad_kernel<HT, GT, 4, false><<<grid, threads, 0, s>>>(a);
    } else if (norm_ept(a.H) == 4) {
        norm_grad_any_kernel<HT, GT, 4><<<grid, threads, 0, s>>>(a);
    } else if (norm_ept(a.H) == 8) {
        norm_grad_any_kernel<HT, GT, 8><<<grid, threads, 0, s>>>(a);
    } else {
        norm_grad_any_kernel<HT, GT, kEpt><<<grid, threads, 0, s>>>(a);
    }
    return cudaPeekAtLastError();
}

}  // namespace

bool norm_supported(int64_t H) { return H >= 1 && H <= kNormMaxH; }

// Rows of partial sums: enough blocks to fill the SMs where a row is short
// (128 columns: 643 us with 512 blocks, 197 so), 8 MB of them at most
int norm_grad_parts(int64_t T, int64_t H)
{
    const int64_t fit = (1 << 21) / H, most = fit < 512 ? 512 : fit > 4096 ? 4096 : fit;
    return (int)(T < most ? T : most);
}

cudaError_t launch_norm(const void *x, bool x_f32, const void *residual, bool res_f32, const float *weight, float eps,
                        int64_t T, int H, void *h_out, void *y, void *codes, void *scales, int n_sm, cudaStream_t s)
{
    const NormArgs a{x, residual, weight, eps, 1.0f / (float)H, T, H, h_out, (__nv_bfloat16 *)y, (uint8_t *)codes,
                     (uint8_t *)scales, mx_scale_bytes(H)};
    const int threads = norm_threads(H);
    const int64_t most = (int64_t)n_sm * (2048 / threads);
    const int grid = (int)(T < most ? T : most);
    const bool mx = codes != nullptr;
    if (!residual)
        return x_f32 ? norm_launch<float, void>(a, mx, grid, threads, s)
                     : norm_launch<__nv_bfloat16, void>(a, mx, grid, threads, s);
    if (res_f32)
        return x_f32 ? norm_launch<float, float>(a, mx, grid, threads, s)
                     : norm_launch<__nv_bfloat16, float>(a, mx, grid, threads, s);
    return x_f32 ? norm_launch<float, __nv_bfloat16>(a, mx, grid, threads, s)
                 : norm_launch<__nv_bfloat16, __nv_bfloat16>(a, mx, grid, threads, s);
}

cudaError_t launch_norm_grad(const void *h, bool h_f32, const float *weight, const void *dy, bool dy_f32,
                             const void *dres, float eps, int64_t T, int H, void *dh, float *dweight, float *partial,
                             int n_sm, cudaStream_t s)
{
    const NormGradArgs a{h, dy, dres, weight, eps, 1.0f / (float)H, T, H, dh, partial};
    const int threads = norm_threads(H);
    const int full = H % 4 == 0 ? 512 : norm_ept(H) == 4 ? 2048 : 1024;
    const int per_sm = threads >= full ? 1 : full / threads;
    int grid = norm_grad_parts(T, H);
    if (grid > n_sm * per_sm) grid = n_sm * per_sm;
    cudaError_t e;
    if (h_f32)
        e = dy_f32 ? norm_grad_launch<float, float>(a, grid, threads, s)
                   : norm_grad_launch<float, __nv_bfloat16>(a, grid, threads, s);
    else
        e = dy_f32 ? norm_grad_launch<__nv_bfloat16, float>(a, grid, threads, s)
                   : norm_grad_launch<__nv_bfloat16, __nv_bfloat16>(a, grid, threads, s);
    if (e != cudaSuccess) return e;
    norm_dweight_kernel<<<(H + 31) / 32, 1024, 0, s>>>(partial, grid, H, dweight);
    return cudaPeekAtLastError();
}

}  // namespace moe
