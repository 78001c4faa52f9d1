// kernels.h -- launchers of the library's kernels (internal to libmoeffn.so).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Grouped path: at most this many assignments (token rows) per GEMM N-chunk.
constexpr int kGemmChunkMax = 64;

// MXFP8 expert weights of a call -- E4M3 codes gq [E, 2I, H] and dq [E, H,
// I], E8M0 scales gs [E, 2I, mx_scale_bytes(H)] and ds [E, H,
// mx_scale_bytes(I)] -- for the decode kernels (the weight pointers are then
// not read).
struct FusedMx {
    const void *gq, *gs, *dq, *ds;
};
// Bytes per scale row for rows of K elements: K / 32 scales padded to 16.
constexpr int mx_scale_bytes(int K) { return (K / 32 + 15) / 16 * 16; }

// A routing that the caller passes instead of logits: [T, k] each.
struct Routing {
    const int32_t *idx;
    const float *w;
};

// routing.cu
cudaError_t routing_init_device();
// tag_size (nullable): the fused decode kernel's size word in a workspace
// that keeps its state; the router lowers it to tag_cap (the call's other
// regions start that many 64-bit words into the tag region).
cudaError_t launch_router(const float *logits, int T, int E, int k, int32_t *idx, float *w, int32_t *idx_copy,
                          float *w_copy, unsigned long long *tag_size, unsigned long long tag_cap, cudaStream_t s);
// logits [T, E] (and logits_copy, nullable) from x [T, H] and the router
// weights wr [E, H] (BF16) plus bias [E] (nullable): the exact sum rounded
// once to FP32
cudaError_t launch_router_gemv(const void *x, const void *wr, const float *bias, int T, int H, int E, float *logits,
                               float *logits_copy, cudaStream_t s);
size_t sort_smem_bytes(int E);
// pad > 1: every expert's segment rounded up to a multiple of pad rows (pad
// rows' perm = -1); counts (nullable): assignments per expert
cudaError_t launch_sort(const int32_t *idx, int n_assign, int E, int chunk_max, int32_t *offs, int32_t *perm,
                        int32_t *pos, int32_t *uexp, int32_t *ucount, int4 *chunks, int32_t *nchunks,
                        cudaStream_t s, int pad = 1, int32_t *counts = nullptr);
// w (nullable): without it the rows are summed unweighted
cudaError_t launch_combine(const float *z, const float *w, const int32_t *pos, int T, int H, int k, float *out,
                           int n_sm, cudaStream_t s, bool drops = false);

// decode.cu
cudaError_t decode_init_device();
int decode_down_tok_tile(int T, int k);
cudaError_t launch_decode_gate_up(const void *x, const void *wgu, const int32_t *uexp, const int32_t *ucount,
                                  const int32_t *offs, const int32_t *perm, int T, int H, int I, int E, int k,
                                  int warps, float *act, const FusedMx *mxw, cudaStream_t s);
cudaError_t launch_decode_down(const float *act, const void *wd, const float *w, const int32_t *uexp,
                               const int32_t *ucount, const int32_t *offs, const int32_t *perm, int T, int H,
                               int I, int k, int warps, float *out, const FusedMx *mxw, cudaStream_t s);

// decode_fused.cu: a decode step of up to four tokens in one cooperative
// kernel.  act: [T*k][I] FP32 scratch; flags: kDecodeFusedFlagWords 64-bit
// words and act_tag: the tag region, both kept between calls (any initial
// contents); act_tag may be null (every call then meets at a grid barrier).
// Word kDecodeFusedSizeWord of flags counts the leading words of the tag
// region known to hold only zeros and tags.  Every call on a workspace that
// keeps state lowers it to its tag_cap, the 64-bit words of the tag region
// before the call's first other region: the fused kernel itself, and the
// router kernel on the other paths.
constexpr int kMaxGridCtas = 1024;
constexpr int kDecodeFusedFlagWords = kMaxGridCtas + 32;
constexpr int kDecodeFusedSizeWord = kMaxGridCtas + 2;
cudaError_t decode_fused_init_device();
cudaError_t read_decode_fused_fault_word(uint32_t *flags, bool clear);
// mx: with MXFP8 expert weights (FusedMx) instead of BF16 ones
bool decode_fused_supported(int T, int H, int I, int E, int k, int n_sm, bool mx = false);
// the same for a call that passes the router weights (its projection's
// scratch must fit too)
bool decode_fused_router_supported(int T, int H, int I, int E, int k, int n_sm);
size_t decode_fused_tag_words(int k, int I);
// exchange_out (nullable, device): CTA 0 stores 1 when the call met at the
// grid barrier, 2 when it exchanged tagged act words.  wait_ns bounds every
// wait; skip_arrival (a test hook) makes the last CTA skip its arrival at
// the grid barrier, so the call's waits run out and it reports a fault.
// router (nullable): the call passes the router weights instead of logits;
// the kernel computes the logits itself, exchanges them through ltag
// (kDecodeFusedLogitCopies copies of T*E words of 16 bytes, any initial
// contents) and writes them to logits_out (nullable).  `logits` is then not
// read.
constexpr int kDecodeFusedLogitCopies = 8;
struct FusedRouter {
    const void *wr;       // [E, H] BF16
    const float *bias;    // [E], nullable
    unsigned long long *ltag;
    float *logits_out;
};
// routing (nullable): the caller's routing instead of logits (then not read);
// not together with router.
// mxw (nullable): MXFP8 expert weights (FusedMx) instead of wgu/wd (then
// not read); not together with router.  prefetch_inputs: fetch x and the
// logits into L2 while the previous launch drains (device memory only).
cudaError_t launch_decode_fused(const void *x, const float *logits, const void *wgu, const void *wd, int T, int H,
                                int I, int E, int k, int n_sm, float *act, unsigned long long *act_tag,
                                unsigned long long tag_cap, unsigned long long *flags, int32_t *idx_out, float *w_out,
                                float *out, int32_t *exchange_out, unsigned long long wait_ns, int skip_arrival,
                                const FusedRouter *router, const FusedMx *mxw, bool prefetch_inputs,
                                cudaStream_t s, const Routing *routing = nullptr);
constexpr unsigned long long kDecodeFusedWaitNs = 2000000000ull;  // default bound of its waits

// moe_ffn_api.cu: an identifier of the calling thread's current CUDA
// context (0 if none can be had), so that per-device set-up is redone in a
// new context, e.g. after cudaDeviceReset.
unsigned long long current_context_id();

// grouped_gemm.cu
// seg, or a third term (lo2) of an operand or a result: the instances that add
// segments of K in FP32 and take FP32 operands as three BF16 terms (the calls
// that take the routing from the caller)
cudaError_t gemm_init_device();
bool gemm_supported(int H, int I, int E);
// gate_up reads the chunk's token rows from x [T, H] by perm (row p of the
// sorted order is token perm[p] / k)
cudaError_t launch_gemm_gate_up(const void *x, const int32_t *perm, int k, const void *wgu, const int4 *chunks,
                                const int32_t *nchunks, const int32_t *offs, int n_assign, int H, int I, int E,
                                void *act_hi, void *act_lo, int ctas, cudaStream_t s, void *act_lo2 = nullptr);
cudaError_t launch_gemm_down(const void *act_hi, const void *act_lo, const void *wd, const int4 *chunks,
                             const int32_t *nchunks, const int32_t *offs, int n_assign, int H, int I, int E, float *z,
                             int ctas, cudaStream_t s, const void *act_lo2 = nullptr);
cudaError_t read_fault_word(uint32_t *flags, bool clear);
// The same two GEMMs with MXFP8 weights: E4M3 codes gq [E, 2I, H] / dq
// [E, H, I] and E8M0 scales gs [E, 2I, mx_scale_bytes(H)] / ds [E, H,
// mx_scale_bytes(I)], converted to exact BF16 tiles inside the kernel.
cudaError_t launch_gemm_gate_up_mx(const void *x, const int32_t *perm, int k, const void *gq, const void *gs,
                                   const int4 *chunks, const int32_t *nchunks, const int32_t *offs, int n_assign, int H,
                                   int I, int E, void *act_hi, void *act_lo, int ctas, cudaStream_t s);
cudaError_t launch_gemm_down_mx(const void *act_hi, const void *act_lo, const void *dq, const void *ds,
                                const int4 *chunks, const int32_t *nchunks, const int32_t *offs, int n_assign, int H,
                                int I, int E, float *z, int ctas, cudaStream_t s);

// Backward pass.  Rows r index the padded sorted order (launch_sort with
// pad 16: each expert's segment rounded up to 16 rows, pad rows zero).
// gate_up_raw: g = W_gate x, u = W_up x [rows][I] FP32.
cudaError_t launch_gemm_gate_up_raw(const void *x, const int32_t *perm, int k, const void *wgu, const int4 *chunks,
                                    const int32_t *nchunks, const int32_t *offs, int n_rows, int H, int I, int E,
                                    float *g, float *u, int ctas, cudaStream_t s, bool seg = false);
// The forward gate_up GEMM (act as a BF16 hi/lo pair) that also keeps g and
// u [n_rows][I] in FP32 for a later backward pass (the training forward).
cudaError_t launch_gemm_gate_up_keep(const void *x, const int32_t *perm, int k, const void *wgu, const int4 *chunks,
                                     const int32_t *nchunks, const int32_t *offs, int n_rows, int H, int I, int E,
                                     void *act_hi, void *act_lo, float *g, float *u, int ctas, cudaStream_t s,
                                     void *act_lo2 = nullptr);
// q = W_down^T dout (dout as ds_hi + ds_lo [rows][H]) and the SwiGLU
// backward: in g, u, w_s; out dgu_hi/lo [rows][2I], wa_hi/lo [rows][I]
// (BF16 pairs) and dwp [rows][I/32] (partial sums of act . q)
struct BwdQOut {
    const float *g, *u, *w_s;
    void *dgu_hi, *dgu_lo, *wa_hi, *wa_lo;
    float *dwp;
};
cudaError_t launch_bwd_q(const void *ds_hi, const void *ds_lo, const void *wd, const int4 *chunks,
                         const int32_t *nchunks, const int32_t *offs, int n_rows, int H, int I, int E,
                         const BwdQOut &o, int ctas, cudaStream_t s);
// q [rows][I] alone, of dout in three terms: launch_bwd_swiglu goes on from it
cudaError_t launch_bwd_q_sums(const void *ds_hi, const void *ds_lo, const void *ds_lo2, const void *wd,
                              const int4 *chunks, const int32_t *nchunks, const int32_t *offs, int n_rows, int H,
                              int I, int E, float *q, int ctas, cudaStream_t s);
// z [rows][H] = W_gate_up^T (dgu_hi + dgu_lo)
cudaError_t launch_bwd_dx(const void *dgu_hi, const void *dgu_lo, const void *wgu, const int4 *chunks,
                          const int32_t *nchunks, const int32_t *offs, int n_rows, int H, int I, int E, float *z,
                          int ctas, cudaStream_t s, const void *dgu_lo2 = nullptr);

// grouped_bwd.cu
cudaError_t bwd_init_device();
cudaError_t read_bwd_fault_word(uint32_t *flags, bool clear);
// per padded row: xs = x[token] (BF16), ds_hi/lo = dout[token] split, w_s =
// routing weight; zeros in pad rows
cudaError_t launch_bwd_prep(const void *x, const float *dout, const float *w, const int32_t *perm,
                            const int32_t *offs, int n_rows_max, int E, int H, int k, void *xs, void *ds_hi,
                            void *ds_lo, float *w_s, int n_sm, cudaStream_t s, void *ds_lo2 = nullptr);
// the SwiGLU backward from q, g, u [rows][I] and w_s: dgu [rows][2I] and wa
// [rows][I] in three BF16 terms, dwp [rows][I/32] as launch_bwd_q's
struct BwdTerms {
    void *dgu_hi, *dgu_lo, *dgu_lo2, *wa_hi, *wa_lo, *wa_lo2;
};
cudaError_t launch_bwd_swiglu(const float *q, const float *g, const float *u, const float *w_s, const int32_t *perm,
                              const int32_t *offs, int n_rows_max, int E, int I, const BwdTerms &o, float *dwp,
                              int n_sm, cudaStream_t s);
// dW_down [E][H][I] = sum_r ds[r] (x) wa[r] over each expert's rows
cudaError_t launch_wgrad_down(const void *ds_hi, const void *ds_lo, const void *wa_hi, const void *wa_lo,
                              const int32_t *offs, const int32_t *counts, int n_rows, int H, int I, int E,
                              float *dwd, int ctas, cudaStream_t s, const void *ds_lo2 = nullptr,
                              const void *wa_lo2 = nullptr);
// dW_gate_up [E][2I][H] = sum_r dgu[r] (x) xs[r]
cudaError_t launch_wgrad_gate_up(const void *dgu_hi, const void *dgu_lo, const void *xs, const int32_t *offs,
                                 const int32_t *counts, int n_rows, int H, int I, int E, float *dwgu, int ctas,
                                 cudaStream_t s, const void *dgu_lo2 = nullptr);
// dlogits [T][E] from dwp (I/32 partial sums per row), pos, idx, w
// Zeroes dW_gate_up[e] and dW_down[e] of every expert with counts[e] == 0
// (the weight-gradient kernels skip those experts).
cudaError_t launch_zero_untouched(const int32_t *counts, int E, int H, int I, float *dwgu, float *dwd,
                                  cudaStream_t s);
cudaError_t launch_dlogits(const float *dwp, const int32_t *pos, const int32_t *idx, const float *w, int T, int E,
                           int k, int I, float *dlogits, cudaStream_t s);


// ---------------------------------------------------------------- the operators around the experts
// moe_ffn_api.cu: the current device's SM count and the pairs of CTAs that
// the orthogonalisation's products can hold at once, after the per-device
// set-up; a MOE_* status
int device_info(int *n_sm, int *pairs);

// rms_norm.cu.  x_f32, res_f32 ...: FP32, else BF16
bool norm_supported(int64_t H);
int norm_grad_parts(int64_t T, int64_t H);
cudaError_t launch_norm(const void *x, bool x_f32, const void *residual, bool res_f32, const float *weight, float eps,
                        int64_t T, int H, void *h_out, void *y, void *codes, void *scales, int n_sm, cudaStream_t s);
// partial: [norm_grad_parts(T, H)][H]
cudaError_t launch_norm_grad(const void *h, bool h_f32, const float *weight, const void *dy, bool dy_f32,
                             const void *dres, float eps, int64_t T, int H, void *dh, float *dweight, float *partial,
                             int n_sm, cudaStream_t s);

// gate.cu
struct GateCall {
    const float *logits, *bias;  // bias nullable
    int64_t T;
    int E, k, groups, topk_groups;
    bool sigmoid, renorm;
    float scale;
    int32_t *idx;
    float *w;
    int32_t *counts;  // nullable
};
cudaError_t launch_gate(const GateCall &c, int n_sm, cudaStream_t s);
cudaError_t launch_gate_grad(const float *logits, const int32_t *idx, const float *dw, int64_t T, int E, int k,
                             bool sigmoid, bool renorm, float scale, float *dlogits, int n_sm, cudaStream_t s);

// routing.cu: the caller's routing as the layer's own (dropped slots marked,
// take_routing_warp); tag_size, tag_cap as for launch_router
cudaError_t launch_take_routing(const int32_t *idx_in, const float *w_in, int T, int E, int k, int32_t *idx, float *w,
                                unsigned long long *tag_size, unsigned long long tag_cap, cudaStream_t s);
// MXFP8 rows [T, H] (codes, scales) widened to BF16
cudaError_t launch_mx_widen(const void *codes, const void *scales, int T, int H, void *x, int n_sm, cudaStream_t s);
// grouped_bwd.cu: dw [T, k] from the q GEMM's partial sums; 0 for a slot
// without a row (dropped)
cudaError_t launch_routed_dw(const float *dwp, const int32_t *pos, int T, int k, int I, float *dw, cudaStream_t s);

// orthogonalize.cu
struct OrthoCall {
    const void *g;
    bool g_f32;
    int64_t B, M, N;
    int steps;
    float a, b, c, eps, out_scale;
    void *out;
};
cudaError_t ortho_init_device(int *pairs);
cudaError_t read_ortho_fault_word(uint32_t *flags, bool clear);
size_t ortho_workspace_bytes(int64_t B, int64_t M, int64_t N);
cudaError_t launch_orthogonalize(const OrthoCall &c, void *workspace, int pairs, cudaStream_t s);

// balance.cu
struct BalanceCall {
    const float *logits;
    const int32_t *idx, *offsets;  // offsets nullable
    int64_t T;
    int S, E, k;
    bool sigmoid;
    float coef, z_coef;
    float *loss, *prob;
    int32_t *counts;
};
struct BalanceGradCall {
    const float *logits, *dloss, *base;  // dloss, base nullable
    const int32_t *counts, *offsets;     // offsets nullable
    int64_t T;
    int S, E, k;
    bool sigmoid;
    float coef, z_coef;
    float *out;
};
size_t balance_workspace_bytes(int64_t T, int64_t S, int64_t E);
cudaError_t launch_balance(const BalanceCall &c, void *workspace, int n_sm, cudaStream_t s);
cudaError_t launch_balance_grad(const BalanceGradCall &c, int n_sm, cudaStream_t s);

// adamw.cu
struct TensorRef {
    const void *data;
    int64_t n;
    bool f32;  // else BF16
};
struct AdamWTensor {
    void *w;
    float *master;  // nullable
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;  // 8-bit states
    int64_t n;
    float lr_factor, weight_decay;
    bool w_f32, grad_f32, bits8;
    uint32_t index;  // its place in the call's list
};
struct AdamWScalars {
    float beta1, one_minus1, beta2, one_minus2, eps, lr;
    float den_scale;            // a power of two that eps, and the quotient's other parts, are taken times
    float2 host;                // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t)
    const float2 *corrections;  // nullable: these, in device memory
    const float *grad_scale, *lr_at;  // nullable
    uint32_t step;                    // this step's number
    const int32_t *step_at;           // nullable: it, in device memory
};
size_t grad_norm_workspace_bytes(int64_t count);
cudaError_t launch_grad_norm(const TensorRef *grads, int count, float max_norm, float *out, void *workspace, int n_sm,
                             cudaStream_t s);
// step nullable: the number of steps so far, in device memory; with it the
// workspace holds a float2.  random: 8-bit codes are rounded at random
cudaError_t launch_adamw(const AdamWTensor *tensors, int count, AdamWScalars sc, double beta1, double beta2,
                         int32_t *step, bool random, void *workspace, cudaStream_t s);

}  // namespace moe
