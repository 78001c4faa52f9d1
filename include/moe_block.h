/*
 * moe_block.h -- C ABI of libmoeffn.so, second part: the operators of a
 * Mixture-of-Experts block around the expert layer of moe_ffn.h, on one
 * GB300 GPU (sm_103a).
 *
 * A block's step on T tokens: the residual stream h takes in the previous
 * layer's output and is normed (moe_rms_norm_forward); the gate scores the
 * experts and chooses k of them for every token (moe_gate_forward); the
 * experts run for that routing (moe_ffn_forward_routed).  Training adds the
 * gradients of the three (moe_ffn_backward_routed, moe_gate_backward,
 * moe_rms_norm_backward), the gate's load-balance loss with its gradient
 * (moe_balance_loss_forward, moe_balance_loss_backward), the clipping of the
 * gradients by their norm (moe_grad_norm) and the updates: orthogonalised for
 * the experts' weight matrices (moe_orthogonalize), AdamW for many tensors of
 * any kind (moe_adamw_step).
 *
 * Conventions: those of moe_ffn.h (row-major contiguous device tensors owned
 * by the caller, 16-byte aligned base pointers, 256-byte aligned workspaces,
 * checks before anything is enqueued, asynchronous on `stream`, status codes
 * MOE_*, deterministic: no floating-point atomics, the same bits from run to
 * run).  Outputs are fully overwritten and must not alias each other or an
 * input, unless a call says otherwise.  T == 0 enqueues nothing unless a
 * call says otherwise.  Every call may be captured into a CUDA graph after
 * one uncaptured call.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors whose type a call lets the caller choose. */
enum { MOE_BF16 = 0, MOE_F32 = 1 };

/*
 * Residual addition and root-mean-square norm.  For each of T rows of H:
 *   h = x + residual                      (FP32; h = x without a residual)
 *   y = h * weight / sqrt(mean(h^2) + eps)
 *   x          [T,H], x_type (the expert layer's FP32 output goes in as it is)
 *   residual   nullable [T,H], res_type
 *   weight_f32 [H]
 *   h_out      nullable [T,H], res_type: h rounded once.  Needs a residual.
 *              It may be the residual itself (in place).
 *   y_bf16     nullable [T,H]: y rounded once
 *   y_e4m3, y_scale  nullable (both or none): y in MXFP8, the layout of
 *              moe_ffn.h's MXFP8 tensors: codes [T,H] and E8M0 scales
 *              [T, MOE_FFN_MX_SCALE_BYTES(H)], one per 32 elements of a row
 *              (2^(floor(log2 amax) - 8), at least 2^-126, 1 for a block of
 *              zeros; the pad bytes are written as zeros), elements rounded to nearest,
 *              ties to even, from the FP32 y and clamped to +-448.  A block
 *              that holds a NaN or an infinity gets the scale 255 (NaN), its
 *              codes then say nothing.
 * The norm is taken of the FP32 h, before h_out is rounded.  Limits: H in
 * 1..16384 (H % 32 == 0 for MXFP8), T * H < 2^40, eps >= 0.  At least one of
 * y_bf16 and y_e4m3 is asked for.  A row of zeros with eps == 0 gives NaN, as
 * the formula does.  Squares are summed in FP32: elements below about 1e-22
 * count as zero in the mean, and a row whose sum of squares is beyond FP32's
 * range (one element of 1.8e19) gives y = 0.
 */
int moe_rms_norm_forward(const void *x, int x_type, const void *residual, int res_type,
                         const float *weight_f32, float eps, int64_t T, int64_t H,
                         void *h_out, void *y_bf16, void *y_e4m3, void *y_scale,
                         cudaStream_t stream);

/*
 * Its gradients at h, from dy = dL/dy.  (The forward call's h_out is h rounded
 * to the stream's type: with a BF16 stream these are the gradients at the
 * rounded h, within BF16's rounding of those at the h of the norm.)
 *   n  = h / sqrt(mean(h^2) + eps),   g = dy * weight
 *   dh = (g - n * mean(g * n)) / sqrt(mean(h^2) + eps) + dres
 *   dweight = sum over the rows of dy * n
 *   h     [T,H], h_type; dy [T,H], dy_type; dres nullable [T,H], h_type: the
 *         gradient that reaches h besides through y (the residual stream's)
 *   dh    [T,H], h_type (rounded once; it may be dres itself, in place): the
 *         gradient of both x and residual
 *   dweight_f32 [H]: summed in FP32 in an order fixed by T, H and the device
 * workspace: at least moe_rms_norm_backward_workspace_bytes.  T == 0 zeroes
 * dweight.  Same limits as the forward call.
 */
size_t moe_rms_norm_backward_workspace_bytes(int64_t T, int64_t H);
int moe_rms_norm_backward(const void *h, int h_type, const float *weight_f32, const void *dy,
                          int dy_type, const void *dres, float eps, int64_t T, int64_t H,
                          void *dh, float *dweight_f32, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* The gate's scores of a token's logits l[0..E). */
enum {
    MOE_SCORE_SOFTMAX = 0, /* s = exp(l - max l) / sum exp(l - max l), all E */
    MOE_SCORE_SIGMOID = 1  /* s = 1 / (1 + exp(-l))                          */
};

/*
 * How the gate chooses.  Zero-initialise and set what you need.
 *   score        MOE_SCORE_*.
 *   groups       0 or 1: one group.  Else the E experts are that many equal
 *                groups of consecutive experts (E % groups == 0, <= 32), and
 *                only the experts of topk_groups of them can be chosen.
 *   topk_groups  1..groups (ignored for one group); topk_groups * E / groups
 *                >= k.
 *   renormalize  != 0: a token's k weights are divided by their sum.
 *   scale        the factor on the weights (0 means 1).
 */
typedef struct moe_gate_opts {
    int32_t score;
    int32_t groups;
    int32_t topk_groups;
    int32_t renormalize;
    float scale;
    int32_t reserved[3]; /* must be zero */
} moe_gate_opts;

/*
 * The gate: the k experts of each of T tokens and their weights.
 *   c[e] = l[e] without a bias (it orders the experts as s does), s[e] +
 *          bias[e] in FP32 with one: the bias moves the choice alone.
 *   With groups: a group's rank is its largest c without a bias and the sum
 *   of its two largest c with one (the one c of a group of one); the
 *   topk_groups groups of highest rank stay, the lower index winning ties.
 *   The k experts of largest c among those that stay are chosen in
 *   descending order, the lower index winning ties (-0.0 == +0.0; a NaN
 *   ranks above every number).  A NaN or +inf among a row's logits makes all
 *   of its softmax scores NaN, so with a bias its first k experts are chosen.
 *   w[j] = scale * s[idx_j]                            renormalize == 0
 *   w[j] = scale * s[idx_j] / sum over m of s[idx_m]   renormalize != 0
 *   A sum of zero gives weights of zero: a sigmoid row of logits that are all
 *   -inf, or so low that every chosen score is zero.  A softmax row whose
 *   logits are all -inf has no largest finite logit; its scores count as zero.
 *   logits_f32 [T,E]; bias_f32 nullable [E]
 *   topk_idx int32 [T,k]; topk_w_f32 [T,k]
 *   counts  nullable int32 [E]: how many tokens chose each expert (integer
 *           atomics; zeroed by the call).  T == 0 zeroes it.
 *   opts    nullable (softmax over all E, one group, not renormalised).
 * Limits: 1 <= E <= 1024, 1 <= k <= min(E, 32), T * E < 2^40, T * k < 2^30.
 */
int moe_gate_forward(const float *logits_f32, const float *bias_f32, int64_t T, int64_t E,
                     int64_t k, const moe_gate_opts *opts, int32_t *topk_idx,
                     float *topk_w_f32, int32_t *counts, cudaStream_t stream);

/*
 * The gate's gradient: dlogits [T,E] from dtopk_w [T,k] = dL/dw, for the
 * choice in topk_idx (piecewise constant in the logits, so the choice and
 * the bias have none).  Scores are computed again from the logits.  With
 * p_j = s[idx_j], P = sum p_m, d_j = scale * dtopk_w_j:
 *   ds_j = d_j (renormalize == 0),  (d_j - sum_m d_m p_m / P) / P (else)
 *   sigmoid: dlogits[idx_j] = ds_j p_j (1 - p_j), 0 elsewhere
 *   softmax: dlogits[e] = s_e (ds_e - sum_m ds_m p_m), ds_e = 0 where e was
 *            not chosen (with renormalize the sum is zero, and so is dlogits
 *            where e was not chosen)
 * P == 0 gives zeros.  A slot whose index is outside [0, E), or that repeats
 * an earlier slot's, counts as one with weight zero: it adds nothing to any
 * sum and gets no gradient.  opts: score, renormalize and scale, as in the
 * forward call.
 */
int moe_gate_backward(const float *logits_f32, const int32_t *topk_idx,
                      const float *dtopk_w_f32, int64_t T, int64_t E, int64_t k,
                      const moe_gate_opts *opts, float *dlogits_f32, cudaStream_t stream);

/*
 * The expert layer for a routing that the caller passes:
 *   out[t] = sum over j ascending of topk_w[t][j] * expert(topk_idx[t][j], x[t])
 * with the experts, shapes, paths, workspace (at least
 * moe_ffn_routed_workspace_bytes; the state and rules of moe_ffn_forward_ex)
 * and options of moe_ffn.h.  topk_w is used as it is.
 *   x        [T,H] BF16; or, with x_scale, E4M3 codes with their E8M0 scales
 *            [T, MOE_FFN_MX_SCALE_BYTES(H)] (moe_rms_norm_forward's MXFP8
 *            output), widened once to BF16 (exact for every value in BF16's
 *            range, and finite codes and scales; a scale of 255 gives NaN)
 *   w_gate_up, w_down: BF16; or, with w_gate_up_scale and w_down_scale (both
 *            or none), MXFP8 as in moe_ffn_forward_mxfp8
 * A slot whose index is outside [0, E), or that repeats the index of an
 * earlier slot of its token, is dropped: it adds nothing to any output, not
 * even where its weight, or the weights of an expert that no slot uses, are
 * infinite or NaN.  So -1 marks an unused slot.  (The fused decode kernel,
 * up to four tokens, reads an unused expert's weights in its place.)
 * Arithmetic with BF16 weights: FP32 sums (on the grouped path in segments of
 * 256 products, added in order) and FP32 intermediates, which the tensor-core
 * products take as three BF16 terms (24 bits): closer to the definition than
 * moe_ffn_forward_ex's grouped path (two terms, one chain), not bit-identical
 * to it.  The decode path, and the calls with MXFP8 weights, give
 * moe_ffn_forward_ex's and moe_ffn_forward_mxfp8's bits for the same routing.
 */
size_t moe_ffn_routed_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k);
int moe_ffn_forward_routed(const void *x, const void *x_scale, const int32_t *topk_idx,
                           const float *topk_w_f32, const void *w_gate_up,
                           const void *w_gate_up_scale, const void *w_down,
                           const void *w_down_scale, int64_t T, int64_t H, int64_t I,
                           int64_t E, int64_t k, float *out_f32, void *workspace,
                           size_t workspace_bytes, moe_ffn_opts *opts, cudaStream_t stream);

/*
 * Its gradients for BF16 x and weights: moe_ffn_backward's dx, dW_gate_up and
 * dW_down, and dtopk_w_f32 [T,k] = dL/dtopk_w (a dropped slot's is 0) in the
 * place of the logits' gradient, with the same arithmetic as above.  workspace:
 * at least moe_ffn_routed_backward_workspace_bytes, and required; the rules
 * are moe_ffn_backward's.  from_state != 0: the workspace is the state that
 * moe_ffn_forward_routed_train left for the same x, routing, weights and
 * shape, and g and u are read from it instead of computed again (same bits).
 * T == 0 zeroes the two weight gradients.
 */
size_t moe_ffn_routed_backward_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E,
                                               int64_t k);
int moe_ffn_backward_routed(const void *x_bf16, const int32_t *topk_idx,
                            const float *topk_w_f32, const void *w_gate_up_bf16,
                            const void *w_down_bf16, const float *dout_f32, int64_t T,
                            int64_t H, int64_t I, int64_t E, int64_t k, float *dx_f32,
                            float *dtopk_w_f32, float *dw_gate_up_f32, float *dw_down_f32,
                            void *workspace, size_t workspace_bytes, int from_state,
                            moe_ffn_opts *opts, cudaStream_t stream);

/*
 * The forward pass that keeps g and u for it in `state` (at least
 * moe_ffn_routed_backward_workspace_bytes), as moe_ffn_forward_train does.
 */
int moe_ffn_forward_routed_train(const void *x_bf16, const int32_t *topk_idx,
                                 const float *topk_w_f32, const void *w_gate_up_bf16,
                                 const void *w_down_bf16, int64_t T, int64_t H, int64_t I,
                                 int64_t E, int64_t k, float *out_f32, void *state,
                                 size_t state_bytes, moe_ffn_opts *opts, cudaStream_t stream);

/*
 * Newton-Schulz orthogonalisation of a batch of B matrices [M,N] (the
 * experts' weight gradients or momenta), as the Muon optimiser's update:
 *   X = G / (||G||_F + eps), transposed if M > N (so that it is wide);
 *   `steps` times:  A = X X^T,  X = a X + (b A + c A A) X;
 *   out = X, transposed back.
 * Every singular value s of X goes through s (a + b s^2 + c s^4) each step;
 * with the usual a, b, c = 3.4445, -4.7750, 2.0315 and five steps all but
 * the smallest end near 1.
 *   g       [B,M,N], g_type
 *   out_bf16 [B,M,N]; scaled by out_scale before it is rounded
 * The products run on the tensor cores with FP16 operands and FP32 sums.  X
 * is kept between steps as a pair of FP16 values (about 22 significant bits),
 * of which the products read the high one; A and b A + c A A are rounded to
 * FP16.  Relative error of a Gaussian matrix in the 2-norm for the usual
 * coefficients and five steps, out's rounding to BF16 (1.7e-3) included: up to
 * 2.9e-3 where the smaller side is 64 or more, 3.8e-3 from 16, 5.9e-3 from 8;
 * the few entries of 1 to 7 rows do not average the roundings out: 1.6e-2.
 * Every further step raises what the roundings left beside small singular
 * values by a (ten steps on a 60 x 40 matrix of rank one: 1.5e-2).
 * A matrix of zeros gives zeros (NaN with eps < 1e-35); a NaN, an infinity or
 * a norm beyond FP32's range makes its whole matrix NaN and no other.
 * Entries below about 1e-28 count as zero in the norm.
 * Limits: M, N in 1..32768, steps in 1..32, B in 0..65535 (0 enqueues
 * nothing), B * M * N <= 2^40, B * ceil(M / 128) * ceil(N / 128) <= 2^24,
 * |a|, |b|, |c| <= 16, eps >= 0.  Coefficients and steps that can take a
 * singular value from [0, 1] to more than 1.9 before the last step, or an
 * eigenvalue of b A + c A A beyond 30, are refused (MOE_ERR_INVALID_ARG): A
 * and b A + c A A would leave FP16's range.  workspace: at least
 * moe_orthogonalize_workspace_bytes (0 for an invalid shape).
 */
size_t moe_orthogonalize_workspace_bytes(int64_t B, int64_t M, int64_t N);
int moe_orthogonalize(const void *g, int g_type, int64_t B, int64_t M, int64_t N, int steps,
                      float a, float b, float c, float eps, float out_scale, void *out_bf16,
                      void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * The load-balance loss of the gate's logits, and what training watches of
 * it: how many tokens chose each expert, and the experts' mean probabilities.
 *   score  MOE_SCORE_SOFTMAX: s_te = softmax(l_t)_e over all E;
 *          MOE_SCORE_SIGMOID: s_te = q_te / sum_e q_te, q = 1 / (1 + exp(-l))
 *   coef, z_coef: the factors of the two losses (0: that part is left out)
 */
typedef struct moe_balance_opts {
    int32_t score;
    float coef;
    float z_coef;
    int32_t reserved[5]; /* must be zero */
} moe_balance_opts;

/*
 * The tokens are S packed sequences: sequence i has the rows
 * [seq_offsets[i], seq_offsets[i+1]), n_i of them, N in all.  Rows before the
 * first sequence and behind the last belong to none: they have no part in
 * anything and are not read, whatever they hold.  Without seq_offsets all T
 * rows are one sequence (S == 1).
 *   counts[i,e] = rows of sequence i among whose k slots e is (a slot outside
 *                 [0, E), and a repeated one, counts for nothing)
 *   prob[i,e]   = mean over its rows of s_te (0 for an empty sequence)
 *   balance     = sum_i n_i / N * E * sum_e counts[i,e] / (k n_i) * prob[i,e]
 *                 (1 where every expert is as likely and as loaded as any)
 *   z           = sum_t logsumexp(l_t)^2 / N
 *   loss_f32[0] = coef * balance + z_coef * z; [1] = balance; [2] = z (0 with
 *                 z_coef == 0).  N == 0 gives zeros.
 *   logits_f32 [T,E]; topk_idx int32 [T,k]; seq_offsets nullable int32 [S+1],
 *   ascending, in 0..T (others give meaningless results, but no access out of
 *   bounds); loss_f32 [3]; counts int32 [S,E]; prob_f32 [S,E]
 * A row of logits that are all -inf has s = 0 and no z.  A sigmoid below 2^-126
 * (logits below -87.3) counts as zero, and so does, in the gradient, its 1 - q
 * there (above 87.3); a row of nothing else has s = 0 (and its z, where its logits
 * are finite).  A NaN among a row's logits, or a +inf with softmax or z, makes its
 * sequence's prob and the losses NaN.
 * Sums are FP32, in an order fixed by T, S, E and the device; exponentials are
 * within three units in the last place of their FP32 argument's, and a fortieth
 * of a unit more for each whole number in it, reciprocals within one.  Limits:
 * those of the gate (E <= 1024, k <= 32, T * E < 2^40, T * k < 2^30), S in
 * 1..2^20, finite coefficients.  T == 0 writes its outputs too.  workspace: at
 * least moe_balance_loss_workspace_bytes (0 for an invalid shape); it needs no
 * initial content.
 */
size_t moe_balance_loss_workspace_bytes(int64_t T, int64_t S, int64_t E);
int moe_balance_loss_forward(const float *logits_f32, const int32_t *topk_idx,
                             const int32_t *seq_offsets, int64_t T, int64_t S, int64_t E,
                             int64_t k, const moe_balance_opts *opts, float *loss_f32,
                             int32_t *counts, float *prob_f32, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/*
 * Its gradient at the logits, added to the one that reaches them besides
 * (moe_gate_backward's):
 *   dlogits = dloss * d loss_f32[0] / d logits + dlogits_in
 * The counts are piecewise constant in the logits and have no gradient:
 *   a_ie = coef * E * counts[i,e] / (k n_i N)
 *   softmax: s_e (a_e - sum a s); sigmoid: (a_e - sum a s) q_e (1 - q_e) / sum q
 *   z: 2 z_coef / N * logsumexp(l) * softmax(l)_e
 * Scores are computed again from the logits.  Rows of no sequence take
 * dlogits_in (0 without one), whatever their logits hold.
 *   counts        the forward call's, or the caller's own (of a larger batch,
 *                 scaled to this one's n_i)
 *   dloss_f32     nullable [1], the gradient at loss_f32[0] (1 without it)
 *   dlogits_in_f32 nullable [T,E]; dlogits_f32 [T,E] may be dlogits_in itself
 * Same limits; T == 0 enqueues nothing.
 */
int moe_balance_loss_backward(const float *logits_f32, const int32_t *counts,
                              const int32_t *seq_offsets, int64_t T, int64_t S, int64_t E,
                              int64_t k, const moe_balance_opts *opts,
                              const float *dloss_f32, const float *dlogits_in_f32,
                              float *dlogits_f32, cudaStream_t stream);

/* One of many tensors: n contiguous elements of a type, 16-byte aligned. */
typedef struct moe_tensor {
    const void *data;
    int64_t n;
    int32_t type;     /* MOE_BF16 or MOE_F32 */
    int32_t reserved; /* must be zero */
} moe_tensor;

/*
 * The norm of many gradients together, and the factor that clips it.
 *   out_f32[0] = sqrt(sum over all elements of g^2)
 *   out_f32[1] = max_norm / norm where norm > max_norm, else 1; NaN where the
 *                norm is no finite FP32 number (moe_adamw_step then leaves its
 *                step out)
 *   grads     host array of `count` descriptors, read before the call returns
 *   max_norm  > 0; infinity for the norm alone
 * Squares are summed in FP32 within a block and in FP64 over the blocks, in an
 * order fixed by the tensors' sizes and the device.  A sum beyond FP32's range is
 * taken of the elements times 2^-64, so the norm holds up to FP32's largest;
 * elements below about 1e-19 lose bits of their squares, and below 1e-22 count as
 * zero.  Limits: count <= 65536, sum of n <= 2^42.  Without elements the norm is 0
 * and the factor 1.  workspace: at least moe_grad_norm_workspace_bytes(count), no
 * initial content.
 */
size_t moe_grad_norm_workspace_bytes(int64_t count);
int moe_grad_norm(const moe_tensor *grads, int64_t count, float max_norm, float *out_f32,
                  void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Elements that share a scale of an 8-bit state. */
#define MOE_ADAMW_STATE_BLOCK 256

/*
 * A tensor of an AdamW step: n elements, contiguous, all updated in place.
 *   w       w_type; with `master` (FP32, nullable) the master is the weight and
 *           w takes its rounding.  A BF16 weight without one is rounded to
 *           nearest after every step: steps below 2^-8 of it can leave it as
 *           it is (half a spacing is 2^-9 to 2^-8 of it)
 *   grad    grad_type, read
 *   m, v    the moments: state_bits 32: FP32.  state_bits 8: E4M3 codes of
 *           m / m_scale and of sqrt(v) / v_scale, one FP32 scale per
 *           MOE_ADAMW_STATE_BLOCK elements (the last block may be shorter):
 *           the block's largest magnitude times the rounded 1 / 448, at least
 *           2^-126.  Codes are
 *           rounded as state_rounding says, but a v above zero takes at
 *           least the lowest code.  The step computes with the values before
 *           they are rounded.  Zeros (of codes and scales) are the initial
 *           state.  A NaN stays with its element, an infinity makes its block
 *           NaN.
 *   lr_factor, weight_decay: this tensor's own
 * All pointers 16-byte aligned, the scales 4-byte.
 */
typedef struct moe_adamw_tensor {
    void *w;
    float *master;
    const void *grad;
    void *m;
    void *v;
    float *m_scale;
    float *v_scale;
    int64_t n;
    int32_t w_type;
    int32_t grad_type;
    int32_t state_bits; /* 32 or 8 */
    float lr_factor;
    float weight_decay;
    int32_t reserved; /* must be zero */
} moe_adamw_tensor;

typedef struct moe_adamw_opts {
    double lr;    /* finite, >= 0 */
    double beta1; /* 0 <= beta < 1 */
    double beta2;
    double eps;   /* >= 0; 0 gives NaN where v is 0, 2^-158 is the least above it */
    int64_t step; /* this step's number, from 1 (ignored with step_i32) */
    int32_t state_rounding; /* MOE_ADAMW_ROUND_*, of 8-bit states' codes */
    int32_t reserved[5]; /* must be zero */
} moe_adamw_opts;

/*
 * How the codes of 8-bit states are rounded.
 *   NEAREST  ties to even.  A code stays where it is while a step changes its
 *            value by less than 3 to 6% of it: moments whose betas are close to 1
 *            stop following their gradients (sqrt(v) 3.4 times too large, for
 *            good, where gradients fall fourfold beside others that do not, with
 *            beta2 = 0.999).  It bears betas up to 0.95, where sqrt(v) is off by
 *            10% rms; a moment without any noise in its gradients can stop there too.
 *   RANDOM   to one of the two codes next to the value, the nearer one the
 *            likelier, so that the mean is the value whatever the betas (16% rms
 *            at beta2 = 0.999).  What is drawn depends on the step's number, the
 *            tensor's place in the list and the element's alone: the same step
 *            gives the same bits again.
 *   AUTO     NEAREST where both betas are at most 0.95, else RANDOM
 */
#define MOE_ADAMW_ROUND_AUTO 0
#define MOE_ADAMW_ROUND_NEAREST 1
#define MOE_ADAMW_ROUND_RANDOM 2

/*
 * One AdamW step of many tensors:
 *   g = grad_scale * grad;  lr_i = lr * lr_factor
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   w = w - lr_i weight_decay w
 *         - lr_i (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 * w is rounded once, after both subtractions.
 *   tensors        host array of `count` descriptors, read before the call
 *                  returns.  What is written (w, master, m, v, scales) must not
 *                  overlap with anything else in the call; gradients may.
 *   grad_scale_f32 nullable device [1] (moe_grad_norm's out_f32 + 1): the
 *                  gradients' factor; where it is NaN or infinite the whole
 *                  step is left out and nothing changes
 *   lr_f32         nullable device [1]: in the place of opts->lr
 *   step_i32       nullable device [1]: the number of steps taken so far; the
 *                  call adds one, unless the step is left out.  With it (and
 *                  lr_f32) a captured graph's replays are successive steps;
 *                  without it they repeat one, what it draws for 8-bit states too.
 *   workspace      with step_i32: at least 256 bytes, else nullable
 * Arithmetic in FP32 but for the corrections by the betas' powers (FP64).
 * Limits: count <= 65536, sum of n <= 2^42.
 */
int moe_adamw_step(const moe_adamw_tensor *tensors, int64_t count, const moe_adamw_opts *opts,
                   const float *grad_scale_f32, const float *lr_f32, int32_t *step_i32,
                   void *workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
