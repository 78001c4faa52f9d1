// moe_block_api.cu -- the C ABI of moe_block.h but for the experts' entry
// points (moe_ffn_api.cu): argument checks and launches.  Host code only.
#include <float.h>
#include <math.h>

#include <vector>

#include "common.cuh"
#include "kernels.h"
#include "moe_block.h"

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

bool is_type(int t) { return t == MOE_BF16 || t == MOE_F32; }

int check_norm(int64_t T, int64_t H, float eps)
{
    if (T < 0 || H < 1 || !(eps >= 0.0f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (!moe::norm_supported(H) || T > ((int64_t)1 << 40) / H) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// The checked options of the gate: one group, scale 1 where they say nothing.
struct Gate {
    int score, groups, topk_groups;
    bool renorm;
    float scale;
};

int check_gate(int64_t T, int64_t E, int64_t k, const moe_gate_opts *o, Gate *g)
{
    if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
    if (E > 1024 || k > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T > ((int64_t)1 << 40) / E || T > ((int64_t)1 << 30) / k) return MOE_ERR_UNSUPPORTED_SHAPE;
    *g = Gate{MOE_SCORE_SOFTMAX, 1, 1, false, 1.0f};
    if (!o) return MOE_OK;
    for (int32_t r : o->reserved)
        if (r != 0) return MOE_ERR_INVALID_ARG;
    if (o->score != MOE_SCORE_SOFTMAX && o->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (!isfinite(o->scale)) return MOE_ERR_INVALID_ARG;
    g->score = o->score;
    g->renorm = o->renormalize != 0;
    if (o->scale != 0.0f) g->scale = o->scale;
    if (o->groups < 0) return MOE_ERR_INVALID_ARG;
    if (o->groups > 1) {
        if (o->groups > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
        if (E % o->groups || o->topk_groups < 1 || o->topk_groups > o->groups) return MOE_ERR_INVALID_ARG;
        if (o->topk_groups * (E / o->groups) < k) return MOE_ERR_INVALID_ARG;
        g->groups = o->groups;
        g->topk_groups = o->topk_groups;
    }
    return MOE_OK;
}

bool ortho_shape(int64_t B, int64_t M, int64_t N)
{
    return B >= 0 && B <= 65535 && M >= 1 && N >= 1 && M <= 32768 && N <= 32768 &&
           B <= ((int64_t)1 << 40) / (M * N) &&
           // the list of tiles, 3 products and 32 steps, is indexed in 32 bits
           B * ((M + 127) / 128) * ((N + 127) / 128) <= ((int64_t)1 << 24);
}

// Whether what the steps store in FP16 stays in its range, whatever the
// matrix: X's singular values lie in [0, top], top = 1 at the start and then
// the largest |s (a + b s^2 + c s^4)| there, one part in a hundred more for
// the roundings; A = X X^T is stored times 2^14 (an entry overflows where top
// reaches 2), b A + c A A times 2^11 (at 32).  The last step's X is not
// stored in FP16.
bool ortho_in_range(double a, double b, double c, int steps)
{
    double top = 1.0;
    for (int i = 0; i < steps; ++i) {
        if (!(top <= 1.9)) return false;
        const double end = top * top;
        auto poly = [&](double t) { return fabs(b * t + c * t * t); };  // of t = s^2
        double most = poly(end);
        if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < end) most = fmax(most, poly(-b / (2.0 * c)));
        if (!(most <= 30.0)) return false;
        auto value = [&](double t) { return fabs(sqrt(t) * (a + b * t + c * t * t)); };
        most = value(end);
        auto at = [&](double t) {  // an extremum, a root of a + 3 b t + 5 c t^2
            if (t > 0.0 && t < end) most = fmax(most, value(t));
        };
        const double root = 9.0 * b * b - 20.0 * a * c;
        if (c != 0.0 && root >= 0.0) {
            at((-3.0 * b - sqrt(root)) / (10.0 * c));
            at((-3.0 * b + sqrt(root)) / (10.0 * c));
        } else if (c == 0.0 && b != 0.0) {
            at(-a / (3.0 * b));
        }
        top = 1.01 * most;
    }
    return true;
}

// The balance loss's limits: the gate's, and the sequences'.
bool balance_shape(int64_t T, int64_t S, int64_t E)
{
    return T >= 0 && S >= 1 && E >= 1 && E <= 1024 && T < ((int64_t)1 << 30) && T <= ((int64_t)1 << 40) / E &&
           S <= (1 << 20);
}

int check_balance(int64_t T, int64_t S, int64_t E, int64_t k, const int32_t *offsets, const moe_balance_opts *o)
{
    if (T < 0 || S < 1 || E < 1 || k < 1 || k > E || !o) return MOE_ERR_INVALID_ARG;
    for (int32_t r : o->reserved)
        if (r != 0) return MOE_ERR_INVALID_ARG;
    if (o->score != MOE_SCORE_SOFTMAX && o->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (!isfinite(o->coef) || !isfinite(o->z_coef)) return MOE_ERR_INVALID_ARG;
    if (!offsets && S != 1) return MOE_ERR_INVALID_ARG;
    if (!balance_shape(T, S, E) || k > 32 || T > ((int64_t)1 << 30) / k) return MOE_ERR_UNSUPPORTED_SHAPE;
    return aligned16(offsets) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

constexpr int64_t kMostTensors = 65536, kMostElements = (int64_t)1 << 42;

// 8-bit moments whose codes are rounded to nearest follow their gradients up to
// these betas.  A step has to change sqrt(v) by 3 to 6% to move its code; with
// Gaussian gradients, sqrt(v) over that of FP32 states, median (and rms error): beta2
// 0.95 1.04 (10%), 0.97 1.10 (17%), 0.99 1.24 (32%); where half of a block's
// gradients then fall fourfold, theirs 1.15, 2.4 and 4.6, at 0.999 3.4 for good.
// Rounded at random: 1.00 to 1.02 in each, 12% rms at 0.95, 16% at 0.99 and 0.999.
// m, with noise as large as its mean, is off by 6% at beta1 0.9, 9% at 0.95, and
// at 0.99 by 1.7 times itself (rounded at random 9%, 12%, 20%).
constexpr double kMostNearest = 0.95;

// The running number of elements of a list of tensors.
int add_elements(int64_t n, int64_t *total)
{
    if (n < 0) return MOE_ERR_INVALID_ARG;
    if (n > kMostElements || (*total += n) > kMostElements) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

bool misses(const void *p, uintptr_t mask) { return !p || ((uintptr_t)p & mask); }

int check_adamw_tensor(const moe_adamw_tensor &t, uint32_t index, moe::AdamWTensor *out)
{
    if (t.reserved != 0 || !is_type(t.w_type) || !is_type(t.grad_type)) return MOE_ERR_INVALID_ARG;
    if (t.state_bits != 32 && t.state_bits != 8) return MOE_ERR_INVALID_ARG;
    if (!isfinite(t.lr_factor) || !isfinite(t.weight_decay)) return MOE_ERR_INVALID_ARG;
    const bool bits8 = t.state_bits == 8;
    if (t.n > 0) {
        if (misses(t.w, 15) || misses(t.grad, 15) || misses(t.m, 15) || misses(t.v, 15)) return MOE_ERR_INVALID_ARG;
        if (t.master && !aligned16(t.master)) return MOE_ERR_INVALID_ARG;
        if (bits8 && (misses(t.m_scale, 3) || misses(t.v_scale, 3))) return MOE_ERR_INVALID_ARG;
    }
    *out = moe::AdamWTensor{t.w,         t.master, t.grad,      t.m,
                            t.v,         t.m_scale, t.v_scale,  t.n,
                            t.lr_factor, t.weight_decay, t.w_type == MOE_F32, t.grad_type == MOE_F32,
                            bits8,       index};
    return MOE_OK;
}

// A list of `count` elements; an empty one where there is no memory for it.
template <typename T>
std::vector<T> list_of(int64_t count)
{
    try {
        return std::vector<T>((size_t)count);
    } catch (...) {
        return {};
    }
}

}  // namespace

extern "C" {

int moe_rms_norm_forward(const void *x, int x_type, const void *residual, int res_type, const float *weight_f32,
                         float eps, int64_t T, int64_t H, void *h_out, void *y_bf16, void *y_e4m3, void *y_scale,
                         cudaStream_t stream)
{
    int st = check_norm(T, H, eps);
    if (st != MOE_OK) return st;
    if (!is_type(x_type) || (residual && !is_type(res_type))) return MOE_ERR_INVALID_ARG;
    if ((y_e4m3 == nullptr) != (y_scale == nullptr)) return MOE_ERR_INVALID_ARG;
    if (y_e4m3 && H % 32) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x || !weight_f32 || (!y_bf16 && !y_e4m3) || (h_out && !residual)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight_f32) || !aligned16(h_out) || !aligned16(y_bf16) ||
        !aligned16(y_e4m3) || !aligned16(y_scale))
        return MOE_ERR_INVALID_ARG;
    int n_sm, pairs;
    st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    return moe::launch_norm(x, x_type == MOE_F32, residual, res_type == MOE_F32, weight_f32, eps, T, (int)H, h_out,
                            y_bf16, y_e4m3, y_scale, n_sm, stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

size_t moe_rms_norm_backward_workspace_bytes(int64_t T, int64_t H)
{
    if (check_norm(T, H, 0.0f) != MOE_OK) return 0;
    const size_t bytes = (size_t)moe::norm_grad_parts(T, H) * (size_t)H * 4;
    return bytes < 256 ? 256 : bytes;
}

int moe_rms_norm_backward(const void *h, int h_type, const float *weight_f32, const void *dy, int dy_type,
                          const void *dres, float eps, int64_t T, int64_t H, void *dh, float *dweight_f32,
                          void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    int st = check_norm(T, H, eps);
    if (st != MOE_OK) return st;
    if (!is_type(h_type) || !is_type(dy_type)) return MOE_ERR_INVALID_ARG;
    if (!dweight_f32 || !aligned16(dweight_f32)) return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        if (!h || !weight_f32 || !dy || !dh) return MOE_ERR_INVALID_ARG;
        if (!aligned16(h) || !aligned16(weight_f32) || !aligned16(dy) || !aligned16(dres) || !aligned16(dh))
            return MOE_ERR_INVALID_ARG;
        if (!workspace || ((uintptr_t)workspace & 255)) return MOE_ERR_INVALID_ARG;
        if (workspace_bytes < moe_rms_norm_backward_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    int n_sm, pairs;
    st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    if (T == 0) return cudaMemsetAsync(dweight_f32, 0, (size_t)H * 4, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    return moe::launch_norm_grad(h, h_type == MOE_F32, weight_f32, dy, dy_type == MOE_F32, dres, eps, T, (int)H, dh,
                                 dweight_f32, (float *)workspace, n_sm, stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

int moe_gate_forward(const float *logits_f32, const float *bias_f32, int64_t T, int64_t E, int64_t k,
                     const moe_gate_opts *opts, int32_t *topk_idx, float *topk_w_f32, int32_t *counts,
                     cudaStream_t stream)
{
    Gate g;
    int st = check_gate(T, E, k, opts, &g);
    if (st != MOE_OK) return st;
    if (!aligned16(counts)) return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        if (!logits_f32 || !topk_idx || !topk_w_f32) return MOE_ERR_INVALID_ARG;
        if (!aligned16(logits_f32) || !aligned16(bias_f32) || !aligned16(topk_idx) || !aligned16(topk_w_f32))
            return MOE_ERR_INVALID_ARG;
    } else if (!counts) {
        return MOE_OK;
    }
    int n_sm, pairs;
    st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    if (T == 0) return cudaMemsetAsync(counts, 0, (size_t)E * 4, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    const moe::GateCall c{logits_f32, bias_f32, T,        (int)E,   (int)k,     g.groups, g.topk_groups,
                          g.score == MOE_SCORE_SIGMOID, g.renorm, g.scale, topk_idx, topk_w_f32, counts};
    return moe::launch_gate(c, n_sm, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_gate_backward(const float *logits_f32, const int32_t *topk_idx, const float *dtopk_w_f32, int64_t T, int64_t E,
                      int64_t k, const moe_gate_opts *opts, float *dlogits_f32, cudaStream_t stream)
{
    Gate g;
    int st = check_gate(T, E, k, opts, &g);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!logits_f32 || !topk_idx || !dtopk_w_f32 || !dlogits_f32) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits_f32) || !aligned16(topk_idx) || !aligned16(dtopk_w_f32) || !aligned16(dlogits_f32))
        return MOE_ERR_INVALID_ARG;
    int n_sm, pairs;
    st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    return moe::launch_gate_grad(logits_f32, topk_idx, dtopk_w_f32, T, (int)E, (int)k, g.score == MOE_SCORE_SIGMOID,
                                 g.renorm, g.scale, dlogits_f32, n_sm, stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

size_t moe_orthogonalize_workspace_bytes(int64_t B, int64_t M, int64_t N)
{
    return ortho_shape(B, M, N) ? moe::ortho_workspace_bytes(B, M, N) : 0;
}

int moe_orthogonalize(const void *g, int g_type, int64_t B, int64_t M, int64_t N, int steps, float a, float b, float c,
                      float eps, float out_scale, void *out_bf16, void *workspace, size_t workspace_bytes,
                      cudaStream_t stream)
{
    if (B < 0 || M < 1 || N < 1 || steps < 1 || !is_type(g_type)) return MOE_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || isinf(eps) || !isfinite(out_scale)) return MOE_ERR_INVALID_ARG;
    if (!ortho_shape(B, M, N) || steps > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
    // NaN coefficients fail these too
    if (!(fabsf(a) <= 16.0f && fabsf(b) <= 16.0f && fabsf(c) <= 16.0f)) return MOE_ERR_INVALID_ARG;
    if (!ortho_in_range(a, b, c, steps)) return MOE_ERR_INVALID_ARG;
    if (B == 0) return MOE_OK;
    if (!g || !out_bf16 || !aligned16(g) || !aligned16(out_bf16)) return MOE_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe::ortho_workspace_bytes(B, M, N)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    int n_sm, pairs;
    const int st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    if (pairs < 1) return MOE_ERR_CUDA;
    const moe::OrthoCall call{g, g_type == MOE_F32, B, M, N, steps, a, b, c, eps, out_scale, out_bf16};
    return moe::launch_orthogonalize(call, workspace, pairs, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_balance_loss_workspace_bytes(int64_t T, int64_t S, int64_t E)
{
    return balance_shape(T, S, E) ? moe::balance_workspace_bytes(T, S, E) : 0;
}

int moe_balance_loss_forward(const float *logits_f32, const int32_t *topk_idx, const int32_t *seq_offsets, int64_t T,
                             int64_t S, int64_t E, int64_t k, const moe_balance_opts *opts, float *loss_f32,
                             int32_t *counts, float *prob_f32, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream)
{
    int st = check_balance(T, S, E, k, seq_offsets, opts);
    if (st != MOE_OK) return st;
    if (!loss_f32 || !counts || !prob_f32 || (T > 0 && (!logits_f32 || !topk_idx))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits_f32) || !aligned16(topk_idx) || !aligned16(loss_f32) || !aligned16(counts) ||
        !aligned16(prob_f32))
        return MOE_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe::balance_workspace_bytes(T, S, E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    int n_sm, pairs;
    st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    const moe::BalanceCall c{logits_f32, topk_idx, seq_offsets, T, (int)S, (int)E, (int)k,
                             opts->score == MOE_SCORE_SIGMOID, opts->coef, opts->z_coef, loss_f32, prob_f32, counts};
    return moe::launch_balance(c, workspace, n_sm, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_balance_loss_backward(const float *logits_f32, const int32_t *counts, const int32_t *seq_offsets, int64_t T,
                              int64_t S, int64_t E, int64_t k, const moe_balance_opts *opts, const float *dloss_f32,
                              const float *dlogits_in_f32, float *dlogits_f32, cudaStream_t stream)
{
    int st = check_balance(T, S, E, k, seq_offsets, opts);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!logits_f32 || !counts || !dlogits_f32) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits_f32) || !aligned16(counts) || !aligned16(dlogits_in_f32) || !aligned16(dlogits_f32) ||
        ((uintptr_t)dloss_f32 & 3))
        return MOE_ERR_INVALID_ARG;
    int n_sm, pairs;
    st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    const moe::BalanceGradCall c{logits_f32, dloss_f32, dlogits_in_f32, counts, seq_offsets, T, (int)S, (int)E, (int)k,
                                 opts->score == MOE_SCORE_SIGMOID, opts->coef, opts->z_coef, dlogits_f32};
    return moe::launch_balance_grad(c, n_sm, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_grad_norm_workspace_bytes(int64_t count)
{
    return count < 0 || count > kMostTensors ? 0 : moe::grad_norm_workspace_bytes(count);
}

int moe_grad_norm(const moe_tensor *grads, int64_t count, float max_norm, float *out_f32, void *workspace,
                  size_t workspace_bytes, cudaStream_t stream)
{
    if (count < 0 || (count > 0 && !grads) || !(max_norm > 0.0f)) return MOE_ERR_INVALID_ARG;
    if (count > kMostTensors) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (misses(out_f32, 3) || misses(workspace, 255)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe::grad_norm_workspace_bytes(count)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    auto refs = list_of<moe::TensorRef>(count);
    if ((int64_t)refs.size() != count) return MOE_ERR_NO_MEMORY;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        const moe_tensor &g = grads[i];
        if (g.reserved != 0 || !is_type(g.type) || (g.n > 0 && misses(g.data, 15))) return MOE_ERR_INVALID_ARG;
        const int st = add_elements(g.n, &total);
        if (st != MOE_OK) return st;
        refs[(size_t)i] = moe::TensorRef{g.data, g.n, g.type == MOE_F32};
    }
    int n_sm, pairs;
    const int st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    return moe::launch_grad_norm(refs.data(), (int)count, max_norm, out_f32, workspace, n_sm, stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

int moe_adamw_step(const moe_adamw_tensor *tensors, int64_t count, const moe_adamw_opts *opts,
                   const float *grad_scale_f32, const float *lr_f32, int32_t *step_i32, void *workspace,
                   size_t workspace_bytes, cudaStream_t stream)
{
    if (count < 0 || (count > 0 && !tensors) || !opts) return MOE_ERR_INVALID_ARG;
    if (count > kMostTensors) return MOE_ERR_UNSUPPORTED_SHAPE;
    const moe_adamw_opts &o = *opts;
    for (int32_t r : o.reserved)
        if (r != 0) return MOE_ERR_INVALID_ARG;
    if (o.state_rounding < MOE_ADAMW_ROUND_AUTO || o.state_rounding > MOE_ADAMW_ROUND_RANDOM) return MOE_ERR_INVALID_ARG;
    // NaN fails these too
    if (!(o.lr >= 0.0) || isinf((float)o.lr) || !(o.eps >= 0.0) || isinf((float)o.eps)) return MOE_ERR_INVALID_ARG;
    if (!(o.beta1 >= 0.0 && o.beta1 < 1.0 && o.beta2 >= 0.0 && o.beta2 < 1.0)) return MOE_ERR_INVALID_ARG;
    if (!step_i32 && o.step < 1) return MOE_ERR_INVALID_ARG;
    if (((uintptr_t)grad_scale_f32 & 3) || ((uintptr_t)lr_f32 & 3) || ((uintptr_t)step_i32 & 3))
        return MOE_ERR_INVALID_ARG;
    if (step_i32 && misses(workspace, 255)) return MOE_ERR_INVALID_ARG;
    if (step_i32 && workspace_bytes < 256) return MOE_ERR_WORKSPACE_TOO_SMALL;
    auto list = list_of<moe::AdamWTensor>(count);
    if ((int64_t)list.size() != count) return MOE_ERR_NO_MEMORY;
    int64_t total = 0;
    bool bits8 = false;
    for (int64_t i = 0; i < count; ++i) {
        int st = check_adamw_tensor(tensors[i], (uint32_t)i, &list[(size_t)i]);
        if (st == MOE_OK) st = add_elements(tensors[i].n, &total);
        if (st != MOE_OK) return st;
        bits8 |= tensors[i].state_bits == 8;
    }
    if (count == 0 && !step_i32) return MOE_OK;
    int n_sm, pairs;
    const int st = moe::device_info(&n_sm, &pairs);
    if (st != MOE_OK) return st;
    const double t = (double)o.step;
    // an eps below FP32's normal numbers, alone in a denominator, would count as
    // zero: numerator and denominator are taken times 2^32, at least 2^-126
    const bool tiny = o.eps > 0.0 && o.eps < FLT_MIN;
    const double den_scale = tiny ? 4294967296.0 : 1.0;
    const double eps = tiny && o.eps * den_scale < FLT_MIN ? FLT_MIN : o.eps * den_scale;
    const moe::AdamWScalars sc{(float)o.beta1,
                               (float)(1.0 - o.beta1),
                               (float)o.beta2,
                               (float)(1.0 - o.beta2),
                               (float)eps,
                               (float)o.lr,
                               (float)den_scale,
                               make_float2((float)(1.0 / (1.0 - pow(o.beta1, t))),
                                           (float)(1.0 / sqrt(1.0 - pow(o.beta2, t)))),
                               nullptr,
                               grad_scale_f32,
                               lr_f32,
                               (uint32_t)o.step,
                               nullptr};
    const bool random = o.state_rounding == MOE_ADAMW_ROUND_AUTO ? o.beta1 > kMostNearest || o.beta2 > kMostNearest
                                                                 : o.state_rounding == MOE_ADAMW_ROUND_RANDOM;
    return moe::launch_adamw(list.data(), (int)count, sc, o.beta1, o.beta2, step_i32, random && bits8, workspace, stream) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // extern "C"
