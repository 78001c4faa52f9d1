// moe_block_api.cu -- the C ABI of moe_block.h but for the experts' entry
// points (moe_ffn_api.cu): argument checks and launches.  Host code only.
#include <math.h>

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

}  // extern "C"
