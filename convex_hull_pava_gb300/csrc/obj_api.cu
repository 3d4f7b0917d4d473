// C ABI of the training objectives (declared in include/iso.h): argument checks.
#include "obj_internal.h"

#include "iso_internal.h"

#include <cmath>

namespace {

constexpr int64_t kMaxN = 2147483647LL;
constexpr int64_t kMaxElems = 1LL << 40;

iso_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ISO_OK : ISO_ERR_CUDA; }

bool dtype_ok(int dtype) { return dtype == ISO_F32 || dtype == ISO_BF16 || dtype == ISO_F16; }

bool span_ok(int64_t rows, int64_t stride) {
    return rows >= 0 && rows <= kMaxN && stride >= 0 && (rows == 0 || stride <= kMaxElems / rows);
}

// One row needs no stride; `least` is what a written row may not be shorter than.
bool rows_ok(int dtype, int64_t rows, int64_t n, int64_t stride, int64_t least) {
    return dtype_ok(dtype) && n >= 1 && n <= kMaxN && span_ok(rows, stride) &&
           (rows <= 1 || stride >= least);
}

float exponent_scale(float t) { return (float)(1.4426950408889634074 / t); }  // log2(e) / t

bool temperature_ok(float t) {
    return std::isfinite(t) && t > 0.f && std::isfinite(1.f / t) && std::isfinite(exponent_scale(t));
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
    return need == 0 || (ws && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0);
}

isodev::ScoreRows score_rows(const void* logits, int64_t rows, int64_t n, int64_t stride,
                             const int64_t* labels, float temperature) {
    return {logits, rows, (int)n, stride, labels, temperature, 1.f / temperature, exponent_scale(temperature)};
}

}  // namespace

extern "C" {

size_t iso_token_logp_workspace_bytes(int64_t rows) {
    return rows < 0 || rows > kMaxN ? 0 : isodev::token_logp_workspace(rows);
}

iso_status iso_token_logp(const void* logits, int dtype, int64_t rows, int64_t n, int64_t stride,
                          const int64_t* labels, float temperature, float* logp, float* norm,
                          void* workspace, size_t workspace_bytes, uint32_t* row_status,
                          void* stream) {
    if (!rows_ok(dtype, rows, n, stride, 0) || !temperature_ok(temperature)) return ISO_ERR_INVALID_ARG;
    if (rows == 0) return ISO_OK;
    if (!logits || !labels || !logp || !norm) return ISO_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, isodev::token_logp_workspace(rows)))
        return ISO_ERR_WORKSPACE;
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::token_logp(dtype, score_rows(logits, rows, n, stride, labels, temperature),
                                        logp, norm, workspace, row_status,
                                        static_cast<cudaStream_t>(stream)));
}

iso_status iso_token_logp_backward(const void* logits, int dtype, int64_t rows, int64_t n,
                                   int64_t stride, const int64_t* labels, float temperature,
                                   const float* norm, const float* grad_logp, float grad_scale,
                                   const float* grad_scale_dev, int changed_only, void* dlogits,
                                   int64_t out_stride, void* stream) {
    if (!rows_ok(dtype, rows, n, stride, 0) || !rows_ok(dtype, rows, n, out_stride, n) ||
        !temperature_ok(temperature) || (changed_only != 0 && changed_only != 1))
        return ISO_ERR_INVALID_ARG;
    if (rows == 0) return ISO_OK;
    if (!logits || !labels || !norm || !grad_logp || !dlogits) return ISO_ERR_INVALID_ARG;
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::token_logp_backward(
        dtype, score_rows(logits, rows, n, stride, labels, temperature), norm, grad_logp,
        grad_scale, grad_scale_dev, changed_only, dlogits, out_stride,
        static_cast<cudaStream_t>(stream)));
}

size_t iso_policy_loss_workspace_bytes(int64_t rows) {
    return rows < 0 || rows > kMaxN ? 0 : isodev::policy_workspace(rows);
}

iso_status iso_policy_loss(const void* logits, int dtype, int64_t rows, int64_t n, int64_t stride,
                           const int64_t* labels, float temperature, const float* old_logp,
                           const float* advantages, const float* ref_logp, const float* weights,
                           float clip_low, float clip_high, float kl_coef, float grad_scale,
                           float* loss, float* stats, float* logp, float* norm, float* coef,
                           void* dlogits, int64_t out_stride, void* workspace,
                           size_t workspace_bytes, uint32_t* row_status, void* stream) {
    if (!rows_ok(dtype, rows, n, stride, 0) || !temperature_ok(temperature) || !loss || !stats ||
        (dlogits && !rows_ok(dtype, rows, n, out_stride, n)))
        return ISO_ERR_INVALID_ARG;
    if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f)) return ISO_ERR_INVALID_ARG;
    if (rows > 0 && (!logits || !labels || !old_logp || !advantages || !logp || !norm || !coef))
        return ISO_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, isodev::policy_workspace(rows)))
        return ISO_ERR_WORKSPACE;
    isodev::PolicyArgs p{};
    p.old_logp = old_logp;
    p.advantages = advantages;
    p.ref_logp = ref_logp;
    p.weights = weights;
    p.low = 1.f - clip_low;
    p.high = 1.f + clip_high;
    p.kl_coef = ref_logp ? kl_coef : 0.f;
    p.grad_scale = grad_scale;
    p.logp = logp;
    p.norm = norm;
    p.coef = coef;
    p.loss = loss;
    p.stats = stats;
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::policy_loss(
        dtype, score_rows(logits, rows, n, stride, labels, temperature), p, dlogits, out_stride, workspace, row_status, static_cast<cudaStream_t>(stream)));
}

size_t iso_preference_loss_workspace_bytes(int64_t rows, int64_t pairs) {
    return rows < 0 || rows > kMaxN || pairs < 0 || pairs > kMaxN
               ? 0
               : isodev::preference_workspace(rows, pairs);
}

iso_status iso_preference_loss(const void* logits, int dtype, int64_t rows, int64_t n,
                               int64_t stride, const int64_t* labels, const int64_t* offsets,
                               int64_t pairs, const float* ref_logp, int kind, float beta,
                               float label_smoothing, int average, float grad_scale, float* loss,
                               float* margins, float* seq_logp, float* logp, float* norm,
                               float* coef, void* dlogits, int64_t out_stride, void* workspace,
                               size_t workspace_bytes, uint32_t* row_status,
                               uint32_t* pair_status, void* stream) {
    if (!rows_ok(dtype, rows, n, stride, 0) || !loss ||
        (dlogits && !rows_ok(dtype, rows, n, out_stride, n)) || pairs < 0 || pairs > kMaxN)
        return ISO_ERR_INVALID_ARG;
    if (kind < ISO_PREFERENCE_SIGMOID || kind > ISO_PREFERENCE_SQUARED ||
        !(std::isfinite(beta) && beta > 0.f) ||
        !(label_smoothing >= 0.f && label_smoothing <= 1.f) || (average != 0 && average != 1))
        return ISO_ERR_INVALID_ARG;
    if (rows > 0 && (!logits || !labels || !logp || !norm || !coef)) return ISO_ERR_INVALID_ARG;
    if (pairs > 0 && (!offsets || !margins || !seq_logp)) return ISO_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, isodev::preference_workspace(rows, pairs)))
        return ISO_ERR_WORKSPACE;
    isodev::PreferenceArgs p{offsets, pairs,   ref_logp, kind,        average, beta,
                             label_smoothing, loss,    margins,  seq_logp,    pair_status, 0, nullptr, nullptr, nullptr};
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::preference_loss(
        dtype, score_rows(logits, rows, n, stride, labels, 1.f), p, logp, norm, coef, grad_scale,
        dlogits, out_stride, workspace, row_status, static_cast<cudaStream_t>(stream)));
}

static bool router_ok(int dtype, int64_t tokens, int64_t experts, int64_t stride, int64_t least,
                      int top_k, int renormalize) {
    return experts <= ISO_MAX_EXPERTS && rows_ok(dtype, tokens, experts, stride, least) &&
           top_k >= 1 && top_k <= experts && top_k <= ISO_MAX_TOP_K &&
           (renormalize == 0 || renormalize == 1);
}

size_t iso_balance_loss_workspace_bytes(int64_t tokens, int64_t experts) {
    return tokens < 0 || tokens > kMaxN || experts < 1 || experts > ISO_MAX_EXPERTS
               ? 0
               : isodev::balance_workspace(tokens, (int)experts);
}

iso_status iso_balance_loss(const void* logits, int dtype, int64_t tokens, int64_t experts,
                            int64_t stride, int top_k, const uint8_t* mask, int renormalize,
                            float* loss, int64_t* counts, int32_t* chosen, float* gates,
                            int64_t* live, void* workspace, size_t workspace_bytes, void* stream) {
    if (!router_ok(dtype, tokens, experts, stride, 0, top_k, renormalize) || !loss || !counts ||
        !live || (tokens > 0 && (!logits || !chosen || !gates)))
        return ISO_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, isodev::balance_workspace(tokens, (int)experts)))
        return ISO_ERR_WORKSPACE;
    const isodev::RouterArgs a{logits, tokens, (int)experts, stride, mask, top_k, renormalize};
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::balance_loss(dtype, a, loss, counts, chosen, gates, live, workspace,
                                          static_cast<cudaStream_t>(stream)));
}

iso_status iso_balance_loss_backward(const void* logits, int dtype, int64_t tokens,
                                     int64_t experts, int64_t stride, int top_k,
                                     const uint8_t* mask, int renormalize, const int64_t* counts,
                                     const int32_t* chosen, const float* gates,
                                     const int64_t* live, const float* grad_gates,
                                     float grad_loss, const float* grad_loss_dev, void* dlogits,
                                     int64_t out_stride, void* stream) {
    if (!router_ok(dtype, tokens, experts, stride, 0, top_k, renormalize) ||
        !rows_ok(dtype, tokens, experts, out_stride, experts))
        return ISO_ERR_INVALID_ARG;
    if (tokens == 0) return ISO_OK;
    if (!logits || !counts || !chosen || !gates || !live || !dlogits) return ISO_ERR_INVALID_ARG;
    const isodev::RouterArgs a{logits, tokens, (int)experts, stride, mask, top_k, renormalize};
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::balance_backward(dtype, a, counts, chosen, gates, live, grad_gates,
                                              grad_loss, grad_loss_dev, dlogits, out_stride,
                                              static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
