// Internal declarations of the training objectives (obj_*.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/iso.h"

namespace isodev {

// Rows of scores of one call: row r starts at x + r * stride elements.
struct ScoreRows {
    const void* x;
    int64_t rows;
    int n;
    int64_t stride;
    const int64_t* labels;
    float t, inv_t, a;  // temperature, 1 / temperature, log2(e) / temperature
};

// At the front of a call's workspace: the CTAs that have come to the end of a kernel, and the rows
// with a label.
struct ListHead {
    unsigned ticket;
    int labelled;
    float inv_count;
};
struct PolicyTerms;

// What the policy loss takes and gives for each row beside its scores.
struct PolicyArgs {
    const float *old_logp, *advantages, *ref_logp, *weights;
    float low, high, kl_coef, grad_scale;
    float *logp, *norm, *coef;
    float *loss, *stats;
    ListHead* head;               // workspace
    struct PolicyTerms* of_team;  // workspace
};

struct PreferenceArgs {
    const int64_t* offsets;
    int64_t pairs;
    const float* ref_logp;
    int kind, average;
    float beta, smooth;
    float *loss, *margins, *seq_logp;
    uint32_t* pair_status;
    int sum_later;     // the gradient's kernel adds up the loss
    unsigned* ticket;  // workspace
    float* rest;       // [rows] workspace: what logp's rounding to float32 has left out
    float* each;       // [pairs] workspace
};

size_t token_logp_workspace(int64_t rows);
cudaError_t token_logp(int dtype, const ScoreRows& s, float* logp, float* norm, void* ws,
                       uint32_t* row_status, cudaStream_t st);
// out = grad_scale * (grad_scale_dev ? *grad_scale_dev : 1) * coef (onehot - p) / T;
// with `changed_only` nothing is written when that device value is 1.
cudaError_t token_logp_backward(int dtype, const ScoreRows& s, const float* norm, const float* coef,
                                float grad_scale, const float* grad_scale_dev, int changed_only,
                                void* out, int64_t out_stride, cudaStream_t st);

size_t policy_workspace(int64_t rows);
cudaError_t policy_loss(int dtype, const ScoreRows& s, const PolicyArgs& p, void* out,
                        int64_t out_stride, void* ws, uint32_t* row_status, cudaStream_t st);

size_t preference_workspace(int64_t rows, int64_t pairs);
cudaError_t preference_loss(int dtype, const ScoreRows& s, PreferenceArgs p, float* logp,
                            float* norm, float* coef, float grad_scale, void* out,
                            int64_t out_stride, void* ws, uint32_t* row_status, cudaStream_t st);

// A router's rows: scores [tokens, experts].
struct RouterArgs {
    const void* x;
    int64_t tokens;
    int experts;
    int64_t stride;
    const uint8_t* mask;
    int top_k, renormalize;
};
size_t balance_workspace(int64_t tokens, int experts);
cudaError_t balance_loss(int dtype, const RouterArgs& a, float* loss, int64_t* counts,
                         int32_t* chosen, float* gates, int64_t* live, void* ws, cudaStream_t st);
cudaError_t balance_backward(int dtype, const RouterArgs& a, const int64_t* counts,
                             const int32_t* chosen, const float* gates, const int64_t* live,
                             const float* grad_gates, float grad_loss, const float* grad_loss_dev,
                             void* out, int64_t out_stride, cudaStream_t st);

}  // namespace isodev
