// Internal declarations of the choices over rows of scores (choice_*.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/iso.h"

namespace isodev {

// A router's rows and how it chooses.
struct RouteArgs {
    const void* x;
    int64_t tokens;
    int experts;
    int64_t stride;
    int top_k;
    const uint8_t* mask;
    const float* bias;
    int score, groups, top_groups, group_best, renormalize;
    float scale;
    float* picked;  // [tokens, top_k] the chosen's scores, written; or NULL
};
cudaError_t route(int dtype, const RouteArgs& a, int64_t* counts, int32_t* chosen, float* gates,
                  cudaStream_t st);
// `picked`: as the forward left them, or NULL: the chosen's scores are read from the rows.
cudaError_t route_backward(int dtype, const RouteArgs& a, const int32_t* chosen, const float* gates,
                           const float* picked, const float* grad_gates, void* out, int64_t out_stride, cudaStream_t st);

// A step of beam search: rows of scores, `beams` of them a batch item.
struct BeamArgs {
    const void* x;
    int64_t batch;
    int beams, n;
    int64_t stride;
    const float* scores;
    const uint8_t* done;
    int64_t end;
    double temperature;
    int keep;
    float* out_scores;
    int32_t* parents;
    int64_t* tokens;
    uint32_t* row_status;
};
size_t beam_workspace(int64_t batch, int beams, int64_t n, int dtype, int keep);
cudaError_t beam_choose(int dtype, const BeamArgs& a, void* ws, cudaStream_t st);

cudaError_t beam_reorder(const iso_state* states, int64_t count, int64_t batch, int beams,
                         const int32_t* parents, cudaStream_t st);

}  // namespace isodev
