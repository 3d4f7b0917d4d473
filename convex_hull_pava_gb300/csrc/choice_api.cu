// C ABI of the choices over rows of scores (declared in include/iso.h): argument checks.
#include "choice_internal.h"

#include "iso_internal.h"

#include <cmath>

namespace {

constexpr int64_t kMaxN = 2147483647LL;
constexpr int64_t kMaxElems = 1LL << 40;
constexpr int64_t kMaxBytes = 1LL << 48;

iso_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ISO_OK : ISO_ERR_CUDA; }

bool rows_ok(int dtype, int64_t rows, int64_t n, int64_t stride, int64_t least) {
    return (dtype == ISO_F32 || dtype == ISO_BF16 || dtype == ISO_F16) && n >= 1 && n <= kMaxN && rows >= 0 &&
           rows <= kMaxN && stride >= 0 && (rows == 0 || stride <= kMaxElems / rows) && (rows <= 1 || stride >= least);
}

bool route_ok(int dtype, int64_t tokens, int64_t experts, int64_t stride, int64_t least, int top_k, int score,
              int renormalize, float scale) {
    return experts <= ISO_MAX_EXPERTS && rows_ok(dtype, tokens, experts, stride, least) && top_k >= 1 &&
           top_k <= experts && top_k <= ISO_MAX_TOP_K && (score == ISO_ROUTE_SOFTMAX || score == ISO_ROUTE_SIGMOID) &&
           (renormalize == 0 || renormalize == 1) && std::isfinite(scale) && scale > 0.f;
}

bool temperature_ok(double t) {
    return std::isfinite(t) && t > 0. && std::isfinite((float)(1. / t)) && (float)(1. / t) > 0.f &&
           std::isfinite((float)(1.4426950408889634074 / t));
}

// The bytes from a row's or run's start to its last one's end, or -1 where they overlap or leave
// the address space.
int64_t span(int64_t count, int64_t stride, int64_t size) {
    if (count <= 1) return size;
    if (stride < size || stride > kMaxBytes / count) return -1;
    return (count - 1) * stride + size;
}

// Rows hold runs, or (a state whose rows are not its first dimension) runs hold rows.
bool state_ok(const iso_state& s, int64_t rows) {
    if (s.runs < 0 || s.run_bytes < 0 || s.runs > kMaxN || s.run_bytes > kMaxBytes) return false;
    if (s.runs == 0 || s.run_bytes == 0) return true;
    if (!s.base || s.row_stride < 0 || s.run_stride < 0) return false;
    const int64_t row = span(s.runs, s.run_stride, s.run_bytes), column = span(rows, s.row_stride, s.run_bytes);
    return (row > 0 && span(rows, s.row_stride, row) > 0) || (column > 0 && span(s.runs, s.run_stride, column) > 0);
}

}  // namespace

extern "C" {

iso_status iso_route(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t stride, int top_k,
                     const uint8_t* mask, const float* bias, int score, int groups, int top_groups, int group_best,
                     int renormalize, float scale, int64_t* counts, int32_t* chosen, float* gates, float* picked,
                     void* stream) {
    if (!route_ok(dtype, tokens, experts, stride, 0, top_k, score, renormalize, scale) || !counts ||
        (tokens > 0 && (!logits || !chosen || !gates)))
        return ISO_ERR_INVALID_ARG;
    if (groups < 1 || groups > ISO_MAX_GROUPS || experts % groups != 0 || top_groups < 1 || top_groups > groups ||
        top_k > top_groups * (experts / groups) || (groups > 1 && group_best != 1 && group_best != 2))
        return ISO_ERR_INVALID_ARG;
    const isodev::RouteArgs a{logits, tokens, (int)experts, stride,     top_k,       mask,  bias,
                              score,  groups, top_groups,   group_best, renormalize, scale, picked};
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::route(dtype, a, counts, chosen, gates, static_cast<cudaStream_t>(stream)));
}

iso_status iso_route_backward(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t stride,
                              int top_k, int score, int renormalize, float scale, const int32_t* chosen,
                              const float* gates, const float* picked, const float* grad_gates, void* dlogits, int64_t out_stride,
                              void* stream) {
    if (!route_ok(dtype, tokens, experts, stride, 0, top_k, score, renormalize, scale) ||
        !rows_ok(dtype, tokens, experts, out_stride, experts))
        return ISO_ERR_INVALID_ARG;
    if (tokens == 0) return ISO_OK;
    if (!logits || !chosen || !gates || !grad_gates || !dlogits) return ISO_ERR_INVALID_ARG;
    isodev::RouteArgs a{};
    a.x = logits;
    a.tokens = tokens;
    a.experts = (int)experts;
    a.stride = stride;
    a.top_k = top_k;
    a.score = score;
    a.renormalize = renormalize;
    a.scale = scale;
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::route_backward(dtype, a, chosen, gates, picked, grad_gates, dlogits, out_stride,
                                            static_cast<cudaStream_t>(stream)));
}

static bool beam_ok(int64_t batch, int64_t beams, int64_t n, int dtype, int64_t stride, int keep) {
    return batch >= 0 && beams >= 1 && beams <= ISO_MAX_BEAMS && batch <= kMaxN / beams &&
           rows_ok(dtype, batch * beams, n, stride, 0) && keep >= 1 && keep <= ISO_MAX_KEEP;
}

size_t iso_beam_choose_workspace_bytes(int64_t batch, int64_t beams, int64_t n, int dtype, int keep) {
    return beam_ok(batch, beams, n, dtype, 0, keep) ? isodev::beam_workspace(batch, (int)beams, n, dtype, keep) : 0;
}

iso_status iso_beam_choose(const void* logits, int dtype, int64_t batch, int64_t beams, int64_t n, int64_t stride,
                           const float* scores, const uint8_t* done, int64_t end, double temperature, int keep,
                           float* out_scores, int32_t* parents, int64_t* tokens, void* workspace,
                           size_t workspace_bytes, uint32_t* row_status, void* stream) {
    if (!beam_ok(batch, beams, n, dtype, stride, keep) || !temperature_ok(temperature) ||
        (done && (end < 0 || end >= n)))
        return ISO_ERR_INVALID_ARG;
    if (batch == 0) return ISO_OK;
    if (!logits || !scores || !out_scores || !parents || !tokens) return ISO_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < isodev::beam_workspace(batch, (int)beams, n, dtype, keep) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return ISO_ERR_WORKSPACE;
    const isodev::BeamArgs a{logits, batch,       (int)beams, (int)n,     stride,  scores, done,
                             end,    temperature, keep,       out_scores, parents, tokens, row_status};
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::beam_choose(dtype, a, workspace, static_cast<cudaStream_t>(stream)));
}

iso_status iso_beam_reorder(const iso_state* states, int64_t count, int64_t batch, int64_t beams,
                            const int32_t* parents, void* stream) {
    if (count < 0 || count > kMaxN || batch < 0 || beams < 1 || beams > ISO_MAX_BEAMS || batch > kMaxN / beams)
        return ISO_ERR_INVALID_ARG;
    if (count == 0 || batch == 0) return ISO_OK;
    if (!states || !parents) return ISO_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i)
        if (!state_ok(states[i], batch * beams)) return ISO_ERR_INVALID_ARG;
    isodev::prof_start(static_cast<cudaStream_t>(stream));
    return from_cuda(isodev::beam_reorder(states, count, batch, (int)beams, parents, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
