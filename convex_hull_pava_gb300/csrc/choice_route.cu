// A router's choice of experts by float32 scores, and the gradient of its gates.
#include "choice_route.cuh"

namespace isodev {

extern template cudaError_t route_rows<__nv_bfloat16>(const RouteArgs&, int64_t*, int32_t*, float*, cudaStream_t);
extern template cudaError_t route_rows<__half>(const RouteArgs&, int64_t*, int32_t*, float*, cudaStream_t);

namespace {

// The gates' part of each gradient element is put together in shared memory, a warp's tokens beside one
// another.  DENSE: softmax without renormalisation, whose gradient has all elements; otherwise only
// the chosen ones' scores are read.
template <class T, int G, int EPL, bool DENSE>
__global__ void __launch_bounds__(256)
route_backward_kernel(RouteArgs a, int whole, const int32_t* chosen, const float* gates, const float* grad_gates,
                      T* out, int64_t out_stride) {
    constexpr int W = 256 / 32, TPW = 32 / G;
    __shared__ __align__(16) float extra[W * TPW][G * EPL];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane & (G - 1), E = a.experts, k = a.top_k;
    float* const mine = extra[warp * TPW + lane / G];
    for (int e = gl; e < G * EPL; e += G) mine[e] = 0.f;
    __syncwarp();
    const int64_t step = (int64_t)gridDim.x * W * TPW;
    const T* const base = static_cast<const T*>(a.x);
    for (int64_t first = ((int64_t)blockIdx.x * W + warp) * TPW; first < a.tokens; first += step) {
        const int64_t t = first + lane / G;
        const bool on = t < a.tokens;
        TokenRow<T, G, EPL> row;
        int slot = -1;
        float g = 0.f, gate = 0.f, x = 0.f;
        if (on) {
            if (DENSE) row.load(base + t * a.stride, gl, E, whole);
            if (gl < k) {
                slot = chosen[t * k + gl];
                gate = gates[t * k + gl];
                g = grad_gates[t * k + gl];
            }
        }
        const bool has = slot >= 0 && slot < E;
        if (!DENSE && has && a.score == ISO_ROUTE_SIGMOID) x = to_f32(base[t * a.stride + slot]);
        const unsigned group = group_lanes<G>();
        const bool any = __ballot_sync(~0u, has) & group;
        const bool bad = __ballot_sync(~0u, has && gate != gate) & group;
        const float dot = group_add<G>(has ? gate * g : 0.f);
        float put;
        if (DENSE) {
            put = a.scale * g;
        } else {
            put = gate * (a.renormalize ? g - dot / a.scale : g);
            if (a.score == ISO_ROUTE_SIGMOID) put *= 1.f / (1.f + expf(x));  // 1 - s
        }
        if (has) mine[slot] = put;
        __syncwarp();
        TokenRow<T, G, EPL> d;
        if (DENSE) {
            float v[EPL], p[EPL];
            row.scores(v, on);
            const SoftState st = token_softmax<G, EPL>(v, p);
            const float inv = 1.f / st.s;
#pragma unroll
            for (int i = 0; i < EPL; ++i) d.v[i] = from_f32<T>(any ? p[i] * inv * (mine[row.expert(gl, i)] - dot) : 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) d.v[i] = from_f32<T>(bad && a.score == ISO_ROUTE_SOFTMAX ? NAN : mine[row.expert(gl, i)]);
        }
        if (on) d.store(out + t * out_stride, gl, E, whole);
        __syncwarp();
        if (has) mine[slot] = 0.f;
        __syncwarp();
    }
}

}  // namespace

cudaError_t route(int dtype, const RouteArgs& a, int64_t* counts, int32_t* chosen, float* gates, cudaStream_t st) {
    return by_type(dtype, [&](auto t) { return route_rows<decltype(t)>(a, counts, chosen, gates, st); });
}

cudaError_t route_backward(int dtype, const RouteArgs& a, const int32_t* chosen, const float* gates,
                           const float* grad_gates, void* out, int64_t out_stride, cudaStream_t st) {
    return by_type(dtype, [&](auto t) {
        return by_experts(a.experts, [&](auto g, auto epl) {
            using T = decltype(t);
            constexpr int G = decltype(g)::value, EPL = decltype(epl)::value, CH = TokenRow<T, G, EPL>::CH;
            const bool dense = a.score == ISO_ROUTE_SOFTMAX && !a.renormalize;
            const int whole = (!dense || chunks_fit(a.x, a.tokens, a.stride, a.experts, CH, sizeof(T))) &&
                              chunks_fit(out, a.tokens, out_stride, a.experts, CH, sizeof(T));
            const int64_t grid = std::min<int64_t>((a.tokens + 256 / G - 1) / (256 / G), 152 * 4);
            auto kernel = dense ? route_backward_kernel<T, G, EPL, true> : route_backward_kernel<T, G, EPL, false>;
            kernel<<<(unsigned)grid, 256, 0, st>>>(a, whole, chosen, gates, grad_gates, static_cast<T*>(out), out_stride);
            const cudaError_t e = cudaGetLastError();
            prof_mark(st, "route_backward");
            return e;
        });
    });
}

}  // namespace isodev
