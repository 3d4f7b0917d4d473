// A router's choice of experts, its gates, and their gradient.
//
//   s[t, e] = softmax of row t over the experts, or 1 / (1 + exp(-x[t, e]));   c = s + bias
//   chosen: the k largest c of the open experts, of the groups with the largest sums of their one or
//   two largest c;   gate[t, i] = scale s[t, e_i], or scale s[t, e_i] / sum_j s[t, e_j]
//
// With w = gate / scale and g the gates' gradient, that of the scores is
//   softmax:               p[e] (scale g[e] - sum_i gate_i g_i)     (g 0 where e is not chosen)
//   softmax, renormalised: gate_i (g_i - sum_j w_j g_j) at the chosen, 0 elsewhere
//   sigmoid:               gate_i (1 - s_i) g_i,  renormalised: gate_i (1 - s_i) (g_i - sum_j w_j g_j)
#include "choice_internal.h"
#include "router_rows.cuh"

namespace isodev {

namespace {

constexpr int kRouteThreads = 256, kRouteWarps = kRouteThreads / 32;

__device__ __forceinline__ double warp_add(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Order-preserving key of a number that is not NaN; both zeros are equal.
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.);
    return b >> 63 ? ~b : b | 1ull << 63;
}

// The choice of one token by a warp in 64 bits: `c` has room for its experts.  Where there is no
// bias the order of c is that of x, which needs no rounding: c holds x then.
template <class T>
__device__ __noinline__ void choose_exact(const RouteArgs& a, const T* x, double* c, int32_t* to, float* gate_to,
                                          uint32_t* counts) {
    const int lane = threadIdx.x & 31, E = a.experts;
    float top = -INFINITY;
    bool bad = false;  // a NaN or +inf: no probabilities
    for (int e = lane; e < E; e += 32) {
        const float v = to_f32(x[e]);
        top = fmaxf(top, v);
        bad |= !(v < INFINITY);
    }
    const bool softmax = a.score == ISO_ROUTE_SOFTMAX;
    bad = __any_sync(~0u, bad) && softmax;
    const double m = warp_max(top);
    double sum = 1.;
    if (softmax) {
        double part = 0.;
        for (int e = lane; e < E; e += 32) part += exp((double)to_f32(x[e]) - m);
        sum = warp_add(part);
    }
    auto share = [&](double v) { return softmax ? (bad ? 0. : exp(v - m) / sum) : 1. / (1. + exp(-v)); };
    for (int e = lane; e < E; e += 32) {
        const float v = to_f32(x[e]), b = a.bias ? a.bias[e] : 0.f;
        c[e] = !(v > -INFINITY) || !(b > -INFINITY) ? -INFINITY : a.bias ? share(v) + (double)b : (double)v;
    }
    __syncwarp();
    if (a.groups > 1) {
        const int size = E / a.groups;
        double value = -INFINITY;
        if (lane < a.groups) {
            double first = -INFINITY, second = -INFINITY;
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const double v = c[e];
                second = fmax(second, fmin(first, v));
                first = fmax(first, v);
            }
            value = first;
            if (a.group_best == 2 && first > -INFINITY) {
                if (!a.bias) value = share(first);
                if (second > -INFINITY) value += a.bias ? second : share(second);
            }
        }
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl_sync(~0u, value, g);
            rank += other > value || (other == value && g < lane) ? 1 : 0;
        }
        const unsigned kept = __ballot_sync(~0u, lane < a.groups && rank < a.top_groups);
        for (int e = lane; e < E; e += 32)
            if (!(kept >> (e / size) & 1u)) c[e] = -INFINITY;
    }
    int mine = -1;  // lane i: the i-th expert
    for (int i = 0; i < a.top_k; ++i) {
        uint64_t best = 0;
        int at = E;
        for (int e = lane; e < E; e += 32) {
            const double v = c[e];
            if (v > -INFINITY && order_key(v) > best) {
                best = order_key(v);
                at = e;
            }
        }
        const uint32_t high = __reduce_max_sync(~0u, (uint32_t)(best >> 32));
        const uint32_t low = __reduce_max_sync(~0u, (uint32_t)(best >> 32) == high ? (uint32_t)best : 0u);
        if (high == 0u && low == 0u) break;
        const bool equal = best == ((uint64_t)high << 32 | low);
        const int winner = (int)__reduce_min_sync(~0u, equal ? (unsigned)at : ~0u);
        if (equal && at == winner) c[at] = -INFINITY;
        if (lane == i) mine = winner;
    }
    // the gates; where they are shares of their sum, against the largest, so that none underflows alone
    const double v = mine >= 0 ? (double)to_f32(x[mine]) : 0.;
    double s = 0.;
    if (!a.renormalize) {
        s = mine >= 0 ? share(v) : 0.;
    } else {
        const double most = (double)warp_max(mine >= 0 ? (float)v : -INFINITY);
        if (softmax)
            s = mine >= 0 ? exp(v - most) : 0.;
        else if (mine >= 0)
            s = v > 0. ? 1. / (1. + exp(-v)) : exp(v - fmin(most, 0.)) / (1. + exp(v));
        s /= warp_add(s);
    }
    if (lane < a.top_k) {
        to[lane] = mine;
        gate_to[lane] = mine < 0 ? 0.f : bad ? NAN : (float)((double)a.scale * s);
        if (mine >= 0) atomicAdd(&counts[mine], 1u);
    }
    __syncwarp();
}

// A warp a token.
template <class T>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(RouteArgs a, int64_t* counts, int32_t* chosen, float* gates) {
    extern __shared__ double values[];  // [kRouteWarps][experts]
    __shared__ uint32_t sh_n[ISO_MAX_EXPERTS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) sh_n[e] = 0u;
    __syncthreads();
    const T* const base = static_cast<const T*>(a.x);
    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        if (a.mask && !a.mask[t]) {
            if (lane < a.top_k) {
                chosen[t * a.top_k + lane] = -1;
                gates[t * a.top_k + lane] = 0.f;
            }
            continue;
        }
        choose_exact(a, base + t * a.stride, values + warp * E, chosen + t * a.top_k, gates + t * a.top_k, sh_n);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads)
        if (sh_n[e]) atomicAdd(reinterpret_cast<unsigned long long*>(counts) + e, (unsigned long long)sh_n[e]);
}

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
    cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)a.experts * sizeof(int64_t), st);
    if (e != cudaSuccess || a.tokens == 0) return e;
    const int64_t grid = std::min<int64_t>((a.tokens + kRouteWarps - 1) / kRouteWarps, 152 * 4);
    const int shared = kRouteWarps * a.experts * (int)sizeof(double);
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (shared > 40 * 1024) {
            const cudaError_t f = cudaFuncSetAttribute(route_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
            if (f != cudaSuccess) return f;
        }
        route_kernel<T><<<(unsigned)grid, kRouteThreads, shared, st>>>(a, counts, chosen, gates);
        const cudaError_t f = cudaGetLastError();
        prof_mark(st, "route");
        return f;
    });
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
