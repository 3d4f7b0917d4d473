// A router's choice of experts, its balance loss and its gradient.
//
//   p[t, e] = softmax of row t over the experts;   n[e] = tokens that chose e
//   L = E / (k T^2) sum_e n[e] sum_t p[t, e]       (E experts, k choices, T live tokens)
//   gate[t, i] = p[t, e_i], or p[t, e_i] / sum_j p[t, e_j]
//   d L / d x[t, e] = p[t, e] (u[e] - sum_f p[t, f] u[f]),   u[e] = E n[e] / (k T^2)
//
// The counts are whole numbers and carry no gradient.  A token is live when its
// mask says so and some expert is open to it (a score above -inf).
#include "obj_internal.h"
#include "obj_device.cuh"

#include <algorithm>

namespace isodev {

namespace {

constexpr int kTokThreads = 256;
constexpr int kTokWarps = kTokThreads / 32;

inline int token_grid(int64_t tokens) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((tokens + kTokWarps - 1) / kTokWarps, 304));
}

// Order-preserving key of a score; 0 for what is never chosen (-inf and NaN),
// equal for both zeros.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Balance {
    float* p;         // [grid][experts] sums of probabilities
    uint32_t* n;      // [grid][experts] counts
    uint32_t* live;   // [grid]
};

// A warp per token; lane l holds experts l, l + 32, ...
template <class T, int EPL>
__global__ void __launch_bounds__(kTokThreads)
balance_tokens_kernel(RouterArgs a, Balance b, int32_t* __restrict__ chosen,
                      float* __restrict__ gates) {
    __shared__ float sh_p[kTokWarps][EPL * 32];
    __shared__ uint32_t sh_n[EPL * 32];
    __shared__ uint32_t sh_live;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
    for (int e = threadIdx.x; e < EPL * 32; e += kTokThreads) sh_n[e] = 0u;
    if (threadIdx.x == 0) sh_live = 0u;
    __syncthreads();
    float psum[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) psum[i] = 0.f;
    uint32_t tokens = 0;
    for (int64_t t = (int64_t)blockIdx.x * kTokWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kTokWarps) {
        const bool on = !a.mask || a.mask[t] != 0;
        float v[EPL];
        SoftState st = soft_empty();
        if (on) {
            const T* x = static_cast<const T*>(a.x) + t * a.stride;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = lane + 32 * i;
                v[i] = e < E ? to_f32(x[e]) : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) soft_raise(st, v[i], kLog2e);
            const SoftRef ref(st.m, kLog2e);
#pragma unroll
            for (int i = 0; i < EPL; ++i) st.s += ref.exp(v[i]);
            st = soft_warp(st, kLog2e);
        }
        if (!on || (st.m == -INFINITY && st.s == 0.f)) {
            if (lane < a.top_k) {
                chosen[t * a.top_k + lane] = -1;
                gates[t * a.top_k + lane] = 0.f;
            }
            continue;
        }
        ++tokens;
        const float inv = 1.f / st.s;
        const SoftRef ref(st.m, kLog2e);
        uint32_t key[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            psum[i] += ref.exp(v[i]) * inv;
            key[i] = choice_key(v[i]);
        }
        int mine = -1;
        float gate = 0.f, total = 0.f;
        for (int c = 0; c < a.top_k; ++c) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) best = max(best, key[i]);
            best = __reduce_max_sync(~0u, best);
            if (best == 0u) break;
            unsigned at = ~0u;
#pragma unroll
            for (int i = EPL - 1; i >= 0; --i)
                if (key[i] == best) at = lane + 32 * i;
            at = __reduce_min_sync(~0u, at);
            float g = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (at == lane + 32 * i) {
                    key[i] = 0u;
                    g = ref.exp(v[i]);
                    atomicAdd(&sh_n[at], 1u);
                }
            g = __shfl_sync(~0u, g, at & 31);
            total += g;
            if (lane == c) {
                mine = (int)at;
                gate = g;
            }
        }
        if (lane < a.top_k) {
            chosen[t * a.top_k + lane] = mine;
            gates[t * a.top_k + lane] = mine < 0 ? 0.f : gate / (a.renormalize ? total : st.s);
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) sh_p[warp][lane + 32 * i] = psum[i];
    if (lane == 0) atomicAdd(&sh_live, tokens);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kTokThreads) {
        float s = 0.f;
        for (int w = 0; w < kTokWarps; ++w) s += sh_p[w][e];
        b.p[(int64_t)blockIdx.x * E + e] = s;
        b.n[(int64_t)blockIdx.x * E + e] = sh_n[e];
    }
    if (threadIdx.x == 0) b.live[blockIdx.x] = sh_live;
}

// The CTAs' sums, in a fixed order; the loss.
__global__ void __launch_bounds__(1024)
balance_finish_kernel(Balance b, int grid, int E, int top_k, float* __restrict__ loss,
                      int64_t* __restrict__ counts, int64_t* __restrict__ live) {
    __shared__ double sh[32];
    double sum = 0.0;
    for (int e = threadIdx.x; e < E; e += 1024) {
        double s = 0.0;
        int64_t c = 0;
        for (int g = 0; g < grid; ++g) {
            s += b.p[(int64_t)g * E + e];
            c += b.n[(int64_t)g * E + e];
        }
        counts[e] = c;
        sum += s * (double)c;
    }
    sum = cta_sum<1024>(sum, sh);
    double t = 0.0;
    for (int g = threadIdx.x; g < grid; g += 1024) t += b.live[g];
    t = cta_sum<1024>(t, sh);
    if (threadIdx.x == 0) {
        *live = (int64_t)t;
        *loss = t > 0.0 ? (float)((double)E / ((double)top_k * t * t) * sum) : 0.f;
    }
}

template <class T, int EPL>
__global__ void __launch_bounds__(kTokThreads)
balance_backward_kernel(RouterArgs a, const int64_t* __restrict__ counts,
                        const int32_t* __restrict__ chosen, const float* __restrict__ gates,
                        const int64_t* __restrict__ live, const float* __restrict__ grad_gates,
                        float grad_loss, const float* __restrict__ grad_loss_dev,
                        T* __restrict__ out, int64_t out_stride) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
    if (grad_loss_dev) grad_loss *= *grad_loss_dev;
    const double tokens = fmax((double)*live, 1.0);
    const float f = (float)((double)grad_loss * E / ((double)a.top_k * tokens * tokens));
    float u[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) u[i] = lane + 32 * i < E ? f * (float)counts[lane + 32 * i] : 0.f;
    for (int64_t t = (int64_t)blockIdx.x * kTokWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kTokWarps) {
        const bool on = !a.mask || a.mask[t] != 0;
        float v[EPL];
        SoftState st = soft_empty();
        if (on) {
            const T* x = static_cast<const T*>(a.x) + t * a.stride;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = lane + 32 * i;
                v[i] = e < E ? to_f32(x[e]) : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) soft_raise(st, v[i], kLog2e);
            const SoftRef ref(st.m, kLog2e);
#pragma unroll
            for (int i = 0; i < EPL; ++i) st.s += ref.exp(v[i]);
            st = soft_warp(st, kLog2e);
        }
        T* o = out + t * out_stride;
        if (!on || (st.m == -INFINITY && st.s == 0.f)) {
            for (int e = lane; e < E; e += 32) o[e] = from_f32<T>(0.f);
            continue;
        }
        int e_own = -1;
        float g_own = 0.f, gate_own = 0.f;
        if (grad_gates && lane < a.top_k) {
            e_own = chosen[t * a.top_k + lane];
            if (e_own >= 0) {
                g_own = grad_gates[t * a.top_k + lane];
                gate_own = gates[t * a.top_k + lane];
            }
        }
        if (a.renormalize) {  // the gates are a softmax of their own over the chosen
            float dot = gate_own * g_own;
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) dot += __shfl_xor_sync(~0u, dot, k);
            g_own = gate_own * (g_own - dot);
        }
        float extra[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) extra[i] = 0.f;
        if (grad_gates)
            for (int c = 0; c < a.top_k; ++c) {
                const int e = __shfl_sync(~0u, e_own, c);
                const float g = __shfl_sync(~0u, g_own, c);
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e == lane + 32 * i) extra[i] = g;
            }
        float dot = 0.f;
        const float inv = 1.f / st.s;
        const SoftRef ref(st.m, kLog2e);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = ref.exp(v[i]) * inv;
            dot += v[i] * (a.renormalize ? u[i] : u[i] + extra[i]);
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) dot += __shfl_xor_sync(~0u, dot, k);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            if (e < E)
                o[e] = from_f32<T>(a.renormalize ? v[i] * (u[i] - dot) + extra[i]
                                                 : v[i] * (u[i] + extra[i] - dot));
        }
    }
}

inline Balance carve_balance(void* ws, int64_t tokens, int experts) {
    const int grid = token_grid(tokens);
    char* at = static_cast<char*>(ws);
    Balance b;
    b.live = reinterpret_cast<uint32_t*>(at);
    at += 4096;
    b.p = reinterpret_cast<float*>(at);
    b.n = reinterpret_cast<uint32_t*>(b.p + (int64_t)grid * experts);
    return b;
}

template <class T, int EPL>
cudaError_t run_balance(const RouterArgs& a, const Balance& b, int32_t* chosen, float* gates,
                        cudaStream_t st) {
    balance_tokens_kernel<T, EPL><<<token_grid(a.tokens), kTokThreads, 0, st>>>(a, b, chosen, gates);
    return cudaGetLastError();
}

template <class T, int EPL>
cudaError_t run_backward(const RouterArgs& a, const int64_t* counts, const int32_t* chosen,
                         const float* gates, const int64_t* live, const float* grad_gates,
                         float grad_loss, const float* grad_loss_dev, void* out,
                         int64_t out_stride, cudaStream_t st) {
    balance_backward_kernel<T, EPL><<<token_grid(a.tokens), kTokThreads, 0, st>>>(
        a, counts, chosen, gates, live, grad_gates, grad_loss, grad_loss_dev, static_cast<T*>(out),
        out_stride);
    return cudaGetLastError();
}

// Experts a lane holds: the smallest power of two with 32 of them covering E.
template <class F>
cudaError_t by_experts(int experts, F f) {
    if (experts <= 32) return f(std::integral_constant<int, 1>{});
    if (experts <= 64) return f(std::integral_constant<int, 2>{});
    if (experts <= 128) return f(std::integral_constant<int, 4>{});
    if (experts <= 256) return f(std::integral_constant<int, 8>{});
    if (experts <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

template <class F>
cudaError_t by_dtype(int dtype, F f) {
    if (dtype == ISO_F32) return f(float{});
    if (dtype == ISO_BF16) return f(__nv_bfloat16{});
    return f(__half{});
}

}  // namespace

size_t balance_workspace(int64_t tokens, int experts) {
    return 4096 + (size_t)token_grid(tokens) * experts * 8;
}

cudaError_t balance_loss(int dtype, const RouterArgs& a, float* loss, int64_t* counts,
                         int32_t* chosen, float* gates, int64_t* live, void* ws, cudaStream_t st) {
    const Balance b = carve_balance(ws, a.tokens, a.experts);
    cudaError_t e = by_dtype(dtype, [&](auto t) {
        return by_experts(a.experts, [&](auto epl) {
            return run_balance<decltype(t), decltype(epl)::value>(a, b, chosen, gates, st);
        });
    });
    if (e != cudaSuccess) return e;
    balance_finish_kernel<<<1, 1024, 0, st>>>(b, token_grid(a.tokens), a.experts, a.top_k, loss,
                                              counts, live);
    return cudaGetLastError();
}

cudaError_t balance_backward(int dtype, const RouterArgs& a, const int64_t* counts,
                             const int32_t* chosen, const float* gates, const int64_t* live,
                             const float* grad_gates, float grad_loss, const float* grad_loss_dev,
                             void* out, int64_t out_stride, cudaStream_t st) {
    if (a.tokens == 0) return cudaSuccess;
    return by_dtype(dtype, [&](auto t) {
        return by_experts(a.experts, [&](auto epl) {
            return run_backward<decltype(t), decltype(epl)::value>(
                a, counts, chosen, gates, live, grad_gates, grad_loss, grad_loss_dev, out,
                out_stride, st);
        });
    });
}

}  // namespace isodev
