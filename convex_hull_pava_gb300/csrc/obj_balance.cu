// A router's choice of experts, its balance loss and its gradient.
//
//   p[t, e] = softmax of row t over the experts;   n[e] = tokens that chose e
//   L = E / (k T^2) sum_e n[e] sum_t p[t, e]       (E experts, k choices, T live tokens)
//   gate[t, i] = p[t, e_i], or p[t, e_i] / sum_j p[t, e_j]
//   d L / d x[t, e] = p[t, e] (u[e] - sum_f p[t, f] u[f]),   u[e] = E n[e] / (k T^2)
//
// The counts are whole numbers and carry no gradient.  A token is live when its mask says so and
// some expert is open to it (a score above -inf).
#include "obj_internal.h"
#include "obj_device.cuh"
#include "obj_launch.h"

#include <type_traits>

namespace isodev {

namespace {

// Threads of a CTA: fewer where a lane holds 32 scores, for its registers and the CTA's shared memory.
template <int EPL>
constexpr int token_threads = EPL == 32 ? 256 : 512;
constexpr int kTokCtas = 304;  // two CTAs for each of 152 SMs: what the workspace has room for
constexpr int kFinishCtas = 8;

// Order-preserving key of a score; 0 for what is never chosen (-inf and NaN), equal for both zeros.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float choice_score(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

struct BalanceParts {
    float* p;        // [grid][experts] sums of probabilities
    uint32_t* n;     // [grid][experts] tokens that chose each
    uint32_t* live;  // [grid]
};

// G lanes hold a token's scores, EPL each, in chunks of CH neighbours: chunk c of lane l holds
// experts (l + G c) CH and on.  Several tokens to a warp where G < 32 (then EPL is 1).
template <class T, int G, int EPL>
struct TokenRow {
    static constexpr int N = 16 / (int)sizeof(T);
    static constexpr int CH = EPL < N ? EPL : N;
    static constexpr int BYTES = CH * (int)sizeof(T);
    T v[EPL];
    static __device__ __forceinline__ int expert(int lane, int i) { return (lane + G * (i / CH)) * CH + i % CH; }
    __device__ __forceinline__ void load(const T* x, int lane, int experts, bool whole) {
#pragma unroll
        for (int c = 0; c < EPL / CH; ++c) {
            const int e = (lane + G * c) * CH;
            if (whole) {
                if (e < experts) {
                    if constexpr (BYTES == 16) {
                        *reinterpret_cast<uint4*>(&v[c * CH]) = *reinterpret_cast<const uint4*>(x + e);
                    } else if constexpr (BYTES == 8) {
                        *reinterpret_cast<uint2*>(&v[c * CH]) = *reinterpret_cast<const uint2*>(x + e);
                    } else if constexpr (BYTES == 4) {
                        *reinterpret_cast<uint32_t*>(&v[c * CH]) = *reinterpret_cast<const uint32_t*>(x + e);
                    } else {
                        v[c] = x[e];
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (e + i < experts) v[c * CH + i] = x[e + i];
            }
        }
    }
    __device__ __forceinline__ void store(T* x, int lane, int experts, bool whole) const {
#pragma unroll
        for (int c = 0; c < EPL / CH; ++c) {
            const int e = (lane + G * c) * CH;
            if (whole) {
                if (e < experts) {
                    if constexpr (BYTES == 16) {
                        store_streaming(x + e, *reinterpret_cast<const uint4*>(&v[c * CH]));
                    } else if constexpr (BYTES == 8) {
                        *reinterpret_cast<uint2*>(x + e) = *reinterpret_cast<const uint2*>(&v[c * CH]);
                    } else if constexpr (BYTES == 4) {
                        *reinterpret_cast<uint32_t*>(x + e) = *reinterpret_cast<const uint32_t*>(&v[c * CH]);
                    } else {
                        x[e] = v[c];
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (e + i < experts) x[e + i] = v[c * CH + i];
            }
        }
    }
    // The scores, -inf past the last expert.
    __device__ __forceinline__ void scores(float (&s)[EPL], int lane, int experts) const {
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = expert(lane, i) < experts ? to_f32(v[i]) : -INFINITY;
    }
};

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
template <int G>
__device__ __forceinline__ float group_add(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// The exponentials of a token's scores, their sum in st.s and the largest score in st.m.
template <int G, int EPL>
__device__ __forceinline__ SoftState token_softmax(const float (&v)[EPL], float (&e)[EPL]) {
    SoftState st;
    float m = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
    st.m = group_max<G>(m);
    const SoftRef ref(st.m, kLog2e);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        e[i] = ref.exp(v[i]);
        s += e[i];
    }
    st.s = group_add<G>(s);
    return st;
}

// Whether a token takes part, given its mask: some score is above -inf (or NaN, which shows).
__device__ __forceinline__ bool token_open(SoftState st) { return !(st.m == -INFINITY && st.s == 0.f); }

// A group of G lanes a token.  The choice: with EPL = 1 each lane counts the scores above its own.
// Otherwise the k-th largest of the lanes' largest scores bounds the k-th largest score from below;
// the scores that reach it (k and a few more) are collected and each counts those above it.  When
// more than 32 reach it, k rounds of one maximum each.
template <class T, int G, int EPL>
__global__ void __launch_bounds__(token_threads<EPL>, EPL <= 8 ? 2 : 1)
balance_tokens_kernel(RouterArgs a, BalanceParts b, int whole, int32_t* __restrict__ chosen,
                      float* __restrict__ gates) {
    constexpr int kTokThreads = token_threads<EPL>, kTokWarps = kTokThreads / 32;
    static_assert(G == 32 || EPL == 1, "several tokens to a warp hold a score a lane");
    __shared__ uint64_t found[EPL == 1 ? 1 : kTokWarps][32];
    __shared__ float sh_p[G * EPL];
    __shared__ uint32_t sh_n[G * EPL];
    __shared__ uint32_t sh_live;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane & (G - 1), E = a.experts, k = a.top_k;
    for (int e = threadIdx.x; e < G * EPL; e += kTokThreads) {
        sh_n[e] = 0u;
        sh_p[e] = 0.f;
    }
    if (threadIdx.x == 0) sh_live = 0u;
    __syncthreads();
    let_next_start();
    float psum[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) psum[i] = 0.f;
    uint32_t tokens = 0;
    const int64_t step = (int64_t)gridDim.x * kTokWarps * (32 / G);
    const int64_t warp_first = ((int64_t)blockIdx.x * kTokWarps + warp) * (32 / G);
    const T* const base = static_cast<const T*>(a.x);
    TokenRow<T, G, EPL> row;
    bool on = false;
    auto fetch = [&](int64_t t) {
        on = t < a.tokens && (!a.mask || a.mask[t] != 0);
        if (on) row.load(base + t * a.stride, gl, E, whole);
    };
    fetch(warp_first + lane / G);
    for (int64_t first = warp_first; first < a.tokens; first += step) {
        const int64_t t = first + lane / G;
        float v[EPL], e[EPL];
        row.scores(v, gl, E);
        const bool was_on = on;
        fetch(t + step);
        if (!was_on) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
        }
        const SoftState st = token_softmax<G, EPL>(v, e);
        const bool open = was_on && token_open(st);
        const float inv = open ? 1.f / st.s : 0.f;
        if (gl == 0 && open) ++tokens;
        const SoftRef ref(st.m, kLog2e);
        if (open) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) psum[i] = fmaf(e[i], inv, psum[i]);
        }
        int32_t* const to = chosen + t * k;
        float* const gate_to = gates + t * k;
        if constexpr (EPL == 1) {
            const uint32_t key = choice_key(v[0]);
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < G; ++j) {
                const uint32_t other = __shfl_sync(~0u, key, (lane & ~(G - 1)) | j);
                rank += other > key || (other == key && j < gl) ? 1 : 0;
            }
            const bool mine = open && key != 0u && rank < k;
            float gate = mine ? e[0] : 0.f;
            gate *= a.renormalize ? 1.f / group_add<G>(gate) : inv;
            if (mine) {
                to[rank] = gl;
                gate_to[rank] = gate;
                atomicAdd(&sh_n[gl], 1u);
            }
            // the places that no open expert takes
            const unsigned in_group = G == 32 ? ~0u : ((1u << (G & 31)) - 1u) << (lane & ~(G - 1));
            const int taken = __popc(__ballot_sync(~0u, mine) & in_group);
            if (t < a.tokens)
                for (int c = taken + gl; c < k; c += G) {
                    to[c] = -1;
                    gate_to[c] = 0.f;
                }
        } else {
            if (!open) {
                if (lane < k) {
                    to[lane] = -1;
                    gate_to[lane] = 0.f;
                }
                continue;
            }
            float top = v[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) top = fmaxf(top, v[i]);
            uint32_t most = choice_key(top), bound = 0u;
            for (int c = 0; c < k; ++c) {
                bound = __reduce_max_sync(~0u, most);
                if (most == bound) most = 0u;
            }
            const float least = bound == 0u ? __uint_as_float(0xff7fffffu) : choice_score(bound);
            int n = 0;
            uint64_t* const list = found[warp];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const bool is = v[i] >= least;
                const unsigned all = __ballot_sync(~0u, is);
                if (all == 0u) continue;
                const int at = n + __popc(all & ((1u << lane) - 1u));
                if (is && at < 32)
                    list[at] = (uint64_t)choice_key(v[i]) << 32 | (0xffffffffu - (uint32_t)row.expert(lane, i));
                n += __popc(all);
            }
            __syncwarp();
            int mine = -1, rank = 32;
            float gate = 0.f;
            if (n <= 32) {
                const uint64_t own = lane < n ? list[lane] : 0u;
                rank = 0;
                for (int j = 0; j < n; ++j) rank += list[j] > own ? 1 : 0;
                if (lane < n && rank < k) {
                    mine = (int)(0xffffffffu - (uint32_t)own);
                    gate = ref.exp(choice_score((uint32_t)(own >> 32)));
                    atomicAdd(&sh_n[mine], 1u);
                }
                n = min(n, k);
            } else {
                unsigned gone = 0u;  // of this lane's scores
                n = 0;
                for (int c = 0; c < k; ++c) {
                    uint32_t key = 0u;
                    int at = -1;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        const uint32_t q = choice_key(v[i]);
                        if (!(gone >> i & 1u) && (q > key || (q == key && q != 0u && row.expert(lane, i) < row.expert(lane, at)))) {
                            key = q;
                            at = i;
                        }
                    }
                    const uint32_t best = __reduce_max_sync(~0u, key);
                    if (best == 0u) break;
                    const unsigned which = key == best ? (unsigned)row.expert(lane, at) : ~0u;
                    const unsigned winner = __reduce_min_sync(~0u, which);
                    if (which == winner) {
                        gone |= 1u << at;
                        atomicAdd(&sh_n[winner], 1u);
                    }
                    if (lane == c) {
                        mine = (int)winner;
                        rank = c;
                        gate = ref.exp(choice_score(best));
                    }
                    n = c + 1;
                }
            }
            gate *= a.renormalize ? 1.f / warp_add(gate) : inv;
            if (mine >= 0) {
                to[rank] = mine;
                gate_to[rank] = gate;
            }
            if (lane >= n && lane < k) {
                to[lane] = -1;
                gate_to[lane] = 0.f;
            }
        }
    }
    // the CTA's sums, in the order of its warps
    if constexpr (G < 32) {
#pragma unroll
        for (int o = 16; o >= G; o >>= 1) psum[0] += __shfl_xor_sync(~0u, psum[0], o);
    }
    for (int w = 0; w < kTokWarps; ++w) {
        if (warp == w && lane < G) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) sh_p[row.expert(gl, i)] += psum[i];
        }
        __syncthreads();
    }
    tokens = __reduce_add_sync(~0u, tokens);
    if (lane == 0) atomicAdd(&sh_live, tokens);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kTokThreads) {
        b.p[(int64_t)blockIdx.x * E + e] = sh_p[e];
        b.n[(int64_t)blockIdx.x * E + e] = sh_n[e];
    }
    if (threadIdx.x == 0) b.live[blockIdx.x] = sh_live;
}

// The CTAs' sums, in a fixed order, by one cluster that shares the experts; the loss.
__global__ void __launch_bounds__(512)
balance_finish_kernel(BalanceParts b, int grid, int E, int top_k, float* __restrict__ loss,
                      int64_t* __restrict__ counts, int64_t* __restrict__ live) {
    __shared__ float sh_p[512];
    __shared__ uint32_t sh_n[512];
    __shared__ float sh_sum[kFinishCtas], sh_warp[16];
    const int rank = (int)cluster_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = (E + kFinishCtas - 1) / kFinishCtas;  // at most 128
    int cols = 1;
    while (cols < share) cols *= 2;
    const int col = tid & (cols - 1), part = tid / cols, parts = 512 / cols;
    const int e = rank * share + col;
    const bool has = col < share && e < E;
    wait_for_previous();
    float p = 0.f;
    uint32_t n = 0u;
    if (has)
        for (int g = part; g < grid; g += parts) {
            p += b.p[(int64_t)g * E + e];
            n += b.n[(int64_t)g * E + e];
        }
    sh_p[tid] = p;
    sh_n[tid] = n;
    __syncthreads();
    float product = 0.f;
    if (part == 0 && has) {
        uint64_t total = n;
        Sum s;
        s.add(p);
        for (int q = 1; q < parts; ++q) {
            s.add(sh_p[q * cols + col]);
            total += sh_n[q * cols + col];
        }
        counts[e] = (int64_t)total;
        product = s.value() * (float)total;
    }
    product = warp_add(product);
    if (lane == 0) sh_warp[warp] = product;
    __syncthreads();
    if (tid == 0) {
        float s = 0.f;
        for (int w = 0; w < 16; ++w) s += sh_warp[w];
        store_remote(&sh_sum[rank], 0, s);
    }
    __syncwarp();
    cluster_sync();
    if (rank == 0 && warp == 0) {
        unsigned long long t = 0;
        for (int g = lane; g < grid; g += 32) t += b.live[g];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
        if (lane == 0) {
            float s = 0.f;
            for (int c = 0; c < kFinishCtas; ++c) s += sh_sum[c];
            const float tokens = (float)t;
            *live = (int64_t)t;
            *loss = t > 0 ? (float)E / ((float)top_k * tokens) * (s / tokens) : 0.f;
        }
    }
}

// The last tokens first: what the forward read last is still in L2.
template <class T, int G, int EPL>
__global__ void __launch_bounds__(token_threads<EPL>, EPL <= 8 ? 2 : 1)
balance_backward_kernel(RouterArgs a, int whole, const int64_t* __restrict__ counts,
                        const int32_t* __restrict__ chosen, const float* __restrict__ gates,
                        const int64_t* __restrict__ live, const float* __restrict__ grad_gates,
                        float grad_loss, const float* __restrict__ grad_loss_dev,
                        T* __restrict__ out, int64_t out_stride) {
    constexpr int kTokThreads = token_threads<EPL>, kTokWarps = kTokThreads / 32;
    // the gates' part of u (or of the gradient), at the chosen experts; zero in between
    __shared__ __align__(16) float extra[kTokWarps * (32 / G)][G * EPL];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane & (G - 1), E = a.experts, k = a.top_k;
    float* const mine = extra[warp * (32 / G) + lane / G];
    for (int e = gl; e < G * EPL; e += G) mine[e] = 0.f;
    wait_for_previous();
    if (grad_loss_dev) grad_loss *= *grad_loss_dev;
    const float tokens = fmaxf((float)*live, 1.f);
    const float f = grad_loss * ((float)E / ((float)k * tokens)) / tokens;
    float u[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = TokenRow<T, G, EPL>::expert(gl, i);
        u[i] = e < E ? f * (float)counts[e] : 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * kTokWarps * (32 / G);
    const int64_t warp_first = ((int64_t)blockIdx.x * kTokWarps + warp) * (32 / G);
    const T* const base = static_cast<const T*>(a.x);
    TokenRow<T, G, EPL> row;
    bool on = false;
    int at = -1;
    float g = 0.f, gate = 0.f;
    // lane gl's first slot of token t beside its scores; further slots (k > G) are read in place
    auto fetch = [&](int64_t t) {
        on = t >= 0 && t < a.tokens && (!a.mask || a.mask[t] != 0);
        at = -1;
        if (!on) return;
        row.load(base + t * a.stride, gl, E, whole);
        if (grad_gates && gl < k) {
            at = chosen[t * k + gl];
            g = grad_gates[t * k + gl];
            gate = gates[t * k + gl];
        }
    };
    fetch(a.tokens - 1 - (warp_first + lane / G));
    for (int64_t first = warp_first; first < a.tokens; first += step) {
        const int64_t t = a.tokens - 1 - (first + lane / G);
        float v[EPL], e[EPL];
        row.scores(v, gl, E);
        const bool was_on = on;
        const int slot = at;
        const float g_slot = g, gate_slot = gate;
        fetch(t - step);
        if (!was_on) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
        }
        const SoftState st = token_softmax<G, EPL>(v, e);
        const bool open = was_on && token_open(st);
        // k <= experts <= G where EPL is 1, and k <= 32 = G otherwise: a slot a lane
        const bool has = open && slot >= 0 && slot < E;
        float put = has ? g_slot : 0.f;
        if (a.renormalize) {  // the gates are a softmax of their own over the chosen
            const float mean = group_add<G>(has ? gate_slot * put : 0.f);
            put = has ? gate_slot * (put - mean) : 0.f;
        }
        __syncwarp();
        if (has) mine[slot] = put;
        __syncwarp();
        float x[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] = mine[row.expert(gl, i)];
        __syncwarp();
        if (has) mine[slot] = 0.f;
        const float inv = 1.f / st.s;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            e[i] *= inv;
            dot = fmaf(e[i], a.renormalize ? u[i] : u[i] + x[i], dot);
        }
        dot = group_add<G>(dot);
        if (t < 0) continue;
        TokenRow<T, G, EPL> d;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            d.v[i] = from_f32<T>(!open ? 0.f : a.renormalize ? fmaf(e[i], u[i] - dot, x[i]) : e[i] * (u[i] + x[i] - dot));
        d.store(out + t * out_stride, gl, E, whole);
    }
}

inline int token_grid(int64_t tokens, int per_warp, int threads) {
    const int64_t per = (int64_t)(threads / 32) * per_warp;
    return (int)std::max<int64_t>(1, std::min<int64_t>((tokens + per - 1) / per, kTokCtas));
}

// Lanes a token and scores a lane: the fewest lanes that hold a score each up to 32 experts, then
// the smallest power of two of scores a lane.
template <class F>
cudaError_t by_experts(int experts, F f) {
    using std::integral_constant;
    if (experts <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (experts <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (experts <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (experts <= 64) return f(integral_constant<int, 32>{}, integral_constant<int, 2>{});
    if (experts <= 128) return f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
    if (experts <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
    if (experts <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
}

// Whether a row is whole chunks of `ch` scores, each aligned to its size.
inline bool chunks_fit(const void* x, int64_t rows, int64_t stride, int experts, int ch, int size) {
    return experts % ch == 0 && reinterpret_cast<uintptr_t>(x) % (unsigned)(ch * size) == 0 &&
           (rows <= 1 || stride % ch == 0);
}

}  // namespace

size_t balance_workspace(int64_t tokens, int experts) {
    return 2048 + (size_t)token_grid(tokens, 1, 256) * experts * 8;
}

cudaError_t balance_loss(int dtype, const RouterArgs& a, float* loss, int64_t* counts,
                         int32_t* chosen, float* gates, int64_t* live, void* ws, cudaStream_t st) {
    BalanceParts b;
    b.live = static_cast<uint32_t*>(ws);
    int grid = 0;
    cudaError_t e = by_type(dtype, [&](auto t) {
        return by_experts(a.experts, [&](auto g, auto epl) {
            using T = decltype(t);
            constexpr int G = decltype(g)::value, EPL = decltype(epl)::value;
            grid = token_grid(a.tokens, 32 / G, token_threads<EPL>);
            b.p = reinterpret_cast<float*>(static_cast<char*>(ws) + 2048);
            b.n = reinterpret_cast<uint32_t*>(b.p + (int64_t)grid * a.experts);
            const int whole = chunks_fit(a.x, a.tokens, a.stride, a.experts, TokenRow<T, G, EPL>::CH, sizeof(T));
            balance_tokens_kernel<T, G, EPL><<<grid, token_threads<EPL>, 0, st>>>(a, b, whole, chosen, gates);
            return cudaGetLastError();
        });
    });
    if (e != cudaSuccess) return e;
    ClusterLaunch l(kFinishCtas, 512, 0, kFinishCtas, true, st);
    return l(balance_finish_kernel, b, grid, a.experts, a.top_k, loss, counts, live);
}

cudaError_t balance_backward(int dtype, const RouterArgs& a, const int64_t* counts,
                             const int32_t* chosen, const float* gates, const int64_t* live,
                             const float* grad_gates, float grad_loss, const float* grad_loss_dev,
                             void* out, int64_t out_stride, cudaStream_t st) {
    if (a.tokens == 0) return cudaSuccess;
    return by_type(dtype, [&](auto t) {
        return by_experts(a.experts, [&](auto g, auto epl) {
            using T = decltype(t);
            constexpr int G = decltype(g)::value, EPL = decltype(epl)::value, CH = TokenRow<T, G, EPL>::CH;
            const int whole = chunks_fit(a.x, a.tokens, a.stride, a.experts, CH, sizeof(T)) &&
                              chunks_fit(out, a.tokens, out_stride, a.experts, CH, sizeof(T));
            ClusterLaunch l(token_grid(a.tokens, 32 / G, token_threads<EPL>), token_threads<EPL>, 0, 1, true, st);
            return l(balance_backward_kernel<T, G, EPL>, a, whole, counts, chosen, gates, live, grad_gates,
                     grad_loss, grad_loss_dev, static_cast<T*>(out), out_stride);
        });
    });
}

}  // namespace isodev
