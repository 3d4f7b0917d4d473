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
constexpr int token_threads = EPL >= 16 ? 256 : 512;
template <int EPL>
constexpr int token_ctas_an_sm = EPL == 32 ? 1 : EPL == 16 ? 3 : 2;
constexpr int kMaxCtas = 3 * 152;  // what the workspace has room for
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
    float2* p;       // [grid][experts] sums of probabilities (Sum's hi and lo)
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
    // -inf everywhere: what is past the last expert keeps it, as no load writes there.
    __device__ __forceinline__ TokenRow() {
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = from_f32<T>(-INFINITY);
    }
    __device__ __forceinline__ void scores(float (&s)[EPL], bool on) const {
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = to_f32(v[i]);
        if (!on) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] = -INFINITY;
        }
    }
};

// The lanes of this lane's group.
template <int G>
__device__ __forceinline__ unsigned group_lanes() {
    return G == 32 ? ~0u : ((1u << (G & 31)) - 1u) << (threadIdx.x & 31 & ~(G - 1));
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
    return warp_max(v, group_lanes<G>());
}
struct BalanceOuts {
    float* loss;
    int64_t *counts, *live;
};

// The loss, from sum_e n[e] sum_t p[t, e].
__device__ __forceinline__ void balance_result(const BalanceOuts& o, unsigned long long live, int E, int k, float sum) {
    const float tokens = (float)live;
    *o.live = (int64_t)live;
    *o.loss = live > 0 ? (float)E / ((float)k * tokens) * (sum / tokens) : 0.f;
}

__device__ __forceinline__ Sum as_sum(float2 v) {
    Sum s;
    s.hi = v.x;
    s.lo = v.y;
    return s;
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
    if (ref.far) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) e[i] = ref.exp(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) e[i] = ex2(fmaf(v[i], kLog2e, -ref.c));
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) s += e[i];
    st.s = group_add<G>(s);
    return st;
}

// Whether a token takes part, given its mask: some score is above -inf (or NaN, which shows).
__device__ __forceinline__ bool token_open(SoftState st) { return !(st.m == -INFINITY && st.s == 0.f); }

// A group of G lanes a token, several tokens to a warp where G < 32 (then EPL is 1).  The choice:
// with EPL = 1 each lane counts the scores above its own, four to a read of shared memory (by shuffles
// 32 experts took 57 us and not 55).  Otherwise the k-th largest of the lanes' largest scores bounds
// the k-th largest score from below; the scores that reach it (k and a few more) are collected and
// each counts those above it.  When more than 32 reach it, k rounds of one maximum each.
// The probabilities of an expert are added in float32 over up to 64 tokens of a lane, those sums to one
// of the warp that keeps what it rounds off (in float32 throughout, the loss of 2^26 equal tokens was
// 1.4e-5 off; the same times).
// Bound by instructions: 443 a token at 256 experts and k = 8 (62 us for 131,072 tokens of float32,
// 2.2 TB/s).  k rounds of one maximum each for all took 214 us, collecting by ballots 69, two tokens
// a warp 80.
template <class T, int G, int EPL>
__global__ void __launch_bounds__(token_threads<EPL>, token_ctas_an_sm<EPL>)
balance_tokens_kernel(RouterArgs a, BalanceParts b, BalanceOuts o, int whole,
                      int32_t* __restrict__ chosen, float* __restrict__ gates) {
    constexpr int kTokThreads = token_threads<EPL>, kTokWarps = kTokThreads / 32, TPW = 32 / G;
    static_assert(G == 32 || EPL == 1, "several tokens to a warp hold a score a lane");
    __shared__ __align__(16) float found[EPL == 1 ? 1 : kTokWarps][36];  // scores that may be among the k largest
    __shared__ int found_at[EPL == 1 ? 1 : kTokWarps][32];               // their experts
    __shared__ int found_n[EPL == 1 ? 1 : kTokWarps];
    __shared__ __align__(16) uint32_t keys[EPL == 1 ? kTokWarps : 1][32];
    extern __shared__ float2 warp_sums[];  // [kTokWarps][G * EPL], Sum's hi and lo
    __shared__ uint32_t sh_n[G * EPL];
    __shared__ uint32_t sh_live;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane & (G - 1), E = a.experts, k = a.top_k;
    const unsigned group = group_lanes<G>(), before = group & ((1u << lane) - 1u);
    for (int e = threadIdx.x; e < G * EPL; e += kTokThreads) sh_n[e] = 0u;
    if (threadIdx.x == 0) sh_live = 0u;
    __syncthreads();
    let_next_start();
    float psum[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) psum[i] = 0.f;
    // takes the lanes' sums to the warp's
    auto gather = [&](bool begun) {
        float2* const mine = warp_sums + warp * G * EPL;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            float p = psum[i];
#pragma unroll
            for (int o = 16; o >= G; o >>= 1) p += __shfl_xor_sync(~0u, p, o);
            if (lane < G) {
                float2& at = mine[TokenRow<T, G, EPL>::expert(gl, i)];
                Sum s = begun ? as_sum(at) : Sum();
                s.add(p);
                at = {s.hi, s.lo};
            }
            psum[i] = 0.f;
        }
    };
    uint32_t tokens = 0;
    const int64_t step = (int64_t)gridDim.x * kTokWarps * TPW;
    const int64_t warp_first = ((int64_t)blockIdx.x * kTokWarps + warp) * TPW;
    const T* const base = static_cast<const T*>(a.x);
    TokenRow<T, G, EPL> row;
    bool on = false;
    auto fetch = [&](int64_t t) {
        on = t < a.tokens && (!a.mask || a.mask[t] != 0);
        if (on) row.load(base + t * a.stride, gl, E, whole);
    };
    fetch(warp_first + lane / G);
    int64_t first = warp_first;
    bool begun = false;
    do {
        const int64_t end = min(a.tokens, first + 64 * step);
        for (; first < end; first += step) {
            const int64_t t = first + lane / G;
            float v[EPL], e[EPL];
            row.scores(v, on);
            const bool was_on = on;
            fetch(t + step);
            const SoftState st = token_softmax<G, EPL>(v, e);
            const bool open = was_on && token_open(st);
            const float inv = open ? __frcp_rn(st.s) : 0.f;
            if (gl == 0 && open) ++tokens;
            if (open) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) psum[i] = fmaf(e[i], inv, psum[i]);
            }
            int32_t* const to = chosen + t * k;
            float* const gate_to = gates + t * k;
            int taken = 0;  // places filled
            if constexpr (EPL == 1) {
                const uint32_t key = choice_key(v[0]);
                keys[warp][lane] = key;
                __syncwarp();
                int rank = 0;
#pragma unroll
                for (int j = 0; j < G; j += 4) {
                    const uint4 q = *reinterpret_cast<const uint4*>(&keys[warp][(lane & ~(G - 1)) + j]);
                    const uint32_t other[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) rank += other[i] > key || (other[i] == key && j + i < gl) ? 1 : 0;
                }
                __syncwarp();
                const bool mine = open && key != 0u && rank < k;
                float gate = mine ? e[0] : 0.f;
                // (0 inv: a token without probabilities has no gates)
                gate *= a.renormalize ? fmaf(0.f, inv, 1.f / group_add<G>(gate)) : inv;
                if (mine) {
                    to[rank] = gl;
                    gate_to[rank] = gate;
                    atomicAdd(&sh_n[gl], 1u);
                }
                taken = __popc(__ballot_sync(~0u, mine) & group);
            } else {
                const SoftRef ref(st.m, kLog2e);
                float most = v[0];
#pragma unroll
                for (int i = 1; i < EPL; ++i) most = fmaxf(most, v[i]);
                float least = 0.f;
#pragma unroll 4
                for (int c = 0; c < k; ++c) {
                    least = group_max<G>(most);
                    if (most == least) most = -INFINITY;
                }
                least = !open ? INFINITY : least > -INFINITY ? least : __uint_as_float(0xff7fffffu);  // (lowest)
                float* const list = found[warp];
                int* const list_at = found_at[warp];
                if (lane == 0) found_n[warp] = 0;
                __syncwarp();
                // in whatever order: the ranks below do not depend on it
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (v[i] >= least) {
                        const int at = atomicAdd(&found_n[warp], 1);
                        if (at < 32) {
                            list[at] = v[i];
                            list_at[at] = row.expert(lane, i);
                        }
                    }
                __syncwarp();
                const int n = found_n[warp];
                if (n <= 32) {
                    if (lane < 4) list[n + lane] = -INFINITY;  // four are read at a time
                    __syncwarp();
                    const float own = lane < n ? list[lane] : 0.f;
                    const int own_at = lane < n ? list_at[lane] : 0;
                    int rank = -1;  // the score itself is counted too
                    for (int j = 0; j < n; j += 4) {
                        const float4 q = *reinterpret_cast<const float4*>(&list[j]);
                        rank += (q.x >= own) + (q.y >= own) + (q.z >= own) + (q.w >= own);
                    }
                    // without equal scores the ranks are 0 .. n - 1
                    if (__reduce_add_sync(~0u, lane < n ? rank : 0) != n * (n - 1) / 2) {
                        rank = 0;
                        for (int j = 0; j < n; ++j) rank += list[j] > own || (list[j] == own && list_at[j] < own_at) ? 1 : 0;
                    }
                    if (lane < n && rank < k) {
                        to[rank] = own_at;
                        gate_to[rank] = ref.exp(own) * inv;
                        atomicAdd(&sh_n[own_at], 1u);
                    }
                    taken = min(n, k);
                } else {
                    unsigned gone = 0u;  // of this lane's scores
                    for (; taken < k; ++taken) {
                        uint32_t key = 0u;
                        int at = -1;
#pragma unroll
                        for (int i = 0; i < EPL; ++i) {
                            const uint32_t q = choice_key(v[i]);
                            if (!(gone >> i & 1u) && (q > key || (q == key && q != 0u && row.expert(gl, i) < row.expert(gl, at)))) {
                                key = q;
                                at = i;
                            }
                        }
                        const uint32_t best = __reduce_max_sync(group, key);
                        if (best == 0u) break;
                        const unsigned which = key == best ? (unsigned)row.expert(gl, at) : ~0u;
                        const unsigned winner = __reduce_min_sync(group, which);
                        if (which == winner) {
                            gone |= 1u << at;
                            to[taken] = (int)winner;
                            gate_to[taken] = ref.exp(choice_score(best)) * inv;
                            atomicAdd(&sh_n[winner], 1u);
                        }
                    }
                }
                __syncwarp();
                if (a.renormalize) {  // the gates over their sum
                    float mine = 0.f;
                    for (int c = gl; c < taken; c += G) mine += gate_to[c];
                    const float scale = 1.f / group_add<G>(mine);
                    for (int c = gl; c < taken; c += G) gate_to[c] *= scale;
                }
            }
            // the places that no open expert takes
            if (t < a.tokens)
                for (int c = taken + gl; c < k; c += G) {
                    to[c] = -1;
                    gate_to[c] = 0.f;
                }
        }
        gather(begun);
        begun = true;
    } while (first < a.tokens);
    tokens = __reduce_add_sync(~0u, tokens);
    if (lane == 0) atomicAdd(&sh_live, tokens);
    __syncthreads();
    // the CTA's sums, in the order of its warps
    for (int e = threadIdx.x; e < E; e += kTokThreads) {
        Sum s;
        for (int w = 0; w < kTokWarps; ++w) s.add(as_sum(warp_sums[w * G * EPL + e]));
        if (gridDim.x > 1) {
            b.p[(int64_t)blockIdx.x * E + e] = {s.hi, s.lo};
            b.n[(int64_t)blockIdx.x * E + e] = sh_n[e];
        } else {
            o.counts[e] = sh_n[e];
            warp_sums[e].x = s.value() * (float)sh_n[e];  // (no other thread reads this place before)
        }
    }
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) b.live[blockIdx.x] = sh_live;
        return;
    }
    // one CTA has had all tokens: the loss
    __syncthreads();
    if (warp == 0) {
        Sum sum;
        for (int e = lane; e < E; e += 32) sum.add(warp_sums[e].x);
        sum = warp_sum(sum);
        if (lane == 0) balance_result(o, sh_live, E, k, sum.value());
    }
}

// The CTAs' sums, in a fixed order, by one cluster that shares the experts; the loss.  Bound by latency:
// 6 us after the choice for 304 CTAs' sums of 256 experts (one CTA alone took 50).
__global__ void __launch_bounds__(512)
balance_finish_kernel(BalanceParts b, BalanceOuts o, int grid, int E, int top_k) {
    __shared__ float2 sh_p[512], sh_sum[kFinishCtas], sh_warp[16];
    __shared__ uint32_t sh_n[512];
    const int rank = (int)cluster_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = (E + kFinishCtas - 1) / kFinishCtas;  // at most 128
    int cols = 1;
    while (cols < share) cols *= 2;
    const int col = tid & (cols - 1), part = tid / cols, parts = min(512 / cols, 32);
    const int e = rank * share + col;
    const bool has = col < share && e < E && part < parts;
    cluster_started();
    wait_for_previous();
    Sum p;
    uint32_t n = 0u;
    if (has)
        for (int g = part; g < grid; g += parts) {
            p.add(as_sum(b.p[(int64_t)g * E + e]));
            n += b.n[(int64_t)g * E + e];
        }
    sh_p[tid] = {p.hi, p.lo};
    sh_n[tid] = n;
    __syncthreads();
    Sum products;
    if (part == 0 && has) {
        uint64_t total = n;
        for (int q = 1; q < parts; ++q) {
            p.add(as_sum(sh_p[q * cols + col]));
            total += sh_n[q * cols + col];
        }
        o.counts[e] = (int64_t)total;
        products.add(p.value() * (float)total);
    }
    products = warp_sum(products);
    if (lane == 0) sh_warp[warp] = {products.hi, products.lo};
    __syncthreads();
    cluster_wait_started();
    if (tid == 0) {
        Sum s;
        for (int w = 0; w < 16; ++w) s.add(as_sum(sh_warp[w]));
        store_remote(&sh_sum[rank].x, 0, s.hi);
        store_remote(&sh_sum[rank].y, 0, s.lo);
    }
    __syncwarp();
    cluster_sync();
    if (rank == 0 && warp == 0) {
        unsigned long long t = 0;
        for (int g = lane; g < grid; g += 32) t += b.live[g];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
        if (lane == 0) {
            Sum s;
            for (int c = 0; c < kFinishCtas; ++c) s.add(as_sum(sh_sum[c]));
            balance_result(o, t, E, top_k, s.value());
        }
    }
}

// The last tokens first: what the forward read last is still in L2.  The softmax is formed again (less
// work than its bytes).  Bound by HBM: 131,072 x 256 float32 in 45 us, 268 MB, 6.0 TB/s.
template <class T, int G, int EPL>
__global__ void __launch_bounds__(token_threads<EPL>, token_ctas_an_sm<EPL>)
balance_backward_kernel(RouterArgs a, int whole, const int64_t* counts, const int32_t* chosen,
                        const float* gates, const int64_t* live, const float* grad_gates,
                        float grad_loss, const float* grad_loss_dev, T* out, int64_t out_stride) {
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
        row.scores(v, on);
        const bool was_on = on;
        const int slot = at;
        const float g_slot = g, gate_slot = gate;
        fetch(t - step);
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
        TokenRow<T, G, EPL> d;  // (its -inf are all written over)
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            d.v[i] = from_f32<T>(!open ? 0.f : a.renormalize ? fmaf(e[i], u[i] - dot, x[i]) : e[i] * (u[i] + x[i] - dot));
        d.store(out + t * out_stride, gl, E, whole);
    }
}

// CTAs for the tokens, `per` at a time each.
inline int token_grid(int64_t tokens, int per, int most) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((tokens + per - 1) / per, most));
}
template <int G, int EPL>
int token_grid(int64_t tokens) {
    return token_grid(tokens, token_threads<EPL> / G, 152 * token_ctas_an_sm<EPL>);
}

// The fewest lanes that hold a score each up to 32 experts, then the smallest power of two of scores
// a lane.
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
    return (2048 + (size_t)token_grid(tokens, 8, kMaxCtas) * experts * 12 + 255) & ~size_t(255);
}

cudaError_t balance_loss(int dtype, const RouterArgs& a, float* loss, int64_t* counts,
                         int32_t* chosen, float* gates, int64_t* live, void* ws, cudaStream_t st) {
    const BalanceOuts o{loss, counts, live};
    BalanceParts b;
    b.live = static_cast<uint32_t*>(ws);
    int grid = 0;
    cudaError_t e = by_type(dtype, [&](auto t) {
        return by_experts(a.experts, [&](auto g, auto epl) {
            using T = decltype(t);
            constexpr int G = decltype(g)::value, EPL = decltype(epl)::value;
            grid = token_grid<G, EPL>(a.tokens);
            b.p = reinterpret_cast<float2*>(static_cast<char*>(ws) + 2048);
            b.n = reinterpret_cast<uint32_t*>(b.p + (int64_t)grid * a.experts);
            const int whole = chunks_fit(a.x, a.tokens, a.stride, a.experts, TokenRow<T, G, EPL>::CH, sizeof(T));
            constexpr int shared = token_threads<EPL> / 32 * G * EPL * (int)sizeof(float2);
            if (shared > 40 * 1024) {  // (what the kernel has besides is within 48 KB of it)
                const cudaError_t e = cudaFuncSetAttribute(balance_tokens_kernel<T, G, EPL>, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
                if (e != cudaSuccess) return e;
            }
            balance_tokens_kernel<T, G, EPL><<<grid, token_threads<EPL>, shared, st>>>(a, b, o, whole, chosen, gates);
            const cudaError_t e = cudaGetLastError();
            prof_mark(st, "balance_tokens");
            return e;
        });
    });
    if (e != cudaSuccess || grid == 1) return e;
    ClusterLaunch l(kFinishCtas, 512, 0, kFinishCtas, true, st);
    e = l(balance_finish_kernel, b, o, grid, a.experts, a.top_k);
    prof_mark(st, "balance_finish");
    return e;
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
            ClusterLaunch l(token_grid<G, EPL>(a.tokens), token_threads<EPL>, 0, 1, true, st);
            const cudaError_t e = l(balance_backward_kernel<T, G, EPL>, a, whole, counts, chosen, gates, live,
                                    grad_gates, grad_loss, grad_loss_dev, static_cast<T*>(out), out_stride);
            prof_mark(st, "balance_backward");
            return e;
        });
    });
}

}  // namespace isodev
