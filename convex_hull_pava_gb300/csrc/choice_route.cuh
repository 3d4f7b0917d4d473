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
#pragma once

#include "choice_device.cuh"
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
__device__ __noinline__ void choose_exact(const RouteArgs& a, int64_t t, double* c, int32_t* chosen, float* gates,
                                          uint32_t* counts) {
    const T* const x = static_cast<const T*>(a.x) + t * a.stride;
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
        const int64_t to = t * a.top_k + lane;
        chosen[to] = mine;
        if (a.picked) a.picked[to] = (float)v;
        gates[to] = mine < 0 ? 0.f : bad ? NAN : (float)((double)a.scale * s);
        if (mine >= 0) atomicAdd(&counts[mine], 1u);
    }
    __syncwarp();
}

// The lanes and shared memory of the choice.  L lanes have a token, each up to EPL neighbouring
// experts of one group: `per_group` lanes a group of `size` experts, `sub` experts a lane.
struct RoutePlan {
    int size, per_group, sub;
    int shift;              // per_group is 1 << shift
    float of_size, of_sub;  // a little over 1 / size and 1 / sub
    int halves;   // sub-teams of the L lanes that give a bound each (1 or 2)
    int mode;
    int vector;   // rows are copied 16 bytes at a time
    int stage;    // bytes of a warp's tile
    int counted;  // one CTA: it writes the counts
};
enum RouteMode { kByScore, kSigmoid, kSoftmax };  // what is ranked: x, sigmoid + bias, softmax + bias

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <int K>
__device__ __forceinline__ float max_nan(const float (&v)[K]) {
    float top = v[0];
#pragma unroll
    for (int i = 1; i + 1 < K; i += 2) top = max_nan(top, v[i], v[i + 1]);
    return K % 2 ? top : max_nan(top, v[K - 1]);
}
template <int K>
__device__ __forceinline__ float min_of(const float (&v)[K]) {
    float low = v[0];
#pragma unroll
    for (int i = 1; i + 1 < K; i += 2) low = min3(low, v[i], v[i + 1]);
    return K % 2 ? low : fminf(low, v[K - 1]);
}
__device__ __forceinline__ void order(float& a, float& b) {  // a the larger
    const float t = fmaxf(a, b);
    b = fminf(a, b);
    a = t;
}
// Sorts numbers that rise and fall once (a bitonic sequence), the largest first.
template <int K>
__device__ __forceinline__ void merge(float (&v)[K]) {
#pragma unroll
    for (int d = K / 2; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (!(i & d)) order(v[i], v[i + d]);
}
// Sorts 8 numbers by a network of 19 comparisons.
__device__ __forceinline__ void sort8(float (&v)[8]) {
    constexpr int at[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6}, {3, 7}, {0, 1}, {2, 3},
                               {4, 5}, {6, 7}, {2, 4}, {3, 5}, {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) order(v[at[i][0]], v[at[i][1]]);
}

// How far apart two ranked values have to be for their float32 order to be that of the exact
// ones: twice what one may be off.  Sigmoid: s is off by s (1 - s) times its exponential's error, 2^-22
// and 2^-24 |x| (s (1 - s) |x| < 0.23), a sum's, a product's and a quotient's rounding (2 of 2^-24, 2^-23),
// together under 3.2e-7.  Softmax: p times the exponential's 2^-22, a sum's 15 roundings and a quotient's
// (1.5e-6), and p |x - m| < 0.37 times 2^-23.  Adding the bias rounds by 2^-24 of the result.
__device__ __forceinline__ float unsure(bool sigmoid, float c, float share) {
    return (sigmoid ? 7e-7f : fmaf(fabsf(share), 3.2e-6f, 1e-7f)) + 1.3e-7f * fabsf(c);
}

// What is ranked, in 64 bits; of softmax with the largest score m and one over the sum.
__device__ __noinline__ double ranked_value(bool sigmoid, float x, float b, float m, double inv) {
    return (sigmoid ? 1. / (1. + exp(-(double)x)) : exp((double)x - (double)m) * inv) + (double)b;
}

// One over the softmax's sum of a token's scores to about 2^-36, of which the team's lanes have `count` each.
template <class T, int L>
__device__ __noinline__ double inverse_sum(const T* x, int count, float m) {
    Sum part;
    for (int i = 0; i < count; ++i) exp_add(part, to_f32(x[i]), m, kLog2e, (float)(1.44269504088896340736 - (double)kLog2e));
    double sum = (double)part.hi + (double)part.lo;
    __syncwarp();
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    return 1. / sum;
}

constexpr int kFound = 32;  // candidates of a token
// Warps of a CTA and CTAs an SM, by shared memory and registers.  float32: 4 and 4 (6 and 3 took 81 us of
// 131,072 x 256 and not 75, 3 and 6 83); 16 bits: 8 and 2, whose fewer CTAs add up fewer counts (16,384 x 128
// in 12.5 us, 4 and 4 14.5).
template <class T>
constexpr int team_warps = sizeof(T) == 4 ? 4 : 8;
template <class T>
constexpr int team_ctas = sizeof(T) == 4 ? 4 : 2;

// Candidates: experts whose ranked value reaches a bound that top_k of them reach, the top_k-th largest of
// the lanes' partial maxima (8 a lane), which the lanes sort and merge (LIST of them).  VALUES: what is
// ranked is formed from the scores; otherwise it is the scores themselves, which nothing rounds.  Where
// candidates' values or groups' sums are nearer to each other than float32 tells they are formed again in
// 64 bits (of 131,072 tokens some hundred); tokens with NaN, without probabilities, or with too many
// candidates are chosen by choose_exact.
// Neighbouring experts to a lane, and not interleaved ones, so that a lane's are of one group and its
// candidates in the experts' order; rows come through shared memory for that, one tile ahead of its turn.
// Bound by instructions: 131,072 x 256 float32, sigmoid with 8 groups and k = 8, in 75 us (1.8 TB/s; 356
// instructions a token, two thirds of them minima, maxima and comparisons at half rate), without groups and
// bias 50 us.  One warp a token in 64 bits throughout took 4.4 ms, 8 lanes a token without the packing of
// sigmoids two to a quotient and with the group's maxima found apart 131.
template <class T, int L, int EPL, bool VALUES, int LIST>
__global__ void __launch_bounds__(32 * team_warps<T>, team_ctas<T>)
route_kernel(const __grid_constant__ RouteArgs a, const __grid_constant__ RoutePlan pl, int64_t* counts, int32_t* chosen, float* gates) {
    constexpr int N = 16 / (int)sizeof(T), TPW = 32 / L, WORDS = EPL / N, LANE = (WORDS | 1) * 16, BIAS = (EPL / 4 | 1) * 4;
    constexpr int kTeamWarps = team_warps<T>, kTeamThreads = 32 * kTeamWarps;
    constexpr int PER = EPL / 8;  // experts of a partial maximum
    extern __shared__ __align__(16) char memory[];
    __shared__ uint32_t sh_n[L * EPL];
    __shared__ int sh_base[L];  // the first expert of a lane
    __shared__ __align__(16) float sh_bias[VALUES ? L * BIAS : 4];
    __shared__ __align__(16) float sh_found[kTeamWarps][TPW][kFound + 4];
    __shared__ float sh_first[kTeamWarps][TPW][kFound];
    __shared__ uint16_t sh_found_at[kTeamWarps][TPW][kFound], sh_first_at[kTeamWarps][TPW][kFound];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane & (L - 1), tw = lane / L;
    const int E = a.experts, k = a.top_k;
    const unsigned team = group_lanes<L>();
    char* const stages = memory + warp * 2 * pl.stage;
    // a token's candidates: values and places (lane EPL + expert of the lane), then those by rank
    float* const found = sh_found[warp][tw];
    float* const first = sh_first[warp][tw];
    uint16_t* const found_at = sh_found_at[warp][tw];
    uint16_t* const first_at = sh_first_at[warp][tw];
    // lane l's first expert and how many it has; the lane of expert e (quotients by products: exact up to 1,024)
    auto base_of = [&](int l) { return (l >> pl.shift) * pl.size + (l & (pl.per_group - 1)) * pl.sub; };
    auto held_by = [&](int l) {
        return l < a.groups << pl.shift ? max(0, min(pl.sub, pl.size - (l & (pl.per_group - 1)) * pl.sub)) : 0;
    };
    auto lane_of = [&](int e) {
        const int g = (int)((float)e * pl.of_size), r = e - g * pl.size;
        return (g << pl.shift) + (int)((float)r * pl.of_sub);
    };
    const bool has_group = gl < a.groups << pl.shift;
    const int own_count = held_by(gl);
    const bool sigmoid = VALUES && pl.mode == kSigmoid;
    const T closed = from_f32<T>(sigmoid ? 0.f : -INFINITY);  // places without an expert (their bias is -inf)
    auto fill = [&](char* stage) {
        for (int i = own_count; i < EPL; ++i) *reinterpret_cast<T*>(stage + (tw * L + gl) * LANE + i * sizeof(T)) = closed;
    };
    for (int e = threadIdx.x; e < E; e += kTeamThreads) sh_n[e] = 0u;
    if (threadIdx.x < L) sh_base[threadIdx.x] = base_of(threadIdx.x);
    if (VALUES)
        for (int i = threadIdx.x; i < L * BIAS; i += kTeamThreads) {
            const int l = i / BIAS, o = i % BIAS;
            const float b = o >= held_by(l) ? -INFINITY : a.bias ? a.bias[base_of(l) + o] : 0.f;
            sh_bias[i] = b > -INFINITY ? b : -INFINITY;
        }
    fill(stages);
    fill(stages + pl.stage);
    __syncthreads();
    const T* const base = static_cast<const T*>(a.x);
    const int64_t tiles = (a.tokens + TPW - 1) / TPW, step = (int64_t)gridDim.x * kTeamWarps;
    // where this lane's words of a row go
    int to[WORDS];
    if (pl.vector) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const int e = (gl + i * L) * N, l = lane_of(e);
            to[i] = e < E ? (tw * L + l) * LANE + (e - base_of(l)) * (int)sizeof(T) : -1;
        }
    }
    auto fetch = [&](int64_t tile, char* stage) {
        const int64_t t = tile * TPW + tw;
        const bool on = t < a.tokens && (!a.mask || a.mask[t] != 0);
        if (on) {
            const T* const x = base + t * a.stride;
            if (pl.vector) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i)
                    if (to[i] >= 0) copy_async(stage + to[i], x + (gl + i * L) * N);
            } else {
                // element by element, the lanes of a token side by side
                T f[EPL];
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (gl + i * L < E) f[i] = x[gl + i * L];
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = gl + i * L;
                    if (e < E) {
                        const int l = lane_of(e);
                        *reinterpret_cast<T*>(stage + (tw * L + l) * LANE + (e - base_of(l)) * (int)sizeof(T)) = f[i];
                    }
                }
            }
        }
        copy_async_commit();
        return on;
    };
    const int64_t tile0 = (int64_t)blockIdx.x * kTeamWarps + warp;
    bool on = fetch(tile0, stages), next_on = fetch(tile0 + step, stages + pl.stage);
    int turn = 0;
    for (int64_t tile = tile0; tile < tiles; tile += step, turn ^= 1) {
        char* const stage = stages + turn * pl.stage;
        const char* const token = stage + tw * L * LANE;
        const int64_t t = tile * TPW + tw;
        copy_async_wait<1>();
        __syncwarp();
        auto score_of = [&](int place) {
            return to_f32(*reinterpret_cast<const T*>(token + place / EPL * LANE + place % EPL * (int)sizeof(T)));
        };
        auto bias_of = [&](int place) { return sh_bias[place / EPL * BIAS + place % EPL]; };
        float v[EPL];
        auto load = [&]() {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                float2 f[N / 2];
                unpack(*reinterpret_cast<const uint4*>(token + gl * LANE + i * 16), f, T());
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    v[i * N + 2 * j] = f[j].x;
                    v[i * N + 2 * j + 1] = f[j].y;
                }
            }
        };
        load();
        const bool summed = a.score == ISO_ROUTE_SOFTMAX && (VALUES || !a.renormalize);
        float top = 0.f, ref = 0.f, inv = 0.f;
        if (!sigmoid) {  // the largest score: NaN shows in it
            top = max_nan(v);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
            ref = top == -INFINITY ? 0.f : top * kLog2e;
        }
        // left to choose_exact: NaN; no probabilities; scores so large that their products lose what counts
        bool exact = top != top || (a.score == ISO_ROUTE_SOFTMAX && top == INFINITY) ||
                     (summed && fabsf(top) >= 2000.f && top != -INFINITY);
        const float low = VALUES ? min_of(v) : 0.f;
        if (summed) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float e = ex2(fmaf(v[i], kLog2e, -ref));
                if (VALUES) v[i] = e;
                part[i & 3] += e;
            }
            inv = 1.f / group_add<L>((part[0] + part[1]) + (part[2] + part[3]));
        }
        if (VALUES) {
            const float* const bias = sh_bias + gl * BIAS;
            // (the product of two must not overflow)
            const bool apart = sigmoid && __any_sync(~0u, low < -40.f);
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                const float4 b = *reinterpret_cast<const float4*>(bias + i);
                if (!sigmoid) {
                    v[i] = fmaf(v[i], inv, b.x);
                    v[i + 1] = fmaf(v[i + 1], inv, b.y);
                    v[i + 2] = fmaf(v[i + 2], inv, b.z);
                    v[i + 3] = fmaf(v[i + 3], inv, b.w);
                } else {
                    float2 p = mul2({v[i], v[i + 1]}, {-kLog2e, -kLog2e}), q = mul2({v[i + 2], v[i + 3]}, {-kLog2e, -kLog2e});
                    p = add2({ex2(p.x), ex2(p.y)}, {1.f, 1.f});
                    q = add2({ex2(q.x), ex2(q.y)}, {1.f, 1.f});
                    if (!apart) {  // two quotients from one
                        const float r = rcp(p.x * p.y), s = rcp(q.x * q.y);
                        v[i] = fmaf(r, p.y, b.x);
                        v[i + 1] = fmaf(r, p.x, b.y);
                        v[i + 2] = fmaf(s, q.y, b.z);
                        v[i + 3] = fmaf(s, q.x, b.w);
                    } else {
                        v[i] = rcp(p.x) + b.x;
                        v[i + 1] = rcp(p.y) + b.y;
                        v[i + 2] = rcp(q.x) + b.z;
                        v[i + 3] = rcp(q.y) + b.w;
                    }
                }
            }
            if (__any_sync(~0u, low == -INFINITY)) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (to_f32(*reinterpret_cast<const T*>(token + gl * LANE + i * (int)sizeof(T))) == -INFINITY) v[i] = -INFINITY;
            }
        }
        // the partial maxima, and the largest of what is second in its part
        float part[8], second = -INFINITY;
        const bool pairs = VALUES && a.groups > 1 && a.group_best == 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* const q = v + i * PER;
            if (PER == 1) {
                part[i] = q[0];
            } else if (PER == 2) {
                part[i] = max_nan(q[0], q[1]);
                if (pairs) second = fmaxf(second, fminf(q[0], q[1]));
            } else {
                const float p = max_nan(q[0], q[1]), r = max_nan(q[2 % PER], q[3 % PER]);
                part[i] = max_nan(p, r);
                if (pairs) second = max3(second, fminf(p, r), fmaxf(fminf(q[0], q[1]), fminf(q[2 % PER], q[3 % PER])));
            }
        }
        static_assert(PER == 1 || PER == 2 || PER == 4, "the parts above");
        if (VALUES) exact |= max_nan(part) != max_nan(part);
        sort8(part);
        bool kept = has_group;
        if (a.groups > 1) {
            float one = part[0], two = pairs ? fmaxf(second, part[1]) : -INFINITY;
            for (int o = 1; o < pl.per_group; o <<= 1) {
                const float p = __shfl_xor_sync(~0u, one, o), q = __shfl_xor_sync(~0u, two, o);
                two = max3(fminf(one, p), two, q);
                one = fmaxf(one, p);
            }
            const float value = pairs && two > -INFINITY ? one + two : one;
            const int own = gl >> pl.shift;
            int rank = 0;
#pragma unroll 1
            for (int g = 0; g < a.groups; ++g) {
                const float other = __shfl_sync(~0u, value, g * pl.per_group, L);
                rank += other > value || (other == value && g < own) ? 1 : 0;
            }
            kept = has_group && rank < a.top_groups;
            if (VALUES && a.top_groups < a.groups) {
                float below = kept ? value : INFINITY, above = has_group && !kept ? value : -INFINITY;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) {
                    below = fminf(below, __shfl_xor_sync(~0u, below, o));
                    above = fmaxf(above, __shfl_xor_sync(~0u, above, o));
                }
                const float least = 2.f * unsure(sigmoid, below, 1.f);
                bool near = on && !exact && above > -INFINITY && !(below - above > least);
                near = (__ballot_sync(~0u, near) & team) != 0u;
                if (__any_sync(~0u, near)) {
                    // the groups' sums in 64 bits, of what may be among their largest
                    const double of_sum = sigmoid ? 0. : inverse_sum<T, L>(reinterpret_cast<const T*>(token + gl * LANE), own_count, top);
                    double p = -INFINITY, q = -INFINITY;
                    unsigned may = 0u;
                    const float least_of = pairs && two > -INFINITY ? two : one;
                    const float from = least_of < INFINITY ? least_of - unsure(sigmoid, least_of, 1.f) : least_of;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) may |= (v[i] >= from && v[i] > -INFINITY ? 1u : 0u) << i;
                    for (; may; may &= may - 1u) {
                        const int place = gl * EPL + __ffs(may) - 1;
                        const double c = ranked_value(sigmoid, score_of(place), bias_of(place), top, of_sum);
                        q = fmax(q, fmin(p, c));
                        p = fmax(p, c);
                    }
                    __syncwarp();
                    for (int o = 1; o < pl.per_group; o <<= 1) {
                        const double r = __shfl_xor_sync(~0u, p, o), s = __shfl_xor_sync(~0u, q, o);
                        q = fmax(fmin(p, r), fmax(q, s));
                        p = fmax(p, r);
                    }
                    const double sum = pairs && q > -INFINITY ? p + q : p;
                    rank = 0;
                    for (int g = 0; g < a.groups; ++g) {
                        const double other = __shfl_sync(~0u, sum, g * pl.per_group, L);
                        rank += other > sum || (other == sum && g < own) ? 1 : 0;
                    }
                    if (near) kept = has_group && rank < a.top_groups;
                }
            }
            if (!kept) {
#pragma unroll
                for (int i = 0; i < 8; ++i) part[i] = -INFINITY;
            }
        }
        // the lanes' maxima merged: the LIST largest of a sub-team's
        float bound;
        if (LIST == 8 && k == 8) {
            // (the most common one.)  4 of each lane, 8 of two; of the last 8 only the least counts
            float list[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                list[i] = part[i];
                list[7 - i] = __shfl_xor_sync(~0u, part[i], 1);
            }
            merge(list);
#pragma unroll
            for (int o = 2; o < L; o <<= 1) {
                float other[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(~0u, list[7 - i], o);
#pragma unroll
                for (int i = 0; i < 8; ++i) list[i] = fmaxf(list[i], other[i]);
                if (2 * o < L) merge(list);
            }
            bound = min_of(list);
        } else {
            float list[LIST];
#pragma unroll
            for (int i = 0; i < LIST; ++i) list[i] = i < 8 ? part[i & 7] : -INFINITY;
            for (int o = 1; o < L / pl.halves; o <<= 1) {
                float other[LIST];
#pragma unroll
                for (int i = 0; i < LIST; ++i) other[i] = __shfl_xor_sync(~0u, list[LIST - 1 - i], o);
#pragma unroll
                for (int i = 0; i < LIST; ++i) list[i] = fmaxf(list[i], other[i]);
                merge(list);
            }
            const int place = (k + pl.halves - 1) / pl.halves - 1;
            bound = list[0];
#pragma unroll
            for (int i = 1; i < LIST; ++i)
                if (i == place) bound = list[i];
            if (pl.halves == 2) bound = fminf(bound, __shfl_xor_sync(~0u, bound, L / 2));
        }
        if (VALUES) bound -= unsure(sigmoid, bound, 1.f);
        bound = fmaxf(bound, __uint_as_float(0xff7fffffu));  // (the lowest)
        unsigned mask = 0u;  // by the signs of v - bound
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i) mask = __funnelshift_l(__float_as_uint(v[i] - bound), mask, 1);
        mask = ~mask & (EPL == 32 ? ~0u : (1u << (EPL & 31)) - 1u);
        exact &= on;
        if (!kept || !on || exact) mask = 0u;
        // the candidates in the order of the experts (loops as short code: it runs from the instruction cache)
        int at = __popc(mask), n;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
            const int q = __shfl_up_sync(~0u, at, o, L);
            if (gl >= o) at += q;
        }
        n = __shfl_sync(~0u, at, L - 1, L);
        at -= __popc(mask);
        if (n > kFound) {
            exact = true;
            mask = 0u;
            n = 0;
        }
        for (; mask; mask &= mask - 1u) found_at[at++] = (uint16_t)(gl * EPL + __ffs(mask) - 1);
        __syncwarp();
#pragma unroll 1
        for (int j = gl; j < ((n + 3) & ~3); j += L) {
            float c = -INFINITY;
            if (j < n) {
                const int place = found_at[j];
                c = score_of(place);
                if (VALUES) c = (sigmoid ? rcp(1.f + ex2(c * -kLog2e)) : ex2(fmaf(c, kLog2e, -ref)) * inv) + bias_of(place);
            }
            found[j] = c;
        }
        __syncwarp();
        int ranks = 0;
#pragma unroll 1
        for (int j = gl; j < n; j += L) {
            const float c = found[j];
            int rank = -1;  // the value itself is counted too
#pragma unroll 1
            for (int q = 0; q < n; q += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&found[q]);
                rank += (f.x >= c) + (f.y >= c) + (f.z >= c) + (f.w >= c);
            }
            ranks += rank;
            rank = max(rank, 0);  // (no candidate is NaN)
            first[rank] = c;
            first_at[rank] = found_at[j];
        }
        // without equal values the ranks are 0 .. n - 1
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ranks += __shfl_xor_sync(~0u, ranks, o);
        __syncwarp();
        if (ranks != n * (n - 1) / 2) {
            for (int j = gl; j < n; j += L) {
                const float c = found[j];
                int rank = 0;
                for (int q = 0; q < n; ++q) rank += found[q] > c || (found[q] == c && q < j) ? 1 : 0;
                first[rank] = c;
                first_at[rank] = found_at[j];
            }
        }
        __syncwarp();
        const int filled = min(k, n);
        if (VALUES) {
            bool near = false;
            for (int i = gl; i < filled && i + 1 < n; i += L) {
                const float c = first[i], gap = c - first[i + 1];
                if (!(gap > unsure(sigmoid, c, 1.f))) {
                    const int p = first_at[i], q = first_at[i + 1];
                    const float b = bias_of(p), d = bias_of(q), share = fmaxf(c - b, c - gap - d) + 1e-6f;
                    near |= !(gap > unsure(sigmoid, c, share)) && (b != d || score_of(p) != score_of(q));
                }
            }
            near = (__ballot_sync(~0u, near) & team) != 0u;
            if (__any_sync(~0u, near)) {
                // the candidates in 64 bits, as two floats
                const double of_sum = sigmoid ? 0. : inverse_sum<T, L>(reinterpret_cast<const T*>(token + gl * LANE), own_count, top);
                if (near) {
                    for (int j = gl; j < n; j += L) {
                        const int place = found_at[j];
                        const double c = ranked_value(sigmoid, score_of(place), bias_of(place), top, of_sum);
                        found[j] = (float)c;
                        first[j] = isfinite(c) ? (float)(c - (double)(float)c) : 0.f;
                    }
                }
                __syncwarp();
                if (near) {
                    for (int j = gl; j < n; j += L) {
                        const float c = found[j], d = first[j];
                        int rank = 0;
                        for (int q = 0; q < n; ++q) {
                            const float e = found[q], f = first[q];
                            rank += e > c || (e == c && (f > d || (f == d && q < j))) ? 1 : 0;
                        }
                        first_at[rank] = found_at[j];
                    }
                }
                __syncwarp();
            }
        }
        // the gates
        float most = 0.f;
        if (a.renormalize && a.score == ISO_ROUTE_SOFTMAX) {  // against the largest score of the chosen
            most = -INFINITY;
            for (int i = gl; i < filled; i += L) most = fmaxf(most, score_of(first_at[i]));
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        }
        float sum = 0.f;
#pragma unroll 1
        for (int i = gl; i < filled; i += L) {
            const float x = score_of(first_at[i]);
            const float s = a.score == ISO_ROUTE_SIGMOID ? rcp(1.f + ex2(x * -kLog2e))
                            : a.renormalize              ? ex2((x - most) * kLog2e)
                                                         : ex2(fmaf(x, kLog2e, -ref)) * inv;
            first[i] = s;
            sum += s;
        }
        if (a.renormalize) {
            sum = group_add<L>(sum);
            if (n > 0 && !(sum > 1e-30f)) exact = true;  // sigmoids that are 0 in float32
        } else {
            sum = 1.f;
        }
        exact = (__ballot_sync(~0u, exact) & team) != 0u;
        if (t < a.tokens && !exact) {
#pragma unroll 1
            for (int i = gl; i < k; i += L) {
                int e = -1;
                float gate = 0.f, x = 0.f;
                if (i < n) {
                    const int place = first_at[i];
                    x = score_of(place);
                    e = sh_base[place / EPL] + place % EPL;
                    gate = a.scale * (first[i] / sum);  // (of one alone the scale itself: its gradient is 0)
                    atomicAdd(&sh_n[e], 1u);
                }
                chosen[t * k + i] = e;
                gates[t * k + i] = gate;
                if (a.picked) a.picked[t * k + i] = x;
            }
        }
        unsigned left = __ballot_sync(~0u, exact && gl == 0);
        __syncwarp();
        if (left) {
            for (; left; left &= left - 1u) {
                const int64_t which = tile * TPW + (__ffs(left) - 1) / L;
                choose_exact<T>(a, which, reinterpret_cast<double*>(stage), chosen, gates, sh_n);
            }
            fill(stage);
            __syncwarp();
        }
        on = next_on;
        next_on = fetch(tile + 2 * step, stage);
    }
    copy_async_wait_all();
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kTeamThreads) {
        if (pl.counted)
            counts[e] = (int64_t)sh_n[e];
        else if (sh_n[e])
            atomicAdd(reinterpret_cast<unsigned long long*>(counts) + e, (unsigned long long)sh_n[e]);
    }
}

// One warp a token, by choose_exact alone: groups whose experts the lanes of no team hold (of 1,000 experts
// 10 groups, of 600 experts 3).
template <class T>
__global__ void __launch_bounds__(kRouteThreads)
route_exact_kernel(const __grid_constant__ RouteArgs a, int64_t* counts, int32_t* chosen, float* gates) {
    extern __shared__ double values[];  // [kRouteWarps][experts]
    __shared__ uint32_t sh_n[ISO_MAX_EXPERTS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) sh_n[e] = 0u;
    __syncthreads();
    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        if (a.mask && !a.mask[t]) {
            if (lane < a.top_k) {
                chosen[t * a.top_k + lane] = -1;
                gates[t * a.top_k + lane] = 0.f;
            }
            continue;
        }
        choose_exact<T>(a, t, values + warp * E, chosen, gates, sh_n);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads)
        if (sh_n[e]) atomicAdd(reinterpret_cast<unsigned long long*>(counts) + e, (unsigned long long)sh_n[e]);
}

// The smallest team whose lanes hold the experts, each of one group.
template <class F>
cudaError_t by_team(int L, int epl, F f) {
    using std::integral_constant;
    if (L == 4 && epl <= 8) return f(integral_constant<int, 4>{}, integral_constant<int, 8>{});
    if (L == 4 && epl <= 16) return f(integral_constant<int, 4>{}, integral_constant<int, 16>{});
    if (L == 4) return f(integral_constant<int, 4>{}, integral_constant<int, 32>{});
    if (L == 8) return f(integral_constant<int, 8>{}, integral_constant<int, 32>{});
    if (L == 16) return f(integral_constant<int, 16>{}, integral_constant<int, 32>{});
    return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
}

// The lanes of a token and what each holds; 0 where no team fits.
int route_team(const RouteArgs& a, int size_of, RoutePlan* p) {
    p->size = a.experts / a.groups;
    p->halves = a.top_k <= 16 ? 1 : 2;
    p->mode = !a.bias && (a.groups == 1 || a.group_best == 1) ? kByScore : a.score == ISO_ROUTE_SIGMOID ? kSigmoid : kSoftmax;
    for (int L = 4; L <= 32; L *= 2) {
        if (L < a.groups) continue;
        int per = L / a.groups;
        while (per & (per - 1)) per &= per - 1;  // (a power of two: the group's lanes are neighbours in a butterfly)
        int sub = (p->size + per - 1) / per;
        const int n = 16 / size_of, whole = (sub + n - 1) / n * n;
        if (whole <= 32 && p->size % n == 0) sub = whole;  // words of 16 bytes are not split between lanes
        if (sub > 32) continue;
        p->per_group = per;
        p->sub = sub;
        p->shift = 0;
        while (1 << p->shift < per) ++p->shift;
        p->of_size = 1.00001f / (float)p->size;  // (e / size is at least 1 / 1,024 below the next whole number)
        p->of_sub = 1.00001f / (float)sub;
        return L;
    }
    return 0;
}

}  // namespace

template <class T>
cudaError_t route_rows(const RouteArgs& a, int64_t* counts, int32_t* chosen, float* gates, cudaStream_t st) {
    RoutePlan p{};
    const int L = route_team(a, sizeof(T), &p);
    constexpr int kTeamWarps = team_warps<T>, kTeamThreads = 32 * kTeamWarps;
    const int warps = L ? kTeamWarps : kRouteWarps;
    const int64_t tiles = L ? (a.tokens + 32 / L - 1) / (32 / L) : a.tokens;
    const int64_t grid = std::min<int64_t>((tiles + warps - 1) / warps, 152 * (L ? team_ctas<T> : 4));
    p.counted = L && grid == 1;
    if (!p.counted) {
        const cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)a.experts * sizeof(int64_t), st);
        if (e != cudaSuccess || a.tokens == 0) return e;
    }
    auto go = [&](auto kernel, int threads, int shared, auto... more) {
        if (shared > 16 * 1024) {  // (what the kernels have besides is within 48 KB of it)
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
            if (e != cudaSuccess) return e;
        }
        kernel<<<(unsigned)grid, threads, shared, st>>>(a, more..., counts, chosen, gates);
        const cudaError_t e = cudaGetLastError();
        prof_mark(st, "route");
        return e;
    };
    if (!L) return go(route_exact_kernel<T>, kRouteThreads, kRouteWarps * a.experts * (int)sizeof(double));
    return by_team(L, p.sub, [&](auto l, auto epl) {
        constexpr int LANES = decltype(l)::value, EPL = decltype(epl)::value, N = Word<T>::N;
        constexpr int tile = 32 * ((EPL / N) | 1) * 16;
        p.stage = std::max(tile, (a.experts + 1) / 2 * 16);
        p.vector = p.sub % N == 0 && p.size % N == 0 && chunks_fit(a.x, a.tokens, a.stride, a.experts, N, sizeof(T));
        const int shared = kTeamWarps * 2 * p.stage;
        if (p.mode == kByScore)
            return a.top_k <= 8 ? go(route_kernel<T, LANES, EPL, false, 8>, kTeamThreads, shared, p) : go(route_kernel<T, LANES, EPL, false, 16>, kTeamThreads, shared, p);
        return a.top_k <= 8 ? go(route_kernel<T, LANES, EPL, true, 8>, kTeamThreads, shared, p) : go(route_kernel<T, LANES, EPL, true, 16>, kTeamThreads, shared, p);
    });
}

}  // namespace isodev
