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

// The lanes and shared memory of the choice.  L lanes have a token, each up to EPL neighbouring
// experts of one group: `per_group` lanes a group of `size` experts, `sub` experts a lane.
struct RoutePlan {
    int size, per_group, sub;
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
// NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
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
// and 2^-24 |x| (s (1 - s) |x| < 0.23), a sum's and a quotient's rounding (2^-24, 2^-23), together under
// 2.7e-7.  Softmax: p times the exponential's 2^-22, a sum's 15 roundings and a quotient's (1.5e-6),
// and p |x - m| < 0.37 times 2^-23.  Adding the bias rounds by 2^-24 of the result.
__device__ __forceinline__ float unsure(int mode, float c, float share) {
    return (mode == kSigmoid ? 6e-7f : fmaf(fabsf(share), 3.2e-6f, 1e-7f)) + 1.3e-7f * fabsf(c);
}

constexpr int kFound = 32;  // candidates of a token

// Candidates: experts whose ranked value reaches a bound that top_k of them reach, the top_k-th largest of
// the lanes' 8 partial maxima, which the lanes sort and merge (LIST of them).  VALUES: what is ranked is
// formed from the scores; otherwise it is the scores themselves, which nothing rounds.  Tokens whose choice float32 does not
// settle, with NaN or infinities, or with too many candidates are chosen by choose_exact.
template <class T, int L, int EPL, bool VALUES, int LIST>
__global__ void __launch_bounds__(kRouteThreads, 3)
route_kernel(RouteArgs a, RoutePlan pl, int64_t* counts, int32_t* chosen, float* gates) {
    constexpr int N = 16 / (int)sizeof(T), TPW = 32 / L, WORDS = EPL / N, LANE = (WORDS | 1) * 16, BIAS = (EPL / 4 | 1) * 4;
    constexpr int PER = EPL / 8;  // experts of a partial maximum
    extern __shared__ __align__(16) char memory[];
    __shared__ uint32_t sh_n[L * EPL];
    __shared__ __align__(16) float sh_bias[VALUES ? L * BIAS : 4];
    __shared__ __align__(16) float found[kRouteWarps][TPW][kFound + 4];
    __shared__ uint16_t found_at[kRouteWarps][TPW][kFound], first_at[kRouteWarps][TPW][kFound + 1];
    __shared__ float first[kRouteWarps][TPW][kFound + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane & (L - 1), tw = lane / L;
    const int E = a.experts, k = a.top_k;
    const unsigned team = group_lanes<L>();
    char* const stages = memory + warp * 2 * pl.stage;
    auto base_of = [&](int l) { return l / pl.per_group * pl.size + l % pl.per_group * pl.sub; };
    auto held_by = [&](int l) { return min(pl.sub, pl.size - l % pl.per_group * pl.sub); };  // may be negative
    const bool has_group = gl < a.groups * pl.per_group;
    const int own_base = base_of(gl), own_count = has_group ? max(0, held_by(gl)) : 0;
    const bool sigmoid = VALUES && pl.mode == kSigmoid;
    const T closed = from_f32<T>(sigmoid ? 0.f : -INFINITY);  // places without an expert (their bias is -inf)
    auto fill = [&](char* stage) {
        for (int i = own_count; i < EPL; ++i) *reinterpret_cast<T*>(stage + (tw * L + gl) * LANE + i * sizeof(T)) = closed;
    };
    for (int e = threadIdx.x; e < E; e += kRouteThreads) sh_n[e] = 0u;
    if (VALUES)
        for (int i = threadIdx.x; i < L * BIAS; i += kRouteThreads) {
            const int l = i / BIAS, o = i % BIAS;
            const bool some = l < a.groups * pl.per_group && o < held_by(l);
            const float b = !some ? -INFINITY : a.bias ? a.bias[base_of(l) + o] : 0.f;
            sh_bias[i] = b > -INFINITY ? b : -INFINITY;
        }
    fill(stages);
    fill(stages + pl.stage);
    __syncthreads();
    const T* const base = static_cast<const T*>(a.x);
    const int64_t tiles = (a.tokens + TPW - 1) / TPW, step = (int64_t)gridDim.x * kRouteWarps;
    // where this lane's words of a row go
    int to[WORDS];
    if (pl.vector) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const int e = (gl + i * L) * N, l = e / pl.size * pl.per_group + e % pl.size / pl.sub;
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
                int g = gl / pl.size, r = gl % pl.size;
                for (int e = gl; e < E; e += L) {
                    const int q = r / pl.sub;
                    *reinterpret_cast<T*>(stage + (tw * L + g * pl.per_group + q) * LANE + (r - q * pl.sub) * (int)sizeof(T)) = x[e];
                    for (r += L; r >= pl.size; r -= pl.size) ++g;
                }
            }
        }
        copy_async_commit();
        return on;
    };
    const int64_t tile0 = (int64_t)blockIdx.x * kRouteWarps + warp;
    bool on = fetch(tile0, stages), next_on = fetch(tile0 + step, stages + pl.stage);
    int turn = 0;
    for (int64_t tile = tile0; tile < tiles; tile += step, turn ^= 1) {
        char* const stage = stages + turn * pl.stage;
        const int64_t t = tile * TPW + tw;
        copy_async_wait<1>();
        __syncwarp();
        const char* const mine = stage + (tw * L + gl) * LANE;
        const float* const own_bias = sh_bias + gl * BIAS;
        float v[EPL];
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            float2 f[N / 2];
            unpack(*reinterpret_cast<const uint4*>(mine + i * 16), f, T());
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                v[i * N + 2 * j] = f[j].x;
                v[i * N + 2 * j + 1] = f[j].y;
            }
        }
        float top = v[0], low = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = max_nan(top, v[i]);
        if (VALUES) {
#pragma unroll
            for (int i = 1; i < EPL; ++i) low = fminf(low, v[i]);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
        // left to choose_exact: NaN; no probabilities; scores so large that their products lose what counts
        const bool summed = a.score == ISO_ROUTE_SOFTMAX && (VALUES || !a.renormalize);
        bool exact = on && (top != top || (a.score == ISO_ROUTE_SOFTMAX && top == INFINITY) ||
                            (summed && fabsf(top) >= 2000.f && top != -INFINITY));
        const float ref = top == -INFINITY ? 0.f : top * kLog2e;
        float inv = 0.f;
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
            unsigned shut = 0u;
            if (__any_sync(~0u, low == -INFINITY)) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    float2 f[N / 2];
                    unpack(*reinterpret_cast<const uint4*>(mine + i * 16), f, T());
#pragma unroll
                    for (int j = 0; j < N / 2; ++j) {
                        shut |= (f[j].x == -INFINITY ? 1u : 0u) << (i * N + 2 * j);
                        shut |= (f[j].y == -INFINITY ? 1u : 0u) << (i * N + 2 * j + 1);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                const float4 b = *reinterpret_cast<const float4*>(own_bias + i);
                const float bias[4] = {b.x, b.y, b.z, b.w};
                if (sigmoid) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i + j] = rcp(1.f + ex2(v[i + j] * -kLog2e)) + bias[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i + j] = fmaf(v[i + j], inv, bias[j]);
                }
            }
            if (shut) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (shut >> i & 1u) v[i] = -INFINITY;
            }
        }
        float part[8];  // the partial maxima
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            part[i] = v[i * PER];
#pragma unroll
            for (int j = 1; j < PER; ++j) part[i] = fmaxf(part[i], v[i * PER + j]);
        }
        sort8(part);
        bool kept = has_group;
        if (a.groups > 1) {
            float one = part[0], two = -INFINITY;
            if (a.group_best == 2) {
                // the second largest: of the largest's maximum, or another one
                float at_most = part[1];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float hi = v[i * PER], second = -INFINITY;
#pragma unroll
                    for (int j = 1; j < PER; ++j) {
                        second = fmaxf(second, fminf(hi, v[i * PER + j]));
                        hi = fmaxf(hi, v[i * PER + j]);
                    }
                    at_most = fmaxf(at_most, second);
                }
                two = at_most;
            }
            for (int o = 1; o < pl.per_group; o <<= 1) {
                const float p = __shfl_xor_sync(~0u, one, o), q = __shfl_xor_sync(~0u, two, o);
                two = fmaxf(fminf(one, p), fmaxf(two, q));
                one = fmaxf(one, p);
            }
            const float value = a.group_best == 2 && two > -INFINITY ? one + two : one;
            const int group = gl / pl.per_group;
            int rank = 0;
            float above = -INFINITY, below = INFINITY;
            for (int g = 0; g < a.groups; ++g) {
                const float other = __shfl_sync(~0u, value, (lane & ~(L - 1)) + g * pl.per_group);
                rank += other > value || (other == value && g < group) ? 1 : 0;
            }
            kept = has_group && rank < a.top_groups;
            if (VALUES && a.top_groups < a.groups) {
                below = has_group && kept ? value : INFINITY;
                above = has_group && !kept ? value : -INFINITY;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) {
                    below = fminf(below, __shfl_xor_sync(~0u, below, o));
                    above = fmaxf(above, __shfl_xor_sync(~0u, above, o));
                }
                if (above > -INFINITY && !(below - above > 2.f * unsure(pl.mode, fmaxf(fabsf(one), fabsf(below)), 1.f))) exact |= on;
            }
            if (!kept) {
#pragma unroll
                for (int i = 0; i < 8; ++i) part[i] = -INFINITY;
            }
        }
        // the lanes' maxima merged: the LIST largest of a sub-team's
        float list[LIST];
#pragma unroll
        for (int i = 0; i < LIST; ++i) list[i] = i < 8 ? part[i] : -INFINITY;
        for (int o = 1; o < L / pl.halves; o <<= 1) {
            float other[LIST];
#pragma unroll
            for (int i = 0; i < LIST; ++i) other[i] = __shfl_xor_sync(~0u, list[LIST - 1 - i], o);
#pragma unroll
            for (int i = 0; i < LIST; ++i) list[i] = fmaxf(list[i], other[i]);
            merge(list);
        }
        const int place = (k + pl.halves - 1) / pl.halves - 1;
        float bound = list[0];
#pragma unroll
        for (int i = 1; i < LIST; ++i)
            if (i == place) bound = list[i];
        if (pl.halves == 2) bound = fminf(bound, __shfl_xor_sync(~0u, bound, L / 2));
        if (VALUES) bound -= unsure(pl.mode, bound, 1.f);
        bound = fmaxf(bound, __uint_as_float(0xff7fffffu));  // (the lowest)
        unsigned mask = 0u;
#pragma unroll
        for (int i = 0; i < EPL; ++i) mask |= (v[i] >= bound ? 1u : 0u) << i;
        if (!kept || !on) mask = 0u;
        // the candidates in the order of the experts
        int at = __popc(mask), n;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
            const int q = __shfl_up_sync(~0u, at, o, L);
            if (gl >= o) at += q;
        }
        n = __shfl_sync(~0u, at, (lane & ~(L - 1)) + L - 1);
        at -= __popc(mask);
        if (n > kFound) {
            exact = true;
            mask = 0u;
            n = 0;
        }
        for (; mask; mask &= mask - 1u) found_at[warp][tw][at++] = (uint16_t)(gl * EPL + __ffs(mask) - 1);
        __syncwarp();
        auto score_of = [&](int code) {
            return to_f32(*reinterpret_cast<const T*>(stage + (tw * L + code / EPL) * LANE + code % EPL * (int)sizeof(T)));
        };
        for (int j = gl; j < ((n + 3) & ~3); j += L) {
            float c = -INFINITY;
            if (j < n) {
                const int code = found_at[warp][tw][j];
                c = score_of(code);
                if (VALUES) {
                    const float b = sh_bias[code / EPL * BIAS + code % EPL];
                    c = sigmoid ? rcp(1.f + ex2(c * -kLog2e)) + b : fmaf(ex2(fmaf(c, kLog2e, -ref)), inv, b);
                }
            }
            found[warp][tw][j] = c;
        }
        __syncwarp();
        for (int j = gl; j < n; j += L) {
            const float c = found[warp][tw][j];
            int rank = 0;
            for (int q = 0; q < n; q += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&found[warp][tw][q]);
                rank += (f.x > c || (f.x == c && q < j)) + (f.y > c || (f.y == c && q + 1 < j)) +
                        (f.z > c || (f.z == c && q + 2 < j)) + (f.w > c || (f.w == c && q + 3 < j));
            }
            first[warp][tw][rank] = c;
            first_at[warp][tw][rank] = found_at[warp][tw][j];
        }
        __syncwarp();
        float most = -INFINITY;  // of the chosen's scores
        bool near = false;
        for (int i = gl; i < min(k, n); i += L) {
            const int code = first_at[warp][tw][i];
            const float x = score_of(code);
            most = fmaxf(most, x);
            if (VALUES && i + 1 < n) {
                const float c = first[warp][tw][i], d = first[warp][tw][i + 1];
                const float b = sh_bias[code / EPL * BIAS + code % EPL];
                if (!(c - d > unsure(pl.mode, fmaxf(fabsf(c), fabsf(d)), fmaxf(c - b, 0.f) + 1e-6f))) {
                    const int other = first_at[warp][tw][i + 1];
                    near |= score_of(other) != x || sh_bias[other / EPL * BIAS + other % EPL] != b;
                }
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        exact |= (__ballot_sync(~0u, near) & team) != 0u;
        // the gates
        auto share_of = [&](float x) {
            if (a.score == ISO_ROUTE_SIGMOID) return rcp(1.f + ex2(x * -kLog2e));
            return a.renormalize ? ex2((x - most) * kLog2e) : ex2(fmaf(x, kLog2e, -ref)) * inv;
        };
        float factor = a.scale;
        if (a.renormalize) {
            float sum = 0.f;
            for (int i = gl; i < min(k, n); i += L) sum += share_of(score_of(first_at[warp][tw][i]));
            sum = group_add<L>(sum);
            if (n > 0 && !(sum > 1e-30f)) exact |= on;  // sigmoids that are 0 in float32
            factor *= 1.f / sum;
        }
        exact = (__ballot_sync(~0u, exact) & team) != 0u;
        if (t < a.tokens && !exact) {
            for (int i = gl; i < k; i += L) {
                int e = -1;
                float gate = 0.f;
                if (i < n) {
                    const int code = first_at[warp][tw][i];
                    e = base_of(code / EPL) + code % EPL;
                    gate = share_of(score_of(code)) * factor;
                    atomicAdd(&sh_n[e], 1u);
                }
                chosen[t * k + i] = e;
                gates[t * k + i] = gate;
            }
        }
        unsigned left = __ballot_sync(~0u, exact && gl == 0);
        __syncwarp();
        if (left) {
            for (; left; left &= left - 1u) {
                const int64_t which = tile * TPW + (__ffs(left) - 1) / L;
                choose_exact(a, base + which * a.stride, reinterpret_cast<double*>(stage), chosen + which * k, gates + which * k, sh_n);
            }
            fill(stage);
            __syncwarp();
        }
        on = next_on;
        next_on = fetch(tile + 2 * step, stage);
    }
    copy_async_wait_all();
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
        if (pl.counted)
            counts[e] = (int64_t)sh_n[e];
        else if (sh_n[e])
            atomicAdd(reinterpret_cast<unsigned long long*>(counts) + e, (unsigned long long)sh_n[e]);
    }
}

// One warp a token, by choose_exact alone: numbers of groups that the lanes of a team do not have, or groups
// larger than its lanes'.
template <class T>
__global__ void __launch_bounds__(kRouteThreads)
route_exact_kernel(RouteArgs a, int64_t* counts, int32_t* chosen, float* gates) {
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
        return L;
    }
    return 0;
}

}  // namespace

template <class T>
cudaError_t route_rows(const RouteArgs& a, int64_t* counts, int32_t* chosen, float* gates, cudaStream_t st) {
    RoutePlan p{};
    const int L = route_team(a, sizeof(T), &p);
    const int64_t tiles = L ? (a.tokens + 32 / L - 1) / (32 / L) : a.tokens;
    const int64_t grid = std::min<int64_t>((tiles + kRouteWarps - 1) / kRouteWarps, 152 * 3);
    p.counted = L && grid == 1;
    if (!p.counted) {
        const cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)a.experts * sizeof(int64_t), st);
        if (e != cudaSuccess || a.tokens == 0) return e;
    }
    auto go = [&](auto kernel, int shared, auto... more) {
        if (shared > 16 * 1024) {  // (what the kernels have besides is within 48 KB of it)
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
            if (e != cudaSuccess) return e;
        }
        kernel<<<(unsigned)grid, kRouteThreads, shared, st>>>(a, more..., counts, chosen, gates);
        const cudaError_t e = cudaGetLastError();
        prof_mark(st, "route");
        return e;
    };
    if (!L) return go(route_exact_kernel<T>, kRouteWarps * a.experts * (int)sizeof(double));
    return by_team(L, p.sub, [&](auto l, auto epl) {
        constexpr int LANES = decltype(l)::value, EPL = decltype(epl)::value, N = Word<T>::N;
        constexpr int tile = 32 * ((EPL / N) | 1) * 16;
        p.stage = std::max(tile, (a.experts + 1) / 2 * 16);
        p.vector = p.sub % N == 0 && p.size % N == 0 && chunks_fit(a.x, a.tokens, a.stride, a.experts, N, sizeof(T));
        const int shared = kRouteWarps * 2 * p.stage;
        if (p.mode == kByScore)
            return a.top_k <= 8 ? go(route_kernel<T, LANES, EPL, false, 8>, shared, p) : go(route_kernel<T, LANES, EPL, false, 16>, shared, p);
        return a.top_k <= 8 ? go(route_kernel<T, LANES, EPL, true, 8>, shared, p) : go(route_kernel<T, LANES, EPL, true, 16>, shared, p);
    });
}

}  // namespace isodev
