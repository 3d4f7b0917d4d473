// A step of beam search: the `keep` best continuations over a batch item's beams and vocabulary.
//
//   total(b, v) = scores_b + x[b, v] / T - lse_b,   lse_b = log sum_u exp(x[b, u] / T)
//
// One pass over the scores: CTAs take a part of a row each and leave its sum of exponentials and its
// `keep` largest scores (the order within a row is that of its scores, whatever lse is); a second
// kernel adds the parts up and ranks an item's continuations.  That order depends on what lse's float32
// sums round, by at most lse_error(n): where two continuations of different beams are nearer to each
// other than that, the rows' sums are formed again to about 2^-36 before they are ranked.
#include "choice_internal.h"
#include "choice_device.cuh"
#include "obj_launch.h"

namespace isodev {

namespace {

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32, kRowCtas = 3;  // CTAs an SM
constexpr int kUnroll = 4;                              // words of a thread at a time
constexpr int kBatch = kRowThreads * kUnroll;           // words of a CTA at a time
constexpr int kMostBatches = 24;                        // of a group of parts
constexpr int kMostWords = kBatch * 17;                 // of a part (2^17 16-bit scores wherever they start)
constexpr int kGroup = 4;                               // parts that are ranked together
constexpr int kList = 520, kHits = 1024;                // a part's candidates, a group's words that may have some
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinList = 512, kRemembered = 1024;
// Exponents are kept against whole numbers c, so that sums are brought to another c without rounding;
// beyond this the float32 product x a has lost its fraction, and the row's sum is formed with the differences (exact_sum).
constexpr float kFar = 8388608.f;

struct PartState {
    float m, c, s, pad;  // largest score; sum s of 2^(x a - c)
};
// How the rows are shared out: each is `stretches` of `words` words, from the 128-byte line that it starts
// in; those of all rows, end to end, are shared evenly among the CTAs, `share` words each.  What a
// CTA has of one stretch is a part; a stretch has room for `most` of them.
struct BeamParts {
    PartState* state;  // [rows][stretches][most]
    float* value;      // [rows][stretches][most][keep], -inf where there are fewer
    int32_t* token;
    int64_t share;
    int stretches, words, most;
};

// How far the log of a row's sum may be off: the hardware's exponential 2^-22; sums of a batch (a tree
// of 6), a warp (5) and a CTA (3) at 2^-24 each, one more when they leave; exponents rounded at
// 2^-24 |v| log 2 with |v| on average at most log2(n), and the scale's own rounding (half of that).
__device__ __forceinline__ float lse_error(int n) {
    return 2.4e-7f + 15 * 6e-8f + 6.3e-8f * (1.f + log2f((float)n)) + 1.5e-7f;
}

// Order-preserving key of a number that is not NaN, and the number; both zeros are equal.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t key) {
    return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}

// 2^d of a whole number d <= 0; 0 below float32's exponents.
__device__ __forceinline__ float power(float d) { return __uint_as_float((uint32_t)(127 + (int)fmaxf(d, -127.f)) << 23); }

// The thread's running sum against the whole number c.
struct PowerSum {
    float m = -INFINITY, c = -kFar;
    Sum s;
    __device__ __forceinline__ void raise(float top, float a) {
        if (top > m) {
            m = top;
            const float to = fminf(fmaxf(ceilf(top * a), -kFar), kFar);
            if (to > c) {
                const float f = power(c - to);
                s.hi *= f;
                s.lo *= f;
                c = to;
            }
        }
    }
};

// Where a row's scores lie: slots of 16 bytes from the 128-byte line that it starts in; slots
// [full, end) are whole words, what is before and behind them (under 2 N scores) is taken one by one.
template <class T>
struct RowSlots {
    static constexpr int N = Word<T>::N;
    const uint4* line;
    int lead, full, end, head, tail;  // head: scores before the words; tail: the first behind them
    __device__ __forceinline__ RowSlots(const T* x, int n) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(x);
        line = reinterpret_cast<const uint4*>(at & ~uintptr_t(127));
        lead = (int)(at & 127) / (int)sizeof(T);
        full = (lead + N - 1) / N;
        end = max((int)(((int64_t)lead + n) / N), full);
        head = min(n, full * N - lead);
        tail = (int)max((int64_t)head, (int64_t)end * N - lead);
    }
    __device__ __forceinline__ int first_of(int slot) const { return (int)((int64_t)slot * N - lead); }
    // the single score of lane e, or -1
    __device__ __forceinline__ int single(int n, int e) const {
        return e < head ? e : e - head < n - tail ? tail + (e - head) : -1;
    }
};

__device__ __forceinline__ bool beam_reads(const BeamArgs& a, int64_t row) {
    return isfinite(a.scores[row]) && !(a.done && a.done[row]);
}

static_assert(kRowThreads == kJoinThreads, "below");
// The k-th largest of the CTA's threads' numbers; 0 where fewer are above 0.  Where some warps have nothing to
// make up a bound of.
__device__ __noinline__ uint32_t largest_of_threads(uint32_t own, int k, uint32_t* all) {
    __syncthreads();
    all[threadIdx.x] = own;
    if (threadIdx.x == 0) all[kRowThreads] = 0u;
    __syncthreads();
    int rank = 0;
    for (int j = 0; j < kRowThreads; ++j) rank += all[j] > own || (all[j] == own && j < (int)threadIdx.x) ? 1 : 0;
    if (rank == k - 1) all[kRowThreads] = own;
    __syncthreads();
    const uint32_t found = all[kRowThreads];
    __syncthreads();
    return found;
}

// The `keep` largest of a part by `keep` rounds of the largest that comes after the last one: where more
// scores than the list holds reach the bound (many equal ones).
template <class T>
__device__ __noinline__ void rows_by_rounds(const RowSlots<T>& slots, int first, int begin, int end, int edge, float edge_x,
                                            int k, float* value, int32_t* token, uint64_t* sh_best) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t last = ~0ull;  // key: the score's order, then the lower token
    for (int i = 0; i < k; ++i) {
        uint64_t best = 0;
        auto look = [&](float v, int at) {
            if (!(v > -INFINITY)) return;
            const uint64_t key = (uint64_t)order_key(v) << 32 | (uint32_t)~at;
            if (key < last && key > best) best = key;
        };
        if (edge >= 0) look(edge_x, edge);
        for (int slot = first + tid; slot < end; slot += kRowThreads) {
            if (slot < begin) continue;
            const uint4 q = slots.line[slot];
            const T* v = reinterpret_cast<const T*>(&q);
#pragma unroll
            for (int j = 0; j < Word<T>::N; ++j) look(to_f32(v[j]), slots.first_of(slot) + j);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(~0u, best, o));
        if (lane == 0) sh_best[warp] = best;
        __syncthreads();
        for (int q = 0; q < kRowWarps; ++q) best = max(best, sh_best[q]);
        __syncthreads();
        if (tid == 0) {
            value[i] = best ? order_value((uint32_t)(best >> 32)) : -INFINITY;
            token[i] = (int32_t)~(uint32_t)best;
        }
        last = best;  // (0: nothing is left, and nothing is found below it)
    }
}

// What a CTA has to know of a part when it ranks it.
struct PartNote {
    int64_t row, slot;
    int begin, end, first;  // words; `first`: thread 0's first one
    int batch, batches;     // of the group's
    int active;             // warps that have words
    int spare, heads;
};

// Parts of rows: their sums of exponentials, and their `keep` largest scores.  Each thread notes the
// largest of every 4 words that it takes; a bound that `keep` scores of a part reach follows from the warps'
// largest, and only words whose largest reaches it are looked at again (from L2).  A CTA reads the words of
// a group of parts first, the next words always on their way, and ranks all of them after that.
// 512 x 131,072 bfloat16 (134 MB) in 36 us, 3.7 TB/s: the reading alone takes 27 us (bound by latency: 64 bytes
// a thread on their way, three CTAs of 74 registers an SM), the ranking the rest.  Not kept: words
// through shared memory by cp.async, three batches ahead (no waits, but a quarter more instructions: 40 us),
// by bulk copies of each warp (no faster), 8 words at a time (40 to 42), CTAs of 128 and 512 threads (46), two or
// four times as many CTAs (47, 60: each part costs 4 us), lists by one addition a warp (42).
template <class T>
__global__ void __launch_bounds__(kRowThreads, kRowCtas)
beam_rows_kernel(const __grid_constant__ BeamArgs a, const __grid_constant__ BeamParts parts, float scale, int rows) {
    constexpr int N = Word<T>::N;
    __shared__ float most[kMostBatches][kRowThreads];
    __shared__ uint8_t part_of[kMostBatches];
    __shared__ int hits[kHits];
    __shared__ float list[kGroup][kList];
    __shared__ int list_at[kGroup][kList];
    __shared__ PartNote note[kGroup];
    __shared__ float sh_m[kGroup][kRowWarps], sh_c[kGroup][kRowWarps], sh_s[kGroup][kRowWarps], sh_least[kGroup][kRowWarps];
    __shared__ float sh_bound[kGroup];
    __shared__ uint64_t sh_best[kRowWarps];
    __shared__ uint32_t sh_all[kRowThreads + 1];
    __shared__ int hit_n, list_n[kGroup];
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.keep;

    struct Part {
        const T* x;
        int64_t slot;            // its place among the parts
        int row;
        int begin, end, first;  // words; `first`: thread 0's first one
        int spare;               // places of its stretch that no part takes, behind its last one
        bool read, heads;        // heads: it begins its row
    };
    // the CTA's words: `left` of them from word `from` of a stretch, the `index`-th of its row, on
    struct Walk {
        int64_t left, stretch;
        int from, row, index, number;
    } walk;
    {
        const int64_t at = blockIdx.x * parts.share;
        walk.left = min(parts.share, (int64_t)rows * parts.stretches * parts.words - at);
        walk.stretch = at / parts.words;
        walk.from = (int)(at - walk.stretch * parts.words);
        walk.row = (int)(walk.stretch / parts.stretches);
        walk.index = (int)(walk.stretch - (int64_t)walk.row * parts.stretches);
        walk.number = walk.from == 0 ? 0 : (int)(blockIdx.x - walk.stretch * parts.words / parts.share);
    }
    auto take = [&](Walk& w) {
        Part p{nullptr, 0, 0, 0, 0, 0, 0, false, false};
        const int size = (int)min((int64_t)(parts.words - w.from), w.left);
        p.read = beam_reads(a, w.row);
        if (p.read) {
            p.row = w.row;
            p.slot = w.stretch * parts.most + w.number;
            p.spare = w.from + size == parts.words ? parts.most - 1 - w.number : 0;
            p.x = static_cast<const T*>(a.x) + w.row * a.stride;
            const RowSlots<T> slots(p.x, a.n);
            const int first = w.index * parts.words + w.from;  // (below 2^29 + 16)
            p.heads = first == 0;
            p.begin = max(first, slots.full);
            p.end = max(p.begin, min(first + size, slots.end));
            p.first = min(first, p.end);
        }
        w.left -= size;
        w.from = w.number = 0;
        ++w.stretch;
        if (++w.index == parts.stretches) {
            w.index = 0;
            ++w.row;
        }
        return p;
    };
    uint4 w[kUnroll];
    auto ask = [&](const Part& p, int b, uint4 (&to)[kUnroll]) {  // words of batch b
        const uint4* const line = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p.x) & ~uintptr_t(127));
        const int slot = p.first + b * kBatch + tid;
        if (p.first + b * kBatch >= p.begin && p.first + (b + 1) * kBatch <= p.end) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) to[u] = load_streaming(line + slot + u * kRowThreads);
            return;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int q = slot + u * kRowThreads;
            to[u] = q >= p.begin && q < p.end ? load_streaming(line + q) : word_closed(T());
        }
    };
    auto batches_of = [&](const Part& p) { return p.read ? (p.end - p.first + kBatch - 1) / kBatch : 0; };
    Part cur = take(walk);
    ask(cur, 0, w);
    bool more = true;
    while (more) {
        // the words of a group
        int group = 0, noted = 0;
        while (more && group < kGroup) {
            const int batches = batches_of(cur);
            if (noted + batches > kMostBatches) break;
            more = walk.left > 0;
            const Part next = more ? take(walk) : Part{nullptr, 0, 0, 0, 0, 0, 0, false, false};
            if (!cur.read) {
                cur = next;
                ask(cur, 0, w);
                continue;
            }
            PowerSum st;
#pragma unroll 1
            for (int b = 0; b < batches; ++b) {
                uint4 ahead[kUnroll];
                if (b + 1 < batches) ask(cur, b + 1, ahead);
                else ask(next, 0, ahead);
                float top = -INFINITY;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) top = fmaxf(top, word_max(w[u], T()));
                most[noted + b][tid] = top;
                st.raise(top, scale);
                float2 sum[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float2 v[N / 2];
                    unpack(w[u], v, T());
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        v[i] = fma2(v[i], {scale, scale}, {-st.c, -st.c});
                        v[i] = {ex2(v[i].x), ex2(v[i].y)};
                    }
#pragma unroll
                    for (int o = N / 4; o > 0; o >>= 1)
#pragma unroll
                        for (int i = 0; i < o; ++i) v[i] = add2(v[i], v[i + o]);
                    sum[u] = v[0];
                }
#pragma unroll
                for (int o = kUnroll / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int u = 0; u < o; ++u) sum[u] = add2(sum[u], sum[u + o]);
                st.s.add(sum[0].x + sum[0].y);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) w[u] = ahead[u];
            }
            if (batches == 0) ask(next, 0, w);
            // the warp's sum, and as many of its threads' largest as make up the bound
            const int active = min(kRowWarps, (cur.end - cur.first + 31) / 32), each = active ? (k + active - 1) / active : 0;
            float v = st.m, least = -INFINITY;  // of the words
            for (int i = 0; i < each; ++i) {
                least = warp_max(v);
                if (lane == __ffs(__ballot_sync(~0u, v == least)) - 1) v = -INFINITY;
            }
            if (cur.heads && warp == 0) {  // the single scores
                const int edge = RowSlots<T>(cur.x, a.n).single(a.n, lane);
                if (edge >= 0) {
                    const float x = to_f32(cur.x[edge]);
                    st.raise(x, scale);
                    st.s.add(ex2(fmaf(x, scale, -st.c)));
                }
            }
            const float m = warp_max(st.m), c = warp_max(st.c);
            const float s = warp_add(st.s.value() * power(st.c - c));
            if (lane == 0) {
                sh_m[group][warp] = m;
                sh_c[group][warp] = c;
                sh_s[group][warp] = s;
                sh_least[group][warp] = warp < active ? least : INFINITY;
            }
            if (tid == 0) {
                note[group] = {cur.row, cur.slot, cur.begin, cur.end, cur.first, noted, batches, active, cur.spare, cur.heads};
                list_n[group] = 0;
                hit_n = 0;
            }
            if (tid < batches) part_of[noted + tid] = (uint8_t)group;
            noted += batches;
            ++group;
            cur = next;
        }
        if (group == 0) break;
        __syncthreads();
        if (warp < group) {  // warp g: the sum of part g, and its bound
            const int i = lane & (kRowWarps - 1);
            const float c = warp_max(sh_c[warp][i]), m = warp_max(sh_m[warp][i]);
            float s = sh_s[warp][i] * power(sh_c[warp][i] - c), least = sh_least[warp][i];
#pragma unroll
            for (int o = kRowWarps / 2; o > 0; o >>= 1) {
                s += __shfl_xor_sync(~0u, s, o);
                least = fminf(least, __shfl_xor_sync(~0u, least, o));
            }
            const PartNote& p = note[warp];
            if (lane == 0) {
                parts.state[p.slot] = {m, c, s, 0.f};
                sh_bound[warp] = p.active ? least : -INFINITY;
            }
            if (lane < p.spare) parts.state[p.slot + 1 + lane] = {-INFINITY, -kFar, 0.f, 0.f};
        }
        __syncthreads();
        for (int g = 0; g < group; ++g)
            if (sh_bound[g] == -INFINITY && note[g].batches > 0) {  // (a part with few words, or closed but for few)
                float own = -INFINITY;
                for (int b = 0; b < note[g].batches; ++b) own = fmaxf(own, most[note[g].batch + b][tid]);
                const uint32_t found = largest_of_threads(own > -INFINITY ? order_key(own) : 0u, k, sh_all);
                if (tid == 0 && found) sh_bound[g] = order_value(found);
                __syncthreads();
            }
        for (int b = 0; b < noted; ++b) {
            const float v = most[b][tid];
            if (v > -INFINITY && v >= sh_bound[part_of[b]]) {
                const int i = atomicAdd(&hit_n, 1);
                if (i < kHits) hits[i] = b << 16 | tid;
            }
        }
        auto put = [&](int g, float v, int at) {
            const int i = atomicAdd(&list_n[g], 1);
            if (i < kList) {
                list[g][i] = v;
                list_at[g][i] = at;
            }
        };
        if (warp < group && note[warp].heads) {
            const T* const x = static_cast<const T*>(a.x) + note[warp].row * a.stride;
            const int edge = RowSlots<T>(x, a.n).single(a.n, lane);
            if (edge >= 0) {
                const float v = to_f32(x[edge]);
                if (v > -INFINITY && v >= sh_bound[warp]) put(warp, v, edge);
            }
        }
        __syncthreads();
        const int looked = min(hit_n, kHits) * kUnroll;
        for (int i = tid; i < looked; i += kRowThreads) {
            const int hit = hits[i / kUnroll], g = part_of[hit >> 16];
            const PartNote& p = note[g];
            const int slot = p.first + ((hit >> 16) - p.batch) * kBatch + (hit & 0xffff) + i % kUnroll * kRowThreads;
            if (slot < p.begin || slot >= p.end) continue;
            const RowSlots<T> slots(static_cast<const T*>(a.x) + p.row * a.stride, a.n);
            const uint4 q = slots.line[slot];
            const T* v = reinterpret_cast<const T*>(&q);
            const float bound = sh_bound[g];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float f = to_f32(v[j]);
                if (f > -INFINITY && f >= bound) put(g, f, slots.first_of(slot) + j);
            }
        }
        __syncthreads();
        const int all_hits = hit_n;
        // a quarter of the threads a part at a time
        for (int g = warp / (kRowWarps / kGroup); g < group; g += kGroup) {
            const int n = list_n[g];
            if (all_hits > kHits || n > kList) continue;
            float* const value = parts.value + note[g].slot * k;
            int32_t* const token = parts.token + note[g].slot * k;
            for (int i = tid % (kRowThreads / kGroup); i < max(n, k); i += kRowThreads / kGroup) {
                if (i < n) {
                    const float v = list[g][i];
                    int above = 0, same = 0;
                    for (int j = 0; j < n; ++j) {
                        above += list[g][j] > v;
                        same += list[g][j] == v;
                    }
                    if (same > 1) {  // the lower tokens first
                        const int at = list_at[g][i];
                        for (int j = 0; j < n; ++j) above += list[g][j] == v && list_at[g][j] < at ? 1 : 0;
                    }
                    if (above < k) {
                        value[above] = v;
                        token[above] = list_at[g][i];
                    }
                } else {
                    value[i] = -INFINITY;
                }
            }
        }
        for (int g = 0; g < group; ++g) {
            const PartNote& p = note[g];
            float* const value = parts.value + p.slot * k;
            for (int i = tid; i < p.spare * k; i += kRowThreads) value[k + i] = -INFINITY;
            if (all_hits > kHits || list_n[g] > kList) {
                const T* const x = static_cast<const T*>(a.x) + p.row * a.stride;
                const RowSlots<T> slots(x, a.n);
                const int edge = p.heads && warp == 0 ? slots.single(a.n, lane) : -1;
                rows_by_rounds(slots, p.first, p.begin, p.end, edge, edge >= 0 ? to_f32(x[edge]) : -INFINITY, k, value,
                               parts.token + p.slot * k, sh_best);
            }
        }
        __syncthreads();
    }
}

// The exponentials of a row's scores against its largest m, summed to about 2^-36 of the sum, in the order
// of the scores, whatever their place in memory.  NaN where a score is NaN or m is not finite.
template <class T>
__device__ __noinline__ double exact_sum(const T* x, int n, float m, float a_hi, float a_lo, Sum* sh) {
    Sum s;
    for (int e = threadIdx.x; e < n; e += kJoinThreads) exp_add(s, to_f32(x[e]), m, a_hi, a_lo);
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    double total = 0.;
    for (int w = 0; w < kJoinWarps; ++w) total += (double)sh[w].hi + (double)sh[w].lo;
    __syncthreads();
    return total;
}

// A total as two floats, hi + lo, hi the larger, and its order: hi's key above lo's.
struct Total {
    float hi, lo;
    __device__ __forceinline__ uint64_t key() const { return (uint64_t)order_key(hi) << 32 | order_key(lo); }
    __device__ __forceinline__ float minus(Total q) const { return __fadd_rn(__fsub_rn(hi, q.hi), __fsub_rn(lo, q.lo)); }
};
__device__ __forceinline__ Total total_of(uint64_t key) { return {order_value((uint32_t)(key >> 32)), order_value((uint32_t)key)}; }
__device__ __forceinline__ Total two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Total normal(float hi, float lo) {
    const float s = __fadd_rn(hi, lo);
    return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}

// A continuation; key 0: none.
struct Continuation {
    uint64_t key;
    float x;
    int beam, token;
};
__device__ __forceinline__ bool before(const Continuation& p, const Continuation& q) {
    if (p.key != q.key) return p.key > q.key;
    if (p.beam != q.beam) return p.beam < q.beam;
    return p.x != q.x ? p.x > q.x : p.token < q.token;
}

// 1 / T and log2(e) / T, each as two floats.
struct BeamScale {
    float inv_hi, inv_lo, a_hi, a_lo;
};

// What a batch item's kernel has of its beams.
struct ItemBeams {
    Total base[ISO_MAX_BEAMS];  // the total of a beam's largest score; -inf: the beam offers nothing
    float off[ISO_MAX_BEAMS];   // how far base may be off
    float largest[ISO_MAX_BEAMS];
    bool ended[ISO_MAX_BEAMS];
    unsigned unsure;            // beams whose sum is to be formed again
};

// Forms the sums of the beams in `unsure` again.
template <class T>
__device__ __noinline__ void settle(const BeamArgs& a, const BeamScale& sc, ItemBeams& beams, Sum* sh) {
    const int64_t row0 = blockIdx.x * (int64_t)a.beams;
    const unsigned which = beams.unsure;
    __syncthreads();
    for (int b = 0; b < a.beams; ++b) {
        if (!(which >> b & 1u)) continue;
        const T* const x = static_cast<const T*>(a.x) + (row0 + b) * a.stride;
        const double sum = exact_sum(x, a.n, beams.largest[b], sc.a_hi, sc.a_lo, sh);
        if (threadIdx.x == 0) {
            const bool bad = !isfinite(sum);
            const double t = (double)a.scores[row0 + b] - log(sum);
            beams.base[b] = bad ? Total{-INFINITY, 0.f} : Total{(float)t, (float)(t - (double)(float)t)};
            beams.off[b] = 0.f;
            if (bad && a.row_status) a.row_status[row0 + b] = ISO_ROW_BAD_Y;
        }
    }
    if (threadIdx.x == 0) beams.unsure = 0u;
    __syncthreads();
}

// Continuation q of all that an item's parts have left, then one of each beam that is done.
struct ItemContinuations {
    const float* value;
    const int32_t* token;
    uint32_t of_beam, left, count;
    int end;
    BeamScale sc;
    __device__ __forceinline__ Continuation operator()(const ItemBeams& beams, uint32_t q) const {
        Continuation c{0, 0.f, 0, 0};
        if (q >= left) {
            if (q >= count) return c;
            c.beam = (int)(q - left);
            if (beams.ended[c.beam] && beams.base[c.beam].hi > -INFINITY) {
                c.key = beams.base[c.beam].key();
                c.token = end;
            }
            return c;
        }
        c.beam = (int)(q / of_beam);
        const Total of = beams.base[c.beam];
        if (!(of.hi > -INFINITY) || beams.ended[c.beam]) return c;
        c.x = value[q];
        c.token = token[q];  // (of no meaning where the value is -inf)
        if (c.x > -INFINITY) {
            // base + (x - m) / T
            const Total d = two_sum(c.x, -beams.largest[c.beam]);
            const float y = __fmul_rn(d.hi, sc.inv_hi), y_low = __fmaf_rn(d.hi, sc.inv_hi, -y) + fmaf(d.hi, sc.inv_lo, d.lo * sc.inv_hi);
            const Total t = two_sum(of.hi, y);
            const Total r = normal(t.hi, t.lo + (of.lo + y_low));
            c.key = isfinite(r.hi) ? r.key() : 0;  // (below float32's range: closed)
        }
        return c;
    }
};

__device__ __forceinline__ void give(const BeamArgs& a, int i, const Continuation& c) {
    const bool some = c.key != 0;
    const int64_t at = blockIdx.x * (int64_t)a.keep + i;
    a.out_scores[at] = some ? total_of(c.key).hi : -INFINITY;
    a.parents[at] = some ? c.beam : -1;
    a.tokens[at] = some ? c.token : -1;
}

// The continuations by `keep` rounds of the first that comes after the last one: where more reach the bound
// than the list holds (many equal ones).  All sums are formed again first.
template <class T>
__device__ __noinline__ void join_by_rounds(const BeamArgs& a, const ItemContinuations& at, ItemBeams& beams, Sum* sh,
                                            Continuation* sh_best) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __syncthreads();
    if (tid == 0) {
        for (int b = 0; b < a.beams; ++b)
            if (beams.off[b] > 0.f) beams.unsure |= 1u << b;
    }
    __syncthreads();
    settle<T>(a, at.sc, beams, sh);
    Continuation last{~0ull, INFINITY, -1, -1};
    for (int i = 0; i < a.keep; ++i) {
        Continuation best{0, 0.f, 0, 0};
        for (uint32_t q = tid; q < at.count; q += kJoinThreads) {
            const Continuation c = at(beams, q);
            if (c.key && before(last, c) && (!best.key || before(c, best))) best = c;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Continuation c;
            c.key = __shfl_xor_sync(~0u, best.key, o);
            c.x = __shfl_xor_sync(~0u, best.x, o);
            c.beam = __shfl_xor_sync(~0u, best.beam, o);
            c.token = __shfl_xor_sync(~0u, best.token, o);
            if (c.key && (!best.key || before(c, best))) best = c;
        }
        if (lane == 0) sh_best[warp] = best;
        __syncthreads();
        for (int w = 0; w < kJoinWarps; ++w) {
            const Continuation c = sh_best[w];
            if (c.key && (!best.key || before(c, best))) best = c;
        }
        __syncthreads();
        if (tid == 0) give(a, i, best);
        if (!best.key) {
            for (int j = i + 1 + tid; j < a.keep; j += kJoinThreads) give(a, j, best);
            return;
        }
        last = best;
    }
}

// A batch item's beams: their parts' sums, and the continuations ranked.  Totals are two floats: beside
// lse's error (off) theirs is nothing (2^-46).  Bound by latency, 9 to 10 us alone (14 with
// totals in float64, 24 with a bound from lists in the order of the beams), part of it behind the rows' kernel.
template <class T>
__global__ void __launch_bounds__(kJoinThreads)
beam_join_kernel(const __grid_constant__ BeamArgs a, const __grid_constant__ BeamParts parts, const __grid_constant__ BeamScale sc) {
    __shared__ ItemBeams beams;
    __shared__ uint64_t key_of[kRemembered];  // the first continuations' keys
    __shared__ Continuation list[kJoinList], sorted[kJoinList];
    __shared__ uint32_t sh_least[kJoinWarps], sh_all[kJoinThreads + 1];
    __shared__ Sum sh_sum[kJoinWarps];
    __shared__ int list_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.keep, P = parts.stretches * parts.most;
    const int64_t row0 = blockIdx.x * (int64_t)a.beams;
    const float may_be = lse_error(a.n), slack = 2.f * may_be;
    constexpr float kLn2Hi = (float)0.693147180559945309417, kLn2Lo = (float)(0.693147180559945309417 - (double)kLn2Hi);
    if (tid == 0) beams.unsure = 0u;
    __syncthreads();
    wait_for_previous();
#pragma unroll 1
    for (int b = warp; b < a.beams; b += kJoinWarps) {
        const float score = a.scores[row0 + b];
        const bool done = a.done && a.done[row0 + b], finite = isfinite(score), read = finite && !done;
        Total of{finite && done ? score : -INFINITY, 0.f};
        float err = 0.f, m = -INFINITY;
        uint32_t status = 0u;
        if (read) {
            const PartState* const s = parts.state + (row0 + b) * P;
            float c = -kFar;
            Sum sum;
            PartState first{-INFINITY, -kFar, 0.f, 0.f};
            if (lane < P) first = s[lane];
            m = first.m;
            c = first.c;
            for (int p = lane + 32; p < P; p += 32) {
                m = fmaxf(m, s[p].m);
                c = fmaxf(c, s[p].c);
            }
            m = warp_max(m);
            c = warp_max(c);
            sum.add(first.s * power(first.c - c));
            for (int p = lane + 32; p < P; p += 32) sum.add(s[p].s * power(s[p].c - c));
            sum = warp_sum(sum);
            const float total = __shfl_sync(~0u, sum.value(), 0);
            const float p = __fmul_rn(m, sc.a_hi);
            if (!isfinite(m)) {
                status = ISO_ROW_BAD_Y;
            } else if (!(fabsf(p) < kFar)) {
                of = {0.f, 0.f};  // (formed below)
                if (lane == 0) atomicOr(&beams.unsure, 1u << b);
            } else if (!isfinite(total)) {
                status = ISO_ROW_BAD_Y;
            } else {
                // score - log 2 (c + log2(total) - m a), a the float32 scale that the sum was formed with;
                // total = f 2^e
                const int e = (__float_as_int(total) - 0x3f3504f3) >> 23;  // 0x3f3504f3: 1 / sqrt(2)
                const float f = __int_as_float(__float_as_int(total) - (e << 23));
                const float p_low = __fmaf_rn(m, sc.a_hi, -p);
                Total d = two_sum(__fadd_rn(c, (float)e), -p);  // c + e is a whole number below 2^24
                d = normal(d.hi, d.lo - p_low);
                const float q = __fmul_rn(d.hi, kLn2Hi), q_low = __fmaf_rn(d.hi, kLn2Hi, -q) + fmaf(d.hi, kLn2Lo, d.lo * kLn2Hi);
                const Total t = two_sum(score, -q), r = two_sum(t.hi, -logf(f));
                of = normal(r.hi, r.lo + (t.lo - q_low));
                err = may_be;
            }
        }
        if (lane == 0) {
            beams.base[b] = of;
            beams.off[b] = err;
            beams.largest[b] = m;
            beams.ended[b] = done;
            if (a.row_status) a.row_status[row0 + b] = status;
        }
    }
    __syncthreads();
    if (beams.unsure) settle<T>(a, sc, beams, sh_sum);

    const uint32_t of_beam = (uint32_t)P * k, left = a.beams * of_beam;
    const ItemContinuations at{parts.value + row0 * P * k, parts.token + row0 * P * k, of_beam, left,
                               left + (a.done ? a.beams : 0), (int)a.end, sc};
    for (;;) {
        // a bound that `keep` continuations reach, as for the parts, by their totals' larger floats.  A lane
        // has `stretch` neighbouring ones, of which the warps take one in turn: each warp has some of all beams
        if (tid == 0) list_n = 0;
        const uint32_t stretch = (at.count + 31) / 32;
        uint32_t most = 0u;
#pragma unroll 1
        for (uint32_t i = warp; i < stretch; i += kJoinWarps) {
            const uint64_t key = at(beams, lane * stretch + i).key;
            most = max(most, (uint32_t)(key >> 32));
            if (i * 32 < kRemembered) key_of[i * 32 + lane] = key;
        }
        const int active = (int)min((uint32_t)kJoinWarps, stretch), each = (k + active - 1) / active;
        uint32_t least = 0u;
#pragma unroll 1
        for (int i = 0; i < each; ++i) {
            least = __reduce_max_sync(~0u, most);
            if (lane == __ffs(__ballot_sync(~0u, most == least)) - 1) most = 0u;
        }
        if (lane == 0) sh_least[warp] = warp < active ? least : ~0u;
        __syncthreads();
        uint32_t high = ~0u;
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) high = min(high, sh_least[i]);
        if (high == 0u && at.count > kJoinThreads) {  // (few of many beams in use)
            most = 0u;
#pragma unroll 1
            for (uint32_t q = tid; q < at.count; q += kJoinThreads) most = max(most, (uint32_t)(at(beams, q).key >> 32));
            high = largest_of_threads(most, k, sh_all);
        }
        // and as far below it as two beams may be off
        const float lowest = high ? order_value(high) : 0.f;
        const uint64_t bound = high ? (uint64_t)order_key(fmaf(fabsf(lowest), -2.4e-7f, lowest - slack)) << 32 : 1;
#pragma unroll 1
        for (uint32_t i = warp; i < stretch; i += kJoinWarps) {
            if (i * 32 < kRemembered && key_of[i * 32 + lane] < bound) continue;
            const Continuation c = at(beams, lane * stretch + i);
            if (c.key < bound) continue;
            const int to = atomicAdd(&list_n, 1);
            if (to < kJoinList) list[to] = c;
        }
        __syncthreads();
        const int n = list_n;
        if (n > kJoinList) {
            join_by_rounds<T>(a, at, beams, sh_sum, sorted);
            return;
        }
        // 4 neighbouring threads rank one
        for (int i = tid >> 2; i < ((n + 7) & ~7); i += kJoinThreads / 4) {
            const Continuation c = i < n ? list[i] : Continuation{0, 0.f, 0, 0};
            int rank = 0;
            for (int j = tid & 3; j < n; j += 4) {
                const uint64_t other = list[j].key;
                if (other == c.key) rank += before(list[j], c) || (!before(c, list[j]) && j < i) ? 1 : 0;
                else rank += other > c.key ? 1 : 0;
            }
            rank += __shfl_xor_sync(~0u, rank, 1);
            rank += __shfl_xor_sync(~0u, rank, 2);
            if (i < n && (tid & 3) == 0) sorted[rank] = c;
        }
        __syncthreads();
        // neighbours of different beams that are nearer than they may be off, down to what may still be chosen
        for (int i = tid; i + 1 < n; i += kJoinThreads) {
            const Continuation p = sorted[i], q = sorted[i + 1];
            const float may = beams.off[p.beam] + beams.off[q.beam];
            if (p.beam == q.beam || !(may > 0.f) || total_of(p.key).minus(total_of(q.key)) > may) continue;
            if (i < k || total_of(sorted[k - 1].key).minus(total_of(q.key)) <= slack)
                atomicOr(&beams.unsure, (beams.off[p.beam] > 0.f ? 1u << p.beam : 0u) | (beams.off[q.beam] > 0.f ? 1u << q.beam : 0u));
        }
        __syncthreads();
        if (!beams.unsure) {
            for (int i = tid; i < k; i += kJoinThreads) give(a, i, i < n ? sorted[i] : Continuation{0, 0.f, 0, 0});
            return;
        }
        settle<T>(a, sc, beams, sh_sum);
    }
}

// CTAs for the rows; a CTA's share is a batch of words at least, or a row where that is less (so that short
// rows get a CTA each).
int64_t share_rows(int64_t rows, int64_t n, int size, BeamParts* p) {
    const int64_t words = ((n * size + 112 + 15) / 16 + 1 + 7) / 8 * 8;  // wherever in 128 bytes a row starts
    p->stretches = (int)((words + kMostWords - 1) / kMostWords);
    p->words = (int)(((words + p->stretches - 1) / p->stretches + 7) / 8 * 8);
    const int64_t all = rows * p->stretches * p->words, held = 152 * kRowCtas;
    p->share = std::max<int64_t>(((all + held - 1) / held + 7) / 8 * 8, std::min(p->words, kBatch));
    p->most = (int)(p->words % p->share == 0 ? p->words / p->share : p->share % p->words == 0 ? 1 : (p->words - 1) / p->share + 2);
    return (all + p->share - 1) / p->share;
}

inline size_t align256c(size_t x) { return (x + 255) & ~size_t(255); }

inline int score_size(int dtype) { return dtype == ISO_F32 ? 4 : 2; }

}  // namespace

size_t beam_workspace(int64_t batch, int beams, int64_t n, int dtype, int keep) {
    BeamParts p;
    share_rows(batch * beams, n, score_size(dtype), &p);
    const size_t all = (size_t)(batch * beams) * p.stretches * p.most;
    return align256c(all * sizeof(PartState)) + 2 * align256c(all * keep * 4);
}

cudaError_t beam_choose(int dtype, const BeamArgs& a, void* ws, cudaStream_t st) {
    const int64_t rows = a.batch * a.beams;
    BeamParts p;
    const int64_t grid = share_rows(rows, a.n, score_size(dtype), &p);
    const size_t all = (size_t)rows * p.stretches * p.most;
    char* at = static_cast<char*>(ws);
    p.state = reinterpret_cast<PartState*>(at);
    p.value = reinterpret_cast<float*>(at += align256c(all * sizeof(PartState)));
    p.token = reinterpret_cast<int32_t*>(at += align256c(all * a.keep * 4));
    const double scale = 1.4426950408889634074 / a.temperature, inv = 1. / a.temperature;
    BeamScale sc{(float)inv, 0.f, (float)scale, 0.f};
    sc.inv_lo = (float)(inv - (double)sc.inv_hi);
    sc.a_lo = (float)(scale - (double)sc.a_hi);
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        beam_rows_kernel<T><<<(unsigned)grid, kRowThreads, 0, st>>>(a, p, sc.a_hi, (int)rows);
        cudaError_t e = cudaGetLastError();
        prof_mark(st, "beam_rows");
        if (e != cudaSuccess) return e;
        ClusterLaunch l(a.batch, kJoinThreads, 0, 1, true, st);
        e = l(beam_join_kernel<T>, a, p, sc);
        prof_mark(st, "beam_join");
        return e;
    });
}

}  // namespace isodev
