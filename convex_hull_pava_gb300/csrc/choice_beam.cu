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
#include "obj_device.cuh"
#include "obj_launch.h"

namespace isodev {

namespace {

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kUnroll = 4;                              // words of a thread at a time
constexpr int kBatch = kRowThreads * kUnroll;           // words of a CTA at a time
constexpr int kMostBatches = 16;                        // of a part
constexpr int kMostWords = kBatch * kMostBatches;       // of a part
constexpr int kList = 512;                              // what is ranked at once
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
// Exponents are kept against whole numbers c, so that sums are brought to another c without rounding;
// beyond this the float32 product x a has lost its fraction, and the row's sum is formed in K2.
constexpr float kFar = 8388608.f;

struct PartState {
    float m, c, s, pad;  // largest score; sum s of 2^(x a - c)
};
struct BeamParts {
    PartState* state;  // [rows * parts]
    float* value;      // [rows * parts][keep], -inf where there are fewer
    int32_t* token;
    int parts, share;  // share: words of a part, from the 128-byte line that the row starts in
};

// How far the log of a row's sum may be off: the hardware's exponential 2^-22; sums of a batch (a tree
// of 6), a warp (5) and a CTA (3) at 2^-24 each, one more when they leave; exponents rounded at
// 2^-24 |v| log 2 with |v| on average at most log2(n), and the scale's own rounding (half of that).
__device__ __forceinline__ double lse_error(int n) {
    return 2.4e-7 + 15 * 6e-8 + 6.3e-8 * (1.0 + (double)log2f((float)n)) + 1e-7;
}

__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double order_value(uint64_t key) {
    return __longlong_as_double((long long)(key >> 63 ? key & ~(1ull << 63) : ~key));
}

// The thread's running sum against the whole number c.
struct PowerSum {
    float m = -INFINITY, c = -kFar;
    Sum s;
    __device__ __forceinline__ void raise(float top, float a) {
        if (top > m) {
            m = top;
            const float to = fminf(fmaxf(ceilf(top * a), -kFar), kFar);
            if (to > c) {
                const float f = ex2(fmaxf(c - to, -200.f));
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

// A part of a row: its sum of exponentials, and its `keep` largest scores.  Each thread notes the
// largest of every 4 words that it takes; a bound that `keep` scores reach follows from the warps'
// largest, and only words whose largest reaches it are looked at again (from L2).
template <class T>
__global__ void __launch_bounds__(kRowThreads, 3)
beam_rows_kernel(BeamArgs a, BeamParts parts, float scale) {
    constexpr int N = Word<T>::N;
    __shared__ float most[kMostBatches][kRowThreads];
    __shared__ int hits[kList];
    __shared__ float list[kList];
    __shared__ int list_at[kList];
    __shared__ float sh_v[kRowWarps], sh_c[kRowWarps], sh_s[kRowWarps];
    __shared__ uint64_t sh_best[kRowWarps];
    __shared__ int hit_n, list_n;
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / parts.parts;
    const int part = (int)(blockIdx.x % parts.parts);
    if (!beam_reads(a, row)) return;
    const T* const x = static_cast<const T*>(a.x) + row * a.stride;
    const RowSlots<T> slots(x, a.n);
    const int64_t from = (int64_t)part * parts.share;
    const int begin = (int)max(from, (int64_t)slots.full);
    const int end = (int)max((int64_t)begin, min(from + parts.share, (int64_t)slots.end));
    const int first = (int)min(from, (int64_t)end);  // the slot of thread 0's first word
    const int batches = (end - first + kBatch - 1) / kBatch;
    if (tid == 0) hit_n = list_n = 0;

    PowerSum st;
    // the single scores
    const int edge = part == 0 && warp == 0 ? slots.single(a.n, lane) : -1;
    const float edge_x = edge >= 0 ? to_f32(x[edge]) : -INFINITY;
    auto word = [&](int slot) {
        return slot >= begin && slot < end ? load_streaming(slots.line + slot) : word_closed(T());
    };
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) w[u] = word(first + tid + u * kRowThreads);
    for (int b = 0; b < batches; ++b) {
        uint4 next[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) next[u] = word(first + (b + 1) * kBatch + tid + u * kRowThreads);
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) top = fmaxf(top, word_max(w[u], T()));
        most[b][tid] = top;
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
        static_assert(kUnroll == 4, "the tree below");
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        st.s.add(sum[0].x + sum[0].y);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) w[u] = next[u];
    }
    const float mine = st.m;  // of the words
    if (edge >= 0) {
        st.raise(edge_x, scale);
        st.s.add(ex2(fmaf(edge_x, scale, -st.c)));
    }
    // the part's sum
    {
        const float m = warp_max(st.m), c = warp_max(st.c);
        const float s = warp_add(st.s.value() * ex2(fmaxf(st.c - c, -200.f)));
        if (lane == 0) {
            sh_v[warp] = m;
            sh_c[warp] = c;
            sh_s[warp] = s;
        }
    }
    __syncthreads();
    if (tid == 0) {
        float m = sh_v[0], c = sh_c[0], s = 0.f;
        for (int i = 1; i < kRowWarps; ++i) {
            m = fmaxf(m, sh_v[i]);
            c = fmaxf(c, sh_c[i]);
        }
        float part_of[kRowWarps];
#pragma unroll
        for (int i = 0; i < kRowWarps; ++i) part_of[i] = sh_s[i] * ex2(fmaxf(sh_c[i] - c, -200.f));
#pragma unroll
        for (int o = kRowWarps / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) part_of[i] += part_of[i + o];
        s = part_of[0];
        parts.state[blockIdx.x] = {m, c, s, 0.f};
    }
    __syncthreads();  // (sh_v is used again)

    // a bound that `keep` scores reach: the warps' largest of their threads', as many of each as it takes
    const int k = a.keep;
    const int active = min(kRowWarps, (end - first + 31) / 32);
    float bound = -INFINITY;
    if (active > 0) {
        const int each = (k + active - 1) / active;
        if (warp < active) {
            float v = mine, least = -INFINITY;
            for (int i = 0; i < each; ++i) {
                least = warp_max(v);
                if (v == least) v = -INFINITY;
            }
            if (lane == 0) sh_v[warp] = least;
        }
        __syncthreads();
        bound = INFINITY;
        for (int i = 0; i < active; ++i) bound = fminf(bound, sh_v[i]);
        __syncthreads();
    }
    auto put = [&](float v, int at) {
        const int i = atomicAdd(&list_n, 1);
        if (i < kList) {
            list[i] = v;
            list_at[i] = at;
        }
    };
    if (edge >= 0 && edge_x > -INFINITY && edge_x >= bound) put(edge_x, edge);
    for (int b = 0; b < batches; ++b) {
        const float v = most[b][tid];
        if (v > -INFINITY && v >= bound) {
            const int i = atomicAdd(&hit_n, 1);
            if (i < kList) hits[i] = b << 16 | tid;
        }
    }
    __syncthreads();
    const int looked = min(hit_n, kList);
    for (int i = tid; i < looked * kUnroll; i += kRowThreads) {
        const int hit = hits[i / kUnroll], slot = first + (hit >> 16) * kBatch + (hit & 0xffff) + i % kUnroll * kRowThreads;
        if (slot < begin || slot >= end) continue;
        const uint4 q = slots.line[slot];
        const T* v = reinterpret_cast<const T*>(&q);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float f = to_f32(v[j]);
            if (f > -INFINITY && f >= bound) put(f, slots.first_of(slot) + j);
        }
    }
    __syncthreads();
    float* const value = parts.value + (int64_t)blockIdx.x * k;
    int32_t* const token = parts.token + (int64_t)blockIdx.x * k;
    const int n = list_n;
    if (hit_n <= kList && n <= kList) {
        for (int i = tid; i < n; i += kRowThreads) {
            const float v = list[i];
            const int at = list_at[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += list[j] > v || (list[j] == v && list_at[j] < at) ? 1 : 0;
            if (rank < k) {
                value[rank] = v;
                token[rank] = at;
            }
        }
        for (int i = n + tid; i < k; i += kRowThreads) value[i] = -INFINITY;
        return;
    }
    // More scores than the list holds reach the bound (many equal ones): `keep` rounds of the largest
    // that comes after the last one.
    uint64_t last = ~0ull;  // key: the score's order, then the lower token
    for (int i = 0; i < k; ++i) {
        uint64_t best = 0;
        auto look = [&](float v, int at) {
            if (!(v > -INFINITY)) return;
            const uint32_t u = __float_as_uint(v + 0.f);
            const uint64_t key = (uint64_t)(u >> 31 ? ~u : u | 0x80000000u) << 32 | (uint32_t)~at;
            if (key < last && key > best) best = key;
        };
        if (edge >= 0) look(edge_x, edge);
        for (int slot = first + tid; slot < end; slot += kRowThreads) {
            if (slot < begin) continue;
            const uint4 q = slots.line[slot];
            const T* v = reinterpret_cast<const T*>(&q);
#pragma unroll
            for (int j = 0; j < N; ++j) look(to_f32(v[j]), slots.first_of(slot) + j);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(~0u, best, o));
        if (lane == 0) sh_best[warp] = best;
        __syncthreads();
        for (int q = 0; q < kRowWarps; ++q) best = max(best, sh_best[q]);
        __syncthreads();
        if (tid == 0) {
            const uint32_t u = (uint32_t)(best >> 32);
            value[i] = best ? __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u) : -INFINITY;
            token[i] = (int32_t)~(uint32_t)best;
        }
        last = best;  // (0: nothing is left, and nothing is found below it)
    }
}

// exp of a row's scores against its largest m, summed to about 2^-36 of the sum: the exponent
// (x - m) log2(e) / T as two floats is split into i / 32 and a rest of at most 1 / 64; 2^(i / 32)
// is a table of two floats, the rest's exponential a polynomial (its z^5 / 120 is under 1.3e-12).
// NaN where a score is NaN or m is not finite.  In the order of the scores, whatever their place in memory.
struct PowerTable {
    float2 of[32];  // 2^(i / 32)
};
template <class T>
__device__ double exact_sum(const T* x, int n, float m, double scale, const PowerTable& table, Sum* sh) {
    const float a_hi = (float)scale, a_lo = (float)(scale - (double)a_hi);
    constexpr float kLn2Hi = (float)0.693147180559945309417, kLn2Lo = (float)(0.693147180559945309417 - (double)kLn2Hi);
    Sum s;
    for (int e = threadIdx.x; e < n; e += kJoinThreads) {
        const float v = to_f32(x[e]);
        // v - m = d + d_low
        const float d = __fsub_rn(v, m), back = __fsub_rn(d, v);
        const float d_low = __fsub_rn(__fsub_rn(v, __fsub_rn(d, back)), __fadd_rn(m, back));
        float y = __fmul_rn(d, a_hi);
        if (!(y > -126.f)) {  // nothing, beside a term of 1 (or NaN)
            s.hi += d == d || v == -INFINITY ? 0.f : NAN;
            continue;
        }
        const float y_low = __fmaf_rn(d, a_hi, -y) + (d * a_lo + d_low * a_hi);
        const float i = rintf(y * 32.f);
        const float r = __fmaf_rn(i, -0.03125f, y);  // exact
        // z = (r + y_low) log 2, two floats
        const float z = __fmul_rn(r, kLn2Hi);
        const float z_low = __fmaf_rn(r, kLn2Hi, -z) + __fmaf_rn(r, kLn2Lo, y_low * kLn2Hi);
        const float rest = __fmaf_rn(z * z, __fmaf_rn(z, __fmaf_rn(z, 1.f / 24, 1.f / 6), 0.5f), z_low * (1.f + z));
        const int k = (int)i;
        const float2 t = table.of[k & 31];
        const float p = __fmul_rn(t.x, z), p_low = __fmaf_rn(t.x, z, -p) + __fmaf_rn(t.x, rest, t.y * (1.f + z));
        const float f = __uint_as_float((uint32_t)(127 + (k >> 5)) << 23);  // 2^(k >> 5); k >= -126 * 32
        s.add(t.x * f);
        s.add(p * f);
        s.lo += p_low * f;
    }
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    double total = 0.;
    for (int w = 0; w < kJoinWarps; ++w) total += (double)sh[w].hi + (double)sh[w].lo;
    __syncthreads();
    return total;
}

struct Continuation {
    uint64_t key;  // order of its total
    float x;
    int beam, token;
};
__device__ __forceinline__ bool before(const Continuation& p, const Continuation& q) {
    if (p.key != q.key) return p.key > q.key;
    if (p.beam != q.beam) return p.beam < q.beam;
    return p.x != q.x ? p.x > q.x : p.token < q.token;
}

// A batch item's beams: their parts' sums, and the continuations ranked.
template <class T>
__global__ void __launch_bounds__(kJoinThreads)
beam_join_kernel(BeamArgs a, BeamParts parts, double scale) {
    __shared__ double base[ISO_MAX_BEAMS];  // the total of a beam's largest score; -inf: the beam offers nothing
    __shared__ double off[ISO_MAX_BEAMS];   // how far base may be off
    __shared__ float largest[ISO_MAX_BEAMS];
    __shared__ Continuation list[kList], sorted[kList];
    __shared__ uint32_t sh_v[kJoinWarps];
    __shared__ Sum sh_sum[kJoinWarps];
    __shared__ PowerTable table;
    __shared__ unsigned unsure;
    __shared__ int list_n;
    __shared__ Continuation sh_best[kJoinWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.keep, P = parts.parts;
    const int64_t item = blockIdx.x, row0 = item * a.beams;
    const double inv_t = 1. / a.temperature;
    const float scale_f = (float)scale;
    const T* const x0 = static_cast<const T*>(a.x) + row0 * a.stride;
    if (tid == 0) {
        unsure = 0u;
        list_n = 0;
    }
    if (tid < 32) {
        const double t = exp2((double)tid * 0.03125);
        table.of[tid] = {(float)t, (float)(t - (double)(float)t)};
    }
    __syncthreads();
    wait_for_previous();
    for (int b = warp; b < a.beams; b += kJoinWarps) {
        const float score = a.scores[row0 + b];
        const bool done = a.done && a.done[row0 + b], read = isfinite(score) && !done;
        double of = -INFINITY, err = 0.;
        float m = -INFINITY;
        uint32_t status = 0u;
        if (isfinite(score) && done) of = score;
        if (read) {
            const PartState* s = parts.state + (row0 + b) * P;
            float c = -kFar;
            for (int p = lane; p < P; p += 32) {
                m = fmaxf(m, s[p].m);
                c = fmaxf(c, s[p].c);
            }
            m = warp_max(m);
            c = warp_max(c);
            double sum = 0.;
            for (int p = lane; p < P; p += 32) sum += (double)s[p].s * (double)ex2(fmaxf(s[p].c - c, -200.f));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (!isfinite(m)) {
                status = ISO_ROW_BAD_Y;
            } else if (fabsf(m * scale_f) >= kFar) {
                of = 0.;  // (set below)
                if (lane == 0) atomicOr(&unsure, 1u << b);
            } else if (!isfinite(sum)) {
                status = ISO_ROW_BAD_Y;
            } else {
                // (against m by the float32 scale that the sums were formed with)
                of = score - ((double)c - (double)m * (double)scale_f + log2(sum)) * 0.693147180559945309417;
                err = lse_error(a.n);
            }
        }
        if (lane == 0) {
            base[b] = of;
            off[b] = err;
            largest[b] = m;
            if (a.row_status) a.row_status[row0 + b] = status;
        }
    }
    __syncthreads();
    auto settle = [&]() {  // forms the sums of the beams in `unsure` again
        const unsigned which = unsure;
        __syncthreads();
        for (int b = 0; b < a.beams; ++b) {
            if (!(which >> b & 1u)) continue;
            const double sum = exact_sum(x0 + b * a.stride, a.n, largest[b], scale, table, sh_sum);
            if (tid == 0) {
                const bool bad = !isfinite(sum);
                base[b] = bad ? -INFINITY : (double)a.scores[row0 + b] - log(sum);
                off[b] = 0.;
                if (bad && a.row_status) a.row_status[row0 + b] = ISO_ROW_BAD_Y;
            }
        }
        if (tid == 0) {
            unsure = 0u;
            list_n = 0;
        }
        __syncthreads();
    };
    if (unsure) settle();

    // continuation q of all that the parts have left, then one of each beam that is done
    const int64_t left = (int64_t)a.beams * P * k, count = left + (a.done ? a.beams : 0);
    auto at = [&](int64_t q) {
        Continuation c{0, 0.f, 0, 0};
        if (q >= left) {
            c.beam = (int)(q - left);
            if (a.done[row0 + c.beam] && base[c.beam] > -INFINITY) {
                c.key = order_key(base[c.beam]);
                c.token = (int)a.end;
            }
            return c;
        }
        c.beam = (int)(q / ((int64_t)P * k));
        if (!(base[c.beam] > -INFINITY) || (a.done && a.done[row0 + c.beam])) return c;
        c.x = parts.value[row0 * P * k + q];
        if (c.x > -INFINITY) {
            c.key = order_key(base[c.beam] + ((double)c.x - (double)largest[c.beam]) * inv_t);
            c.token = parts.token[row0 * P * k + q];
        }
        return c;
    };
    float* const out_scores = a.out_scores + item * k;
    int32_t* const parents = a.parents + item * k;
    int64_t* const tokens = a.tokens + item * k;
    auto give = [&](int i, const Continuation& c) {
        const bool some = c.key != 0;
        out_scores[i] = some ? (float)order_value(c.key) : -INFINITY;
        parents[i] = some ? c.beam : -1;
        tokens[i] = some ? c.token : -1;
    };
    for (;;) {
        // a bound that `keep` continuations reach, as for the parts, from the upper halves of their keys
        uint32_t most = 0u;
        for (int64_t q = tid; q < count; q += kJoinThreads) most = max(most, (uint32_t)(at(q).key >> 32));
        const int active = (int)min((int64_t)kJoinWarps, (count + 31) / 32), each = (k + active - 1) / active;
        uint32_t least = 0u;
        for (int i = 0; i < each; ++i) {
            least = __reduce_max_sync(~0u, most);
            if (most == least) most = 0u;
        }
        if (lane == 0) sh_v[warp] = least;
        __syncthreads();
        uint32_t high = ~0u;
        for (int i = 0; i < active; ++i) high = min(high, sh_v[i]);
        // and as far below it as two beams may be off
        const double slack = 2. * lse_error(a.n);
        const uint64_t bound = high ? order_key(order_value((uint64_t)high << 32) - slack) : 1;
        for (int64_t q = tid; q < count; q += kJoinThreads) {
            const Continuation c = at(q);
            if (c.key >= bound) {
                const int i = atomicAdd(&list_n, 1);
                if (i < kList) list[i] = c;
            }
        }
        __syncthreads();
        const int n = list_n;
        if (n > kList) break;
        for (int i = tid; i < n; i += kJoinThreads) {
            const Continuation c = list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += before(list[j], c);
            sorted[rank] = c;
        }
        __syncthreads();
        // neighbours of different beams that are nearer than they may be off
        if (n > k) {
            const double last = order_value(sorted[k - 1].key) - slack;
            for (int i = tid; i + 1 < n; i += kJoinThreads) {
                const Continuation p = sorted[i], q = sorted[i + 1];
                const double gap = order_value(p.key) - order_value(q.key), may = off[p.beam] + off[q.beam];
                if (p.beam != q.beam && may > 0. && !(gap > may) && order_value(q.key) >= last)
                    atomicOr(&unsure, (off[p.beam] > 0. ? 1u << p.beam : 0u) | (off[q.beam] > 0. ? 1u << q.beam : 0u));
            }
        } else {
            for (int i = tid; i + 1 < n; i += kJoinThreads) {
                const Continuation p = sorted[i], q = sorted[i + 1];
                const double gap = order_value(p.key) - order_value(q.key), may = off[p.beam] + off[q.beam];
                if (p.beam != q.beam && may > 0. && !(gap > may))
                    atomicOr(&unsure, (off[p.beam] > 0. ? 1u << p.beam : 0u) | (off[q.beam] > 0. ? 1u << q.beam : 0u));
            }
        }
        __syncthreads();
        if (!unsure) {
            for (int i = tid; i < k; i += kJoinThreads) give(i, i < n ? sorted[i] : Continuation{0, 0.f, 0, 0});
            return;
        }
        settle();
    }
    // More continuations than the list holds reach the bound (many equal ones): all sums formed again,
    // and `keep` rounds of the first that comes after the last one.
    __syncthreads();
    if (tid == 0) {
        for (int b = 0; b < a.beams; ++b)
            if (off[b] > 0.) unsure |= 1u << b;
    }
    __syncthreads();
    settle();
    Continuation last{~0ull, INFINITY, -1, -1};
    for (int i = 0; i < k; ++i) {
        Continuation best{0, 0.f, 0, 0};
        for (int64_t q = tid; q < count; q += kJoinThreads) {
            const Continuation c = at(q);
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
        if (tid == 0) give(i, best);
        if (!best.key) {
            for (int j = i + 1 + tid; j < k; j += kJoinThreads) give(j, best);
            return;
        }
        last = best;
    }
}

// Parts of a row: enough CTAs for the GPU, each with a batch of words at least, and no more words
// than a part has room to note.
int row_parts(int64_t rows, int64_t n, int size, int* share) {
    const int64_t slots = (n * size + 112 + 15) / 16 + 1;
    const int64_t want = (152 * 4 + rows - 1) / std::max<int64_t>(rows, 1);
    int64_t parts = std::min<int64_t>(want, (slots + kBatch - 1) / kBatch);
    parts = std::max<int64_t>(parts, (slots + kMostWords - 1) / kMostWords);
    *share = (int)(((slots + parts - 1) / parts + 7) / 8 * 8);
    if (*share > kMostWords) *share = kMostWords;
    return (int)((slots + *share - 1) / *share);
}

inline size_t align256c(size_t x) { return (x + 255) & ~size_t(255); }

inline int score_size(int dtype) { return dtype == ISO_F32 ? 4 : 2; }

}  // namespace

size_t beam_workspace(int64_t batch, int beams, int64_t n, int dtype, int keep) {
    int share;
    const size_t all = (size_t)(batch * beams) * row_parts(batch * beams, n, score_size(dtype), &share);
    return align256c(all * sizeof(PartState)) + align256c(all * keep * 4) + align256c(all * keep * 4);
}

cudaError_t beam_choose(int dtype, const BeamArgs& a, void* ws, cudaStream_t st) {
    const int64_t rows = a.batch * a.beams;
    BeamParts p;
    p.parts = row_parts(rows, a.n, score_size(dtype), &p.share);
    const size_t all = (size_t)rows * p.parts;
    if (all > 2147483647u) return cudaErrorInvalidConfiguration;
    char* at = static_cast<char*>(ws);
    p.state = reinterpret_cast<PartState*>(at);
    p.value = reinterpret_cast<float*>(at += align256c(all * sizeof(PartState)));
    p.token = reinterpret_cast<int32_t*>(at += align256c(all * a.keep * 4));
    const double scale = 1.4426950408889634074 / a.temperature;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        beam_rows_kernel<T><<<(unsigned)all, kRowThreads, 0, st>>>(a, p, (float)scale);
        cudaError_t e = cudaGetLastError();
        prof_mark(st, "beam_rows");
        if (e != cudaSuccess) return e;
        ClusterLaunch l(a.batch, kJoinThreads, 0, 1, true, st);
        e = l(beam_join_kernel<T>, a, p, scale);
        prof_mark(st, "beam_join");
        return e;
    });
}

}  // namespace isodev
