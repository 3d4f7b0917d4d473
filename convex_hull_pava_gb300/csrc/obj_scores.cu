// Objectives over rows of scores x[r, 0..n): the log-probability of one label
// a row, a clipped policy loss and a preference loss, each with its gradient
// in the scores.
//
//   lp_r = (x[r, l_r] - m) / T - log s,   m = max_j x[r, j],  s = sum_j exp((x[r, j] - m) / T)
//   d L / d x[r, j] = c_r / T * ([j == l_r] - exp((x[r, j] - m) / T) / s),   c_r = d L / d lp_r
//
// The policy loss's c_r follows from row r alone; the preference loss's from
// all tokens of a pair.  A row without a label (l_r < 0) is not read: its
// log-probability and its gradient are 0.
#include "obj_internal.h"
#include "obj_device.cuh"
#include "iso_internal.h"

#include <algorithm>
#include <type_traits>
#define MINB 3

namespace isodev {

namespace {


inline __host__ __device__ size_t align256o(size_t x) { return (x + 255) & ~size_t(255); }

inline int row_grid(int64_t rows) { return (int)std::min<int64_t>(rows, 1 << 20); }

// One row's part of the policy loss, from its log-probability.
struct PolicyRow {
    float coef, pg, kl, cut;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& p, float logp, float old,
                                                float adv, float ref, float w) {
    const float ratio = expf(logp - old);
    const float free = -adv * ratio;
    const float held = -adv * fminf(fmaxf(ratio, p.low), p.high);
    const bool cut = held > free;
    PolicyRow q;
    q.coef = cut ? 0.f : w * free;
    q.pg = w * (cut ? held : free);
    q.cut = cut ? w : 0.f;
    q.kl = 0.f;
    if (p.ref_logp) {
        // exp(d) - 1 - d without its cancellation at small d
        const float d = ref - logp, e = expm1f(d);
        q.kl = w * (e - d);
        q.coef -= p.kl_coef * w * e;
    }
    return q;
}

// The gradient of a row: h exp(...) throughout, and g more at the label.
template <class T>
struct RowGrad {
    float g, h;
    SoftRef ref;
    template <bool FAR>
    __device__ __forceinline__ uint4 word(const uint4& w) const {
        float2 v[Word<T>::N / 2];
        word_exp<T, FAR>(w, ref, v);
#pragma unroll
        for (int i = 0; i < Word<T>::N / 2; ++i) v[i] = mul2(v[i], {h, h});
        return pack(v, T());
    }
    __device__ __forceinline__ T one(float x, bool label) const {
        return from_f32<T>(h * ref.exp(x) + (label ? g : 0.f));
    }
};

__device__ __forceinline__ uint32_t norm_status(SoftState st) {
    return isfinite(st.m) && isfinite(st.s) ? 0u : ISO_ROW_BAD_Y;
}

// What is asked of a row's scores.
enum class Ask { kLogp, kPolicy };

struct RowOuts {
    float *logp, *norm, *coef;
    void* out;
    int64_t out_stride;
    int out_words;  // the gradient's rows are aligned as the scores' rows: words can be stored
    uint32_t* status;
};

// A row as words of 16 bytes between at most 2 (N - 1) single scores (N a word), of which a CTA
// of a cluster takes an equal share.
template <class T>
struct RowShape {
    int head, words, tail;  // single scores before the words, words, single scores after
    int first, count;       // this CTA's words
    // ctas: a power of two of which `shift` is the exponent, or any number with shift < 0
    __device__ __forceinline__ RowShape(const T* x, int n, int rank, int ctas, int shift = -1) {
        constexpr int N = Word<T>::N;
        const int at = (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (N - 1);
        head = min(n, (N - at) & (N - 1));
        words = (n - head) / N;
        tail = n - head - words * N;
        const int share = shift < 0 ? (words + ctas - 1) / ctas : (words + ctas - 1) >> shift;
        first = min(words, rank * share);
        count = min(words, first + share) - first;
    }
    // The thread of a team that has the label's word, or -1.
    __device__ __forceinline__ int owner(int64_t label, int team) const {
        const int64_t j = label - head - (int64_t)first * Word<T>::N;
        return j >= 0 && j < (int64_t)count * Word<T>::N ? (int)(j / Word<T>::N) % team : -1;
    }
    // The single score that lane e of the row's first warp takes, or -1.
    __device__ __forceinline__ int edge(int n, int e) const {
        return e < head ? e : e < head + tail ? n - tail + (e - head) : -1;
    }
};

// A word of a gradient, whole or score by score.
template <class T>
__device__ __forceinline__ void store_word(T* at, const uint4& w, bool whole) {
    if (whole) {
        store_streaming(at, w);
    } else {
        const T* v = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int i = 0; i < Word<T>::N; ++i) at[i] = v[i];
    }
}

// What a team has of its next row before that row's turn; the scores' words are on their way to
// shared memory.
struct RowAhead {
    int64_t label;
    float at_label, edge, old, adv, ref, w;
};

// Teams of TEAM threads (a warp; a CTA; the CTAs of a cluster) take the rows in turn.  Each thread
// copies its words of the next row (up to K) to a place of its own in shared memory while it works
// on the current one, which it holds in registers from the maximum to the gradient: the scores are
// read once.  A thread reads only what it has copied, so the one thing that a team shares is the
// row's (maximum, sum); the warps of a cluster write theirs to every CTA and meet once a row.
// LONG: rows longer than the team's registers are read twice, the second time from L2.
template <class T, Ask ASK, int NT, int TEAM, int K, bool LONG>
__global__ void __launch_bounds__(NT, NT * K >= 4096 ? 2 : NT == 128 ? 6 : 3)
score_rows_kernel(ScoreRows sc, PolicyArgs p, RowOuts o) {
    constexpr int N = Word<T>::N, W = NT / 32;
    extern __shared__ uint4 ahead_words[];
    __shared__ SoftState part[2][TEAM == 32 ? 1 : 8 * W];
    const int ctas = TEAM == 32 ? 1 : (int)cluster_size(), rank = TEAM == 32 ? 0 : (int)cluster_rank();
    const int shift = 31 - __clz(ctas);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tt = TEAM == 32 ? lane : threadIdx.x;
    const int64_t teams = TEAM == 32 ? (int64_t)gridDim.x * W : gridDim.x >> shift;
    int64_t r = TEAM == 32 ? (int64_t)blockIdx.x * W + warp : blockIdx.x >> shift;
    uint4* mine = ahead_words + (TEAM == 32 ? warp * 32 * K : 0) + tt;
    const float a = kLog2e * sc.inv_t;
    const int n = sc.n;
    const bool edges = rank == 0 && tt < 32;
    const T* const base = static_cast<const T*>(sc.x);

    auto start = [&](int64_t row, int64_t label) {
        RowAhead h;
        h.label = label;
        h.at_label = h.edge = h.old = h.adv = h.ref = h.w = 0.f;
        if (label >= 0) {
            const T* x = base + row * sc.stride;
            const RowShape<T> s(x, n, rank, ctas, shift);
            if (!LONG) {
                const uint4* src = reinterpret_cast<const uint4*>(x + s.head) + s.first + tt;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (tt + k * TEAM < s.count) copy_async(mine + k * TEAM, src + k * TEAM);
            }
            h.at_label = label < n ? to_f32(x[label]) : NAN;
            const int e = edges ? s.edge(n, tt) : -1;
            h.edge = e >= 0 ? to_f32(x[e]) : -INFINITY;
            if (ASK == Ask::kPolicy) {
                h.old = p.old_logp[row];
                h.adv = p.advantages[row];
                if (p.ref_logp) h.ref = p.ref_logp[row];
                if (p.weights) h.w = p.weights[row];
            }
        }
        copy_async_commit();
        return h;
    };

    if (r >= sc.rows) return;
    int64_t label_next = r + teams < sc.rows ? sc.labels[r + teams] : -1;
    RowAhead cur = start(r, sc.labels[r]), next;
    const float inv_count = ASK == Ask::kPolicy && !p.weights ? *p.inv_count : 0.f;
    for (int turn = 0; r < sc.rows; r += teams, cur = next) {
        const int64_t after = r + 2 * teams;
        const int64_t label_after = after < sc.rows ? sc.labels[after] : -1;
        const T* x = base + r * sc.stride;
        const RowShape<T> s(x, n, rank, ctas, shift);
        const int rounds = (s.count + TEAM - 1) / TEAM;  // the same in all threads, as is what depends on it
        T* out = static_cast<T*>(o.out) + r * o.out_stride;
        uint4 w[K];
        float top = -INFINITY;
        if (cur.label >= 0) {
            copy_async_wait_all();
            top = cur.edge;
            if (!LONG) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k < rounds) {
                        w[k] = mine[k * TEAM];
                        if (tt + k * TEAM >= s.count) w[k] = word_closed(T());
                        top = fmaxf(top, word_max(w[k], T()));
                    }
            }
        }
        next = start(r + teams, label_next);
        label_next = label_after;
        if (cur.label < 0) {
            if (rank == 0 && tt == 0) {
                o.logp[r] = 0.f;
                o.norm[2 * r] = 0.f;
                o.norm[2 * r + 1] = 1.f;
                if (o.coef) o.coef[r] = 0.f;
                if (o.status) o.status[r] = 0u;
                if (ASK == Ask::kPolicy)
                    for (int i = 0; i < 3; ++i) p.terms[i * sc.rows + r] = 0.f;
            }
            if (ASK == Ask::kPolicy && o.out) {
                if (o.out_words) {
                    uint4* dst = reinterpret_cast<uint4*>(out + s.head) + s.first;
                    for (int j = tt; j < s.count; j += TEAM) store_streaming(dst + j, uint4{0, 0, 0, 0});
                    const int e = edges ? s.edge(n, tt) : -1;
                    if (e >= 0) out[e] = from_f32<T>(0.f);
                } else {
                    for (int j = rank * TEAM + tt; j < n; j += ctas * TEAM) out[j] = from_f32<T>(0.f);
                }
            }
            continue;
        }

        // the warp's sum, against the warp's maximum
        SoftState st;
        float2 sum{0.f, 0.f};
        if (!LONG) {
            st.m = warp_max(top);
            const SoftRef ref(st.m, a);
            auto add = [&](auto far) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k < rounds) {
                        float2 v[N / 2];
                        word_exp<T, decltype(far)::value>(w[k], ref, v);
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) sum = add2(sum, v[i]);
                    }
            };
            ref.far ? add(std::true_type()) : add(std::false_type());
            st.s = warp_add((edges ? ref.exp(cur.edge) : 0.f) + sum.x + sum.y);
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(x + s.head) + s.first;
            st.m = cur.edge;
            st.s = edges ? SoftRef(st.m, a).exp(cur.edge) : 0.f;
            for (int j = tt; j < s.count; j += K * TEAM) {
                float m = -INFINITY;
#pragma unroll
                for (int k = 0; k < K; ++k) w[k] = j + k * TEAM < s.count ? src[j + k * TEAM] : word_closed(T());
#pragma unroll
                for (int k = 0; k < K; ++k) m = fmaxf(m, word_max(w[k], T()));
                soft_raise(st, m, a);
                const SoftRef ref(st.m, a);
                sum = {0.f, 0.f};
                auto add = [&](auto far) {
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        float2 v[N / 2];
                        word_exp<T, decltype(far)::value>(w[k], ref, v);
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) sum = add2(sum, v[i]);
                    }
                };
                ref.far ? add(std::true_type()) : add(std::false_type());
                st.s += sum.x + sum.y;
            }
            st = soft_warp(st, a);
        }
        if (TEAM != 32) {
            // Two sets of places in turn: a CTA that writes to one again has been through the
            // meeting in between, for which every thread had read the first.
            SoftState* slot = part[turn++ & 1];
            if (ctas == 1) {
                if (lane == 0) slot[warp] = st;
                __syncthreads();
            } else {
                if (lane < ctas) store_remote(&slot[rank * W + warp], lane, st);
                __syncwarp();
                cluster_sync();
            }
            constexpr int P = 8 * W / 32;
            SoftState q[P];
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                q[i] = lane + 32 * i < ctas * W ? slot[lane + 32 * i] : soft_empty();
                m = fmaxf(m, q[i].m);
            }
            st.m = warp_max(m);
            const SoftRef ref(st.m, a);
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) t += q[i].s * ref.factor(q[i].m);
            st.s = warp_add(t);
        }

        const SoftRef ref(st.m, a);
        const float lp = ref.of(cur.at_label) * kLn2 - logf(st.s);
        PolicyRow q{};
        if (ASK == Ask::kPolicy)
            q = policy_row(p, lp, cur.old, cur.adv, cur.ref, p.weights ? cur.w : inv_count);
        if (rank == 0 && tt == 0) {
            o.logp[r] = lp;
            o.norm[2 * r] = st.m;
            o.norm[2 * r + 1] = st.s;
            if (o.coef) o.coef[r] = q.coef;
            if (o.status) o.status[r] = norm_status(st) | (cur.label >= n ? ISO_ROW_BAD_LABEL : 0u);
            if (ASK == Ask::kPolicy) {
                p.terms[r] = q.pg;
                p.terms[sc.rows + r] = q.kl;
                p.terms[2 * sc.rows + r] = q.cut;
            }
        }
        if (ASK == Ask::kLogp || !o.out) continue;

        const float g = q.coef * p.grad_scale * sc.inv_t;
        const RowGrad<T> grad{g, -g / st.s, ref};
        if (!LONG && o.out_words) {
            uint4* dst = reinterpret_cast<uint4*>(out + s.head) + s.first + tt;
            auto give = [&](auto far) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k < rounds) {
                        const uint4 d = grad.template word<decltype(far)::value>(w[k]);
                        if (tt + k * TEAM < s.count) store_streaming(dst + k * TEAM, d);
                    }
            };
            ref.far ? give(std::true_type()) : give(std::false_type());
        } else {
            // read again: the row is long, or its gradient lies at other places within 16 bytes
            const uint4* src = reinterpret_cast<const uint4*>(x + s.head) + s.first;
            T* dst = out + s.head + (int64_t)s.first * N;
            for (int j = tt; j < s.count; j += TEAM) {
                const uint4 word = src[j];
                store_word(dst + (int64_t)j * N, ref.far ? grad.template word<true>(word) : grad.template word<false>(word), o.out_words);
            }
        }
        const int e = edges ? s.edge(n, tt) : -1;
        if (e >= 0) out[e] = grad.one(cur.edge, e == cur.label);
        // the label's score again, by the thread that has just written its word
        if (s.owner(cur.label, TEAM) == tt) out[cur.label] = grad.one(cur.at_label, true);
    }
    copy_async_wait_all();
}

// out = g (onehot - p) with g from the rows' coefficients: a CTA takes K words a thread of one
// row, from the last row to the first (the forward has read them in order, so that the last
// ones are in L2).
template <class T, int NT, int K>
__global__ void __launch_bounds__(NT)
score_backward_kernel(ScoreRows sc, const float* __restrict__ norm, const float* __restrict__ coef,
                      float grad_scale, const float* grad_scale_dev, int changed_only, RowOuts o,
                      int parts) {
    constexpr int N = Word<T>::N;
    if (grad_scale_dev) {
        const float g = *grad_scale_dev;
        if (changed_only && g == 1.f) return;
        grad_scale *= g;
    }
    const float a = kLog2e * sc.inv_t;
    const int n = sc.n, tt = threadIdx.x;
    for (int64_t unit = blockIdx.x; unit < sc.rows * parts; unit += gridDim.x) {
        const int64_t r = sc.rows - 1 - unit / parts;
        const int part = (int)(unit % parts);
        const T* x = static_cast<const T*>(sc.x) + r * sc.stride;
        T* out = static_cast<T*>(o.out) + r * o.out_stride;
        const RowShape<T> s(x, n, part, parts);
        const int64_t label = sc.labels[r];
        const uint4* src = reinterpret_cast<const uint4*>(x + s.head) + s.first;
        uint4* dst = reinterpret_cast<uint4*>(out + s.head) + s.first;
        const int e = part == 0 && tt < 32 ? s.edge(n, tt) : -1;
        if (label < 0) {
            if (o.out_words) {
                for (int j = tt; j < s.count; j += NT) store_streaming(dst + j, uint4{0, 0, 0, 0});
            } else {
                for (int j = tt; j < s.count * N; j += NT) out[s.head + (int64_t)s.first * N + j] = from_f32<T>(0.f);
            }
            if (e >= 0) out[e] = from_f32<T>(0.f);
            continue;
        }
        const float edge = e >= 0 ? to_f32(x[e]) : 0.f;
        const float m = norm[2 * r], sum = norm[2 * r + 1];
        const float g = coef[r] * grad_scale * sc.inv_t;
        const RowGrad<T> grad{g, -g / sum, SoftRef(m, a)};
        const bool owner = s.owner(label, NT) == tt;
        const float at_label = owner ? to_f32(x[label]) : 0.f;
        for (int j = tt; j < s.count; j += K * NT) {
            uint4 w[K];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (j + k * NT < s.count) w[k] = load_streaming(src + j + k * NT);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (j + k * NT < s.count) {
                    const uint4 d = grad.ref.far ? grad.template word<true>(w[k]) : grad.template word<false>(w[k]);
                    store_word(out + s.head + (int64_t)(s.first + j + k * NT) * N, d, o.out_words);
                }
        }
        if (e >= 0) out[e] = grad.one(edge, e == label);
        if (owner) out[label] = grad.one(at_label, true);
    }
}

// 1 / (number of labelled rows), for the mean over them; 0 when there are none.
__global__ void __launch_bounds__(1024)
count_labels_kernel(const int64_t* __restrict__ labels, int64_t rows, float* __restrict__ inv) {
    __shared__ double sh[32];
    double c = 0.0;
    for (int64_t r = threadIdx.x; r < rows; r += 1024) c += labels[r] >= 0 ? 1.0 : 0.0;
    c = cta_sum<1024>(c, sh);
    if (threadIdx.x == 0) *inv = c > 0.0 ? (float)(1.0 / c) : 0.f;
}

// The rows' terms, summed in 64 bits in a fixed order.
__global__ void __launch_bounds__(1024)
policy_finish_kernel(const float* __restrict__ terms, int64_t rows, float kl_coef,
                     float* __restrict__ loss, float* __restrict__ stats) {
    __shared__ double sh[32];
    double v[3];
    for (int i = 0; i < 3; ++i) {
        double c = 0.0;
        for (int64_t r = threadIdx.x; r < rows; r += 1024) c += terms[i * rows + r];
        v[i] = cta_sum<1024>(c, sh);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) stats[i] = (float)v[i];
        *loss = (float)(v[0] + (double)kl_coef * v[1]);
    }
}

// One CTA per pair: the two sequences' sums, the pair's loss and the
// coefficient of every labelled token of the two.
__global__ void __launch_bounds__(256)
preference_pairs_kernel(PreferenceArgs p, const int64_t* __restrict__ labels, int64_t rows,
                        const float* __restrict__ logp, float* __restrict__ coef) {
    __shared__ double sh[8];
    __shared__ float sh_each[2];
    for (int64_t q = blockIdx.x; q < p.pairs; q += gridDim.x) {
        double seq[2], gain[2], count[2];
        bool bad = false;
        for (int i = 0; i < 2; ++i) {
            const int64_t a = p.offsets[2 * q + i], b = p.offsets[2 * q + i + 1];
            const bool ok = a >= 0 && b >= a && b <= rows;
            bad = bad || !ok;
            double s = 0.0, g = 0.0, c = 0.0;
            if (ok)
                for (int64_t r = a + threadIdx.x; r < b; r += 256)
                    if (labels[r] >= 0) {
                        const double lp = logp[r];
                        s += lp;
                        g += p.ref_logp ? lp - (double)p.ref_logp[r] : lp;
                        c += 1.0;
                    }
            seq[i] = cta_sum<256>(s, sh);
            gain[i] = cta_sum<256>(g, sh);
            count[i] = cta_sum<256>(c, sh);
        }
        if (threadIdx.x == 0) {
            double share[2];
            for (int i = 0; i < 2; ++i) {
                share[i] = p.average ? 1.0 / fmax(count[i], 1.0) : 1.0;
                seq[i] *= share[i];
                gain[i] *= share[i];
                p.seq_logp[2 * q + i] = bad ? NAN : (float)seq[i];
            }
            const double h = gain[0] - gain[1], beta = p.beta, z = beta * h;
            double each, slope;  // the pair's loss and its derivative in h
            if (p.kind == ISO_PREFERENCE_SIGMOID) {
                const double e = exp(-fabs(z)), over = log1p(e);
                const double up = z >= 0 ? 1.0 / (1.0 + e) : e / (1.0 + e);  // sigmoid(z)
                const double dn = z >= 0 ? e / (1.0 + e) : 1.0 / (1.0 + e);  // sigmoid(-z)
                each = over + (1.0 - p.smooth) * (z < 0 ? -z : 0.0) + p.smooth * (z > 0 ? z : 0.0);
                slope = beta * (p.smooth * up - (1.0 - p.smooth) * dn);
            } else if (p.kind == ISO_PREFERENCE_HINGE) {
                each = z < 1.0 ? 1.0 - z : (z >= 1.0 ? 0.0 : z);
                slope = z < 1.0 ? -beta : 0.0;
            } else {
                const double d = h - 0.5 / beta;
                each = d * d;
                slope = 2.0 * d;
            }
            if (bad) each = slope = NAN;
            p.margins[q] = bad ? NAN : (float)z;
            p.each[q] = (float)each;
            if (p.pair_status) p.pair_status[q] = bad ? ISO_ROW_BAD_SHAPE : 0u;
            sh_each[0] = (float)(slope * share[0] / (double)p.pairs);
            sh_each[1] = (float)(-slope * share[1] / (double)p.pairs);
        }
        __syncthreads();
        if (coef)
            for (int i = 0; i < 2; ++i) {
                const int64_t a = p.offsets[2 * q + i], b = p.offsets[2 * q + i + 1];
                if (a < 0 || b < a || b > rows) continue;
                for (int64_t r = a + threadIdx.x; r < b; r += 256)
                    if (labels[r] >= 0) coef[r] = sh_each[i];
            }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256)
preference_finish_kernel(const float* __restrict__ each, int64_t pairs, float* __restrict__ loss) {
    __shared__ double sh[8];
    double c = 0.0;
    for (int64_t q = threadIdx.x; q < pairs; q += 256) c += each[q];
    c = cta_sum<256>(c, sh);
    if (threadIdx.x == 0) *loss = pairs > 0 ? (float)(c / (double)pairs) : 0.f;
}

template <class T, Ask ASK, int NT, int TEAM, int K, bool LONG>
cudaError_t launch_rows(const ScoreRows& s, const PolicyArgs& p, const RowOuts& o, int ctas, cudaStream_t st) {
    auto* kernel = score_rows_kernel<T, ASK, NT, TEAM, K, LONG>;
    constexpr size_t shared = LONG ? 0 : (size_t)NT * K * 16;
    cudaLaunchConfig_t c{};
    c.blockDim = dim3(NT);
    c.dynamicSmemBytes = shared;
    c.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = TEAM == 32 ? 0 : 1;
    // the clusters of this size that the GPU holds at once (a cluster's CTAs share a group of SMs,
    // so that they are fewer than its SMs alone would take); asked once
    static int held[64][4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int& fit = held[dev][ctas == 1 ? 0 : ctas == 2 ? 1 : ctas == 4 ? 2 : 3];
    if (fit == 0) {
        if (shared > 48 * 1024 &&
            (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared)) != cudaSuccess)
            return e;
        int n = 0;
        c.gridDim = dim3((unsigned)(device_sms() * ctas));
        if (ctas == 1) {
            if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, NT, shared)) != cudaSuccess) return e;
            n *= device_sms();
        } else if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &c)) != cudaSuccess) {
            return e;
        }
        fit = std::max(1, n);
    }
    const int64_t wanted = TEAM == 32 ? (s.rows + NT / 32 - 1) / (NT / 32) : s.rows;
    c.gridDim = dim3((unsigned)(std::min<int64_t>(wanted, fit) * ctas));
    return cudaLaunchKernelEx(&c, kernel, s, p, o);
}

// By a row's bytes: a warp holds up to 4 KB, a CTA 16, 32 or 64 KB and a cluster up to 8 times that;
// longer rows are read twice.
template <class T, Ask ASK>
cudaError_t run_rows(const ScoreRows& s, const PolicyArgs& p, const RowOuts& o, cudaStream_t st) {
    if (s.rows == 0) return cudaSuccess;
    const int64_t words = (s.n + Word<T>::N - 1) / Word<T>::N;
    if (words <= 32 * 8) return launch_rows<T, ASK, 256, 32, 8, false>(s, p, o, 1, st);
    if (words > 8 * 256 * 16) return launch_rows<T, ASK, 256, 256, 8, true>(s, p, o, 8, st);
    int ctas = 1;
    while (words > (int64_t)ctas * 256 * 16) ctas *= 2;
    // few rows: more CTAs for each, down to a word a thread
    while (ctas < 8 && s.rows * ctas < device_sms() && words > (int64_t)ctas * 256) ctas *= 2;
    if (words <= ctas * 128 * 8) return launch_rows<T, ASK, 128, 128, 8, false>(s, p, o, ctas, st);
    if (words <= ctas * 256 * 8) return launch_rows<T, ASK, 256, 256, 8, false>(s, p, o, ctas, st);
    return launch_rows<T, ASK, 256, 256, 16, false>(s, p, o, ctas, st);
}

template <class F>
cudaError_t by_type(int dtype, F f) {
    switch (dtype) {
        case ISO_F32: return f(float{});
        case ISO_BF16: return f(__nv_bfloat16{});
        default: return f(__half{});
    }
}

// Whether the gradient's rows start at the same place within 16 bytes as the scores' rows.
inline int words_agree(const ScoreRows& s, const void* out, int64_t out_stride, int dtype) {
    const int64_t size = dtype == ISO_F32 ? 4 : 2;
    const uintptr_t off = reinterpret_cast<uintptr_t>(s.x) ^ reinterpret_cast<uintptr_t>(out);
    return (off & 15u) == 0 && (s.rows <= 1 || ((s.stride - out_stride) * size) % 16 == 0);
}

}  // namespace

cudaError_t token_logp(int dtype, const ScoreRows& s, float* logp, float* norm, float* zero_coef,
                       uint32_t* row_status, cudaStream_t st) {
    const RowOuts o{logp, norm, zero_coef, nullptr, 0, 0, row_status};
    return by_type(dtype, [&](auto t) {
        return run_rows<decltype(t), Ask::kLogp>(s, PolicyArgs{}, o, st);
    });
}

cudaError_t token_logp_backward(int dtype, const ScoreRows& s, const float* norm, const float* coef,
                                float grad_scale, const float* grad_scale_dev, int changed_only,
                                void* out, int64_t out_stride, cudaStream_t st) {
    if (s.rows == 0) return cudaSuccess;
    const RowOuts o{nullptr, nullptr, nullptr, out, out_stride, words_agree(s, out, out_stride, dtype), nullptr};
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int NT = 256, K = 4;
        const int64_t words = (s.n + Word<T>::N - 1) / Word<T>::N;
        const int parts = (int)std::max<int64_t>(1, (words + NT * K - 1) / (NT * K));
        score_backward_kernel<T, NT, K><<<(unsigned)std::min<int64_t>(s.rows * parts, 1 << 30), NT, 0, st>>>(
            s, norm, coef, grad_scale, grad_scale_dev, changed_only, o, parts);
        return cudaGetLastError();
    });
}

size_t policy_workspace(int64_t rows) { return 256 + align256o((size_t)rows * 12); }

cudaError_t policy_loss(int dtype, const ScoreRows& s, const PolicyArgs& args, float* loss,
                        float* stats, void* out, int64_t out_stride, void* ws,
                        uint32_t* row_status, cudaStream_t st) {
    PolicyArgs p = args;
    float* inv = static_cast<float*>(ws);
    p.inv_count = inv;
    p.terms = inv + 64;
    cudaError_t e = cudaSuccess;
    if (!p.weights) {
        count_labels_kernel<<<1, 1024, 0, st>>>(s.labels, s.rows, inv);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const RowOuts o{p.logp, p.norm, p.coef, out, out_stride, out ? words_agree(s, out, out_stride, dtype) : 0, row_status};
    e = by_type(dtype, [&](auto t) { return run_rows<decltype(t), Ask::kPolicy>(s, p, o, st); });
    if (e != cudaSuccess) return e;
    policy_finish_kernel<<<1, 1024, 0, st>>>(p.terms, s.rows, p.kl_coef, loss, stats);
    return cudaGetLastError();
}

size_t preference_workspace(int64_t, int64_t pairs) { return align256o((size_t)pairs * 4) + 256; }

cudaError_t preference_loss(int dtype, const ScoreRows& s, PreferenceArgs p, float* logp,
                            float* norm, float* coef, float grad_scale, void* out,
                            int64_t out_stride, void* ws, uint32_t* row_status, cudaStream_t st) {
    p.each = static_cast<float*>(ws);
    cudaError_t e = token_logp(dtype, s, logp, norm, coef, row_status, st);
    if (e != cudaSuccess) return e;
    if (p.pairs > 0) {
        preference_pairs_kernel<<<row_grid(p.pairs), 256, 0, st>>>(p, s.labels, s.rows, logp, coef);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    preference_finish_kernel<<<1, 256, 0, st>>>(p.each, p.pairs, p.loss);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (!out) return cudaSuccess;
    return token_logp_backward(dtype, s, norm, coef, grad_scale, nullptr, 0, out, out_stride, st);
}

}  // namespace isodev
