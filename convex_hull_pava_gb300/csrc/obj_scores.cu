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
#include "obj_launch.h"

#include <type_traits>

namespace isodev {

namespace {


inline __host__ __device__ size_t align256o(size_t x) { return (x + 255) & ~size_t(255); }

// The most teams of a launch: what the workspace has room for.
constexpr int64_t kMaxTeams = 32768;

}  // namespace

// Partial sums of the policy loss: policy term, KL term, clipped weight.
struct PolicyTerms {
    Sum v[3];
};

namespace {

// Which rows a team takes: first the row of its own number, whose scores it can ask for at once; then,
// where there are more rows than teams, of the rows behind those, which another kernel lists
// meanwhile: the labelled ones in order from the list's front, the others in order from its back, so
// that teams have equal work.
struct RowList {
    const ListHead* head;
    const int32_t* list;  // or NULL: no more rows than teams
    int64_t rows;         // listed, with and without a label
};

// One row's part of the policy loss, from its log-probability.
struct PolicyRow {
    float coef, pg, kl, cut;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& p, LogP logp, float old,
                                                float adv, float ref, float w) {
    const float ratio = expf(logp.minus(old));
    // (an advantage of 0 leaves nothing, also of a ratio past float32's range)
    const float free = adv == 0.f && ratio == INFINITY ? 0.f : -adv * ratio;
    const float held = -adv * fminf(fmaxf(ratio, p.low), p.high);
    const bool cut = held > free;
    PolicyRow q;
    q.coef = cut ? 0.f : w * free;
    q.pg = w * (cut ? held : free);
    q.cut = cut ? w : 0.f;
    q.kl = 0.f;
    if (p.ref_logp) {
        // exp(d) - 1 - d without its cancellation at small d
        const float d = -logp.minus(ref), e = expm1f(d);
        q.kl = w * (e - d);
        if (p.kl_coef != 0.f) q.coef -= p.kl_coef * w * e;  // (0 of an exponential past float32's range is 0)
    }
    return q;
}

// The gradient of a row: h exp(...) throughout, and g more at the label; h = -g / s by __fdividef (2
// units in the last place, beside ex2's; s is far from where that instruction gives 0).
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

// A preference loss that the backward adds up (loss NULL: none).
struct PairSum {
    const float* each;
    int64_t pairs;
    float* loss;
};

struct RowOuts {
    float *logp, *norm, *coef;
    float* rest;  // or NULL: what logp's rounding to float32 has left out
    void* out;
    int64_t out_stride;
    int out_words;  // the gradient's rows are aligned as the scores' rows: words can be stored
    uint32_t* status;
};

// A row as words of 16 bytes between at most 2 (N - 1) single scores (N a word), shared out to a number
// of readers (CTAs) in stretches that start where 128 bytes do; a reader's threads take its words
// so that those of 8 neighbouring threads share 128 bytes: thread t has words t - skew, t - skew +
// threads, ... of its stretch.  Rows that start elsewhere (an odd number of scores) would otherwise
// have every 128 bytes asked for twice: in 32,771-score rows of bfloat16, 14.8 million sectors of 32
// bytes for 9.0 million.
template <class T>
struct RowShape {
    int head, words, tail;   // single scores before the words, words, single scores after
    int first, count, skew;  // this reader's words, and the threads before the first one's
    // 1 << shift readers, or stretches of `fixed` words (a multiple of 8) if that is not 0.
    __device__ __forceinline__ RowShape(const T* x, int n, int rank, int shift, int fixed = 0) {
        constexpr int N = Word<T>::N;
        const uintptr_t at = reinterpret_cast<uintptr_t>(x) / sizeof(T);
        head = min(n, (int)(-at & (N - 1)));
        words = (n - head) / N;
        tail = n - head - words * N;
        const int before = (int)((at + head) / N) & 7, total = words + before;
        const int share = fixed ? fixed : (((total + (1 << shift) - 1) >> shift) + 7) & ~7;
        const int from = min(total, rank * share), end = min(total, from + share);
        first = max(from, before) - before;
        skew = max(before - from, 0);
        count = max(end - max(from, before), 0);
    }
    // Whether this reader has a word of index j; the rounds that its threads take their words in.
    __device__ __forceinline__ bool has(int j) const { return (unsigned)j < (unsigned)count; }
    __device__ __forceinline__ int rounds(int threads) const { return (count + skew + threads - 1) / threads; }
    // The thread of a team that has the label's word, or -1.
    __device__ __forceinline__ int owner(int64_t label, int team) const {
        const int64_t j = label - head - (int64_t)first * Word<T>::N;
        return j >= 0 && j < (int64_t)count * Word<T>::N ? ((int)(j / Word<T>::N) + skew) % team : -1;
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

// What a team has of its next row before that row's turn, beside its words, which are on their way
// to shared memory.
struct RowAhead {
    int row;     // -1: none
    int label;   // -1: none; n where it is not below n
    float edge;  // the single score that this lane takes, or -inf
};

// A row without a label: zeros.
__device__ __forceinline__ void unlabelled_row(const RowOuts& o, int64_t r) {
    o.logp[r] = 0.f;
    *reinterpret_cast<float2*>(o.norm + 2 * r) = {0.f, 1.f};
    if (o.coef) o.coef[r] = 0.f;
    if (o.status) o.status[r] = 0u;
}

// Teams of TEAM threads (a warp; a CTA; the CTAs of a cluster) take the rows in turn.  Each thread
// copies its words of the next row (up to K) to a place of its own in shared memory while it works
// on the current one, which it holds in registers from the maximum to the gradient: the scores are
// read once.  A thread reads only what it has copied, so the one thing that a team shares is the
// row's (maximum, sum); the warps of a cluster write theirs to every CTA and meet once a row.
// LONG: rows longer than the team's registers are read twice, the second time from L2.
// Bound by HBM where rows are long (8,192 x 131,072 bf16, 3.65 GB: 605 us, 6.0 TB/s; 8,192 x 65,536:
// 321 us, 6.4 TB/s), by a row's chain of steps where its stretch is short: a turn of a 50 KB stretch
// takes 6.3 us with two CTAs an SM, of which the exponentials are a third (2,047 x 50,021: 85 us,
// 4.5 TB/s).  Registers hold the row because shared memory holds the next one: together they keep
// 256 KB an SM on the chip.  16 words a thread and not 8: what a row costs each warp beside its
// words, some 600 instructions, is then half as much a score (21.6 instructions a score became 13.4).
template <class T, int NT, int TEAM, int K, bool LONG>
__global__ void __launch_bounds__(NT, NT * K > 4096 ? 1 : NT * K == 4096 ? 2 : NT == 128 ? 6 : 3)
policy_rows_kernel(ScoreRows sc, PolicyArgs p, RowOuts o, RowList rl) {
    constexpr int N = Word<T>::N, W = NT / 32;
    extern __shared__ uint4 ahead_words[];
    __shared__ SoftState part[2][TEAM == 32 ? 2 : 8 * W];
    __shared__ uint64_t come[2];
    __shared__ bool any_lost;
    const int ctas = TEAM == 32 ? 1 : (int)cluster_size(), rank = TEAM == 32 ? 0 : (int)cluster_rank();
    const int shift = 31 - __clz(ctas);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tt = TEAM == 32 ? lane : threadIdx.x;
    const uint32_t teams = TEAM == 32 ? gridDim.x * W : gridDim.x >> shift;
    const uint32_t team = TEAM == 32 ? blockIdx.x * W + warp : blockIdx.x >> shift;
    uint4* mine = ahead_words + (TEAM == 32 ? warp * 32 * K : 0) + tt;
    const float a = sc.a;
    const int n = sc.n;
    const bool edges = rank == 0 && tt < 32;
    const T* const base = static_cast<const T*>(sc.x);

    auto start = [&](int row, int64_t label) {
        RowAhead h{row, label < 0 ? -1 : label < n ? (int)label : n, -INFINITY};
        if (label >= 0) {
            const T* x = base + row * sc.stride;
            const RowShape<T> s(x, n, rank, shift);
            if (!LONG) {
                const int j = tt - s.skew;
                const uint4* src = reinterpret_cast<const uint4*>(x + s.head) + s.first + j;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (s.has(j + k * TEAM)) copy_async(mine + k * TEAM, src + k * TEAM);
            }
            const int e = edges ? s.edge(n, tt) : -1;
            if (e >= 0) h.edge = to_f32(x[e]);
        }
        copy_async_commit();
        return h;
    };
    auto zero_row = [&](int64_t row) {
        if (rank == 0 && tt == 0) unlabelled_row(o, row);
        if (!o.out) return;
        T* out = static_cast<T*>(o.out) + row * o.out_stride;
        const RowShape<T> s(o.out_words ? base + row * sc.stride : out, n, rank, shift);
        uint4* dst = reinterpret_cast<uint4*>(out + s.head) + s.first;
        for (int j = tt - s.skew; j < s.count; j += TEAM)
            if (j >= 0) store_streaming(dst + j, uint4{0, 0, 0, 0});
        const int e = edges ? s.edge(n, tt) : -1;
        if (e >= 0) out[e] = from_f32<T>(0.f);
    };

    if (ctas > 1) {
        if (threadIdx.x == 0) {
            any_lost = false;
            for (int i = 0; i < 2; ++i) {
                bytes_init(&come[i]);
                bytes_expect(&come[i], ctas * W * (int)sizeof(SoftState));
            }
            bytes_fence_init();
        }
        cluster_sync();
    }
    bool lost = false;  // a wait for the other CTAs has run out
    let_next_start();
    auto label_of = [&](int row) { return row >= 0 ? sc.labels[row] : (int64_t)-1; };
    const int row0 = team < sc.rows ? (int)team : -1;
    RowAhead cur = start(row0, label_of(row0)), next;
    wait_for_previous();
    // the team's rows: the current one, the next (its words copied while the current one's turn
    // lasts), the one after (its label known), and the one after that
    const uint32_t items = rl.list ? (uint32_t)rl.head->labelled : 0u;
    auto item = [&](uint32_t i) { return i >= items ? -1 : rl.list[i]; };
    uint32_t at = team;
    int row1 = item(at), row2 = item(at + teams), row3;
    int64_t label1 = label_of(row1);
    const float inv_count = p.weights ? 0.f : rl.head->inv_count;
    // rows without a label are spread between the labelled ones, from the last team to the first
    // (those have had fewer labelled ones)
    uint32_t zeros = (uint32_t)rl.rows - items, zero_at = teams - 1 - team;
    int64_t due = (int64_t)items * team / teams;
    PolicyTerms terms;
    for (int turn = 0; cur.row >= 0; row1 = row2, row2 = row3, at += teams, cur = next) {
        const int r = cur.row;
        const int64_t label2 = label_of(row2);
        row3 = item(at + 2 * teams);
        float at_label = NAN, old = 0.f, adv = 0.f, base_lp = 0.f, weight = 0.f;
        if (cur.label >= 0) {
            if (lane == 0 && cur.label < n) at_label = to_f32(base[r * sc.stride + cur.label]);
            old = p.old_logp[r];
            adv = p.advantages[r];
            if (p.ref_logp) base_lp = p.ref_logp[r];
            weight = p.weights ? p.weights[r] : inv_count;
        }
        const T* x = base + r * sc.stride;
        const RowShape<T> s(x, n, rank, shift);
        const int rounds = s.rounds(TEAM), j0 = tt - s.skew;  // rounds: the same in all threads, as is what depends on it
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
                        if (!s.has(j0 + k * TEAM)) w[k] = word_closed(T());
                        top = fmaxf(top, word_max(w[k], T()));
                    }
            }
        }
        next = start(row1, label1);
        label1 = label2;
        if (cur.label < 0) {
            zero_row(r);
            continue;
        }
        for (due += zeros; items > 0 && due >= items && zero_at < zeros; due -= items, zero_at += teams) zero_row(rl.list[rl.rows - 1 - zero_at]);

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
            for (int j = j0; j < s.count; j += K * TEAM) {
#pragma unroll
                for (int k = 0; k < K; ++k) w[k] = s.has(j + k * TEAM) ? src[j + k * TEAM] : word_closed(T());
                add_words<T, K>(st, w, a);
            }
            st = soft_warp(st, a);
        }
        // Every warp has the label's score before it lets the others go on, who may write the gradient
        // over it.
        at_label = __shfl_sync(~0u, at_label, 0);
        if (TEAM != 32) {
            // Two sets of places in turn: a CTA that writes to one again has been through the
            // meeting in between, for which every thread had read the first.
            SoftState* slot = part[turn & 1];
            if (ctas == 1) {
                if (lane == 0) slot[warp] = st;
                __syncthreads();
            } else {
                // Not a barrier of the cluster: that would wait for the last row's gradient to be written.
                uint64_t* bar = &come[turn & 1];
                if (lane < ctas) send_remote(&slot[rank * W + warp], bar, lane, st);
                if (!lost) {
                    if (!bytes_wait(bar, turn >> 1 & 1)) lost = any_lost = true;
                    else if (threadIdx.x == 0) bytes_expect(bar, ctas * W * (int)sizeof(SoftState));  // for the row after next
                }
            }
            ++turn;
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
            st.s = lost ? NAN : warp_add(t);
        }

        const SoftRef ref(st.m, a);
        const LogP logp = log_p(ref, at_label, st.s, sc.t, sc.inv_t);
        const float lp = logp.value();
        const PolicyRow q = policy_row(p, logp, old, adv, base_lp, weight);
        if (rank == 0 && tt == 0) {
            o.logp[r] = lp;
            *reinterpret_cast<float2*>(o.norm + 2 * r) = {st.m, st.s};
            o.coef[r] = q.coef;
            if (o.status)
                o.status[r] = norm_status(st) | (cur.label >= n ? ISO_ROW_BAD_LABEL : 0u) | (lost ? ISO_ROW_TIMEOUT : 0u);
            terms.v[0].add(q.pg);
            terms.v[1].add(q.kl);
            terms.v[2].add(q.cut);
        }
        if (!o.out) continue;

        const float g = q.coef * p.grad_scale * sc.inv_t;
        const RowGrad<T> grad{g, __fdividef(-g, st.s), ref};
        if (!LONG && o.out_words) {
            uint4* dst = reinterpret_cast<uint4*>(out + s.head) + s.first + j0;
            auto give = [&](auto far) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k < rounds) {
                        const uint4 d = grad.template word<decltype(far)::value>(w[k]);
                        if (s.has(j0 + k * TEAM)) store_streaming(dst + k * TEAM, d);
                    }
            };
            ref.far ? give(std::true_type()) : give(std::false_type());
        } else {
            // read again: the row is long, or its gradient lies at other places within 16 bytes
            const uint4* src = reinterpret_cast<const uint4*>(x + s.head) + s.first;
            T* dst = out + s.head + (int64_t)s.first * N;
            for (int j = j0; j < s.count; j += TEAM) {
                if (j < 0) continue;
                const uint4 word = src[j];
                store_word(dst + (int64_t)j * N, ref.far ? grad.template word<true>(word) : grad.template word<false>(word), o.out_words);
            }
        }
        const int e = edges ? s.edge(n, tt) : -1;
        if (e >= 0) out[e] = grad.one(cur.edge, e == cur.label);
        // the label's score again, by the thread that has just written its word
        if (s.owner(cur.label, TEAM) == tt) out[cur.label] = grad.one(at_label, true);
    }
    copy_async_wait_all();
    for (; zero_at < zeros; zero_at += teams) zero_row(rl.list[rl.rows - 1 - zero_at]);

    // the teams' sums, by the last CTA, in the teams' order
    if (rank == 0 && tt == 0) p.of_team[team] = terms;
    const bool last = last_to_come(&p.head->ticket, gridDim.x);
    // This CTA's shared memory outlives what it has stopped waiting for: the others send all they have
    // to, then end or come here (who has ended counts as here); the last of it is on its way by then.
    if (ctas > 1 && any_lost) {
        cluster_sync();
        __nanosleep(100000);
    }
    if (!last) return;
    Sum* const total = reinterpret_cast<Sum*>(part);
    if (warp < 3) {
        Sum v;
        for (uint32_t i = lane; i < teams; i += 32) {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(&p.of_team[i].v[warp]));
            Sum q;
            q.hi = f.x;
            q.lo = f.y;
            v.add(q);
        }
        v = warp_sum(v);
        if (lane == 0) total[warp] = v;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) p.stats[i] = total[i].value();
        // the KL term's product rounds once
        *p.loss = p.kl_coef != 0.f ? fmaf(p.kl_coef, total[1].value(), total[0].value()) : total[0].value();
    }
}

// A team's labelled rows in turn (see RowList).
struct TeamRows {
    RowList rl;
    const int64_t* labels;
    int64_t rows, teams, at, items, upcoming;
    bool begun, listed;
    __device__ __forceinline__ TeamRows(const ScoreRows& sc, const RowList& list, int64_t team, int64_t step)
        : rl(list), labels(sc.labels), rows(sc.rows), teams(step), at(team), items(0), upcoming(-1), begun(false), listed(false) {}
    // The next row, or -1 when there are none left.
    __device__ __forceinline__ int64_t next() {
        if (!begun) {
            begun = true;
            if (at < rows && labels[at] >= 0) return at;
        }
        if (!rl.list) return -1;
        if (!listed) {
            wait_for_previous();
            listed = true;
            items = rl.head->labelled;
            upcoming = at < items ? rl.list[at] : -1;
        }
        const int64_t r = upcoming;
        at += teams;
        upcoming = at < items ? rl.list[at] : -1;
        return r;
    }
};

// Log-probabilities alone: a stream of the rows' words through a ring in shared memory, D groups of
// U words a thread in flight across the ends of rows, a running (maximum, sum) a thread, and one
// meeting of the CTA (or of a cluster's CTAs) a row, after which all warps but the first go on.
// Short rows are a warp's each.  Bound by HBM: 3,072 labelled rows of 65,536 bf16 (403 MB) in 63 us,
// 6.4 TB/s; by registers alone (a row held as by the policy loss) it was 89 us, the meetings being in
// the way of the loads.  U D = 16 words a thread and 3 CTAs keep 192 KB an SM in flight.
template <class T, int NT, int TEAM, int U, int D>
__global__ void __launch_bounds__(NT, 3)
score_stream_kernel(ScoreRows sc, RowOuts o, RowList rl, unsigned* zero_ticket) {
    constexpr int W = NT / 32;
    extern __shared__ uint4 ring[];
    __shared__ SoftState part[2][TEAM == 32 ? 1 : 8 * W];
    const int ctas = TEAM == 32 ? 1 : (int)cluster_size(), rank = TEAM == 32 ? 0 : (int)cluster_rank();
    const int shift = 31 - __clz(ctas);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tt = TEAM == 32 ? lane : threadIdx.x;
    const int64_t teams = TEAM == 32 ? (int64_t)gridDim.x * W : gridDim.x >> shift;
    const int64_t team = TEAM == 32 ? (int64_t)blockIdx.x * W + warp : blockIdx.x >> shift;
    uint4* mine = ring + (TEAM == 32 ? warp * 32 * U * D : 0) + tt;
    const float a = sc.a;
    const int n = sc.n;
    const bool edges = rank == 0 && tt < 32;
    const T* const base = static_cast<const T*>(sc.x);
    if (ctas > 1) cluster_started();
    let_next_start();
    if (zero_ticket && blockIdx.x == 0 && threadIdx.x == 0) *zero_ticket = 0u;

    // what is copied next: group `at` of row `row`
    TeamRows ahead(sc, rl, team, teams);
    int64_t row = 0;
    int at = 0, groups = 0, count = 0, skew = 0;
    const uint4* src = nullptr;
    auto copy_group = [&](int slot) {
        if (at == groups && row >= 0) {
            row = ahead.next();
            if (row >= 0) {
                const T* x = base + row * sc.stride;
                const RowShape<T> s(x, n, rank, shift);
                src = reinterpret_cast<const uint4*>(x + s.head) + s.first;
                count = s.count;
                skew = s.skew;
                at = 0;
                groups = max(1, s.rounds(TEAM * U));
            }
        }
        if (at < groups && row >= 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = tt - skew + (at * U + u) * TEAM;
                if ((unsigned)j < (unsigned)count) copy_async(mine + (slot * U + u) * TEAM, src + j);
            }
            ++at;
        }
        copy_async_commit();
    };
#pragma unroll
    for (int d = 0; d < D; ++d) copy_group(d);
    __syncwarp();
    if (ctas > 1) cluster_wait_started();

    TeamRows here(sc, rl, team, teams);
    int slot = 0, turn = 0;
    for (int64_t r = here.next(); r >= 0; r = here.next()) {
        const T* x = base + r * sc.stride;
        const RowShape<T> s(x, n, rank, shift);
        int64_t label = 0;
        float at_label = 0.f, edge = -INFINITY;
        if (edges) {
            label = sc.labels[r];
            at_label = label < n ? to_f32(x[label]) : NAN;
            const int e = s.edge(n, lane);
            if (e >= 0) edge = to_f32(x[e]);
        }
        SoftState st = soft_empty();
        const int end = max(1, s.rounds(TEAM * U));
        for (int g = 0; g < end; ++g) {
            copy_async_wait<D - 1>();
            uint4 w[U];
            float m = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = s.has(tt - s.skew + (g * U + u) * TEAM) ? mine[(slot * U + u) * TEAM] : word_closed(T());
                m = fmaxf(m, word_max(w[u], T()));  // (read, before the place is copied to again)
            }
            copy_group(slot);
            slot = slot + 1 == D ? 0 : slot + 1;
            add_words<T, U>(st, w, a, m);
        }
        if (edges) {
            soft_raise(st, edge, a);
            st.s += SoftRef(st.m, a).exp(edge);
        }
        st = soft_warp(st, a);
        if (TEAM != 32) {
            SoftState* place = part[turn++ & 1];  // as in policy_rows_kernel
            if (ctas == 1) {
                if (lane == 0) place[warp] = st;
                __syncthreads();
            } else {
                if (lane == 0) store_remote(&place[rank * W + warp], 0, st);
                __syncwarp();
                cluster_sync();
            }
            if (!edges) continue;
            st = soft_empty();
            for (int i = lane; i < ctas * W; i += 32) {
                const SoftState q = place[i];
                soft_raise(st, q.m, a);
                st.s += q.s * SoftRef(st.m, a).factor(q.m);
            }
            st = soft_warp(st, a);
        }
        if (lane == 0) {
            const LogP lp = log_p(SoftRef(st.m, a), at_label, st.s, sc.t, sc.inv_t);
            o.logp[r] = lp.value();
            if (o.rest) o.rest[r] = lp.rest();
            *reinterpret_cast<float2*>(o.norm + 2 * r) = {st.m, st.s};
            if (o.coef) o.coef[r] = 0.f;
            if (o.status) o.status[r] = norm_status(st) | (label >= n ? ISO_ROW_BAD_LABEL : 0u);
        }
    }
    copy_async_wait_all();
    // the rows without a label
    const int64_t thread = (int64_t)blockIdx.x * NT + threadIdx.x, threads = (int64_t)gridDim.x * NT;
    if (rl.list)  // (which next() has waited for)
        for (int64_t j = thread; j < rl.rows - rl.head->labelled; j += threads) unlabelled_row(o, rl.list[rl.rows - 1 - j]);
    if (rank == 0 && tt == 0 && team < sc.rows && sc.labels[team] < 0) unlabelled_row(o, team);
    __syncwarp();
    if (ctas > 1) cluster_sync();  // the first CTA's shared memory outlives the others' writes
}

// The pairs' mean loss, by a warp, in a fixed order.
__device__ __forceinline__ void sum_pairs(const float* each, int64_t pairs, float* loss) {
    const int lane = threadIdx.x & 31;
    Sum v;
    for (int64_t q = lane; q < pairs; q += 32) v.add(__ldcg(each + q));
    v = warp_sum(v);
    if (lane == 0) *loss = v.value() / (float)pairs;
}

// out = g (onehot - p) with g from the rows' coefficients: a CTA (or, of a short row, a warp) takes
// K words a thread of one row, from the last row to the first (the forward has read them in order,
// so that the last ones are in L2).  One unit a CTA and no loop: the loads of six CTAs an SM overlap
// the stores of others.  Bound by HBM: of a batch of 92 MB twice the size takes 25.7 us more for 184 MB
// more, 7.2 TB/s, beside 6 us of start and end; 8 words a thread 3% slower, 2 words 9%.
template <class T, int NT, int TEAM, int K, bool PAIRS>
__global__ void __launch_bounds__(NT, K == 4 ? 6 : 3)
score_backward_kernel(ScoreRows sc, const float* norm, const float* coef, float grad_scale,
                      const float* grad_scale_dev, int changed_only, RowOuts o, PairSum pairs) {
    constexpr int N = Word<T>::N;
    wait_for_previous();
    if (PAIRS && blockIdx.x == gridDim.x - 1) {  // a column of CTAs of its own
        if ((blockIdx.y | blockIdx.z) == 0 && threadIdx.x < 32) sum_pairs(pairs.each, pairs.pairs, pairs.loss);
        return;
    }
    if (grad_scale_dev) {
        const float g = *grad_scale_dev;
        if (changed_only && g == 1.f) return;
        grad_scale *= g;
    }
    const int n = sc.n, part = blockIdx.x, tt = threadIdx.x & (TEAM - 1);
    const int64_t r = sc.rows - 1 - ((blockIdx.z * (int64_t)gridDim.y + blockIdx.y) * (NT / TEAM) + threadIdx.x / TEAM);
    if (r < 0) return;
    const T* x = static_cast<const T*>(sc.x) + r * sc.stride;
    T* out = static_cast<T*>(o.out) + r * o.out_stride;
    const int64_t label = sc.labels[r];
    if (label < 0) {
        const RowShape<T> s(o.out_words ? x : out, n, part, 0, TEAM * K);
        T* dst = out + s.head + (int64_t)s.first * N;
        const int e = part == 0 && tt < 32 ? s.edge(n, tt) : -1, j = tt - s.skew;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (s.has(j + k * TEAM)) store_streaming(dst + (int64_t)(j + k * TEAM) * N, uint4{0, 0, 0, 0});
        if (e >= 0) out[e] = from_f32<T>(0.f);
        return;
    }
    const RowShape<T> s(x, n, part, 0, TEAM * K);
    const uint4* src = reinterpret_cast<const uint4*>(x + s.head) + s.first;
    T* dst = out + s.head + (int64_t)s.first * N;
    const int e = part == 0 && tt < 32 ? s.edge(n, tt) : -1, j = tt - s.skew;
    uint4 w[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (s.has(j + k * TEAM)) w[k] = load_streaming(src + j + k * TEAM);
    const float edge = e >= 0 ? to_f32(x[e]) : 0.f;
    const bool owner = s.owner(label, TEAM) == tt;
    const float at_label = owner ? to_f32(x[label]) : 0.f;
    const float2 ms = *reinterpret_cast<const float2*>(norm + 2 * r);
    const float g = label < n ? coef[r] * grad_scale * sc.inv_t : NAN;  // (no log-probability, no gradient)
    const RowGrad<T> grad{g, __fdividef(-g, ms.y), SoftRef(ms.x, sc.a)};
    auto give = [&](auto far) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (s.has(j + k * TEAM))
                store_word(dst + (int64_t)(j + k * TEAM) * N, grad.template word<decltype(far)::value>(w[k]), o.out_words);
    };
    grad.ref.far ? give(std::true_type()) : give(std::false_type());
    if (e >= 0) out[e] = grad.one(edge, e == label);
    if (owner) out[label] = grad.one(at_label, true);
}

// The list of the rows behind the first `skip` (see RowList), its counts, 1 / (number of all labelled
// rows), and a zeroed ticket; with list == NULL the counts alone.  One CTA, or one cluster of which each CTA has a stretch of the rows, so that nothing has
// to be zeroed first.  Bound by latency: 3.5 us for 8,192 rows.
__global__ void __launch_bounds__(1024)
row_list_kernel(const int64_t* __restrict__ labels, int64_t rows, int64_t skip, ListHead* __restrict__ head,
                int32_t* __restrict__ list) {
    __shared__ int of_cta[8], of_warp[2][32], skipped[32];
    const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
    if (ctas > 1) cluster_started();
    let_next_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t behind = rows - skip, share = (behind + ctas - 1) / ctas;
    const int64_t first = skip + min(behind, rank * share), end = min(rows, first + share);
    int c = 0;
    if (rank == 0)
        for (int64_t r = threadIdx.x; r < skip; r += 1024) c += labels[r] >= 0 ? 1 : 0;
    c = __reduce_add_sync(~0u, c);
    if (lane == 0) skipped[warp] = c;
    c = 0;
    bool mine_has = false;  // of the stretch's first 1,024 rows
    for (int64_t r = first + threadIdx.x; r < end; r += 1024) {
        const bool has = labels[r] >= 0;
        if (r == first + threadIdx.x) mine_has = has;
        c += has ? 1 : 0;
    }
    c = __reduce_add_sync(~0u, c);
    if (lane == 0) of_warp[0][warp] = c;
    __syncthreads();
    c = __reduce_add_sync(~0u, of_warp[0][lane]);
    if (ctas > 1) cluster_wait_started();
    if (warp == 0 && lane < ctas) store_remote(&of_cta[rank], lane, c);
    __syncwarp();
    cluster_sync();
    int run = 0, labelled = 0;  // labelled rows before this CTA's; of all
    for (int q = 0; q < ctas; ++q) {
        if (q < rank) run += of_cta[q];
        labelled += of_cta[q];
    }
    if (rank == 0 && warp == 0) {
        const int all = labelled + __reduce_add_sync(~0u, skipped[lane]);
        if (lane == 0) {
            head->ticket = 0u;
            head->labelled = labelled;
            head->inv_count = all > 0 ? 1.f / (float)all : 0.f;
        }
    }
    if (!list) return;
    int turn = 1;
    for (int64_t from = first; from < end; from += 1024, turn ^= 1) {
        const int64_t r = from + threadIdx.x;
        const bool has = from == first ? mine_has : r < end && labels[r] >= 0;
        const unsigned all = __ballot_sync(~0u, has);
        if (lane == 0) of_warp[turn][warp] = __popc(all);
        __syncthreads();  // (of_warp's other half is written after the next one)
        const int mine = of_warp[turn][lane];
        const int before = __reduce_add_sync(~0u, lane < warp ? mine : 0) + __popc(all & ((1u << lane) - 1u));
        if (has) list[run + before] = (int32_t)r;
        else if (r < end) list[behind - 1 - (r - skip - (run + before))] = (int32_t)r;
        run += __reduce_add_sync(~0u, mine);
    }
}

// No rows: the losses of none.
__global__ void zero_kernel(float* a, int na, float* b, int nb) {
    if ((int)threadIdx.x < na) a[threadIdx.x] = 0.f;
    if ((int)threadIdx.x < nb) b[threadIdx.x] = 0.f;
}

// CTAs an SM of the kernel below: one wave of them, since each looks through all offsets (4,096 pairs of
// single tokens 43 us, with as many CTAs as pairs up to 1,024 47; without looking 43).
constexpr int kPairCtas = 3;

// Whether pair q's own offsets are in order and within the rows; o: its three offsets.
__device__ __forceinline__ bool pair_in_order(const int64_t* offsets, int64_t q, int64_t rows, int64_t (&o)[3]) {
    for (int i = 0; i < 3; ++i) o[i] = offsets[2 * q + i];
    return o[0] >= 0 && o[1] >= o[0] && o[2] >= o[1] && o[2] <= rows;
}

// One CTA per pair, half of it for each of the two sequences: their sums, the pair's loss and the
// coefficient of every labelled token.  Each row's coefficient has one writer: a pair out of order
// writes none, and where some pair is, one that starts before the end of an earlier pair in order
// counts as out of order too (in order throughout, pairs share no rows; every CTA looks through all
// offsets, before the log-probabilities are there, and at most once more).  Bound by latency: 3.2 us
// after the log-probabilities' end for 16 pairs of 300 tokens (in float64, and adding up the loss
// itself, it was 12.5).
__global__ void __launch_bounds__(512, kPairCtas)
preference_pairs_kernel(PreferenceArgs p, const int64_t* __restrict__ labels, int64_t rows,
                        const float* logp, float* coef) {
    constexpr int W = 16;
    __shared__ Sum sh[3][W];
    __shared__ float sh_coef[2];
    __shared__ int sh_end[W];
    let_next_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, side = threadIdx.x >> 8, tt = threadIdx.x & 255;
    bool off = threadIdx.x == 0 && (p.offsets[0] < 0 || p.offsets[2 * p.pairs] > rows);
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < 2 * p.pairs; i += 512) off |= p.offsets[i] > p.offsets[i + 1];
    const bool disorder = __syncthreads_or(off);
    bool waited = false;
    int64_t looked = 0;  // pairs that `end` has taken in: this thread's part of the largest end of one in order
    int end = 0;
    for (int64_t q = blockIdx.x; q < p.pairs; q += gridDim.x) {
        int64_t o[3];
        bool bad = !pair_in_order(p.offsets, q, rows, o);
        if (disorder) {
            for (int64_t e = looked + threadIdx.x; e < q; e += 512) {
                int64_t before[3];
                if (pair_in_order(p.offsets, e, rows, before) && before[0] < before[2]) end = max(end, (int)before[2]);
            }
            looked = q;
            const int most = __reduce_max_sync(~0u, end);
            if (lane == 0) sh_end[warp] = most;
            __syncthreads();  // (read before the next one, written behind it)
            bad |= o[0] < o[2] && o[0] < __reduce_max_sync(~0u, sh_end[lane & (W - 1)]);
        }
        const bool ok = !bad;
        const int64_t a = side ? o[1] : o[0], b = side ? o[2] : o[1];
        if (!waited) wait_for_previous();
        waited = true;
        Sum seq, gain, count;
        if (ok)
            for (int64_t r = a + tt; r < b; r += 256)
                if (labels[r] >= 0) {
                    const float lp = logp[r];
                    seq.add(lp);
                    gain.add(p.ref_logp ? lp - p.ref_logp[r] : lp);
                    gain.add(p.rest[r]);
                    count.add(1.f);
                }
        seq = warp_sum(seq);
        gain = warp_sum(gain);
        count = warp_sum(count);
        if (lane == 0) {
            sh[0][warp] = seq;
            sh[1][warp] = gain;
            sh[2][warp] = count;
        }
        __syncthreads();
        if (warp == 0) {
            // lanes 0 and 8 end up with the two sequences' sums
            float total[3];
            for (int v = 0; v < 3; ++v) {
                Sum s = sh[v][lane & (W - 1)];
#pragma unroll
                for (int o = W / 4; o > 0; o >>= 1) {
                    Sum other;
                    other.hi = __shfl_down_sync(~0u, s.hi, o);
                    other.lo = __shfl_down_sync(~0u, s.lo, o);
                    s.add(other);
                }
                total[v] = s.value();
            }
            const float own_share = p.average ? 1.f / fmaxf(total[2], 1.f) : 1.f;
            if (lane == 0 || lane == W / 2) p.seq_logp[2 * q + (lane != 0)] = bad ? NAN : total[0] * own_share;
            const float gained = total[1] * own_share;
            const float h = gained - __shfl_down_sync(~0u, gained, W / 2);
            const float share[2] = {own_share, __shfl_down_sync(~0u, own_share, W / 2)};
            const float beta = p.beta, z = beta * h;  // lane 0's are meant from here on
            float each, slope;  // the pair's loss and its derivative in h
            if (p.kind == ISO_PREFERENCE_SIGMOID) {
                const float e = expf(-fabsf(z)), over = log1pf(e);
                const float up = (z >= 0.f ? 1.f : e) / (1.f + e);  // sigmoid(z)
                const float down = (z >= 0.f ? e : 1.f) / (1.f + e);  // sigmoid(-z)
                // (a side without weight has no part, also where z is infinite)
                each = over + (z < 0.f && p.smooth < 1.f ? (1.f - p.smooth) * -z : 0.f) + (z > 0.f && p.smooth > 0.f ? p.smooth * z : 0.f);
                slope = beta * (p.smooth * up - (1.f - p.smooth) * down);
            } else if (p.kind == ISO_PREFERENCE_HINGE) {
                each = z < 1.f ? 1.f - z : z >= 1.f ? 0.f : z;
                slope = z < 1.f ? -beta : 0.f;
            } else {
                const float d = h - 0.5f / beta;
                each = d * d;
                slope = 2.f * d;
            }
            if (bad) each = slope = NAN;
            if (lane == 0) {
                p.margins[q] = bad ? NAN : z;
                p.each[q] = each;
                if (p.pair_status) p.pair_status[q] = bad ? ISO_ROW_BAD_SHAPE : 0u;
                sh_coef[0] = slope * share[0] / (float)p.pairs;
                sh_coef[1] = -slope * share[1] / (float)p.pairs;
            }
        }
        __syncthreads();
        if (ok)
            for (int64_t r = a + tt; r < b; r += 256)
                if (labels[r] >= 0) coef[r] = sh_coef[side];
    }
    if (!waited) wait_for_previous();
    // with a gradient to follow, its kernel adds up the loss, and need not wait for that here
    if (p.sum_later || !last_to_come(p.ticket, gridDim.x)) return;
    if (warp == 0) sum_pairs(p.each, p.pairs, p.loss);
}

// Rows that log-probabilities alone need no list for.
constexpr int64_t kNoList = 64;

// The words that a reader's threads have to hold, of the rows of a call (see RowShape): their number,
// with the threads before the first one's.
template <class T>
struct RowWords {
    int64_t words, before;
    explicit RowWords(const ScoreRows& s) {
        words = (s.n + Word<T>::N - 1) / Word<T>::N;
        const bool aligned = reinterpret_cast<uintptr_t>(s.x) % 128 == 0 && (s.rows <= 1 || s.stride * sizeof(T) % 128 == 0);
        before = aligned ? 0 : 7;
    }
    int64_t share(int64_t readers) const { return ((words + before + readers - 1) / readers + 7) & ~int64_t(7); }
};

// The workspace: a head, the list of rows, what follows.
inline size_t list_bytes(int64_t rows) { return 256 + align256o((size_t)rows * 4); }
inline ListHead* list_head(void* ws) { return static_cast<ListHead*>(ws); }
inline int32_t* list_rows(void* ws) { return reinterpret_cast<int32_t*>(static_cast<char*>(ws) + 256); }
inline char* after_list(void* ws, int64_t rows) { return static_cast<char*>(ws) + list_bytes(rows); }

// With `teams` fewer than the rows: the list of those behind the teams' own.
cudaError_t make_list(const ScoreRows& s, void* ws, int64_t teams, RowList* rl, cudaStream_t st) {
    const bool list = s.rows > teams;
    *rl = RowList{list_head(ws), list ? list_rows(ws) : nullptr, list ? s.rows - teams : 0};
    const int ctas = s.rows > 1024 ? 8 : 1;
    ClusterLaunch l(ctas, 1024, 0, ctas, false, st);
    const cudaError_t e = l(row_list_kernel, s.labels, s.rows, list ? teams : 0, list_head(ws), list ? list_rows(ws) : nullptr);
    prof_mark(st, "row_list");
    return e;
}

template <class T, int NT, int TEAM, int K, bool LONG>
cudaError_t launch_policy(const ScoreRows& s, PolicyArgs p, const RowOuts& o, int ctas, void* ws, cudaStream_t st) {
    auto* kernel = policy_rows_kernel<T, NT, TEAM, K, LONG>;
    ClusterLaunch l(1, NT, LONG ? 0 : (size_t)NT * K * 16, ctas, true, st);
    static Held held;
    int fit = 0;
    cudaError_t e = clusters_held(kernel, l.c, ctas, held, &fit);
    if (e != cudaSuccess) return e;
    constexpr int per_cta = TEAM == 32 ? NT / 32 : 1;
    const int64_t grid = std::min<int64_t>({(s.rows + per_cta - 1) / per_cta, fit, kMaxTeams / per_cta});
    RowList rl;
    if ((e = make_list(s, ws, grid * per_cta, &rl, st)) != cudaSuccess) return e;
    p.head = list_head(ws);
    p.of_team = reinterpret_cast<PolicyTerms*>(after_list(ws, s.rows));
    l.c.gridDim = dim3((unsigned)(grid * ctas));
    e = l(kernel, s, p, o, rl);
    prof_mark(st, "policy_rows");
    return e;
}

// By a row's bytes: a warp holds up to 4 KB, a CTA of 128 or 256 threads 16, 32 or 64 KB, a pair of
// the latter 128 KB, and up to 8 CTAs of 512 threads 128 KB each; rows over 1 MB are read twice.
// Several small CTAs an SM are better than one (8,192 x 65,536 bf16: 321 us by pairs of 256 threads,
// 363 by one CTA of 512), but two wide ones better than four: 8,192 x 131,072 bf16 took 615 us on
// every GPU by pairs of 512 threads, and by fours of 256 between 588 and 705, as the chip's groups
// of SMs happened to lie.
template <class T>
cudaError_t run_policy(const ScoreRows& s, const PolicyArgs& p, const RowOuts& o, void* ws, cudaStream_t st) {
    const RowWords<T> w(s);
    if (w.share(1) <= 32 * 8) return launch_policy<T, 256, 32, 8, false>(s, p, o, 1, ws, st);
    if (w.share(8) > 512 * 16) return launch_policy<T, 256, 256, 8, true>(s, p, o, 8, ws, st);
    int ctas = w.share(1) <= 256 * 16 ? 1 : 2;
    while (w.share(ctas) > (ctas == 1 ? 256 : 512) * 16) ctas *= 2;
    // few rows: more CTAs for each, down to a word a thread
    while (ctas < 8 && s.rows * ctas < device_sms() && w.share(ctas) > 256) ctas *= 2;
    if (w.share(ctas) <= 128 * 8) return launch_policy<T, 128, 128, 8, false>(s, p, o, ctas, ws, st);
    if (w.share(ctas) <= 256 * 8) return launch_policy<T, 256, 256, 8, false>(s, p, o, ctas, ws, st);
    if (w.share(ctas) <= 256 * 16) return launch_policy<T, 256, 256, 16, false>(s, p, o, ctas, ws, st);
    return launch_policy<T, 512, 512, 16, false>(s, p, o, ctas, ws, st);
}

// Rows of up to 4 KB by warps; longer ones by as many CTAs a row (up to 8) as make the slowest
// team's share smallest: a row costs a team its groups and about one more for the meeting at its end.
template <class T>
cudaError_t run_logp(const ScoreRows& s, const RowOuts& o, void* ws, bool zero_ticket, cudaStream_t st) {
    constexpr int NT = 256, U = 4, D = 4;
    constexpr size_t shared = (size_t)NT * U * D * 16;
    const RowWords<T> w(s);
    const bool warps = w.share(1) <= 32 * 8;
    const int per_cta = warps ? NT / 32 : 1;
    auto* kernel = warps ? score_stream_kernel<T, NT, 32, U, D> : score_stream_kernel<T, NT, NT, U, D>;
    static Held held[2];
    int best = 1, best_fit = 1;
    double least = 0.0;
    for (int ctas = 1; ctas <= 8 && (ctas == 1 || (!warps && w.words >= (int64_t)ctas * NT)); ctas *= 2) {
        ClusterLaunch l(1, NT, shared, ctas, false, st);
        int fit = 0;
        const cudaError_t e = clusters_held(kernel, l.c, ctas, held[warps], &fit);
        if (e != cudaSuccess) return e;
        const int64_t groups = (w.share(ctas) + NT * U - 1) / (NT * U);
        const double cost = (double)((s.rows + fit - 1) / fit) * (double)(groups + 1);
        if (ctas == 1 || cost < 0.97 * least) {
            best = ctas;
            best_fit = fit;
            least = cost;
        }
    }
    const int64_t grid = std::min<int64_t>((s.rows + per_cta - 1) / per_cta, std::max<int64_t>(best_fit, kNoList));
    const bool list = s.rows > grid * per_cta;  // (never for up to kNoList rows)
    RowList rl{};
    if (list) {
        const cudaError_t e = make_list(s, ws, grid * per_cta, &rl, st);
        if (e != cudaSuccess) return e;
    }
    ClusterLaunch l(grid * best, NT, shared, best, list, st);
    const cudaError_t e = l(kernel, s, o, rl,
                            zero_ticket && !list ? &list_head(ws)->ticket : nullptr);
    prof_mark(st, "score_stream");
    return e;
}

// Whether the gradient's rows start at the same place within 16 bytes as the scores' rows.
inline int words_agree(const ScoreRows& s, const void* out, int64_t out_stride, int dtype) {
    const int64_t size = dtype == ISO_F32 ? 4 : 2;
    const uintptr_t off = reinterpret_cast<uintptr_t>(s.x) ^ reinterpret_cast<uintptr_t>(out);
    return (off & 15u) == 0 && (s.rows <= 1 || ((s.stride - out_stride) * size) % 16 == 0);
}

}  // namespace

size_t token_logp_workspace(int64_t rows) { return rows <= kNoList ? 0 : list_bytes(rows); }

cudaError_t token_logp(int dtype, const ScoreRows& s, float* logp, float* norm, void* ws,
                       uint32_t* row_status, cudaStream_t st) {
    const RowOuts o{logp, norm, nullptr, nullptr, nullptr, 0, 0, row_status};
    return by_type(dtype, [&](auto t) { return run_logp<decltype(t)>(s, o, ws, false, st); });
}

namespace {
cudaError_t run_backward(int dtype, const ScoreRows& s, const float* norm, const float* coef, float grad_scale,
                         const float* grad_scale_dev, int changed_only, void* out, int64_t out_stride,
                         const PairSum& pairs, cudaStream_t st) {
    const RowOuts o{nullptr, nullptr, nullptr, nullptr, out, out_stride, words_agree(s, out, out_stride, dtype), nullptr};
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int NT = 256, K = 4;
        RowWords<T> w(s);
        if (!o.out_words) w.before = 7;  // zeros are shared out as the gradient's own rows lie
        const bool warps = w.share(1) <= 32 * 8;
        const int64_t parts = warps ? 1 : (w.share(1) + NT * K - 1) / (NT * K);  // at most 2^19
        const int64_t row_ctas = warps ? (s.rows + NT / 32 - 1) / (NT / 32) : s.rows;
        const bool sum = pairs.loss != nullptr;
        ClusterLaunch l(parts + (sum ? 1 : 0), NT, 0, 1, true, st);
        l.c.gridDim.y = (unsigned)std::min<int64_t>(row_ctas, 65535);
        l.c.gridDim.z = (unsigned)((row_ctas + 65534) / 65535);
        auto* kernel = warps ? (sum ? score_backward_kernel<T, NT, 32, 8, true> : score_backward_kernel<T, NT, 32, 8, false>)
                             : (sum ? score_backward_kernel<T, NT, NT, K, true> : score_backward_kernel<T, NT, NT, K, false>);
        const cudaError_t e = l(kernel, s, norm, coef, grad_scale, grad_scale_dev, changed_only, o, pairs);
        prof_mark(st, "score_backward");
        return e;
    });
}
}  // namespace

cudaError_t token_logp_backward(int dtype, const ScoreRows& s, const float* norm, const float* coef,
                                float grad_scale, const float* grad_scale_dev, int changed_only,
                                void* out, int64_t out_stride, cudaStream_t st) {
    if (s.rows == 0) return cudaSuccess;
    return run_backward(dtype, s, norm, coef, grad_scale, grad_scale_dev, changed_only, out, out_stride, PairSum{}, st);
}

size_t policy_workspace(int64_t rows) {
    return list_bytes(rows) + align256o((size_t)std::min<int64_t>((rows + 7) / 8 * 8, kMaxTeams) * sizeof(PolicyTerms));
}

cudaError_t policy_loss(int dtype, const ScoreRows& s, const PolicyArgs& p, void* out,
                        int64_t out_stride, void* ws, uint32_t* row_status, cudaStream_t st) {
    if (s.rows == 0) {
        zero_kernel<<<1, 32, 0, st>>>(p.loss, 1, p.stats, 3);
        return cudaGetLastError();
    }
    const RowOuts o{p.logp, p.norm, p.coef, nullptr, out, out_stride, out ? words_agree(s, out, out_stride, dtype) : 0, row_status};
    return by_type(dtype, [&](auto t) { return run_policy<decltype(t)>(s, p, o, ws, st); });
}

size_t preference_workspace(int64_t rows, int64_t pairs) {
    return list_bytes(rows) + align256o((size_t)rows * 4) + align256o((size_t)pairs * 4);
}

cudaError_t preference_loss(int dtype, const ScoreRows& s, PreferenceArgs p, float* logp,
                            float* norm, float* coef, float grad_scale, void* out,
                            int64_t out_stride, void* ws, uint32_t* row_status, cudaStream_t st) {
    p.ticket = &list_head(ws)->ticket;
    p.rest = reinterpret_cast<float*>(after_list(ws, s.rows));
    p.each = p.rest + align256o((size_t)s.rows * 4) / 4;
    cudaError_t e = cudaSuccess;
    if (s.rows > 0) {
        const RowOuts o{logp, norm, coef, p.rest, nullptr, 0, 0, row_status};
        e = by_type(dtype, [&](auto t) { return run_logp<decltype(t)>(s, o, ws, true, st); });
    } else {  // pairs of empty sequences: the ticket's zero
        zero_kernel<<<1, 32, 0, st>>>(reinterpret_cast<float*>(p.ticket), 1, nullptr, 0);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    if (p.pairs == 0) {
        zero_kernel<<<1, 32, 0, st>>>(p.loss, 1, nullptr, 0);
        e = cudaGetLastError();
    } else {
        p.sum_later = out && s.rows > 0;
        ClusterLaunch l(std::min<int64_t>(p.pairs, kPairCtas * device_sms()), 512, 0, 1, true, st);
        e = l(preference_pairs_kernel, p, s.labels, s.rows, logp, coef);
        prof_mark(st, "preference_pairs");
    }
    if (e != cudaSuccess || !out || s.rows == 0) return e;
    return run_backward(dtype, s, norm, coef, grad_scale, nullptr, 0, out, out_stride,
                        PairSum{p.each, p.pairs, p.pairs > 0 ? p.loss : nullptr}, st);
}

}  // namespace isodev
