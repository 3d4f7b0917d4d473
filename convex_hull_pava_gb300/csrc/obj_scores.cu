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

#include <algorithm>

namespace isodev {

namespace {

constexpr int kRowThreads = 256;

inline __host__ __device__ size_t align256o(size_t x) { return (x + 255) & ~size_t(255); }

inline int row_grid(int64_t rows) { return (int)std::min<int64_t>(rows, 1 << 20); }

// One row's part of the policy loss, from its log-probability.
struct PolicyRow {
    float coef, pg, kl, cut;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& p, int64_t r, float logp) {
    const float w = p.weights ? p.weights[r] : *p.inv_count;
    const float adv = p.advantages[r];
    const float ratio = expf(logp - p.old_logp[r]);
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
        const float d = p.ref_logp[r] - logp, e = expm1f(d);
        q.kl = w * (e - d);
        q.coef -= p.kl_coef * w * e;
    }
    return q;
}

__device__ __forceinline__ uint32_t norm_status(SoftState st) {
    return isfinite(st.m) && isfinite(st.s) ? 0u : ISO_ROW_BAD_Y;
}

// What is asked of a row's scores.
enum class Ask { kLogp, kPolicy, kBackward };

// One CTA per row: a pass for the norm (kLogp, kPolicy) and a pass for the gradient.
template <class T, Ask ASK>
__global__ void __launch_bounds__(kRowThreads)
score_rows_kernel(ScoreRows sc, PolicyArgs p, float* __restrict__ logp, float* __restrict__ norm,
                  float* __restrict__ coef, float grad_scale, const float* grad_scale_dev,
                  int changed_only, T* __restrict__ out, int64_t out_stride,
                  uint32_t* __restrict__ row_status) {
    __shared__ SoftState sh[kRowThreads / 32];
    __shared__ float sh_coef;
    const float a = kLog2e * sc.inv_t;
    const int n = sc.n;
    if (ASK == Ask::kBackward && grad_scale_dev) {
        const float g = *grad_scale_dev;
        if (changed_only && g == 1.f) return;
        grad_scale *= g;
    }
    for (int64_t r = blockIdx.x; r < sc.rows; r += gridDim.x) {
        const T* __restrict__ x = static_cast<const T*>(sc.x) + r * sc.stride;
        const int64_t label = sc.labels[r];
        if (label < 0) {
            if (ASK != Ask::kBackward && threadIdx.x == 0) {
                logp[r] = 0.f;
                norm[2 * r] = 0.f;
                norm[2 * r + 1] = 1.f;
                if (coef) coef[r] = 0.f;
                if (row_status) row_status[r] = 0u;
                if (ASK == Ask::kPolicy)
                    for (int i = 0; i < 3; ++i) p.terms[i * sc.rows + r] = 0.f;
            }
            if (out)
                for (int j = threadIdx.x; j < n; j += kRowThreads) out[r * out_stride + j] = from_f32<T>(0.f);
            continue;
        }
        SoftState st;
        if (ASK != Ask::kBackward) {
            st = soft_empty();
            for (int j = threadIdx.x; j < n; j += kRowThreads) {
                const float v = to_f32(x[j]);
                soft_raise(st, v, a);
                st.s += ex2((v - soft_ref(st.m)) * a);
            }
            st = soft_cta<kRowThreads>(st, a, sh);
            if (threadIdx.x == 0) {
                const bool bad = label >= n;
                const float lp = bad ? NAN : (to_f32(x[label]) - st.m) * sc.inv_t - logf(st.s);
                logp[r] = lp;
                norm[2 * r] = st.m;
                norm[2 * r + 1] = st.s;
                if (row_status) row_status[r] = norm_status(st) | (bad ? ISO_ROW_BAD_LABEL : 0u);
                if (ASK == Ask::kPolicy) {
                    const PolicyRow q = policy_row(p, r, lp);
                    p.terms[r] = q.pg;
                    p.terms[sc.rows + r] = q.kl;
                    p.terms[2 * sc.rows + r] = q.cut;
                    coef[r] = q.coef;
                    sh_coef = q.coef;
                } else if (coef) {
                    coef[r] = 0.f;
                }
            }
            if (ASK == Ask::kLogp || !out) continue;
            __syncthreads();
        } else {
            st = {norm[2 * r], norm[2 * r + 1]};
        }
        const float g = (ASK == Ask::kBackward ? coef[r] : sh_coef) * grad_scale * sc.inv_t;
        const float h = -g / st.s;
        for (int j = threadIdx.x; j < n; j += kRowThreads) {
            float d = h * ex2((to_f32(x[j]) - st.m) * a);
            if (j == label) d += g;
            out[r * out_stride + j] = from_f32<T>(d);
        }
        __syncthreads();  // sh_coef is read before the next row writes it
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

template <class T, Ask ASK>
cudaError_t run_rows(const ScoreRows& s, const PolicyArgs& p, float* logp, float* norm, float* coef,
                     float grad_scale, const float* grad_scale_dev, int changed_only, void* out,
                     int64_t out_stride, uint32_t* row_status, cudaStream_t st) {
    if (s.rows == 0) return cudaSuccess;
    score_rows_kernel<T, ASK><<<row_grid(s.rows), kRowThreads, 0, st>>>(
        s, p, logp, norm, coef, grad_scale, grad_scale_dev, changed_only, static_cast<T*>(out),
        out_stride, row_status);
    return cudaGetLastError();
}

template <Ask ASK, class... A>
cudaError_t by_type(int dtype, A... args) {
    switch (dtype) {
        case ISO_F32: return run_rows<float, ASK>(args...);
        case ISO_BF16: return run_rows<__nv_bfloat16, ASK>(args...);
        default: return run_rows<__half, ASK>(args...);
    }
}

}  // namespace

cudaError_t token_logp(int dtype, const ScoreRows& s, float* logp, float* norm, float* zero_coef,
                       uint32_t* row_status, cudaStream_t st) {
    return by_type<Ask::kLogp>(dtype, s, PolicyArgs{}, logp, norm, zero_coef, 1.f,
                               (const float*)nullptr, 0, (void*)nullptr, (int64_t)0, row_status, st);
}

cudaError_t token_logp_backward(int dtype, const ScoreRows& s, const float* norm, const float* coef,
                                float grad_scale, const float* grad_scale_dev, int changed_only,
                                void* out, int64_t out_stride, cudaStream_t st) {
    return by_type<Ask::kBackward>(dtype, s, PolicyArgs{}, (float*)nullptr,
                                   const_cast<float*>(norm), const_cast<float*>(coef), grad_scale,
                                   grad_scale_dev, changed_only, out, out_stride,
                                   (uint32_t*)nullptr, st);
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
    e = by_type<Ask::kPolicy>(dtype, s, p, p.logp, p.norm, p.coef, p.grad_scale,
                              (const float*)nullptr, 0, out, out_stride, row_status, st);
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
