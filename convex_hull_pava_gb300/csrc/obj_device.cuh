// Device helpers of the training objectives: words of scores, the softmax's reference and
// running state, and their reductions.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

namespace isodev {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^v by the hardware's instruction: relative error about 2^-22, results under
// 2^-126 become 0 (a probability that small adds nothing to a float32 sum).
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 two(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t two(float2 v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(two(a)), "l"(two(b)), "l"(two(c)));
    return two(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(two(a)), "l"(two(b)));
    return two(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(two(a)), "l"(two(b)));
    return two(d);
}

// A word: 16 bytes of scores.
template <class T>
struct Word {
    static constexpr int N = 16 / (int)sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4& w, float2 (&v)[2], float) {
    v[0] = {__uint_as_float(w.x), __uint_as_float(w.y)};
    v[1] = {__uint_as_float(w.z), __uint_as_float(w.w)};
}
__device__ __forceinline__ void unpack(const uint4& w, float2 (&v)[4], __nv_bfloat16) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = {__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u)};
}
__device__ __forceinline__ void unpack(const uint4& w, float2 (&v)[4], __half) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[2], float) {
    return {__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y)};
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[4], __nv_bfloat16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return {u[0], u[1], u[2], u[3]};
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[4], __half) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return {u[0], u[1], u[2], u[3]};
}

// A word of closed entries.
__device__ __forceinline__ uint4 word_closed(float) { return {0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u}; }
__device__ __forceinline__ uint4 word_closed(__nv_bfloat16) { return {0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u}; }
__device__ __forceinline__ uint4 word_closed(__half) { return {0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u}; }

// The largest score of a word (NaN are passed over, as by fmaxf).
__device__ __forceinline__ float word_max(const uint4& w, float) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                 fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
template <class H2>
__device__ __forceinline__ H2 word_max2(const uint4& w) {
    const H2* h = reinterpret_cast<const H2*>(&w);
    return __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
}
__device__ __forceinline__ float word_max(const uint4& w, __nv_bfloat16) {
    const __nv_bfloat162 m = word_max2<__nv_bfloat162>(w);
    return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float word_max(const uint4& w, __half) {
    const __half2 m = word_max2<__half2>(w);
    return fmaxf(__low2float(m), __high2float(m));
}

// Loads and stores of what this call touches once.
__device__ __forceinline__ void store_streaming(void* p, const uint4& w) {
    asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}
__device__ __forceinline__ uint4 load_streaming(const void* p) {
    uint4 w;
    asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
    return w;
}

// 16 bytes from global memory into shared memory, behind the caller's back.
__device__ __forceinline__ void copy_async(void* shared, const void* global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(shared)), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void copy_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Every thread of the cluster arrives and waits: shared-memory writes before it, in any of its
// CTAs, are seen after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Another CTA's shared memory may be written to once that CTA runs: all CTAs say so as they start,
// and wait for the others' word before they write.
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_started() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// What scores are taken against in a softmax, a = log2(e) / temperature: exp2(x a - c), with c the
// float32 product of the largest score m and a.  The one fused operation rounds the difference
// only, and c's own rounding, r = m a - c, is the same in every term, in the sum and in the label's:
// it cancels in a probability, and log_p puts it right to first order.  |r| is at most 2^-24 |c|, so
// that this holds for |c| < 2^12 (a score of 2,839 at a temperature of 1; the second order is then
// under 4e-9).  Beyond, "far", the difference is formed first, exp2((x - m) a): no such rest, one more
// rounding, and no product that could leave float32's range (a row of a mask's large negative number,
// or of the type's lowest value, is a softmax as any other).  With nothing but -inf seen, m counts as
// 0: every -inf then adds 0, and a NaN still shows.
struct SoftRef {
    float m, c, a;
    bool far;
    static __device__ __forceinline__ bool is_far(float c) { return !(fabsf(c) < 4096.f); }
    __device__ __forceinline__ SoftRef(float top, float scale) {
        m = top == -INFINITY ? 0.f : top;
        a = scale;
        c = __fmul_rn(m, a);
        far = is_far(c);
    }
    // The exponent of a score.
    __device__ __forceinline__ float of(float x) const { return far ? (x - m) * a : fmaf(x, a, -c); }
    __device__ __forceinline__ float exp(float x) const { return ex2(of(x)); }
    // What turns a sum that was taken against the score `top` into one against this.  Near terms are
    // against c, far ones against m a itself: where one is near and the other far, r counts.
    __device__ __forceinline__ float factor(float top) const {
        if (top == -INFINITY) return 0.f;
        const float of_top = __fmul_rn(top, a);
        const bool top_far = is_far(of_top);
        if (far == top_far) return ex2(far ? (top - m) * a : of_top - c);
        return ex2(far ? fmaf(-m, a, of_top) : fmaf(top, a, -c));
    }
};

// A log-probability as the unevaluated sum of two floats, hi the larger.  About 3e-8 off beside the
// sum's own error, where one float32 of its size would be up to 5e-7: a policy's ratio and a
// preference's margin are differences of such numbers.
struct LogP {
    float hi, lo;
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
    // what value() leaves out
    __device__ __forceinline__ float rest() const {
        const float v = value();
        return isfinite(v) ? (hi - v) + lo : 0.f;
    }
    // this minus a float, which is near it
    __device__ __forceinline__ float minus(float v) const { return isfinite(hi) ? (hi - v) + lo : hi - v; }
};

// log p of a score x, given the sum of all against `ref`:
//   (x - m) / T - log sum',   sum' = sum 2^(c - m a): c's rounding put right (to first order: it is
//   under 2^-24 of c),   log sum' = k high + (k low + log f),  sum' = f 2^k,  1/2 <= f / sqrt(2) < 1,
// with high + low = log 2 and so few bits in high that k high is exact.  The exponentials are low by
// 5.1e-8 of themselves in the mean (ex2 against 64 bits, 2^22 arguments in each of -2..-26's pairs of
// octaves; not the largest score's, which is 1), and so is the rest of their sum; hundreds of tokens'
// log-probabilities add up in a margin.  (A mean: a row of a few equal scores, whose exponentials are
// exact, is put off by up to that much.)
__device__ __forceinline__ LogP log_p(const SoftRef& ref, float x, float sum, float temperature, float inv_t) {
    constexpr float kHigh = 2839.f / 4096.f, kLow = (float)(0.693147180559945309417 - 2839.0 / 4096.0);
    // x - m = d + d_low, d / T = q + q_low
    const float d = __fsub_rn(x, ref.m), back = __fsub_rn(d, x);
    const float d_low = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(ref.m, back));
    const float q = d * inv_t, q_low = (fmaf(-q, temperature, d) + d_low) * inv_t;
    const float total = ref.far ? sum : fmaf(sum, -kLn2 * fmaf(ref.m, ref.a, -ref.c), sum);
    // a sum is at least about 1 and at most n; anything else (0, NaN, infinity) is for logf alone
    const bool usual = total > 0.5f && total < 1e30f;
    const int k = usual ? (__float_as_int(total) - 0x3f3504f3) >> 23 : 0;  // 0x3f3504f3: 1 / sqrt(2)
    const float f = usual ? __int_as_float(__float_as_int(total) - (k << 23)) : total;
    const float high = (float)k * kHigh, low = fmaf((float)k, kLow, logf(f)) + 5.1e-8f * (1.f - __fdividef(1.f, total));
    // q - high exactly, as hi + err
    const float hi = __fsub_rn(q, high), b = __fsub_rn(hi, q);
    const float err = __fsub_rn(__fsub_rn(q, __fsub_rn(hi, b)), __fadd_rn(high, b));
    LogP lp{hi, err + q_low - low};
    if (!usual) lp = {q - low, 0.f};
    return lp;
}

// A softmax's running state: the largest score m seen so far and the sum s of the exponentials
// against it.  A state that has seen nothing, or only -inf, is (-inf, 0); a NaN or +inf among the
// scores leaves NaN in s.
struct alignas(8) SoftState {
    float m, s;
};

__device__ __forceinline__ SoftState soft_empty() { return {-INFINITY, 0.f}; }

// Raises the state's maximum to at least `top`.
__device__ __forceinline__ void soft_raise(SoftState& st, float top, float a) {
    if (top > st.m) {
        st.s *= SoftRef(top, a).factor(st.m);
        st.m = top;
    }
}

// The exponentials of a word's scores, in pairs; FAR is ref.far.
template <class T, bool FAR>
__device__ __forceinline__ void word_exp(const uint4& w, const SoftRef& ref, float2 (&v)[Word<T>::N / 2]) {
    unpack(w, v, T());
    const float2 a2{ref.a, ref.a};
#pragma unroll
    for (int i = 0; i < Word<T>::N / 2; ++i) {
        v[i] = FAR ? mul2(add2(v[i], {-ref.m, -ref.m}), a2) : fma2(v[i], a2, {-ref.c, -ref.c});
        v[i] = {ex2(v[i].x), ex2(v[i].y)};
    }
}

// Over the lanes of a warp (or the given ones, which all call with the same), in one instruction;
// NaN are passed over.
__device__ __forceinline__ float warp_max(float v, unsigned lanes = ~0u) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(lanes));
    return r;
}

// Takes U words into a state whose scores' maximum is `top`.
template <class T, int U>
__device__ __forceinline__ void add_words(SoftState& st, const uint4 (&w)[U], float a, float top) {
    soft_raise(st, top, a);
    const SoftRef ref(st.m, a);
    float2 sum{0.f, 0.f};
    auto add = [&](auto far) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 v[Word<T>::N / 2];
            word_exp<T, decltype(far)::value>(w[u], ref, v);
#pragma unroll
            for (int i = 0; i < Word<T>::N / 2; ++i) sum = add2(sum, v[i]);
        }
    };
    ref.far ? add(std::true_type()) : add(std::false_type());
    st.s += sum.x + sum.y;
}
template <class T, int U>
__device__ __forceinline__ void add_words(SoftState& st, const uint4 (&w)[U], float a) {
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, word_max(w[u], T()));
    add_words<T, U>(st, w, a, top);
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Over a warp: the maximum first, then one rescaling of each lane's sum.  Every lane gets the
// same bits.
__device__ __forceinline__ SoftState soft_warp(SoftState st, float a) {
    const float m = warp_max(st.m);
    return {m, warp_add(st.s * SoftRef(m, a).factor(st.m))};
}

// Writes a state to the same place of another CTA of the cluster.
__device__ __forceinline__ void store_remote(SoftState* place, int cta, SoftState st) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(place)), "r"(cta));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(st.m), "f"(st.s) : "memory");
}

__device__ __forceinline__ void store_remote(int* place, int cta, int v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(place)), "r"(cta));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ void store_remote(float* place, int cta, float v) {
    store_remote(reinterpret_cast<int*>(place), cta, __float_as_int(v));
}

// Barriers in shared memory that count bytes: what the CTAs of a cluster send one another without
// waiting for their stores to global memory, as a barrier of the whole cluster would.
__device__ __forceinline__ void bytes_init(uint64_t* bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"((uint32_t)__cvta_generic_to_shared(bar)) : "memory");
}
__device__ __forceinline__ void bytes_fence_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
// The current phase ends when `bytes` have come.
__device__ __forceinline__ void bytes_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"((uint32_t)__cvta_generic_to_shared(bar)), "r"(bytes) : "memory");
}
// Waits for the end of the phase of that parity; false when it has not come within two seconds.
__device__ __forceinline__ bool bytes_wait(uint64_t* bar, uint32_t parity) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(bar);
    uint64_t since = 0;
    for (uint32_t i = 1;; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(at), "r"(parity) : "memory");
        if (done) return true;
        if ((i & 255u) == 0u) {
            uint64_t now;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
            if (since == 0) since = now;
            if (now - since > 2000000000ull) return false;
        }
    }
}
// Sends a state to the same place of another CTA, and its 8 bytes to that CTA's barrier.
__device__ __forceinline__ void send_remote(SoftState* place, uint64_t* bar, int cta, SoftState st) {
    uint32_t at, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(place)), "r"(cta));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(b) : "r"((uint32_t)__cvta_generic_to_shared(bar)), "r"(cta));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
                 ::"r"(at), "r"(__float_as_uint(st.m)), "r"(__float_as_uint(st.s)), "r"(b) : "memory");
}

// A float32 sum that keeps what its additions round off: about 48 bits, without 64-bit arithmetic
// (of which this GPU has little).
struct alignas(8) Sum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
        hi = s;
    }
    __device__ __forceinline__ void add(const Sum& q) {
        add(q.hi);
        lo += q.lo;
    }
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

// Over a warp; valid in lane 0.
__device__ __forceinline__ Sum warp_sum(Sum v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sum q;
        q.hi = __shfl_down_sync(~0u, v.hi, o);
        q.lo = __shfl_down_sync(~0u, v.lo, o);
        v.add(q);
    }
    return v;
}

// The kernel that follows in the stream may be launched (it waits for this one's results where it
// needs them), and such a wait.  It runs while those are written: it takes them through pointers
// that are not const __restrict__ (which would allow loads that assume that nobody writes, also in
// front of the wait).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Whether this CTA is the last of `ctas` to come here; the others' writes to global memory before
// it are seen by the last one's threads.  Called by all threads of a CTA.
__device__ __forceinline__ bool last_to_come(unsigned* ticket, unsigned ctas) {
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(ticket, 1u) == ctas - 1;
    __syncthreads();
    __threadfence();
    return last;
}

}  // namespace isodev
