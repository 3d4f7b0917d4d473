// Device helpers of the training objectives: element types, the running
// maximum and sum of a softmax, and their reductions.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace isodev {

constexpr float kLog2e = 1.4426950408889634f;

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

// A softmax's running state: the largest score m seen so far and the sum s of
// exp2((x - m) a), a = log2(e) / temperature.  Differences are formed before
// the scaling, so that the type's lowest value minus itself is 0 and not an
// overflow.  A state that has seen nothing, or only -inf, is (-inf, 0); a NaN
// or +inf among the scores leaves NaN in s.
struct SoftState {
    float m, s;
};

__device__ __forceinline__ SoftState soft_empty() { return {-INFINITY, 0.f}; }

// The reference that scores are taken against: with only -inf seen, 0 (every
// -inf then adds 0, and a NaN still shows).
__device__ __forceinline__ float soft_ref(float m) { return m == -INFINITY ? 0.f : m; }

// Raises the state's maximum to at least mc.
__device__ __forceinline__ void soft_raise(SoftState& st, float mc, float a) {
    if (mc > st.m) {
        st.s *= ex2((st.m - mc) * a);
        st.m = mc;
    }
}

__device__ __forceinline__ SoftState soft_merge(SoftState p, SoftState q, float a) {
    const float m = fmaxf(p.m, q.m), r = soft_ref(m);
    // each product rounded by itself: the same bits whichever of the two comes first
    return {m, __fadd_rn(__fmul_rn(p.s, ex2((p.m - r) * a)), __fmul_rn(q.s, ex2((q.m - r) * a)))};
}

__device__ __forceinline__ SoftState soft_warp(SoftState st, float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        SoftState q{__shfl_xor_sync(~0u, st.m, o), __shfl_xor_sync(~0u, st.s, o)};
        st = soft_merge(st, q, a);
    }
    return st;
}

// Over a CTA of NT threads; `sh` holds NT / 32 states.  Every thread gets the
// result; ends with the CTA in step, so that `sh` may be used again.
template <int NT>
__device__ __forceinline__ SoftState soft_cta(SoftState st, float a, SoftState* sh) {
    st = soft_warp(st, a);
    if (NT == 32) return st;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sh[warp] = st;
    __syncthreads();
    st = lane < NT / 32 ? sh[lane] : soft_empty();
    st = soft_warp(st, a);
    __syncthreads();
    return st;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Sum over a CTA of NT threads, in a fixed order; valid in thread 0.
template <int NT>
__device__ __forceinline__ double cta_sum(double v, double* sh) {
    v = warp_sum(v);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    v = lane < NT / 32 ? sh[lane] : 0.0;
    if (warp == 0) v = warp_sum(v);
    __syncthreads();
    return v;
}

}  // namespace isodev
