// Rows of a router's scores: the lanes that hold a token's, their softmax, and the launch by experts.
#pragma once

#include "obj_device.cuh"
#include "obj_launch.h"

#include <type_traits>

namespace isodev {

// Order-preserving key of a score; 0 for what is never chosen (-inf and NaN), equal for both zeros.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float choice_score(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

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

}  // namespace isodev
