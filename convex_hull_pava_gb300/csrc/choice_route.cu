// A router's choice of experts by float32 scores, and the gradient of its gates.
#include "choice_route.cuh"

namespace isodev {

extern template cudaError_t route_rows<__nv_bfloat16>(const RouteArgs&, int64_t*, int32_t*, float*, cudaStream_t);
extern template cudaError_t route_rows<__half>(const RouteArgs&, int64_t*, int32_t*, float*, cudaStream_t);

namespace {

// Softmax without renormalisation: all elements have a gradient.  The gates' part of each is put together in
// shared memory, a warp's tokens beside one another; the next tokens' scores are on their way meanwhile.
// Bound by HBM: 131,072 x 256 float32 in 44.6 us (268 MB, 6.0 TB/s; a plain copy of them takes 41.2).
template <class T, int G, int EPL>
__global__ void __launch_bounds__(256)
route_dense_backward_kernel(const __grid_constant__ RouteArgs a, int whole, const int32_t* chosen, const float* gates, const float* grad_gates,
                            T* out, int64_t out_stride) {
    constexpr int W = 256 / 32, TPW = 32 / G;
    __shared__ __align__(16) float extra[W * TPW][G * EPL];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane & (G - 1), E = a.experts, k = a.top_k;
    const unsigned group = group_lanes<G>();
    float* const mine = extra[warp * TPW + lane / G];
    for (int e = gl; e < G * EPL; e += G) mine[e] = 0.f;
    __syncwarp();
    const int64_t step = (int64_t)gridDim.x * W * TPW;
    const T* const base = static_cast<const T*>(a.x);
    TokenRow<T, G, EPL> row;
    int slot = -1;
    float g = 0.f, gate = 0.f;
    bool on = false;
    auto fetch = [&](int64_t t) {
        on = t < a.tokens;
        slot = -1;
        if (!on) return;
        row.load(base + t * a.stride, gl, E, whole);
        if (gl < k) {
            slot = chosen[t * k + gl];
            gate = gates[t * k + gl];
            g = grad_gates[t * k + gl];
        }
    };
    int64_t first = ((int64_t)blockIdx.x * W + warp) * TPW;
    fetch(first + lane / G);
    for (; first < a.tokens; first += step) {
        const int64_t t = first + lane / G;
        float v[EPL], p[EPL];
        row.scores(v, on);
        const int at = slot;
        const bool has = at >= 0 && at < E, write = on;
        const float dot = group_add<G>(has ? gate * g : 0.f), put = a.scale * g;
        fetch(t + step);
        if (has) mine[at] = put;
        __syncwarp();
        const bool any = __ballot_sync(~0u, has) & group;
        const SoftState st = token_softmax<G, EPL>(v, p);
        const float inv = 1.f / st.s;
        TokenRow<T, G, EPL> d;
#pragma unroll
        for (int i = 0; i < EPL; ++i) d.v[i] = from_f32<T>(any ? p[i] * inv * (mine[row.expert(gl, i)] - dot) : 0.f);
        if (write) d.store(out + t * out_stride, gl, E, whole);
        __syncwarp();
        if (has) mine[at] = 0.f;
    }
}

// The others: the chosen alone have a gradient.  A warp has as many tokens at a time as its lanes have
// places (`places` lanes a token, a power of two); their rows, zero but for the chosen, lie in shared memory
// in the output's type and are stored from there, 16 bytes a lane.  The next tokens' choice is asked
// for one turn ahead, and (where the forward has not kept them) its scores as soon as that is there.  `chunk`: bytes of a store.
// Bound by HBM's writes: 131,072 x 256 float32 in 20.3 us (6.6 TB/s; zeroing them takes 19.4).  With the
// chosen's scores gathered from the rows 43 us, with float32 rows in shared memory and a token a group of
// lanes 53.
template <class T>
__global__ void __launch_bounds__(256)
route_sparse_backward_kernel(const __grid_constant__ RouteArgs a, int places, int tokens, int chunk, const int32_t* chosen, const float* gates,
                             const float* picked, const float* grad_gates, T* out, int64_t out_stride) {
    extern __shared__ __align__(16) char rows[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts, k = a.top_k;
    const int place = lane & (places - 1), tw = lane / places;
    const int pitch = (E * (int)sizeof(T) + 15) / 16 * 16;  // bytes of a row in shared memory
    char* const mine = rows + warp * tokens * pitch;
    for (int i = lane * 16; i < tokens * pitch; i += 512) *reinterpret_cast<uint4*>(mine + i) = uint4{0, 0, 0, 0};
    const T* const base = static_cast<const T*>(a.x);
    const bool sigmoid = a.score == ISO_ROUTE_SIGMOID;
    const int64_t step = (int64_t)gridDim.x * 8 * tokens;
    int slot = -1;
    float gate = 0.f, g = 0.f, x = 0.f;
    auto fetch = [&](int64_t first) {
        const int64_t t = first + tw;
        slot = -1;
        if (tw < tokens && place < k && t < a.tokens) {
            slot = chosen[t * k + place];
            gate = gates[t * k + place];
            g = grad_gates[t * k + place];
            if (picked) x = picked[t * k + place];
            if (slot < 0 || slot >= E) slot = -1;
        }
    };
    auto score = [&](int64_t first) {
        if (sigmoid && !picked && slot >= 0) x = to_f32(base[(first + tw) * a.stride + slot]);
    };
    int64_t first = ((int64_t)blockIdx.x * 8 + warp) * tokens;
    fetch(first);
    score(first);
    __syncwarp();
    for (; first < a.tokens; first += step) {
        const int at = slot;
        const float own = gate, of = g, own_x = x;
        fetch(first + step);
        float dot = at >= 0 ? own / a.scale * of : 0.f;  // (of one alone the gradient itself)
        for (int o = places / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
        float put = own * (a.renormalize ? __fsub_rn(of, dot) : of);
        if (sigmoid) put *= 1.f / (1.f + expf(own_x));  // 1 - s
        T* const row = reinterpret_cast<T*>(mine + tw * pitch);
        if (at >= 0) row[at] = from_f32<T>(put);
        // without probabilities nothing has a gradient
        unsigned bad = __ballot_sync(~0u, at >= 0 && own != own);
        if (sigmoid) bad = 0u;
        __syncwarp();
        const int live = (int)min((int64_t)tokens, a.tokens - first);
        const int chunks = E * (int)sizeof(T) / chunk;  // of a row
        if (chunk == 16) {
            for (int r = lane / chunks, c = lane % chunks; r < live;) {
                store_streaming(reinterpret_cast<char*>(out + (first + r) * out_stride) + c * 16,
                                *reinterpret_cast<const uint4*>(mine + r * pitch + c * 16));
                for (c += 32; c >= chunks; c -= chunks) ++r;
            }
        } else {
            for (int r = 0; r < live; ++r)
                for (int e = lane; e < E; e += 32)
                    out[(first + r) * out_stride + e] = reinterpret_cast<const T*>(mine + r * pitch)[e];
        }
        __syncwarp();
        if (bad) {
            for (int r = 0; r < live; ++r)
                if (bad >> (r * places) & (places == 32 ? ~0u : (1u << places) - 1u))
                    for (int e = lane; e < E; e += 32) out[(first + r) * out_stride + e] = from_f32<T>(NAN);
        }
        if (at >= 0) row[at] = from_f32<T>(0.f);
        score(first + step);
        __syncwarp();
    }
}

}  // namespace

cudaError_t route(int dtype, const RouteArgs& a, int64_t* counts, int32_t* chosen, float* gates, cudaStream_t st) {
    return by_type(dtype, [&](auto t) { return route_rows<decltype(t)>(a, counts, chosen, gates, st); });
}

cudaError_t route_backward(int dtype, const RouteArgs& a, const int32_t* chosen, const float* gates,
                           const float* picked, const float* grad_gates, void* out, int64_t out_stride, cudaStream_t st) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int N = Word<T>::N;
        T* const to = static_cast<T*>(out);
        if (a.score == ISO_ROUTE_SOFTMAX && !a.renormalize)
            return by_experts(a.experts, [&](auto g, auto epl) {
                constexpr int G = decltype(g)::value, EPL = decltype(epl)::value, CH = TokenRow<T, G, EPL>::CH;
                const int whole = chunks_fit(a.x, a.tokens, a.stride, a.experts, CH, sizeof(T)) &&
                                  chunks_fit(out, a.tokens, out_stride, a.experts, CH, sizeof(T));
                const int64_t grid = std::min<int64_t>((a.tokens + 256 / G - 1) / (256 / G), 152 * 4);
                route_dense_backward_kernel<T, G, EPL><<<(unsigned)grid, 256, 0, st>>>(a, whole, chosen, gates, grad_gates, to, out_stride);
                const cudaError_t e = cudaGetLastError();
                prof_mark(st, "route_backward");
                return e;
            });
        int places = 1;
        while (places < a.top_k) places *= 2;
        const int pitch = (a.experts * (int)sizeof(T) + 15) / 16 * 16;
        const int tokens = std::max(1, std::min(32 / places, 4096 / pitch));  // of a warp at a time: up to 4 KB
        const int chunk = chunks_fit(out, a.tokens, out_stride, a.experts, N, sizeof(T)) ? 16 : (int)sizeof(T);
        const int64_t grid = std::min<int64_t>((a.tokens + 8 * tokens - 1) / (8 * tokens), 152 * 24);  // (152 * 6: 22.3 us and not 20.6)
        route_sparse_backward_kernel<T><<<(unsigned)grid, 256, 8 * tokens * pitch, st>>>(a, places, tokens, chunk, chosen, gates, picked, grad_gates, to, out_stride);
        const cudaError_t e = cudaGetLastError();
        prof_mark(st, "route_backward");
        return e;
    });
}

}  // namespace isodev
