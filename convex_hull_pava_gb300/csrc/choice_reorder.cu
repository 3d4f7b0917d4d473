// The states of beams put, in place, where their continuations are.
//
//   row (item, b) of each state becomes what row (item, parents[item, b]) was
//
// A thread holds one word (up to 16 bytes) of every beam that moves, in registers, before it stores
// any: no second buffer, and each row that moves is written, each row that is taken over read, once.
#include "choice_internal.h"
#include "obj_device.cuh"
#include "obj_launch.h"

namespace isodev {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveStates = 32;  // states of a launch

// A state of one launch: words of `width` bytes, `tail` single bytes behind each run's words.
struct MoveState {
    char* base;
    int64_t row_stride, run_stride;
    int64_t words, units_of_run;  // of a run, the tail's bytes counted as words
    int64_t first_unit;           // the launch's units before this state's
    int32_t runs, tail, width;
};
struct MoveArgs {
    MoveState state[kMoveStates];
    const int32_t* parents;
    int64_t units;
    int32_t count, beams;
};

template <int W> struct MoveWord;
template <> struct MoveWord<16> { using type = uint4; };
template <> struct MoveWord<8> { using type = uint2; };
template <> struct MoveWord<4> { using type = uint32_t; };
template <> struct MoveWord<2> { using type = uint16_t; };
template <> struct MoveWord<1> { using type = uint8_t; };

template <int B, int W>
__device__ __forceinline__ void move_words(char* at, int64_t row_stride, int moved, const int (&to)[B], const int (&from)[B]) {
    using V = typename MoveWord<W>::type;
    V v[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
        if (i < moved) v[i] = *reinterpret_cast<const V*>(at + from[i] * row_stride);
#pragma unroll
    for (int i = 0; i < B; ++i)
        if (i < moved) *reinterpret_cast<V*>(at + to[i] * row_stride) = v[i];
}

// A unit is kMoveThreads words of a run, of all beams of an item.
template <int B>
__global__ void __launch_bounds__(kMoveThreads)
beam_reorder_kernel(const __grid_constant__ MoveArgs a) {
    __shared__ int sh_to[32], sh_from[32], sh_moved;
    for (int64_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        int s = 0;
        for (int i = 1; i < a.count; ++i)
            if (unit >= a.state[i].first_unit) s = i;
        const MoveState& st = a.state[s];
        int64_t u = unit - st.first_unit;
        const int64_t block = u % st.units_of_run;
        u /= st.units_of_run;
        const int run = (int)(u % st.runs);
        const int64_t item = u / st.runs;
        __syncthreads();
        if (threadIdx.x < 32) {
            const int b = threadIdx.x;
            const int p = b < a.beams ? a.parents[item * a.beams + b] : b;
            const bool moves = p != b && p >= 0 && p < a.beams;
            const unsigned all = __ballot_sync(~0u, moves);
            if (moves) {
                const int i = __popc(all & ((1u << b) - 1u));
                sh_to[i] = b;
                sh_from[i] = p;
            }
            if (b == 0) sh_moved = __popc(all);
        }
        __syncthreads();
        const int moved = sh_moved;
        const int64_t word = block * kMoveThreads + threadIdx.x;
        if (moved == 0 || word >= st.words) continue;
        int to[B], from[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            to[i] = i < moved ? sh_to[i] : 0;
            from[i] = i < moved ? sh_from[i] : 0;
        }
        const int64_t whole = st.words - st.tail;
        char* at = st.base + item * a.beams * st.row_stride + run * st.run_stride;
        if (word < whole) {
            at += word * st.width;
            switch (st.width) {
                case 16: move_words<B, 16>(at, st.row_stride, moved, to, from); break;
                case 8: move_words<B, 8>(at, st.row_stride, moved, to, from); break;
                case 4: move_words<B, 4>(at, st.row_stride, moved, to, from); break;
                case 2: move_words<B, 2>(at, st.row_stride, moved, to, from); break;
                default: move_words<B, 1>(at, st.row_stride, moved, to, from);
            }
        } else {
            move_words<B, 1>(at + whole * st.width + (word - whole), st.row_stride, moved, to, from);
        }
    }
}

// The largest power of two up to 16 that divides the address and the strides.
int common_width(const iso_state& s, int64_t rows) {
    uint64_t v = reinterpret_cast<uintptr_t>(s.base) | 16u;
    if (rows > 1) v |= (uint64_t)s.row_stride;
    if (s.runs > 1) v |= (uint64_t)s.run_stride;
    return (int)(v & (~v + 1));
}

}  // namespace

cudaError_t beam_reorder(const iso_state* states, int64_t count, int64_t batch, int beams, const int32_t* parents,
                         cudaStream_t st) {
    if (beams == 1) return cudaSuccess;
    MoveArgs a;
    a.parents = parents;
    a.beams = beams;
    a.count = 0;
    a.units = 0;
    auto go = [&]() {
        if (a.count == 0) return cudaSuccess;
        const unsigned grid = (unsigned)std::min<int64_t>(a.units, 152 * 32);
        auto kernel = beams <= 4 ? beam_reorder_kernel<4> : beams <= 8 ? beam_reorder_kernel<8>
                    : beams <= 16 ? beam_reorder_kernel<16> : beam_reorder_kernel<32>;
        kernel<<<grid, kMoveThreads, 0, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        prof_mark(st, "beam_reorder");
        a.count = 0;
        a.units = 0;
        return e;
    };
    for (int64_t i = 0; i < count; ++i) {
        const iso_state& s = states[i];
        if (s.runs == 0 || s.run_bytes == 0) continue;
        MoveState& m = a.state[a.count++];
        m.base = static_cast<char*>(s.base);
        m.row_stride = s.row_stride;
        m.run_stride = s.run_stride;
        m.runs = (int32_t)s.runs;
        m.width = common_width(s, batch * beams);
        m.tail = (int32_t)(s.run_bytes % m.width);
        m.words = s.run_bytes / m.width + m.tail;
        m.units_of_run = (m.words + kMoveThreads - 1) / kMoveThreads;
        m.first_unit = a.units;
        a.units += (int64_t)m.units_of_run * m.runs * batch;
        if (a.count == kMoveStates) {
            const cudaError_t e = go();
            if (e != cudaSuccess) return e;
        }
    }
    return go();
}

}  // namespace isodev
