// The states of beams put, in place, where their continuations are.
//
//   row (item, b) of each state becomes what row (item, parents[item, b]) was
//
// A thread holds one word (up to 16 bytes) of every beam that moves, in registers, before it stores
// any: no second buffer, and each row that moves is written, each row that is taken over read, once.
// Bound by HBM: 16 caches of 64 rows of 2 MB, 6 of 8 beams moved from 4, in 387 us (2.6 GB, 6.8 TB/s, the copy
// rate); 32 caches of 4 rows, 184 MB, in 30 us (6.1 TB/s).  With a barrier a unit and one word of each beam a
// thread at a time 487 and 47 us, with all word widths in one kernel 485 and 41.
#include "choice_internal.h"
#include "obj_device.cuh"
#include "obj_launch.h"

namespace isodev {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveStates = 64;  // states of a launch, a power of two

// A state of one launch: words of `width` bytes, `tail` single bytes behind each run's words.
struct MoveState {
    char* base;
    int64_t row_stride, run_stride;
    int64_t words;          // of a run
    uint32_t units_of_run;  // one at least
    uint32_t first_unit;    // the launch's units before this state's
    uint32_t runs;
    int32_t tail, width;
};
struct MoveArgs {
    MoveState state[kMoveStates];
    const int32_t* parents;
    uint32_t units;
    int32_t count, beams;
};

template <int W> struct MoveWord;
template <> struct MoveWord<16> { using type = uint4; };
template <> struct MoveWord<8> { using type = uint2; };
template <> struct MoveWord<4> { using type = uint32_t; };
template <> struct MoveWord<2> { using type = uint16_t; };
template <> struct MoveWord<1> { using type = uint8_t; };

// What a warp has to know of its item's beams that move: byte offsets of their rows.
struct Move {
    int64_t to, from;
};

// M words of each of up to B beams that move, `apart` bytes apart; the first `mine` of them are there.
template <int B, int M, int W>
__device__ __forceinline__ void move_words(char* at, int apart, int mine, int moved, const Move* moves) {
    using V = typename MoveWord<W>::type;
    V v[B][M];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        if (i < moved) {
            const char* const p = at + moves[i].from;
#pragma unroll
            for (int m = 0; m < M; ++m)
                if (m < mine) v[i][m] = *reinterpret_cast<const V*>(p + m * apart);
        }
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
        if (i < moved) {
            char* const p = at + moves[i].to;
#pragma unroll
            for (int m = 0; m < M; ++m)
                if (m < mine) *reinterpret_cast<V*>(p + m * apart) = v[i][m];
        }
    }
}

// A unit is 32 M words of a run, of all beams of an item; warps take them in turn.  WIDE: all states' words
// are of 16 bytes (with the other widths beside it the kernel needs twice the registers).
template <int B, int M, bool WIDE>
__global__ void __launch_bounds__(kMoveThreads)
beam_reorder_kernel(const __grid_constant__ MoveArgs a) {
    __shared__ Move sh_moves[kMoveThreads / 32][B];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Move* const moves = sh_moves[warp];
    for (uint32_t unit = blockIdx.x * (kMoveThreads / 32) + warp; unit < a.units; unit += gridDim.x * (kMoveThreads / 32)) {
        int s = 0;
        for (int step = kMoveStates / 2; step > 0; step >>= 1)
            if (s + step < a.count && unit >= a.state[s + step].first_unit) s += step;
        const MoveState& st = a.state[s];
        const uint32_t u = unit - st.first_unit, line = u / st.units_of_run, block = u - line * st.units_of_run;
        const uint32_t item = line / st.runs, run = line - item * st.runs;
        const int p = lane < a.beams ? a.parents[(int64_t)item * a.beams + lane] : lane;
        const bool moving = p != lane && p >= 0 && p < a.beams;
        const unsigned all = __ballot_sync(~0u, moving);
        const int moved = __popc(all);
        if (moving) moves[__popc(all & ((1u << lane) - 1u))] = {lane * st.row_stride, p * st.row_stride};
        __syncwarp();
        char* const base = st.base + (int64_t)item * a.beams * st.row_stride + run * st.run_stride;
        const int64_t first = (int64_t)block * (32 * M), whole = st.words;
        const int64_t word = first + lane;
        if (moved > 0 && word < whole) {
            const int mine = (int)min((int64_t)M, (whole - word + 31) / 32), apart = 32 * st.width;
            char* const at = base + word * st.width;
            if constexpr (WIDE) {
                move_words<B, M, 16>(at, apart, mine, moved, moves);
            } else switch (st.width) {
                case 16:
                    if constexpr (B <= 16) move_words<B, M, 16>(at, apart, mine, moved, moves);
                    break;
                case 8: move_words<B, M, 8>(at, apart, mine, moved, moves); break;
                case 4: move_words<B, M, 4>(at, apart, mine, moved, moves); break;
                case 2: move_words<B, M, 2>(at, apart, mine, moved, moves); break;
                default: move_words<B, M, 1>(at, apart, mine, moved, moves);
            }
        }
        // the bytes behind the last word, with the last unit
        if (moved > 0 && block == st.units_of_run - 1 && lane < st.tail)
            move_words<B, 1, 1>(base + whole * st.width + lane, 0, 1, moved, moves);
        __syncwarp();
    }
}

// The largest power of two up to `most` that divides the address and the strides.
int common_width(const iso_state& s, int64_t rows, unsigned most) {
    uint64_t v = reinterpret_cast<uintptr_t>(s.base) | most;
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
    // The states of 16-byte words first, those of others in launches of their own.
    for (int wide = 1; wide >= 0; --wide) {
        // words of a thread at a time, 16 of all beams (8 beams: one each took 485 us of the largest case and not 387)
        const int words = wide && beams <= 8 ? 2 : 1;
        a.count = 0;
        a.units = 0;
        auto go = [&]() {
            if (a.count == 0) return cudaSuccess;
            constexpr int kWarps = kMoveThreads / 32;
            const unsigned grid = std::min<uint32_t>((a.units + kWarps - 1) / kWarps, 152 * 32);
            auto kernel = beam_reorder_kernel<32, 1, false>;
            if (beams <= 4)
                kernel = wide ? beam_reorder_kernel<4, 2, true> : beam_reorder_kernel<4, 1, false>;
            else if (beams <= 8)
                kernel = wide ? beam_reorder_kernel<8, 2, true> : beam_reorder_kernel<8, 1, false>;
            else if (beams <= 16)
                kernel = wide ? beam_reorder_kernel<16, 1, true> : beam_reorder_kernel<16, 1, false>;
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
            const int width = common_width(s, batch * beams, beams <= 16 ? 16 : 8);  // (a thread holds 32 of 8 bytes)
            if ((width == 16) != (wide == 1)) continue;
            const int64_t whole = s.run_bytes / width, of_run = std::max<int64_t>(1, (whole + 32 * words - 1) / (32 * words));
            // (states that are really there are far below this)
            if (of_run > 0x7fffffff / s.runs || of_run * s.runs > 0x7fffffff / batch) return cudaErrorInvalidValue;
            const uint32_t units = (uint32_t)(of_run * s.runs * batch);
            if (a.count == kMoveStates || a.units + units > 0x7fffffffu) {
                const cudaError_t e = go();
                if (e != cudaSuccess) return e;
            }
            MoveState& m = a.state[a.count++];
            m.base = static_cast<char*>(s.base);
            m.row_stride = s.row_stride;
            m.run_stride = s.run_stride;
            m.runs = (uint32_t)s.runs;
            m.width = width;
            m.tail = (int32_t)(s.run_bytes % width);
            m.words = whole;
            m.units_of_run = (uint32_t)of_run;
            m.first_unit = a.units;
            a.units += units;
        }
        const cudaError_t e = go();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace isodev
