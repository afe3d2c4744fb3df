// reorder.cu -- states that follow their beams (spec_reorder_beams) and the
// rows of an accepted tree path (spec_commit_path), moved in place.
//
// Both are permutations with repetition of rows that are far longer than a
// vector.  A thread owns one column (the same vector of every row) and no
// two threads share one, so moving in place needs no barrier and no second
// buffer: it reads what moves before it writes.  Memory traffic bounds both:
// every row that moves is read once (a parent with several children once
// for all of them) and written once per child.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/specverify.h"

namespace sv {
namespace {

constexpr int kMoveThreads = 128;

struct States {
    char *at[SPEC_MAX_STATES];
};

struct MoveArgs {
    int64_t request_stride, row_stride, segment_stride, unit_bytes;  // bytes
    int segments, capacity, batch, rows, width;
    const int32_t *begin, *end;  // reorder: window; commit: begin = base
    const int32_t *map;          // [B][width]
    int32_t *out_lens;           // commit only
    int32_t *status;
};

// Copies global -> shared of one vector; types below 4 bytes have no
// asynchronous form.
template <class T>
__device__ __forceinline__ void stage(T *dst, const char *src)
{
    if constexpr (sizeof(T) == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(
                         static_cast<unsigned>(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
    } else if constexpr (sizeof(T) == 4 || sizeof(T) == 8) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(
                         static_cast<unsigned>(__cvta_generic_to_shared(dst))), "l"(src), "n"(sizeof(T)) : "memory");
    } else {
        *dst = *reinterpret_cast<const T *>(src);
    }
}

// The moves of request b, in shared memory: the distinct parents of the
// beams that move, and for each beam that moves its parent's slot.
struct BeamMoves {
    int nsrc, ndst;
    short src[SPEC_MAX_BEAMS], dst[SPEC_MAX_BEAMS], slot[SPEC_MAX_BEAMS];
};

// One warp builds the moves; false if a parent is malformed.
__device__ bool beam_moves(const int32_t *parents, int width, int beams, BeamMoves &mv)
{
    const int lane = threadIdx.x & 31;
    uint64_t used = 0, moving = 0;  // bit masks over beams
    bool ok = true;
    int par[2];
    for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        par[h] = j < width ? __ldg(parents + j) : -1;
        ok &= par[h] >= -1 && par[h] < beams;
    }
    if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    for (int h = 0; h < 2; ++h) {
        const bool mine = par[h] >= 0 && par[h] != lane + 32 * h;
        moving |= static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, mine)) << (32 * h);
        const uint64_t bit = mine ? uint64_t(1) << par[h] : 0;
        used |= static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(bit))) |
                static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(bit >> 32))) << 32;
    }
    for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        const uint64_t below = (uint64_t(1) << j) - 1;
        if (used >> j & 1) mv.src[__popcll(used & below)] = static_cast<short>(j);
        if (moving >> j & 1) {
            const int at = __popcll(moving & below);
            mv.dst[at] = static_cast<short>(j);
            mv.slot[at] = static_cast<short>(__popcll(used & ((uint64_t(1) << par[h]) - 1)));
        }
    }
    if (lane == 0) {
        mv.nsrc = __popcll(used);
        mv.ndst = __popcll(moving);
    }
    return true;
}

// Grid (x: columns, y: requests, z: states).  A thread stages its column
// of every distinct parent in its own words of shared memory, then writes
// the children.  Asynchronous copies keep all of a thread's reads in flight
// whatever the number of parents is, which registers could not (64 vectors).
// (Eight bf16 states, 4 requests x 8 beams, 8 heads, windows of 524 to 1048
// positions of 128: 111 us, 90 % of the copy bandwidth over the bytes that
// have to move.)
template <class T>
__global__ void __launch_bounds__(kMoveThreads)
    k_reorder_beams(const __grid_constant__ States st, const __grid_constant__ MoveArgs a)
{
    extern __shared__ __align__(16) unsigned char staged_raw[];
    T *mine = reinterpret_cast<T *>(staged_raw) + threadIdx.x;
    __shared__ BeamMoves mv;
    __shared__ int go;
    char *state = st.at[blockIdx.z];
    const bool first = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0;
    for (int b = blockIdx.y; b < a.batch; b += gridDim.y) {
        const int begin = a.begin ? __ldg(a.begin + b) : 0;
        const int end = a.end ? __ldg(a.end + b) : a.capacity;
        const bool fits = 0 <= begin && begin <= end && end <= a.capacity;
        __syncthreads();  // the last request's moves are read
        if (threadIdx.x < 32) {
            const bool ok = beam_moves(a.map + static_cast<int64_t>(b) * a.width, a.width, a.rows, mv);
            if (threadIdx.x == 0) go = ok ? 1 : 0;
        }
        __syncthreads();
        if (first && a.status && !(fits && go))
            atomicOr(a.status, (fits ? 0 : SPEC_STATUS_CAPACITY) | (go ? 0 : SPEC_STATUS_TREE));
        if (!fits || !go || mv.ndst == 0) continue;
        const int64_t per_seg = (static_cast<int64_t>(end) - begin) * a.unit_bytes / static_cast<int64_t>(sizeof(T));
        const int64_t columns = per_seg * a.segments;
        char *req = state + b * a.request_stride + begin * a.unit_bytes;
        for (int64_t c = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; c < columns;
             c += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
            const int64_t seg = c / per_seg;
            char *col = req + seg * a.segment_stride + (c - seg * per_seg) * static_cast<int64_t>(sizeof(T));
            for (int i = 0; i < mv.nsrc; ++i) stage<T>(mine + i * kMoveThreads, col + mv.src[i] * a.row_stride);
            asm volatile("cp.async.wait_all;\n" ::: "memory");
            for (int i = 0; i < mv.ndst; ++i)
                *reinterpret_cast<T *>(col + mv.dst[i] * a.row_stride) = mine[mv.slot[i] * kMoveThreads];
        }
    }
}

// Grid as above.  Path entries rise, so entry i's source lies at or after
// unit i: groups of entries move in order, each read before it is written.
// (32 requests, 60-node trees: 7 us under a profiler, a chain of three
// dependent reads; the rows' 6.7 MB would take 1.)
template <class T>
__global__ void __launch_bounds__(kMoveThreads)
    k_commit_path(const __grid_constant__ States st, const __grid_constant__ MoveArgs a)
{
    constexpr int kGroup = 8;
    __shared__ int nodes;  // entries before the first -1
    char *state = st.at[blockIdx.z];
    const bool first = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0;
    for (int b = blockIdx.y; b < a.batch; b += gridDim.y) {
        const int32_t *path = a.map + static_cast<int64_t>(b) * a.width;
        const int base = a.begin ? __ldg(a.begin + b) : 0;
        const bool fits = base >= 0 && static_cast<int64_t>(base) + a.rows <= a.capacity;
        __syncthreads();
        if (threadIdx.x == 0) nodes = a.width;
        __syncthreads();
        for (int i = threadIdx.x; i < a.width; i += kMoveThreads)
            if (__ldg(path + i) < 0) atomicMin(&nodes, i);
        __syncthreads();
        const int n = nodes;
        bool ok = true;
        for (int i = threadIdx.x; i < a.width; i += kMoveThreads) {
            const int v = __ldg(path + i);
            if (v < -1) ok = false;
            if (i < n) ok &= v < a.rows && (i == 0 || v > __ldg(path + i - 1));
        }
        ok = __syncthreads_and(ok);
        if (first) {
            if (a.out_lens) a.out_lens[b] = fits && ok ? base + n : base;
            if (a.status && !(fits && ok))
                atomicOr(a.status, (fits ? 0 : SPEC_STATUS_CAPACITY) | (ok ? 0 : SPEC_STATUS_TREE));
        }
        if (!fits || !ok || !state) continue;
        const int64_t per_unit = a.unit_bytes / static_cast<int64_t>(sizeof(T));
        const int64_t columns = per_unit * a.segments;
        char *req = state + b * a.request_stride + base * a.unit_bytes;
        for (int64_t c = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; c < columns;
             c += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
            const int64_t seg = c / per_unit;
            char *col = req + seg * a.segment_stride + (c - seg * per_unit) * static_cast<int64_t>(sizeof(T));
            for (int i0 = 0; i0 < n; i0 += kGroup) {
                T x[kGroup];
#pragma unroll
                for (int i = 0; i < kGroup; ++i)
                    if (i0 + i < n) x[i] = *reinterpret_cast<const T *>(col + __ldg(path + i0 + i) * a.unit_bytes);
#pragma unroll
                for (int i = 0; i < kGroup; ++i)
                    if (i0 + i < n && __ldg(path + i0 + i) != i0 + i)
                        *reinterpret_cast<T *>(col + (i0 + i) * a.unit_bytes) = x[i];
            }
        }
    }
}

// The widest vector that every address and length is a multiple of.
int vector_bytes(const States &st, int n, uint64_t strides)
{
    uint64_t bits = strides;
    for (int i = 0; i < n; ++i) bits |= reinterpret_cast<uintptr_t>(st.at[i]);
    return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}

// Blocks along x: eight waves of what fits the GPU at once (`per_sm` blocks a
// SM) over all requests and states, no more than the columns need: mostly one
// column a thread, and no tail.  (Eight beams, 773 MB moved: 122 us, 6.35 TB/s;
// 131 us with a third as many blocks, 143 us with exactly one wave.  64 beams,
// one block a SM: 190 us, 207 us with 16 times as many.)
unsigned column_blocks(int64_t columns, int64_t others, int per_sm)
{
    const int64_t want = std::max<int64_t>(1, 8 * 148 * per_sm / std::max<int64_t>(1, others));
    const int64_t need = std::max<int64_t>(1, (columns + kMoveThreads - 1) / kMoveThreads);
    return static_cast<unsigned>(std::min({need, want, int64_t(65535)}));
}

std::mutex g_move_mu;
bool g_move_attr[64][5];

template <class T>
int launch_beams(const States &st, int n, const MoveArgs &a, int slot, cudaStream_t stream)
{
    const size_t smem = sizeof(T) * kMoveThreads * static_cast<size_t>(a.rows);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ECUDA;
    {
        std::lock_guard<std::mutex> lock(g_move_mu);
        if (!g_move_attr[dev][slot]) {
            if (cudaFuncSetAttribute(k_reorder_beams<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(sizeof(T) * kMoveThreads * SPEC_MAX_BEAMS)) != cudaSuccess)
                return SPEC_ECUDA;
            g_move_attr[dev][slot] = true;
        }
    }
    const unsigned gy = static_cast<unsigned>(std::min(a.batch, 65535));
    const int64_t columns = a.capacity * (a.unit_bytes / static_cast<int64_t>(sizeof(T))) * a.segments;
    const int per_sm = static_cast<int>(std::min<size_t>(2048 / kMoveThreads, (227 * 1024) / (smem + 2048)));
    const dim3 grid(column_blocks(columns, static_cast<int64_t>(gy) * n, std::max(1, per_sm)), gy, static_cast<unsigned>(n));
    k_reorder_beams<T><<<grid, kMoveThreads, smem, stream>>>(st, a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

template <class T>
int launch_path(const States &st, int n, const MoveArgs &a, cudaStream_t stream)
{
    const unsigned gy = static_cast<unsigned>(std::min(a.batch, 65535));
    const int64_t columns = a.unit_bytes / static_cast<int64_t>(sizeof(T)) * a.segments;
    // without states the lengths alone are written
    const dim3 grid(column_blocks(columns, static_cast<int64_t>(gy) * n, 2048 / kMoveThreads), gy,
                    static_cast<unsigned>(std::max(n, 1)));
    k_commit_path<T><<<grid, kMoveThreads, 0, stream>>>(st, a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

// Sizes and strides of a state, bounded so that their products (at most
// 2^16 segments of 2^46 bytes) stay below 2^63.
int check_state(int num_states, int64_t request_stride, int segments, int64_t segment_stride,
                int64_t unit_bytes, int capacity, int batch)
{
    constexpr int64_t kMost = int64_t(1) << 46;
    if (num_states < 0 || segments < 1 || unit_bytes < 1 || capacity < 1 || batch < 0) return SPEC_EINVAL;
    if (request_stride < 0 || segment_stride < 0) return SPEC_EINVAL;
    if (num_states > SPEC_MAX_STATES || unit_bytes > INT_MAX || segments > (1 << 16) ||
        request_stride > kMost || segment_stride > kMost || unit_bytes * capacity > kMost)
        return SPEC_EUNSUPPORTED;
    return SPEC_OK;
}

// The addresses; false if one is null or comes twice (blocks of different
// states run at once, and the moves of one would read those of the other).
bool take_states(void *const *states, int n, States &st)
{
    std::memset(&st, 0, sizeof st);
    for (int i = 0; i < n; ++i) {
        if (!states[i]) return false;
        st.at[i] = static_cast<char *>(states[i]);
    }
    States sorted = st;
    std::sort(sorted.at, sorted.at + n);
    return std::adjacent_find(sorted.at, sorted.at + n) == sorted.at + n;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_reorder_beams(void *const *states, int num_states, int64_t request_stride,
                                  int64_t beam_stride, int segments, int64_t segment_stride,
                                  int64_t unit_bytes, int capacity, const int32_t *begin,
                                  const int32_t *end, const int32_t *parents, int batch, int beams,
                                  int width, int32_t *status, cudaStream_t stream)
{
    if (beams < 1 || width < 1 || width > beams) return SPEC_EINVAL;
    if (beam_stride < 0) return SPEC_EINVAL;
    if (beams > SPEC_MAX_BEAMS || beam_stride > (int64_t(1) << 46)) return SPEC_EUNSUPPORTED;
    const int rc = check_state(num_states, request_stride, segments, segment_stride, unit_bytes, capacity, batch);
    if (rc != SPEC_OK) return rc;
    // rows may not overlap: a segment fits its stride, a beam's segments the
    // beam stride (whichever of the two is the outer one), the beams the request's
    const int64_t seg = unit_bytes * capacity;
    if (segments > 1 && segment_stride < seg) return SPEC_EINVAL;
    if (beams > 1 && beam_stride < (segments - 1) * segment_stride + seg) return SPEC_EINVAL;
    if (batch > 1 && request_stride < (beams - 1) * beam_stride + (segments - 1) * segment_stride + seg)
        return SPEC_EINVAL;
    if (batch == 0 || num_states == 0) return SPEC_OK;
    if (!states || !parents) return SPEC_EINVAL;
    States st;
    if (!take_states(states, num_states, st)) return SPEC_EINVAL;
    const MoveArgs a{request_stride, beam_stride, segment_stride, unit_bytes, segments, capacity, batch,
                     beams, width, begin, end, parents, nullptr, status};
    // strides that nothing steps over do not narrow the vector
    const uint64_t strides = static_cast<uint64_t>(unit_bytes) | (batch > 1 ? request_stride : 0) |
                             (beams > 1 ? beam_stride : 0) | (segments > 1 ? segment_stride : 0);
    switch (vector_bytes(st, num_states, strides)) {
    case 16: return launch_beams<uint4>(st, num_states, a, 0, stream);
    case 8: return launch_beams<uint2>(st, num_states, a, 1, stream);
    case 4: return launch_beams<uint32_t>(st, num_states, a, 2, stream);
    case 2: return launch_beams<uint16_t>(st, num_states, a, 3, stream);
    default: return launch_beams<uint8_t>(st, num_states, a, 4, stream);
    }
}

extern "C" int spec_commit_path(void *const *states, int num_states, int64_t request_stride, int segments,
                                int64_t segment_stride, int64_t unit_bytes, int capacity,
                                const int32_t *base, const int32_t *path, int batch, int num_nodes,
                                int width, int32_t *out_lens, int32_t *status, cudaStream_t stream)
{
    if (num_nodes < 1 || width < 1) return SPEC_EINVAL;
    if (num_nodes > SPEC_MAX_NODES || width > SPEC_MAX_NODES) return SPEC_EUNSUPPORTED;
    const int rc = check_state(num_states, request_stride, segments, segment_stride, unit_bytes, capacity, batch);
    if (rc != SPEC_OK) return rc;
    const int64_t seg = unit_bytes * capacity;
    if (segments > 1 && segment_stride < seg) return SPEC_EINVAL;
    if (batch > 1 && request_stride < (segments - 1) * segment_stride + seg) return SPEC_EINVAL;
    if (batch == 0 || (num_states == 0 && !out_lens)) return SPEC_OK;
    if ((num_states > 0 && !states) || !path || (out_lens && out_lens == base)) return SPEC_EINVAL;
    States st;
    if (!take_states(states, num_states, st)) return SPEC_EINVAL;
    const MoveArgs a{request_stride, 0, segment_stride, unit_bytes, segments, capacity, batch,
                     num_nodes, width, base, nullptr, path, out_lens, status};
    const uint64_t strides = static_cast<uint64_t>(unit_bytes) | (batch > 1 ? request_stride : 0) |
                             (segments > 1 ? segment_stride : 0);
    switch (vector_bytes(st, num_states, strides)) {
    case 16: return launch_path<uint4>(st, num_states, a, stream);
    case 8: return launch_path<uint2>(st, num_states, a, stream);
    case 4: return launch_path<uint32_t>(st, num_states, a, stream);
    case 2: return launch_path<uint16_t>(st, num_states, a, stream);
    default: return launch_path<uint8_t>(st, num_states, a, stream);
    }
}
