// evict.cu -- spec_cache_evict: a cache past its budget gives up the slots of
// the least accumulated attention weight, in every head by itself.
//
// The `budget` best of n slots are found by selection over 32-bit keys of the
// documented order (protected slots above every score, NaN below), not by
// sorting.  Only slots from `budget` on that stay move, each into a place
// that was given up below, so sources and targets are disjoint: no ordering
// between the moves is needed and a serving step that is a few slots over
// moves a few rows instead of half the cache.  Latency bounds the small
// calls (a chain of block-wide steps per head), the moved rows the large ones.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "../../include/specverify.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kPickThreads = 512;  // two blocks a SM: with 1024 threads only some 14 clusters of 8 fit the GPU at once
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kClusterMax = 8;
constexpr int kSliceMax = SPEC_MAX_SLOTS / kClusterMax;  // keys of a block: 128 KB at most
constexpr int kBins = 2048;                              // 11 bits a pass
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kMoveGroup = 4;                            // rows a warp moves at a time

struct EvictArgs {
    char *k, *v;
    int64_t k_req, k_head, k_slot, k_row, v_req, v_head, v_slot, v_row;  // bytes
    const float *scores;
    const int32_t *positions, *lens;
    int B, H, C, budget, sinks, recent;
    int most;  // moves a head can have: min(budget, C - budget)
    float *out_scores;
    int32_t *out_positions, *out_lens;
    int32_t *status;
    int32_t *count;  // [B * H] moves
    int32_t *src, *dst;  // [B * H][most]
};

// Scores as unsigned integers of the same order: protected slots on top,
// then +inf .. -inf (both zeros equal), NaN at the bottom.
__device__ __forceinline__ uint32_t slot_key(float score, bool safe)
{
    if (safe) return 0xFFFFFFFFu;
    if (score != score) return 0u;
    const uint32_t u = __float_as_uint(score + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int warp_inclusive(int x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// ------------------------------------------------------------ large caches
// A cluster of blocks per head with the keys in shared memory; three radix
// passes of 11, 11 and 10 bits over counts that the blocks read from one
// another through distributed shared memory.  Each exchange has its own
// words, so it costs one cluster barrier.  (16 heads of 32768 slots: about 20
// us, the latency of seven cluster-wide steps; their 4.2 MB would take 1.)
struct alignas(16) Shown {
    int hist[3][kBins];
    int newest;
    int counts[2][2];  // of this block's slice, for cluster-wide prefixes
};

__global__ void __launch_bounds__(kPickThreads, 2) k_evict_pick(const __grid_constant__ EvictArgs a)
{
    extern __shared__ uint32_t keys[];
    __shared__ Shown sh;
    __shared__ int warp_sum[2][kPickWarps];
    __shared__ int pick_bin, pick_above;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t head = blockIdx.x / blocks;
    const int b = static_cast<int>(head / a.H);
    const int n = __ldg(a.lens + b);
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid == 0 && rank == 0) a.count[head] = 0;
    const bool fits = n >= 0 && n <= a.C;
    if (!fits) {  // the whole cluster leaves
        if (tid == 0 && rank == 0 && a.status) atomicOr(a.status, SPEC_STATUS_CAPACITY);
        return;
    }
    const float *scores = a.scores + head * a.C;
    const int32_t *positions = a.positions + head * a.C;
    float *out_scores = a.out_scores + head * a.C;
    int32_t *out_positions = a.out_positions + head * a.C;
    // the block's slice of slots
    const int slice = (n + blocks - 1) / blocks;
    const int s0 = min(n, rank * slice), s1 = min(n, s0 + slice), len = s1 - s0;
    if (n <= a.budget) {
        for (int i = s0 + tid; i < s1; i += kPickThreads) {
            const float sc = scores[i];
            const int po = positions[i];
            out_scores[i] = sc;
            out_positions[i] = po;
        }
        return;
    }

    // the head's newest position
    int newest = INT_MIN;
#pragma unroll 4
    for (int i = s0 + tid; i < s1; i += kPickThreads) newest = max(newest, positions[i]);
    newest = __reduce_max_sync(kAll, newest);
    if (lane == 0) warp_sum[0][warp] = newest;
    for (int i = tid; i < 3 * kBins; i += kPickThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    if (warp == 0) {
        newest = __reduce_max_sync(kAll, warp_sum[0][lane % kPickWarps]);
        if (lane == 0) sh.newest = newest;
    }
    cluster.sync();
    newest = INT_MIN;
#pragma unroll
    for (int r = 0; r < kClusterMax; ++r)
        if (r < blocks) newest = max(newest, cluster.map_shared_rank(&sh, r)->newest);
    const int64_t fresh = static_cast<int64_t>(newest) - a.recent;

    bool nan = false;
#pragma unroll 4
    for (int i = tid; i < len; i += kPickThreads) {
        const float sc = scores[s0 + i];
        const int po = positions[s0 + i];
        nan |= sc != sc;
        keys[i] = slot_key(sc, po < a.sinks || po > fresh);
    }
    if (nan && a.status) atomicOr(a.status, SPEC_STATUS_LOGIT);

    // radix selection of the budget-th largest key
    uint32_t prefix = 0, mask = 0;
    int want = a.budget;  // still to take among the keys that match the prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < len; i += kPickThreads) {  // a thread counts the keys it wrote
            const uint32_t key = keys[i];
            if ((key & mask) == prefix) atomicAdd(&sh.hist[pass][(key >> shift) & digit], 1);
        }
        cluster.sync();
        // four bins a thread from the top, hi .. hi - 3, over all blocks
        static_assert(kBins == 4 * kPickThreads, "four bins a thread");
        const int hi = kBins - 1 - 4 * tid;
        int c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < kClusterMax; ++r)
            if (r < blocks) {
                const int4 x = *reinterpret_cast<const int4 *>(&cluster.map_shared_rank(&sh, r)->hist[pass][hi - 3]);
                c[0] += x.w;
                c[1] += x.z;
                c[2] += x.y;
                c[3] += x.x;
            }
        const int sum = c[0] + c[1] + c[2] + c[3], incl = warp_inclusive(sum);
        if (lane == 31) warp_sum[0][warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const int w = lane < kPickWarps ? warp_sum[0][lane] : 0;
            const int before = warp_inclusive(w) - w;
            if (lane < kPickWarps) warp_sum[1][lane] = before;
        }
        __syncthreads();
        int above = incl - sum + warp_sum[1][warp];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (above < want && above + c[x] >= want) {
                pick_bin = hi - x;
                pick_above = above;
            }
            above += c[x];
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(pick_bin) << shift;
        mask |= digit << shift;
        want -= pick_above;
    }
    // keys above `prefix` stay; of those equal to it, the `want` lowest slots

    // exclusive prefixes over the cluster's slots: each warp owns a
    // contiguous part of the slice
    const int per_warp = ((len + kPickWarps - 1) / kPickWarps + 31) / 32 * 32;
    const int w0 = min(len, warp * per_warp), w1 = min(len, w0 + per_warp);
    auto prefixes = [&](int call, int mine0, int mine1, int &before0, int &before1) {
        // mine: this warp's counts (uniform over the warp)
        __syncthreads();
        if (lane == 0) {
            warp_sum[0][warp] = mine0;
            warp_sum[1][warp] = mine1;
        }
        __syncthreads();
        if (warp < 2) {
            const int w = lane < kPickWarps ? warp_sum[warp][lane] : 0;
            const int incl = warp_inclusive(w);
            __syncwarp();
            if (lane < kPickWarps) warp_sum[warp][lane] = incl - w;
            if (lane == 31) sh.counts[call][warp] = incl;
        }
        cluster.sync();
        before0 = warp_sum[0][warp];
        before1 = warp_sum[1][warp];
#pragma unroll
        for (int r = 0; r < kClusterMax; ++r)
            if (r < rank) {
                before0 += cluster.map_shared_rank(&sh, r)->counts[call][0];
                before1 += cluster.map_shared_rank(&sh, r)->counts[call][1];
            }
    };
    int equal = 0;
    for (int i = w0; i < w1; i += 32) {
        const int j = i + lane;
        equal += __popc(__ballot_sync(kAll, j < w1 && keys[j] == prefix));
    }
    int ties, none;
    prefixes(0, equal, 0, ties, none);
    // which slots stay; count sources (stay, at or past the budget) and
    // targets (given up, below it)
    auto walk = [&](auto &&visit) {
        int seen = ties;
        for (int i = w0; i < w1; i += 32) {
            const int j = i + lane;
            const uint32_t key = j < w1 ? keys[j] : 0u;
            const unsigned eq = __ballot_sync(kAll, j < w1 && key == prefix);
            const int at = seen + __popc(eq & ((1u << lane) - 1));
            const bool stays = j < w1 && (key > prefix || (key == prefix && at < want));
            seen += __popc(eq);
            const int slot = s0 + j;
            visit(slot, j < w1, __ballot_sync(kAll, stays && slot >= a.budget),
                  __ballot_sync(kAll, j < w1 && !stays && slot < a.budget), stays);
        }
    };
    int nsrc = 0, ndst = 0, fsrc, fdst;
    walk([&](int, bool, unsigned s, unsigned d, bool) {
        nsrc += __popc(s);
        ndst += __popc(d);
    });
    prefixes(1, nsrc, ndst, fsrc, fdst);
    int32_t *src = a.src + head * a.most, *dst = a.dst + head * a.most;
    walk([&](int slot, bool in, unsigned s, unsigned d, bool stays) {
        const unsigned below = (1u << lane) - 1;
        if (s >> lane & 1) src[fsrc + __popc(s & below)] = slot;
        if (d >> lane & 1) dst[fdst + __popc(d & below)] = slot;
        fsrc += __popc(s);
        fdst += __popc(d);
        if (in && stays && slot < a.budget) {
            const float sc = scores[slot];
            const int po = positions[slot];
            out_scores[slot] = sc;
            out_positions[slot] = po;
        }
    });
    // fsrc is now this warp's inclusive count: the last warp of the last
    // block holds the total
    if (rank == blocks - 1 && warp == kPickWarps - 1 && lane == 0) a.count[head] = fsrc;
    cluster.sync();  // no block leaves while another reads its counts
}

// Move n <= kMoveGroup rows of a head, one warp: all loads, then all stores.
template <class T>
__device__ __forceinline__ void move_rows(const EvictArgs &a, int64_t head, const int *src, const int *dst, int n, int lane)
{
    const int b = static_cast<int>(head / a.H), h = static_cast<int>(head % a.H);
    const int mine = lane < n ? lane : 0;
    const int s = src[mine], d = dst[mine];
    char *k = a.k + b * a.k_req + h * a.k_head, *v = a.v + b * a.v_req + h * a.v_head;
    const int nk = static_cast<int>(a.k_row / static_cast<int64_t>(sizeof(T)));
    const int nv = a.v ? static_cast<int>(a.v_row / static_cast<int64_t>(sizeof(T))) : 0;
    for (int i = lane; i < (nk + nv + 31) / 32 * 32; i += 32) {
        char *row = i < nk ? k : v;
        const int64_t pitch = i < nk ? a.k_slot : a.v_slot, at = static_cast<int64_t>(i < nk ? i : i - nk) * sizeof(T);
        const bool in = i < nk + nv;
        T x[kMoveGroup];
#pragma unroll
        for (int u = 0; u < kMoveGroup; ++u) {
            const int from = __shfl_sync(kAll, s, u);
            if (in && u < n) x[u] = *reinterpret_cast<const T *>(row + from * pitch + at);
        }
#pragma unroll
        for (int u = 0; u < kMoveGroup; ++u) {
            const int to = __shfl_sync(kAll, d, u);
            if (in && u < n) *reinterpret_cast<T *>(row + to * pitch + at) = x[u];
        }
    }
    if (lane < n) {
        a.out_scores[head * a.C + d] = a.scores[head * a.C + s];
        a.out_positions[head * a.C + d] = a.positions[head * a.C + s];
    }
}

// Move: kMoveGroup moves a warp (grid x: moves, y: heads).  (256 heads, 2048
// moves of two 256-byte rows each, pick and moves: 148 us with four rows a
// warp, 182 with eight, whose registers leave half the warps, 177 with two.)
template <class T>
__global__ void __launch_bounds__(256) k_evict_move(const __grid_constant__ EvictArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    for (int64_t head = blockIdx.y; head < static_cast<int64_t>(a.B) * a.H; head += gridDim.y) {
        const int b = static_cast<int>(head / a.H);
        if (head % a.H == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
            const int n = a.lens[b];
            a.out_lens[b] = n >= 0 && n <= a.C ? min(n, a.budget) : n;
        }
        const int moves = __ldcg(a.count + head);
        for (int m = (blockIdx.x * 8 + warp) * kMoveGroup; m < moves; m += gridDim.x * 8 * kMoveGroup)
            move_rows<T>(a, head, a.src + head * a.most + m, a.dst + head * a.most + m, min(kMoveGroup, moves - m), lane);
    }
}

// ------------------------------------------------------------ small caches
// Heads of up to kSmallSlots slots: one block a head, the keys in registers
// (slot j * threads + tid), the budget-th largest by a search with three
// pivots a step, two bits each; it ends early where a pivot has exactly
// `budget` keys above.  With kFused the block also moves the rows.  (8 heads
// of 4000 slots 9.0 us, 256 of 2057 12.4; the cluster form takes 17 and 19.)
constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallKeys = 8;
constexpr int kSmallSlots = kSmallThreads * kSmallKeys;
constexpr int kFusedMoves = kSmallSlots / 2;  // at most min(budget, capacity - budget)

template <class T, bool kFused>
__global__ void __launch_bounds__(kSmallThreads, 2) k_evict_small(const __grid_constant__ EvictArgs a)
{
    __shared__ uint32_t sums[2][kSmallWarps];
    __shared__ int newest_sh[kSmallWarps];
    __shared__ __align__(16) int counts[2][kSmallKeys * kSmallWarps];
    __shared__ int moves_sh;
    __shared__ int src_sh[kFusedMoves], dst_sh[kFusedMoves];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t head = blockIdx.x;
    const int b = static_cast<int>(head / a.H);
    const int n = __ldg(a.lens + b);
    const bool fits = n >= 0 && n <= a.C;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid == 0) {
        if (kFused) {
            if (head % a.H == 0) a.out_lens[b] = fits ? min(n, a.budget) : n;
        } else {
            a.count[head] = 0;
        }
        if (!fits && a.status) atomicOr(a.status, SPEC_STATUS_CAPACITY);
    }
    if (!fits) return;
    const float *scores = a.scores + head * a.C;
    const int32_t *positions = a.positions + head * a.C;
    float *out_scores = a.out_scores + head * a.C;
    int32_t *out_positions = a.out_positions + head * a.C;
    float sc[kSmallKeys];
    int po[kSmallKeys];
    uint32_t key[kSmallKeys];
    int newest = INT_MIN;
#pragma unroll
    for (int j = 0; j < kSmallKeys; ++j) {
        const int slot = j * kSmallThreads + tid;
        sc[j] = 0.f;
        po[j] = INT_MIN;
        if (slot < n) {
            sc[j] = scores[slot];
            po[j] = positions[slot];
        }
        newest = max(newest, po[j]);
    }
    bool keep_all = n <= a.budget;
    uint32_t t = 0;
    int want = INT_MAX;  // keys equal to t that stay
    if (!keep_all) {
        newest = __reduce_max_sync(kAll, newest);
        if (lane == 0) newest_sh[warp] = newest;
        __syncthreads();
        newest = __reduce_max_sync(kAll, newest_sh[lane % kSmallWarps]);
        const int64_t fresh = static_cast<int64_t>(newest) - a.recent;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < kSmallKeys; ++j) {
            const bool in = j * kSmallThreads + tid < n;
            nan |= in && sc[j] != sc[j];
            key[j] = in ? slot_key(sc[j], po[j] < a.sinks || po[j] > fresh) : 0u;
        }
        if (nan && a.status) atomicOr(a.status, SPEC_STATUS_LOGIT);
        // slots past n count as key 0, the lowest: [lo, hi] holds the largest
        // t that at least `budget` keys reach
        uint32_t lo = 0, hi = 0xFFFFFFFFu;
        int buf = 0;
        auto reach = [&](uint32_t p1, uint32_t p2, uint32_t p3, int &c1, int &c2, int &c3) {
            uint32_t c = 0;  // three fields of ten bits: a warp has 256 keys
#pragma unroll
            for (int j = 0; j < kSmallKeys; ++j)
                c += (key[j] >= p1 ? 1u : 0u) + (key[j] >= p2 ? 1u << 10 : 0u) + (key[j] >= p3 ? 1u << 20 : 0u);
            c = __reduce_add_sync(kAll, c);
            if (lane == 0) sums[buf][warp] = c;
            __syncthreads();
            c = lane < kSmallWarps ? sums[buf][lane] : 0u;
            // the block's fields need 13 bits
            const uint32_t x = __reduce_add_sync(kAll, (c & 1023u) | (c >> 20) << 16);
            c1 = static_cast<int>(x & 0xFFFFu);
            c3 = static_cast<int>(x >> 16);
            c2 = static_cast<int>(__reduce_add_sync(kAll, c >> 10 & 1023u));
            buf ^= 1;
        };
        bool done = false;
        while (lo < hi && !done) {
            // pivots in (lo, hi], equal ones where few are left
            const uint32_t span = hi - lo;
            const uint32_t p2 = lo + span / 2 + (span & 1), p1 = lo + (p2 - lo + 1) / 2, p3 = p2 + (hi - p2 + 1) / 2;
            int c1, c2, c3;
            reach(p1, p2, p3, c1, c2, c3);
            if (c1 == a.budget || c2 == a.budget || c3 == a.budget) {
                lo = c3 == a.budget ? p3 : c2 == a.budget ? p2 : p1;
                done = true;
            } else if (c3 >= a.budget) {
                lo = p3;
            } else if (c2 >= a.budget) {
                lo = p2;
                hi = p3 - 1;
            } else if (c1 >= a.budget) {
                lo = p1;
                hi = p2 - 1;
            } else {
                hi = p1 - 1;
            }
        }
        t = lo;
        if (!done) {
            // keys above t stay, and the first of those equal to it
            int c1, c2, c3;
            reach(t + 1, t + 1, t + 1, c1, c2, c3);
            want = t == 0xFFFFFFFFu ? a.budget : a.budget - c1;
        }
    }
    // exclusive prefixes over slots of per-warp counts[x][j * warps + warp]
    static_assert(kSmallKeys * kSmallWarps == 128, "four counts a lane");
    auto scan = [&](int x) {  // one warp
        int4 v = *reinterpret_cast<int4 *>(&counts[x][4 * lane]);
        const int sum = v.x + v.y + v.z + v.w;
        const int before = warp_inclusive(sum) - sum;
        const int total = __shfl_sync(kAll, before + sum, 31);
        v = make_int4(before, before + v.x, before + v.x + v.y, before + v.x + v.y + v.z);
        *reinterpret_cast<int4 *>(&counts[x][4 * lane]) = v;
        return total;
    };
    unsigned stays = 0;
#pragma unroll
    for (int j = 0; j < kSmallKeys; ++j)
        if (keep_all ? j * kSmallThreads + tid < n : j * kSmallThreads + tid < n && key[j] >= t) stays |= 1u << j;
    if (want != INT_MAX) {  // ties: the lowest `want` slots
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSmallKeys; ++j) {
            const unsigned eq = __ballot_sync(kAll, j * kSmallThreads + tid < n && key[j] == t);
            if (lane == 0) counts[0][j * kSmallWarps + warp] = __popc(eq);
        }
        __syncthreads();
        if (warp == 0) scan(0);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSmallKeys; ++j) {
            const bool mine = j * kSmallThreads + tid < n && key[j] == t;
            const unsigned eq = __ballot_sync(kAll, mine);
            if (mine && counts[0][j * kSmallWarps + warp] + __popc(eq & ((1u << lane) - 1)) >= want) stays &= ~(1u << j);
        }
        __syncthreads();
    }
    // what stays below the budget keeps its place
#pragma unroll
    for (int j = 0; j < kSmallKeys; ++j) {
        const int slot = j * kSmallThreads + tid;
        if ((stays >> j & 1) && slot < a.budget) {
            out_scores[slot] = sc[j];
            out_positions[slot] = po[j];
        }
    }
    if (keep_all) return;
    // the i-th source goes to the i-th target
#pragma unroll
    for (int j = 0; j < kSmallKeys; ++j) {
        const int slot = j * kSmallThreads + tid;
        const unsigned s = __ballot_sync(kAll, (stays >> j & 1) && slot >= a.budget);
        const unsigned d = __ballot_sync(kAll, !(stays >> j & 1) && slot < a.budget);
        if (lane == 0) {
            counts[0][j * kSmallWarps + warp] = __popc(s);
            counts[1][j * kSmallWarps + warp] = __popc(d);
        }
    }
    __syncthreads();
    if (warp < 2) {
        const int total = scan(warp);
        if (tid == 0) {
            moves_sh = total;
            if (!kFused) a.count[head] = total;
        }
    }
    __syncthreads();
    int *src = kFused ? src_sh : a.src + head * a.most, *dst = kFused ? dst_sh : a.dst + head * a.most;
#pragma unroll
    for (int j = 0; j < kSmallKeys; ++j) {
        const int slot = j * kSmallThreads + tid;
        const bool is = (stays >> j & 1) && slot >= a.budget, id = !(stays >> j & 1) && slot < a.budget;
        const unsigned s = __ballot_sync(kAll, is), d = __ballot_sync(kAll, id), below = (1u << lane) - 1;
        if (is) src[counts[0][j * kSmallWarps + warp] + __popc(s & below)] = slot;
        if (id) dst[counts[1][j * kSmallWarps + warp] + __popc(d & below)] = slot;
    }
    if (kFused) {
        __syncthreads();
        const int moves = moves_sh;
        for (int m = warp * kMoveGroup; m < moves; m += kSmallWarps * kMoveGroup)
            move_rows<T>(a, head, src_sh + m, dst_sh + m, min(kMoveGroup, moves - m), lane);
    }
}

constexpr size_t kEvictAlign = 256;
size_t align_up(size_t x) { return (x + kEvictAlign - 1) / kEvictAlign * kEvictAlign; }

struct EvictLayout {
    size_t count, src, dst, total;
    int most;
};
bool evict_layout(int B, int H, int C, int budget, EvictLayout &L)
{
    if (B < 0 || H < 1 || C < 1 || budget < 1) return false;
    L.most = std::max(0, std::min(budget, C - budget));
    const size_t heads = static_cast<size_t>(B) * H;
    L.count = 0;
    L.src = align_up(sizeof(int32_t) * heads);
    L.dst = L.src + align_up(sizeof(int32_t) * heads * L.most);
    L.total = std::max(kEvictAlign, L.dst + align_up(sizeof(int32_t) * heads * L.most));
    return true;
}

// Whether no two rows overlap: from the inside out, each stride steps over
// all that lies inside it.  (Heads that share rows would move them twice.)
bool rows_apart(int64_t row_bytes, const int64_t *strides, const int64_t *sizes)
{
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return strides[x] < strides[y]; });
    double extent = static_cast<double>(row_bytes);  // strides of 2^42 times sizes of 2^31 pass 64 bits
    for (int i : order) {
        if (sizes[i] <= 1) continue;
        if (static_cast<double>(strides[i]) < extent) return false;
        extent += static_cast<double>(sizes[i] - 1) * static_cast<double>(strides[i]);
    }
    return true;
}

std::mutex g_evict_mu;
bool g_evict_attr[64];

// Blocks a head is shared by: slices of about 4096 slots.
int cluster_blocks(int C)
{
    int n = 1;
    while (n < kClusterMax && static_cast<int64_t>(n) * 4096 < C) n *= 2;
    return n;
}

// Launches: small caches in one block a head, large ones in a cluster a head,
// then the moves as a programmatic dependent.
template <class T>
int launch_evict(const EvictArgs &a, cudaStream_t stream)
{
    const int64_t heads = static_cast<int64_t>(a.B) * a.H;
    if (a.C <= kSmallSlots) {
        // One kernel while a block a head moves its rows as fast as the whole
        // GPU would: few moves, or heads for most SMs.  (One kernel / two, us.  32
        // heads: 100 moves 8.1 / 9.9, 200 9.1 / 10.1, 400 11.1 / 11.0, 650 13.5 /
        // 12.2; 64 of 4096 slots: 400 16.9 / 14.9, 512 19.8 / 16.4; 128: 200 9.3 /
        // 11.7, 512 14.6 / 17.2, 1024 22.8 / 20.9, 2048 37.2 / 29.9; 192: 1024 29.8 /
        // 28.8, 2048 49.1 / 42.6; 256: 1024 31.4 / 33.3, 2048 53.3 / 52.6; 512: 2048
        // 90.2 / 96.3.)  The lengths must not be overwritten while other heads read
        // them.
        const bool one = a.most <= 128 || (heads >= 128 && a.most <= 512) || heads >= 256;
        if (one && a.out_lens != a.lens) {
            k_evict_small<T, true><<<static_cast<unsigned>(heads), kSmallThreads, 0, stream>>>(a);
            return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
        }
        k_evict_small<T, false><<<static_cast<unsigned>(heads), kSmallThreads, 0, stream>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SPEC_ECUDA;
    } else {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ECUDA;
        {
            std::lock_guard<std::mutex> lock(g_evict_mu);
            if (!g_evict_attr[dev]) {
                if (cudaFuncSetAttribute(k_evict_pick, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(sizeof(uint32_t) * kSliceMax)) != cudaSuccess)
                    return SPEC_ECUDA;
                g_evict_attr[dev] = true;
            }
        }
        const int G = cluster_blocks(a.C);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(G);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(heads * G));
        cfg.blockDim = dim3(kPickThreads);
        cfg.dynamicSmemBytes = sizeof(uint32_t) * static_cast<size_t>((a.C + G - 1) / G);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, k_evict_pick, a) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
    }
    const unsigned gy = static_cast<unsigned>(std::min<int64_t>(heads, 65535));
    const int64_t need = std::max<int64_t>(1, (static_cast<int64_t>(a.most) + 8 * kMoveGroup - 1) / (8 * kMoveGroup));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(need, std::max<int64_t>(1, 148 * 16 / gy))), gy);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_evict_move<T>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_evict_workspace_size(int batch, int heads, int capacity, int budget)
{
    EvictLayout L;
    return evict_layout(batch, heads, capacity, budget, L) ? L.total : 0;
}

extern "C" int spec_cache_evict(void *k, void *v, int64_t k_request_stride, int64_t k_head_stride,
                                int64_t k_slot_stride, int64_t k_row_bytes, int64_t v_request_stride,
                                int64_t v_head_stride, int64_t v_slot_stride, int64_t v_row_bytes,
                                const float *scores, const int32_t *positions, const int32_t *lens,
                                int batch, int heads, int capacity, int budget, int sinks, int recent,
                                float *out_scores, int32_t *out_positions, int32_t *out_lens,
                                int32_t *status, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream)
{
    if (batch < 0 || heads < 1 || capacity < 1 || budget < 1 || sinks < 0 || recent < 0 ||
        static_cast<int64_t>(sinks) + recent > budget)
        return SPEC_EINVAL;
    const int64_t row[8] = {k_request_stride, k_head_stride, k_slot_stride, k_row_bytes,
                            v_request_stride, v_head_stride, v_slot_stride, v_row_bytes};
    for (int i = 0; i < (v ? 8 : 4); ++i) {
        if (row[i] < 0) return SPEC_EINVAL;
        if (row[i] > (int64_t(1) << 42)) return SPEC_EUNSUPPORTED;
    }
    if (k_row_bytes < 1 || (capacity > 1 && k_slot_stride < k_row_bytes)) return SPEC_EINVAL;
    if (v && (v_row_bytes < 1 || (capacity > 1 && v_slot_stride < v_row_bytes))) return SPEC_EINVAL;
    if (capacity > SPEC_MAX_SLOTS || k_row_bytes > (1 << 30) || (v && v_row_bytes > (1 << 30)) ||
        static_cast<int64_t>(batch) * heads > INT_MAX / kClusterMax)
        return SPEC_EUNSUPPORTED;
    const int64_t sizes[3] = {batch, heads, capacity};
    if (!rows_apart(k_row_bytes, row, sizes) || (v && !rows_apart(v_row_bytes, row + 4, sizes))) return SPEC_EINVAL;
    if (batch == 0) return SPEC_OK;
    if (!k || !scores || !positions || !lens || !out_scores || !out_positions || !out_lens) return SPEC_EINVAL;
    EvictLayout L;
    if (!evict_layout(batch, heads, capacity, budget, L)) return SPEC_EINVAL;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kEvictAlign) != 0 || workspace_bytes < L.total)
        return SPEC_EWORKSPACE;
    char *ws = static_cast<char *>(workspace);
    EvictArgs a{static_cast<char *>(k), static_cast<char *>(v), k_request_stride, k_head_stride, k_slot_stride,
                k_row_bytes, v_request_stride, v_head_stride, v_slot_stride, v_row_bytes, scores, positions, lens,
                batch, heads, capacity, budget, sinks, recent, L.most, out_scores, out_positions, out_lens, status,
                reinterpret_cast<int32_t *>(ws + L.count), reinterpret_cast<int32_t *>(ws + L.src),
                reinterpret_cast<int32_t *>(ws + L.dst)};
    uint64_t bits = reinterpret_cast<uintptr_t>(k) | static_cast<uint64_t>(k_request_stride | k_head_stride | k_slot_stride | k_row_bytes);
    if (v) bits |= reinterpret_cast<uintptr_t>(v) | static_cast<uint64_t>(v_request_stride | v_head_stride | v_slot_stride | v_row_bytes);
    if (bits % 16 == 0) return launch_evict<uint4>(a, stream);
    if (bits % 4 == 0) return launch_evict<uint32_t>(a, stream);
    return launch_evict<uint8_t>(a, stream);
}
