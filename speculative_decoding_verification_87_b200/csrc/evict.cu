// evict.cu -- spec_cache_evict: a cache past its budget gives up the slots of
// the least accumulated attention weight, in every head by itself.
//
// The `budget` best of n slots are found by radix selection over 32-bit keys
// of the documented order (protected slots above every score, NaN below),
// not by sorting: three counting passes over keys held in shared memory, a
// cluster of blocks per head sharing counts through distributed shared
// memory.  Only slots from `budget` on that stay move, each into a place
// that was given up below, so sources and targets are disjoint: no ordering
// between the moves is needed and a serving step that is a few slots over
// moves a few rows instead of half the cache.
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

constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kClusterMax = 8;
constexpr int kSliceMax = SPEC_MAX_SLOTS / kClusterMax;  // keys of a block: 128 KB at most
constexpr int kBins = 2048;                              // 11 bits a pass
constexpr unsigned kAll = 0xFFFFFFFFu;

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

// What the blocks of a cluster show one another.
struct Shown {
    int hist[kBins];
    int newest;
    int counts[2];  // of this block's slice, for cluster-wide prefixes
};

// Pick: a cluster of blocks per (request, head).
__global__ void __launch_bounds__(kPickThreads, 1) k_evict_pick(const __grid_constant__ EvictArgs a)
{
    extern __shared__ uint32_t keys[];
    __shared__ Shown sh;
    __shared__ int total[kBins];
    __shared__ int warp_sum[2][kPickWarps + 1];
    __shared__ int pick_bin, pick_above;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t head = blockIdx.x / blocks;
    const int b = static_cast<int>(head / a.H);
    const int n = __ldg(a.lens + b);
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
    for (int i = s0 + tid; i < s1; i += kPickThreads) newest = max(newest, positions[i]);
    newest = __reduce_max_sync(kAll, newest);
    if (lane == 0) warp_sum[0][warp] = newest;
    __syncthreads();
    if (warp == 0) {
        newest = __reduce_max_sync(kAll, warp_sum[0][lane]);
        if (lane == 0) sh.newest = newest;
    }
    cluster.sync();
    newest = INT_MIN;
    for (int r = 0; r < blocks; ++r) newest = max(newest, cluster.map_shared_rank(&sh, r)->newest);
    const int64_t fresh = static_cast<int64_t>(newest) - a.recent;

    bool nan = false;
    for (int i = tid; i < len; i += kPickThreads) {
        const float sc = scores[s0 + i];
        const int po = positions[s0 + i];
        nan |= sc != sc;
        keys[i] = slot_key(sc, po < a.sinks || po > fresh);
    }
    if (nan && a.status) atomicOr(a.status, SPEC_STATUS_LOGIT);

    // radix selection of the budget-th largest key, 11 + 11 + 10 bits
    uint32_t prefix = 0, mask = 0;
    int want = a.budget;  // still to take among the keys that match the prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit = pass == 2 ? 1023u : 2047u;
        __syncthreads();
        for (int i = tid; i < kBins; i += kPickThreads) sh.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < len; i += kPickThreads) {
            const uint32_t key = keys[i];
            if ((key & mask) == prefix) atomicAdd(&sh.hist[(key >> shift) & digit], 1);
        }
        cluster.sync();
        for (int i = tid; i < kBins; i += kPickThreads) {
            int t = 0;
            for (int r = 0; r < blocks; ++r) t += cluster.map_shared_rank(&sh, r)->hist[i];
            total[i] = t;
        }
        cluster.sync();  // counts read everywhere before they are cleared
        // suffix sums, two bins a thread from the top: bins 2047 - 2 tid, 2046 - 2 tid
        const int hi = kBins - 1 - 2 * tid, c0 = total[hi], c1 = total[hi - 1];
        int incl = warp_inclusive(c0 + c1);
        if (lane == 31) warp_sum[0][warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const int w = warp_sum[0][lane];
            warp_sum[1][lane] = warp_inclusive(w) - w;
        }
        __syncthreads();
        const int above = incl - (c0 + c1) + warp_sum[1][warp];
        if (above < want && above + c0 >= want) {
            pick_bin = hi;
            pick_above = above;
        } else if (above + c0 < want && above + c0 + c1 >= want) {
            pick_bin = hi - 1;
            pick_above = above + c0;
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
    auto prefixes = [&](int mine0, int mine1, int &before0, int &before1) {
        // mine: this warp's counts (uniform over the warp)
        __syncthreads();
        if (lane == 0) {
            warp_sum[0][warp] = mine0;
            warp_sum[1][warp] = mine1;
        }
        __syncthreads();
        if (warp < 2) {
            const int w = warp_sum[warp][lane];
            const int incl = warp_inclusive(w);
            __syncwarp();
            warp_sum[warp][lane] = incl - w;
            if (lane == 31) sh.counts[warp] = incl;
        }
        cluster.sync();
        before0 = warp_sum[0][warp];
        before1 = warp_sum[1][warp];
        for (int r = 0; r < rank; ++r) {
            before0 += cluster.map_shared_rank(&sh, r)->counts[0];
            before1 += cluster.map_shared_rank(&sh, r)->counts[1];
        }
        cluster.sync();  // read everywhere before the next use
    };
    int equal = 0;
    for (int i = w0; i < w1; i += 32) {
        const int j = i + lane;
        equal += __popc(__ballot_sync(kAll, j < w1 && keys[j] == prefix));
    }
    int ties, none;
    prefixes(equal, 0, ties, none);
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
    prefixes(nsrc, ndst, fsrc, fdst);
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
}

// Move: a warp per move and head (grid x: moves, y: heads).
template <class T>
__global__ void __launch_bounds__(256) k_evict_move(const __grid_constant__ EvictArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t head = blockIdx.y; head < static_cast<int64_t>(a.B) * a.H; head += gridDim.y) {
        const int b = static_cast<int>(head / a.H), h = static_cast<int>(head % a.H);
        if (h == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
            const int n = a.lens[b];
            a.out_lens[b] = n >= 0 && n <= a.C ? min(n, a.budget) : n;
        }
        const int moves = __ldcg(a.count + head);
        char *k = a.k + b * a.k_req + h * a.k_head, *v = a.v + b * a.v_req + h * a.v_head;
        const int nk = static_cast<int>(a.k_row / static_cast<int64_t>(sizeof(T)));
        const int nv = a.v ? static_cast<int>(a.v_row / static_cast<int64_t>(sizeof(T))) : 0;
        for (int m = blockIdx.x * 8 + warp; m < moves; m += gridDim.x * 8) {
            const int64_t s = __ldcg(a.src + head * a.most + m), d = __ldcg(a.dst + head * a.most + m);
            for (int i = lane; i < nk + nv; i += 32) {
                const int j = i < nk ? i : i - nk;
                char *row = i < nk ? k : v;
                const int64_t pitch = i < nk ? a.k_slot : a.v_slot;
                reinterpret_cast<T *>(row + d * pitch)[j] = reinterpret_cast<const T *>(row + s * pitch)[j];
            }
            if (lane == 0) a.out_scores[head * a.C + d] = a.scores[head * a.C + s];
            if (lane == 1) a.out_positions[head * a.C + d] = a.positions[head * a.C + s];
        }
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

std::mutex g_evict_mu;
bool g_evict_attr[64];

// Blocks a head is shared by: slices of about 4096 slots.
int cluster_blocks(int C)
{
    int n = 1;
    while (n < kClusterMax && static_cast<int64_t>(n) * 4096 < C) n *= 2;
    return n;
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
    const int G = cluster_blocks(capacity);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(G);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(batch * heads * G));
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = sizeof(uint32_t) * static_cast<size_t>((capacity + G - 1) / G);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_evict_pick, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    const int64_t bh = static_cast<int64_t>(batch) * heads;
    const unsigned gy = static_cast<unsigned>(std::min<int64_t>(bh, 65535));
    const int64_t need = std::max<int64_t>(1, (static_cast<int64_t>(L.most) + 7) / 8);
    const unsigned gx = static_cast<unsigned>(std::min(need, std::max<int64_t>(1, 148 * 16 / gy)));
    uint64_t bits = reinterpret_cast<uintptr_t>(k) | static_cast<uint64_t>(k_request_stride | k_head_stride | k_slot_stride | k_row_bytes);
    if (v) bits |= reinterpret_cast<uintptr_t>(v) | static_cast<uint64_t>(v_request_stride | v_head_stride | v_slot_stride | v_row_bytes);
    const dim3 grid(gx, gy);
    if (bits % 16 == 0) k_evict_move<uint4><<<grid, 256, 0, stream>>>(a);
    else if (bits % 4 == 0) k_evict_move<uint32_t><<<grid, 256, 0, stream>>>(a);
    else k_evict_move<uint8_t><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}
