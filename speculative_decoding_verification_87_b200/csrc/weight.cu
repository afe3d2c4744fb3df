// weight.cu -- spec_cache_score: the attention weight that a step's queries
// give the slots of a cache, added up per key head and slot.
//
// Mathematics.  With s_rt = scale q_r . k_t over the rows r = (query i,
// head g of the group), slot t gains sum_r exp(s_rt - L_r) where L_r is the
// row's log-sum-exp over the slots it sees (t <= begin + i).  L_r needs every
// slot of the row before the first weight can be formed, hence three steps:
// partial (max, sum) per row and chunk of slots, their merge into L_r, the
// weights.  A slot's weights are summed by one thread in row order, so the
// result does not depend on the schedule.  Everything is in units of log2
// (scale log2 e folded into the products), sums and statistics in fp32.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/specverify.h"
#include "sv_common.cuh"

namespace sv {
namespace {

constexpr int kTile = 128;      // slots per tile, a thread each
constexpr int kRows = 8;        // rows per register tile
constexpr int kChunksMax = 64;  // chunks of slots per row

struct ScoreArgs {
    const void *q, *k;
    int64_t q_req, q_tok, q_head, k_req, k_head, k_slot;  // elements
    const int32_t *begin, *end;
    int B, Q, H, G, D, C;  // H key heads, C capacity
    int R;                 // Q * G
    int chunk, chunks;     // slots per chunk, chunks per row
    float scale2;          // scale * log2(e)
    const float *in;
    float *out;
    int32_t *status;
    float2 *part;          // [B][H][R][chunks]
    float *lse;            // [B][H][R], log2 units
};

// Filled slots and queries of request b; false: left as it was.
struct Span {
    int begin, end;
    bool ok;
};
__device__ __forceinline__ Span span_of(const ScoreArgs &a, int b)
{
    Span s;
    s.begin = __ldg(a.begin + b);
    s.end = __ldg(a.end + b);
    s.ok = 0 <= s.begin && s.begin <= s.end && s.end <= a.C && s.end - s.begin <= a.Q;
    return s;
}

// Row r = i * G + g of head h: its first element.
template <class Tag>
__device__ __forceinline__ const typename Tag::elem *row_at(const ScoreArgs &a, int b, int h, int r)
{
    const int i = r / a.G, g = r - i * a.G;
    return static_cast<const typename Tag::elem *>(a.q) + b * a.q_req + i * a.q_tok +
           (static_cast<int64_t>(h) * a.G + g) * a.q_head;
}

// Rows [r0, r0 + kRows) below `rows` into shared memory as fp32, times
// scale2; the rest as zeros.
template <class Tag>
__device__ __forceinline__ void stage_rows(const ScoreArgs &a, int b, int h, int r0, int rows, float *sq)
{
    constexpr int kVec = Tag::kVec;
    const int nv = a.D / kVec;
    for (int i = threadIdx.x; i < kRows * nv; i += kTile) {
        const int r = i / nv, v = i - r * nv;
        float x[kVec];
        if (r0 + r < rows) unpack<Tag>(ldg_vec(row_at<Tag>(a, b, h, r0 + r) + v * kVec), x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) sq[r * a.D + v * kVec + e] = r0 + r < rows ? x[e] * a.scale2 : 0.f;
    }
}

// Slots [t0, t0 + kTile) below `end` into shared memory as fp32 (pitch
// D + 4 words), the rest as zeros.
template <class Tag>
__device__ __forceinline__ void stage_slots(const ScoreArgs &a, int b, int h, int t0, int end, float *sk)
{
    constexpr int kVec = Tag::kVec;
    const int nv = a.D / kVec, pitch = a.D + 4;
    const auto *base = static_cast<const typename Tag::elem *>(a.k) + b * a.k_req + h * a.k_head;
    for (int i = threadIdx.x; i < kTile * nv; i += kTile) {
        const int t = i / nv, v = i - t * nv;
        float x[kVec];
        if (t0 + t < end) {
            unpack<Tag>(ldg_vec(base + (t0 + t) * a.k_slot + v * kVec), x);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) sk[t * pitch + v * kVec + e] = x[e];
    }
}

// This thread's slot against the staged rows.
__device__ __forceinline__ void products(const float *sq, const float *sk, int D, float (&s)[kRows])
{
    const float *mine = sk + threadIdx.x * (D + 4);
#pragma unroll
    for (int r = 0; r < kRows; ++r) s[r] = 0.f;
    for (int d = 0; d < D; d += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(mine + d);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float4 y = *reinterpret_cast<const float4 *>(sq + r * D + d);
            s[r] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[r]))));
        }
    }
}

// Merge (m, l) pairs, l relative to 2^m; an empty pair is (-inf, 0).
__device__ __forceinline__ void merge(float &m, float &l, float om, float ol)
{
    const float n = max_nan(m, om);
    if (n == -INFINITY) return;
    l = l * exp2f(m - n) + ol * exp2f(om - n);
    m = n;
}

// Partial statistics: grid (row tile * chunks + chunk, head, request).
template <class Tag>
__global__ void __launch_bounds__(kTile) k_score_stats(const __grid_constant__ ScoreArgs a)
{
    extern __shared__ __align__(16) float smem[];
    float *sq = smem, *sk = smem + kRows * a.D;
    __shared__ float2 warp_part[kTile / 32][kRows];
    const int b = blockIdx.z, h = blockIdx.y;
    const int r0 = static_cast<int>(blockIdx.x / a.chunks) * kRows, chunk = blockIdx.x % a.chunks;
    const Span sp = span_of(a, b);
    const int rows = (sp.end - sp.begin) * a.G;
    if (!sp.ok || r0 >= rows) return;
    const int t_begin = chunk * a.chunk, t_end = min(sp.end, t_begin + a.chunk);
    float m[kRows], l[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    stage_rows<Tag>(a, b, h, r0, rows, sq);
    for (int t0 = t_begin; t0 < t_end; t0 += kTile) {
        __syncthreads();
        stage_slots<Tag>(a, b, h, t0, t_end, sk);
        __syncthreads();
        float s[kRows];
        products(sq, sk, a.D, s);
        const int t = t0 + threadIdx.x;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (t < t_end && t <= sp.begin + (r0 + r) / a.G) merge(m[r], l[r], s[r], 1.f);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            merge(m[r], l[r], __shfl_xor_sync(kFull, m[r], o), __shfl_xor_sync(kFull, l[r], o));
        if (lane == 0) warp_part[warp][r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    if (threadIdx.x < kRows && r0 + threadIdx.x < rows) {
        float2 x = warp_part[0][threadIdx.x];
        for (int w = 1; w < kTile / 32; ++w) merge(x.x, x.y, warp_part[w][threadIdx.x].x, warp_part[w][threadIdx.x].y);
        a.part[((static_cast<int64_t>(b) * a.H + h) * a.R + r0 + threadIdx.x) * a.chunks + chunk] = x;
    }
}

// L_r of every row: a warp each.
__global__ void __launch_bounds__(256) k_score_merge(const __grid_constant__ ScoreArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
    if (row >= static_cast<int64_t>(a.B) * a.H * a.R) return;
    const int b = static_cast<int>(row / (static_cast<int64_t>(a.H) * a.R)), r = static_cast<int>(row % a.R);
    const Span sp = span_of(a, b);
    if (!sp.ok || r >= (sp.end - sp.begin) * a.G) return;
    const int n = (sp.end + a.chunk - 1) / a.chunk;
    float m = -INFINITY, l = 0.f;
    for (int c = lane; c < n; c += 32) {
        const float2 x = __ldcg(a.part + row * a.chunks + c);
        merge(m, l, x.x, x.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) merge(m, l, __shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, l, o));
    if (lane == 0) a.lse[row] = m + log2f(l);
}

// The weights: grid (tile of slots, head, request).
template <class Tag>
__global__ void __launch_bounds__(kTile) k_score_apply(const __grid_constant__ ScoreArgs a)
{
    extern __shared__ __align__(16) float smem[];
    float *sq = smem, *sk = smem + kRows * a.D;
    __shared__ float lse[kRows];
    const int b = blockIdx.z, h = blockIdx.y, t0 = static_cast<int>(blockIdx.x) * kTile;
    const Span sp = span_of(a, b);
    if (!sp.ok) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0 && a.status) atomicOr(a.status, SPEC_STATUS_CAPACITY);
        return;
    }
    if (t0 >= sp.end) return;
    const int rows = (sp.end - sp.begin) * a.G;
    const int t = t0 + threadIdx.x;
    const int64_t at = (static_cast<int64_t>(b) * a.H + h) * a.C + t;
    float sum = 0.f;
    stage_slots<Tag>(a, b, h, t0, sp.end, sk);
    for (int r0 = 0; r0 < rows; r0 += kRows) {
        __syncthreads();
        stage_rows<Tag>(a, b, h, r0, rows, sq);
        if (threadIdx.x < kRows)
            lse[threadIdx.x] = r0 + threadIdx.x < rows
                                   ? __ldcg(a.lse + (static_cast<int64_t>(b) * a.H + h) * a.R + r0 + threadIdx.x)
                                   : 0.f;
        __syncthreads();
        float s[kRows];
        products(sq, sk, a.D, s);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (r0 + r < rows && t <= sp.begin + (r0 + r) / a.G) sum += exp2f(s[r] - lse[r]);
    }
    if (t < sp.end) a.out[at] = (t < sp.begin ? a.in[at] : 0.f) + sum;
}

constexpr size_t kScoreAlign = 256;
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t align_up(size_t x) { return (x + kScoreAlign - 1) / kScoreAlign * kScoreAlign; }

// Slots per chunk: at most kChunksMax chunks, whole tiles.
int chunk_slots(int C) { return static_cast<int>(ceil_div(ceil_div(C, kChunksMax), kTile) * kTile); }

struct ScoreLayout {
    size_t part, lse, total;
};
bool score_layout(int B, int Q, int Hq, int H, int C, ScoreLayout &L)
{
    if (B < 0 || Q < 1 || H < 1 || Hq < H || Hq % H != 0 || C < 1) return false;
    const size_t rows = static_cast<size_t>(B) * Hq * Q;
    L.part = 0;
    L.lse = align_up(sizeof(float2) * rows * ceil_div(C, chunk_slots(C)));
    L.total = std::max(kScoreAlign, L.lse + align_up(sizeof(float) * rows));
    return true;
}

std::mutex g_score_mu;
bool g_score_attr[64][2];

template <class Tag>
int launch_score(const ScoreArgs &a, int dtype_index, cudaStream_t st)
{
    const size_t smem = sizeof(float) * (static_cast<size_t>(kRows) * a.D + static_cast<size_t>(kTile) * (a.D + 4));
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ECUDA;
    {
        std::lock_guard<std::mutex> lock(g_score_mu);
        if (!g_score_attr[dev][dtype_index]) {
            const int most = static_cast<int>(sizeof(float) * (kRows * SPEC_MAX_HEAD_DIM + kTile * (SPEC_MAX_HEAD_DIM + 4)));
            if (cudaFuncSetAttribute(k_score_stats<Tag>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
                cudaFuncSetAttribute(k_score_apply<Tag>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
                return SPEC_ECUDA;
            g_score_attr[dev][dtype_index] = true;
        }
    }
    const unsigned H = static_cast<unsigned>(a.H), B = static_cast<unsigned>(a.B);
    const unsigned tiles = static_cast<unsigned>(ceil_div(a.R, kRows) * a.chunks);
    k_score_stats<Tag><<<dim3(tiles, H, B), kTile, smem, st>>>(a);
    k_score_merge<<<static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.B) * a.H * a.R, 8)), 256, 0, st>>>(a);
    k_score_apply<Tag><<<dim3(static_cast<unsigned>(ceil_div(a.C, kTile)), H, B), kTile, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_score_workspace_size(int batch, int queries, int q_heads, int kv_heads, int capacity)
{
    ScoreLayout L;
    return score_layout(batch, queries, q_heads, kv_heads, capacity, L) ? L.total : 0;
}

extern "C" int spec_cache_score(const void *q, const void *k, spec_dtype_t dtype, int64_t q_request_stride,
                                int64_t q_token_stride, int64_t q_head_stride, int64_t k_request_stride,
                                int64_t k_head_stride, int64_t k_slot_stride, const int32_t *begin,
                                const int32_t *end, int batch, int queries, int q_heads, int kv_heads,
                                int head_dim, int capacity, float scale, const float *scores,
                                float *out_scores, int32_t *status, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream)
{
    if (batch < 0 || queries < 1 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 ||
        head_dim < 1 || capacity < 1)
        return SPEC_EINVAL;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EINVAL;
    if (!std::isfinite(scale)) return SPEC_EINVAL;
    const int vec = dtype == SPEC_BF16 ? 8 : 4;
    if (head_dim % vec != 0) return SPEC_EALIGN;
    if (head_dim < 8 || head_dim > SPEC_MAX_HEAD_DIM || batch > 65535 || kv_heads > 65535 ||
        static_cast<int64_t>(queries) * (q_heads / kv_heads) > 65535 || capacity > (1 << 30) ||
        static_cast<int64_t>(batch) * queries * q_heads > INT_MAX)
        return SPEC_EUNSUPPORTED;
    const int64_t strides[6] = {q_request_stride, q_token_stride, q_head_stride,
                                k_request_stride, k_head_stride, k_slot_stride};
    for (int64_t s : strides) {
        if (s < 0) return SPEC_EINVAL;
        if (s % vec != 0) return SPEC_EALIGN;
        if (s > (int64_t(1) << 40)) return SPEC_EUNSUPPORTED;
    }
    if (batch == 0) return SPEC_OK;
    if (!q || !k || !begin || !end || !scores || !out_scores) return SPEC_EINVAL;
    if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k)) & 15u) != 0) return SPEC_EALIGN;
    ScoreLayout L;
    if (!score_layout(batch, queries, q_heads, kv_heads, capacity, L)) return SPEC_EINVAL;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kScoreAlign) != 0 || workspace_bytes < L.total)
        return SPEC_EWORKSPACE;
    ScoreArgs a;
    std::memset(&a, 0, sizeof a);
    a.q = q;
    a.k = k;
    a.q_req = q_request_stride;
    a.q_tok = q_token_stride;
    a.q_head = q_head_stride;
    a.k_req = k_request_stride;
    a.k_head = k_head_stride;
    a.k_slot = k_slot_stride;
    a.begin = begin;
    a.end = end;
    a.B = batch;
    a.Q = queries;
    a.H = kv_heads;
    a.G = q_heads / kv_heads;
    a.D = head_dim;
    a.C = capacity;
    a.R = a.Q * a.G;
    a.chunk = chunk_slots(capacity);
    a.chunks = static_cast<int>(ceil_div(capacity, a.chunk));
    a.scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    a.in = scores;
    a.out = out_scores;
    a.status = status;
    a.part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + L.part);
    a.lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + L.lse);
    return dtype == SPEC_BF16 ? launch_score<Bf16>(a, 1, stream) : launch_score<F32>(a, 0, stream);
}
