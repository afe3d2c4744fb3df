// weight.cu -- spec_cache_score: the attention weight that a step's queries
// give the slots of a cache, added up per key head and slot.
//
// Mathematics.  With s_rt = scale q_r . k_t over the rows r = (query i,
// head g of the group), slot t gains sum_r exp(s_rt - m_r) / l_r where m_r is
// the row's maximum over the slots it sees (t <= begin + i) and l_r the sum of
// exp(s_rt - m_r).  They need every slot of the row before the first weight can
// be formed.  They stay two numbers: m + ln l as one would be rounded to a step
// of its size, and every weight of the row off by as much (2.6e-6 for products
// of 44 to 88).  Everything is in units of log2 (scale log2 e multiplies the
// products), sums and statistics in fp32.
//
// Bounds: the keys' bytes while rows are few, the tensor cores and the
// exponentials (one a row and slot in either sweep) when they are many.
//
// Two forms.  Few rows (decoding): the keys are read once, their products
// stored and added up by a second kernel.  Many rows (a prompt's last
// queries): two sweeps over the keys that keep everything in registers.  Both
// spread a head's slots over the whole GPU and merge the chunks' (max, sum)
// per row in between.
//
// Products run on mma.sync m16n8k16 with 16 rows as A and 8 slots as B.  The
// sum over d may run in any order, so a lane's 16 contiguous bytes (8
// elements) of a key serve as its two k-steps' elements, straight from global
// memory as B fragments (two registers that follow one another); the queries
// are laid out in shared memory so that one 16-byte load is an A fragment.
// (With the slots as A every product needed four register moves.)  fp32
// inputs are split into three bf16 parts (24 bits in all) and the six
// products above 2^-24 are added up.
//
// A slot's weights are summed by one thread in row order and the parts are
// merged in a fixed order, so results do not depend on the schedule.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/specverify.h"
#include "sv_common.cuh"

namespace sv {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kPartSlots = 128;     // the shortest chunk of slots: 16 a warp

struct ScoreArgs {
    const void *q, *k;
    int64_t q_req, q_tok, q_head, k_req, k_head, k_slot;  // elements
    const int32_t *begin, *end;
    int B, Q, H, G, D, C;  // H key heads, C capacity
    int R;                 // Q * G
    int part, chunks;      // slots of a chunk of the statistics, chunks
    float scale2;          // scale * log2(e)
    const float *in;
    float *out;
    int32_t *status;
    int slots;             // slots of a block (weights), of a warp's stage (statistics)
    float2 *stats;         // [B][H][R][chunks]
    float2 *norm;          // many rows: -m, 1 / l [B][H][R]
    int pitch;             // few rows: words between rows of products
    int head0;             // few rows: the launch's first head (of B * H)
    float *held;           // few rows: products [heads of the launch][R][pitch]; so are stats
};

// Filled slots and queries of request b; !ok: left as it was.
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

// (m, 1 / l) of a row as its weights take them.  A row whose products are all
// -inf weighs nothing anywhere: (0, 0); l is at least 1 otherwise, or NaN.
__device__ __forceinline__ float2 norm_of(float m, float l)
{
    return l == 0.f ? make_float2(0.f, 0.f) : make_float2(m, 1.f / l);
}

// Where a running maximum starts: below it there is only -inf, which then
// weighs 2^-inf without a case of its own.
constexpr float kNoMax = -FLT_MAX;

// Merge (m, l) pairs, l relative to 2^m; an empty pair is (-inf or kNoMax, 0).
__device__ __forceinline__ void merge(float &m, float &l, float om, float ol)
{
    const float n = max_nan(m, om);
    if (n == -INFINITY) return;
    l = l * ex2_approx(m - n) + ol * ex2_approx(om - n);
    m = n;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero accumulator.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%10,%10,%10,%10};\n"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ unsigned long long f2_ex2(unsigned long long x)
{
    float lo, hi;
    f2_unpack(x, lo, hi);
    return f2_pack(ex2_approx(lo), ex2_approx(hi));
}

// Eight elements of a vector as bf16 pairs: themselves, or the three parts
// of fp32 values (x = p0 + p1 + p2 to 24 bits, each difference exact).
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <class Tag>
struct Parts;
template <>
struct Parts<Bf16> {
    static constexpr int kRaw = 1;   // uint4 of raw data per 8 elements
    static constexpr int kParts = 1;
    static __device__ __forceinline__ void split(const uint4 (&raw)[1], uint4 (&p)[1]) { p[0] = raw[0]; }
};
template <>
struct Parts<F32> {
    static constexpr int kRaw = 2;
    static constexpr int kParts = 3;
    static __device__ __forceinline__ void split(const uint4 (&raw)[2], uint4 (&p)[3])
    {
        float x[8] = {__uint_as_float(raw[0].x), __uint_as_float(raw[0].y), __uint_as_float(raw[0].z),
                      __uint_as_float(raw[0].w), __uint_as_float(raw[1].x), __uint_as_float(raw[1].y),
                      __uint_as_float(raw[1].z), __uint_as_float(raw[1].w)};
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = pack2(x[2 * e], x[2 * e + 1]);
                x[2 * e] -= bf16_lo(w[e]);
                x[2 * e + 1] -= bf16_hi(w[e]);
            }
            p[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// Elements d .. d + 7 of a row of D elements (zeros past D).
template <class Tag>
__device__ __forceinline__ void load8(const typename Tag::elem *row, int d, int D, uint4 (&raw)[Parts<Tag>::kRaw])
{
#pragma unroll
    for (int i = 0; i < Parts<Tag>::kRaw; ++i) {
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (d + i * Tag::kVec < D) raw[i] = ldg_vec(row + d + i * Tag::kVec);
    }
}

// A warp's 16 slots: lane (g = lane / 4, t = lane % 4) holds elements
// 32 j + 8 t .. + 7 of slots g and g + 8.  Up to 128 bf16 elements are held
// in registers, loaded ahead of use (kHeld); longer or fp32 rows, which would
// not fit beside the accumulators, are read where they are used, from L1
// after the first group of rows.
template <class Tag, int NB>
struct Slots {
    static constexpr bool kHeld = Parts<Tag>::kParts == 1 && NB <= 4;
    uint4 raw[kHeld ? NB : 1][2][Parts<Tag>::kRaw];
    const typename Tag::elem *row[2];
    int width[2];  // D, or 0 past the last slot
    __device__ __forceinline__ void load(const ScoreArgs &a, const typename Tag::elem *keys, int t0, int end)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int slot = t0 + (lane >> 2) + 8 * half;
            row[half] = keys + slot * a.k_slot;
            width[half] = slot < end ? a.D : 0;
            if (kHeld) {
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    load8<Tag>(row[half], 32 * j + 8 * (lane & 3), width[half], raw[kHeld ? j : 0][half]);
            }
        }
    }
    __device__ __forceinline__ void part(int j, int half, uint4 (&p)[Parts<Tag>::kParts]) const
    {
        if (kHeld) {
            Parts<Tag>::split(raw[kHeld ? j : 0][half], p);
        } else {
            uint4 x[Parts<Tag>::kRaw];
            load8<Tag>(row[half], 32 * j + 8 * (threadIdx.x & 3), width[half], x);
            Parts<Tag>::split(x, p);
        }
    }
};

// Rows [r0, r0 + 16 * tiles) of head h below `rows` as A fragments: 1024 bytes
// per (16 rows, 32 elements, part), 512 a k-step, a lane's 16 bytes in place.
// Past `rows` the last row comes again: zeros would make NaN of an infinite
// key, where the last row, which sees every slot, makes what its weights show.
template <class Tag>
__device__ __forceinline__ void stage_rows(const ScoreArgs &a, int b, int h, int r0, int rows, int tiles, int nb, uint4 *sq)
{
    constexpr int kP = Parts<Tag>::kParts;
    constexpr int kBatch = 2;  // four loads in flight a thread
    const int threads = blockDim.x;
    for (int i0 = threadIdx.x; i0 < tiles * nb * 32; i0 += kBatch * threads) {
        uint4 raw[kBatch][2][Parts<Tag>::kRaw];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const int i = i0 + x * threads, lane = i & 31, j = (i >> 5) % nb, tile = (i >> 5) / nb;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = min(r0 + tile * 16 + (lane >> 2) + 8 * half, rows - 1), q = r / a.G, g = r - q * a.G;
                const auto *row = static_cast<const typename Tag::elem *>(a.q) + b * a.q_req + q * a.q_tok +
                                  (static_cast<int64_t>(h) * a.G + g) * a.q_head;
                load8<Tag>(row, tile < tiles ? 32 * j + 8 * (lane & 3) : a.D, a.D, raw[x][half]);
            }
        }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const int i = i0 + x * threads;
            uint4 u[kP], v[kP];
            Parts<Tag>::split(raw[x][0], u);
            Parts<Tag>::split(raw[x][1], v);
            if (i < tiles * nb * 32)
#pragma unroll
                for (int y = 0; y < kP; ++y) {
                    uint4 *to = sq + ((i >> 5) * kP + y) * 64 + (i & 31);
                    to[0] = make_uint4(u[y].x, v[y].x, u[y].y, v[y].y);
                    to[32] = make_uint4(u[y].z, v[y].z, u[y].w, v[y].w);
                }
        }
    }
}

// ------------------------------------------------- fp32 numbers past bf16's range
// The parts of an fp32 number that is infinite, or above bf16's largest, are
// infinities of both signs, so its products come out as NaN; and so do sums
// that pass fp32's range in one part before another.  A row's statistics and
// a slot's weights are NaN then, and are formed once more from products in
// plain fp32: a number where there is one, and NaN if it stays.  (One check a
// row and chunk and one a slot: checking every product cost the sweeps 10 %.
// bf16 products are what they are.)
template <class Tag>
constexpr bool kSplit = (Parts<Tag>::kParts > 1);

// Row `row` (a query and head of the group) times slot `slot`, in units of log2.
template <class Tag>
__device__ __forceinline__ float plain_product(const ScoreArgs &a, int b, int h, int row, int slot)
{
    const int n = row / a.G;
    const auto *q = static_cast<const typename Tag::elem *>(a.q) + b * a.q_req + n * a.q_tok +
                    (static_cast<int64_t>(h) * a.G + row - n * a.G) * a.q_head;
    const auto *k = static_cast<const typename Tag::elem *>(a.k) + b * a.k_req + h * a.k_head + slot * a.k_slot;
    float sum = 0.f;
#pragma unroll 4
    for (int d = 0; d < a.D; ++d) sum = fmaf(__ldg(q + d), __ldg(k + d), sum);
    return __fmul_rn(sum, a.scale2);
}

// (max, sum) of a row over slots [t0, t1), one warp.  `held`: the row's stored
// products, of which those that are NaN are formed and stored again.
template <class Tag>
__device__ __noinline__ float2 plain_row(const ScoreArgs &a, int b, int h, int row, int t0, int t1, float *held)
{
    float m = kNoMax, l = 0.f;
#pragma unroll 1
    for (int t = t0 + static_cast<int>(threadIdx.x & 31); t < t1; t += 32) {
        float x = held ? held[t] : NAN;
        if (x != x) {
            x = plain_product<Tag>(a, b, h, row, t);
            if (held) held[t] = x;
        }
        if (x > m) {
            l *= ex2_approx(m - x);
            m = x;
        }
        l += ex2_approx(x - m);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float om = __shfl_xor_sync(kFull, m, o), ol = __shfl_xor_sync(kFull, l, o);
        merge(m, l, om, ol);
    }
    return make_float2(m, l);
}

// What rows [r0, r0 + nr) give a slot, from row `first` on; `norm` as k_score_slots holds it.
template <class Tag>
__device__ __noinline__ float plain_slot(const ScoreArgs &a, int b, int h, int r0, int first, int nr, int slot, const float2 *norm)
{
    float sum = 0.f;
#pragma unroll 1
    for (int r = first; r < nr; ++r)
        sum = fmaf(ex2_approx(plain_product<Tag>(a, b, h, r0 + r, slot) + norm[r].x), norm[r].y, sum);
    return sum;
}

// The products of a warp's 16 slots with the 16-row tiles [tile0, tile0 + MT):
// c[i][half] holds slots 8 half + 2 t, + 1 of rows g ([0], [1]) and g + 8.
template <class Tag, int NB, int MT>
__device__ __forceinline__ void products(const Slots<Tag, NB> &k, const uint4 *sq, int nb, int tile0, int tiles,
                                         float (&c)[MT][2][4])
{
    constexpr int kP = Parts<Tag>::kParts;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) c[i][half][0] = c[i][half][1] = c[i][half][2] = c[i][half][3] = 0.f;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        if (j < nb) {
            uint4 y[2][kP];
            k.part(j, 0, y[0]);
            k.part(j, 1, y[1]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if (tile0 + i < tiles) {
                    uint4 lo[kP], hi[kP];
#pragma unroll
                    for (int x = 0; x < kP; ++x) {
                        const uint4 *at = sq + (((tile0 + i) * nb + j) * kP + x) * 64 + lane;
                        lo[x] = at[0];
                        hi[x] = at[32];
                    }
                    // the smaller products first
#pragma unroll
                    for (int s = kP - 1; s >= 0; --s)
#pragma unroll
                        for (int x = s; x >= 0; --x)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint4 w = y[half][s - x];
                                mma_bf16(c[i][half], lo[x].x, lo[x].y, lo[x].z, lo[x].w, w.x, w.y);
                                mma_bf16(c[i][half], hi[x].x, hi[x].y, hi[x].z, hi[x].w, w.z, w.w);
                            }
                }
            }
        }
    }
}

// ------------------------------------------------------------------ few rows
// Decoding and small verifications: reading the keys bounds the step, so they
// are read once.  k_score_few forms the products, stores them and the
// statistics of its chunk; k_score_sum merges the statistics and adds up the
// weights from the stored products.  No cluster, no wait: a head of any length
// spreads over the whole GPU.  (32 requests of 2050 to 4096 slots, 8 heads of
// 4 rows, D = 128 bf16, 203 MB of keys: 46 us, 4.4 TB/s; of these the keys'
// read takes about 36 and its start and the second kernel the rest.)
constexpr int kFewRows = 32;

// Products and statistics of one chunk of slots: grid (chunk, head - head0).  A warp
// takes every eighth 16 slots of the chunk, the next ones in flight; the
// running (max, sum) of a row stays in the four lanes that hold it.
template <class Tag, int NB, int MT>
__global__ void __launch_bounds__(kScoreThreads, 2) k_score_few(const __grid_constant__ ScoreArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *sq = reinterpret_cast<uint4 *>(smem);
    __shared__ float2 stat[kScoreWarps][16 * MT];
    const int64_t kept = blockIdx.y, head = a.head0 + kept;
    const int b = static_cast<int>(head / a.H), h = static_cast<int>(head % a.H);
    const Span sp = span_of(a, b);
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int rows = (sp.end - sp.begin) * a.G;
    const int t_begin = blockIdx.x * a.part, t_end = min(sp.end, t_begin + a.part);
    if (!sp.ok || rows == 0 || t_begin >= t_end) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t2 = 2 * (lane & 3);
    const int nb = (a.D + 31) / 32, tiles = (rows + 15) / 16;
    const auto *keys = static_cast<const typename Tag::elem *>(a.k) + b * a.k_req + h * a.k_head;
    float *held = a.held + kept * a.R * a.pitch;
    float2 *stats = a.stats + kept * a.R * a.chunks + blockIdx.x;
    Slots<Tag, NB> cur, next;
    int t0 = t_begin + warp * 16;
    if (t0 < t_end) cur.load(a, keys, t0, t_end);
    stage_rows<Tag>(a, b, h, 0, rows, tiles, nb, sq);
    __syncthreads();
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) m[i][0] = m[i][1] = kNoMax, l[i][0] = l[i][1] = 0.f;
    for (; t0 < t_end; t0 += kScoreWarps * 16) {
        if (t0 + kScoreWarps * 16 < t_end) next.load(a, keys, t0 + kScoreWarps * 16, t_end);
        float c[MT][2][4];
        products<Tag, NB, MT>(cur, sq, nb, 0, tiles, c);
        const bool whole = t0 + 16 <= min(t_end, sp.begin + 1);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int low = 0; low < 2; ++low) {
                const int r = 16 * i + g + 8 * low;
                if (r < rows) {
                    float x[4];  // slots t0 + t2, + 1, + 8, + 9
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = __fmul_rn(c[i][e >> 1][2 * low + (e & 1)], a.scale2);
                    float *to = held + static_cast<int64_t>(r) * a.pitch + t0 + t2;
                    if (whole) {
                        *reinterpret_cast<float2 *>(to) = make_float2(x[0], x[1]);
                        *reinterpret_cast<float2 *>(to + 8) = make_float2(x[2], x[3]);
                    } else {
                        const int last = sp.begin + r / a.G;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int at = (e >> 1) * 8 + (e & 1), t = t0 + t2 + at;
                            if (!(t < t_end && t <= last)) x[e] = -INFINITY;
                            if (t < t_end) to[at] = x[e];
                        }
                    }
                    const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    if (top > m[i][low]) {
                        l[i][low] *= ex2_approx(m[i][low] - top);
                        m[i][low] = top;
                    }
                    const float mm = m[i][low];
                    l[i][low] += (ex2_approx(x[0] - mm) + ex2_approx(x[1] - mm)) + (ex2_approx(x[2] - mm) + ex2_approx(x[3] - mm));
                }
            }
        cur = next;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int low = 0; low < 2; ++low) {
            float mm = m[i][low], ll = l[i][low];
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const float om = __shfl_xor_sync(kFull, mm, o), ol = __shfl_xor_sync(kFull, ll, o);
                merge(mm, ll, om, ol);
                if (ol != ol) ll = ol;
            }
            if (t2 == 0) stat[warp][16 * i + g + 8 * low] = make_float2(mm, ll);
        }
    __syncthreads();
    const int r = threadIdx.x;
    bool again = false;
    if (r < rows) {
        float mm = -INFINITY, ll = 0.f;
        for (int w = 0; w < kScoreWarps; ++w) {
            const float2 y = stat[w][r];
            merge(mm, ll, y.x, y.y);
            if (y.y != y.y) ll = y.y;
        }
        again = ll != ll;
        __stcg(stats + static_cast<int64_t>(r) * a.chunks, make_float2(mm, ll));
    }
    if constexpr (kSplit<Tag>) {
        if (again) stat[0][r].y = NAN;
        if (!__syncthreads_or(again)) return;
        for (int x = warp; x < rows; x += kScoreWarps) {
            if (stat[0][x].y == stat[0][x].y) continue;
            const float2 y = plain_row<Tag>(a, b, h, x, t_begin, min(t_end, sp.begin + x / a.G + 1), held + static_cast<int64_t>(x) * a.pitch);
            if (lane == 0) __stcg(stats + static_cast<int64_t>(x) * a.chunks, y);
        }
    }
}

// The weights of kSumSlots slots: grid (slots, head - head0), four slots a thread
// (with one, four times as many blocks merge the statistics: 17 us of the
// decode call's 59 under a profiler).
constexpr int kSumSlots = 4 * kScoreThreads;

__global__ void __launch_bounds__(kScoreThreads) k_score_sum(const __grid_constant__ ScoreArgs a)
{
    __shared__ float2 norm[kFewRows];  // m, 1 / l
    const int64_t kept = blockIdx.y, head = a.head0 + kept;
    const int b = static_cast<int>(head / a.H);
    const Span sp = span_of(a, b);
    if (!sp.ok) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && head % a.H == 0 && a.status) atomicOr(a.status, SPEC_STATUS_CAPACITY);
        return;
    }
    const int rows = (sp.end - sp.begin) * a.G, t_begin = blockIdx.x * kSumSlots;
    if (t_begin >= sp.end) return;
    const int t = t_begin + 4 * threadIdx.x;
    const float *in = a.in + head * a.C;
    float *out = a.out + head * a.C;
    float sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = t + i < sp.begin ? in[t + i] : 0.f;
    const int chunks = (sp.end + a.part - 1) / a.part;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    {  // eight lanes a row merge the chunks' statistics
        const int r = threadIdx.x >> 3;
        float mm = -INFINITY, ll = 0.f;
        if (r < rows)
            for (int c = threadIdx.x & 7; c < chunks; c += 8) {
                const float2 y = __ldcg(a.stats + (kept * a.R + r) * a.chunks + c);
                merge(mm, ll, y.x, y.y);
                if (y.y != y.y) ll = y.y;
            }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            const float om = __shfl_xor_sync(kFull, mm, o), ol = __shfl_xor_sync(kFull, ll, o);
            merge(mm, ll, om, ol);
            if (ol != ol) ll = ol;
        }
        if ((threadIdx.x & 7) == 0) norm[r] = norm_of(mm, ll);
    }
    __syncthreads();
    if (t >= sp.end) return;
    // the step's weight by itself, in row order, then the old value
    const float4 *s = reinterpret_cast<const float4 *>(a.held + kept * a.R * a.pitch + t);
    const int64_t pitch = a.pitch / 4;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    if (t + 3 <= sp.begin) {  // seen by every row
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const float4 x = __ldcg(s + r * pitch);
            const float2 y = norm[r];
            w[0] = fmaf(ex2_approx(x.x - y.x), y.y, w[0]);
            w[1] = fmaf(ex2_approx(x.y - y.x), y.y, w[1]);
            w[2] = fmaf(ex2_approx(x.z - y.x), y.y, w[2]);
            w[3] = fmaf(ex2_approx(x.w - y.x), y.y, w[3]);
        }
    } else {
        for (int r = max(0, (t - sp.begin) * a.G); r < rows; ++r) {
            const float4 x = __ldcg(s + r * pitch);  // past the last slot: not used
            const float2 y = norm[r];
            const float z[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r >= (t + i - sp.begin) * a.G) w[i] = fmaf(ex2_approx(z[i] - y.x), y.y, w[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t + i < sp.end) out[t + i] = sum[i] + w[i];
}

// ------------------------------------------------------------------ many rows
// Where a key head has many rows (a prompt's last queries, a verification with
// wide groups) the products no longer fit shared memory and the exponentials
// and the tensor pipe bound the step, not the keys.  Two sweeps:
//   k_score_rows   a warp holds 16 rows as A fragments in registers, the keys
//                  stream through shared memory as B fragments for all warps; the
//                  running (max, sum) of a row stays in its four lanes (its
//                  chunks are merged by k_score_merge);
//   k_score_slots  a warp holds 32 slots as B fragments in registers, the rows
//                  are A fragments in shared memory; a slot's sum over the
//                  rows stays in the eight lanes of its column.
// tcgen05 accumulators were built and measured for this step: they would
// halve its time, but drop what falls below the running sum at each of the
// D / 16 steps, and the weights came out 6e-6 off (2-norm, against 3e-7 here)
// on peaked keys; mma.sync keeps fp32 accuracy.  (8 heads of 65536 slots, 128
// rows, D = 128 bf16: 134 us; the two sweeps keep the tensor pipe 42 % and 56 %
// busy, where mma.sync alone peaked at 555 TFLOP/s, 62 us for both.  The rest
// is the running statistics and exponentials between the products.)
// Rows of a row tile, tiles of 8 slots a warp of the weights sweep and blocks a
// SM: fp32 rows take three times a bf16 row's shared memory and fp32 slots
// twice the registers.
template <class Tag>
struct Many;
template <>
struct Many<Bf16> {
    static constexpr int kRows = 128, kBlocks = 2;
    template <int NB>
    static constexpr int kTiles = NB <= 4 ? 4 : 2;
};
template <>
struct Many<F32> {
    static constexpr int kRows = 64, kBlocks = 1;
    template <int NB>
    static constexpr int kTiles = NB <= 2 ? 4 : NB <= 4 ? 2 : 1;
};
constexpr int kRowStages = 3;

// Slots [t0, t0 + slots) below `end` as B fragments (512 bytes per 8 slots and
// 32 elements, 1024 for fp32: a lane's first and second 16 bytes apart),
// NB * 32 elements a slot, asynchronously; the rest as zeros.
template <class Tag, int NB>
__device__ __forceinline__ void copy_slots(const ScoreArgs &a, const typename Tag::elem *keys, int t0, int slots, int end,
                                           uint4 *dst)
{
    constexpr int kRaw = Parts<Tag>::kRaw, kChunks = 4 * NB * kRaw;
    for (int i = threadIdx.x; i < slots * kChunks; i += blockDim.x) {
        const int slot = i / kChunks, c = i % kChunks;
        const bool in = t0 + slot < end && c * Tag::kVec < a.D;
        const auto *from = in ? keys + (t0 + slot) * a.k_slot + c * Tag::kVec : keys;
        uint4 *to = dst + ((slot >> 3) * NB + c / (4 * kRaw)) * 32 * kRaw + c % kRaw * 32 + (slot & 7) * 4 + c / kRaw % 4;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                     "l"(from), "r"(in ? 16 : 0)
                     : "memory");
    }
}

// c += the products of a row tile's parts (two k-steps lo, hi) with 8 slots'
// parts, the smaller ones first; FIRST: c = for bf16.
template <class Tag, bool FIRST>
__device__ __forceinline__ void tile_products(float (&c)[4], const uint4 (&lo)[Parts<Tag>::kParts],
                                              const uint4 (&hi)[Parts<Tag>::kParts], const uint4 (&w)[Parts<Tag>::kParts])
{
    constexpr int kP = Parts<Tag>::kParts;
    if (FIRST && kP > 1) c[0] = c[1] = c[2] = c[3] = 0.f;
#pragma unroll
    for (int s = kP - 1; s >= 0; --s)
#pragma unroll
        for (int x = s; x >= 0; --x) {
            const uint4 u = lo[x], v = hi[x], y = w[s - x];
            if (FIRST && kP == 1) mma_bf16_first(c, u.x, u.y, u.z, u.w, y.x, y.y);
            else mma_bf16(c, u.x, u.y, u.z, u.w, y.x, y.y);
            mma_bf16(c, v.x, v.y, v.z, v.w, y.z, y.w);
        }
}

// Statistics of the rows of one tile over one chunk of slots: grid (chunk,
// row tile, request and head).
template <class Tag, int NB>
__global__ void __launch_bounds__(kScoreThreads, Many<Tag>::kBlocks) k_score_rows(const __grid_constant__ ScoreArgs a)
{
    constexpr int kP = Parts<Tag>::kParts, kRaw = Parts<Tag>::kRaw, kRows = Many<Tag>::kRows;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *ring = reinterpret_cast<uint4 *>(smem);
    __shared__ float2 stat[kScoreWarps][16];
    const int64_t head = blockIdx.z;
    const int b = static_cast<int>(head / a.H), h = static_cast<int>(head % a.H);
    const Span sp = span_of(a, b);
    const int rows = (sp.end - sp.begin) * a.G, r0 = blockIdx.y * kRows;
    const int t_begin = blockIdx.x * a.part, t_end = min(sp.end, t_begin + a.part);
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (!sp.ok || r0 >= rows || t_begin >= t_end) return;
    const int nr = min(rows - r0, kRows);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int wr = (min(a.R, kRows) + 15) / 16;  // warps over the rows
    const int groups = (blockDim.x >> 5) / wr;   // groups of them over the slots
    const int row_slots = a.slots;               // of a stage, for each group
    const int rw = (warp % wr) * 16, sg = warp / wr;
    const auto *keys = static_cast<const typename Tag::elem *>(a.k) + b * a.k_req + h * a.k_head;
    const int stage_slots = row_slots * groups, stage = stage_slots / 8 * NB * 32 * kRaw;  // uint4
    const int stages = (t_end - t_begin + stage_slots - 1) / stage_slots;
    // This warp's rows: lane (g, t) holds rows g and g + 8.  bf16: in
    // registers, by way of the ring; fp32: read from behind the ring.
    uint4 *sq = kP == 1 ? ring : ring + kRowStages * stage;
    stage_rows<Tag>(a, b, h, r0, rows, (nr + 15) / 16, NB, sq);
    __syncthreads();
    const uint4 *own = sq + rw / 16 * NB * kP * 64 + lane;  // (j * kP + part) * 64 + 32 * k-step
    uint4 q[kP == 1 ? NB : 1][2];
    int last[2];  // the last slot a row sees
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        last[half] = sp.begin + (r0 + rw + g + 8 * half) / a.G;
        if (kP == 1) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
                q[kP == 1 ? j : 0][half] = rw < nr ? own[j * 64 + half * 32] : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (kP == 1) __syncthreads();
    for (int s = 0; s < kRowStages - 1; ++s) {
        if (s < stages) copy_slots<Tag, NB>(a, keys, t_begin + s * stage_slots, stage_slots, t_end, ring + s * stage);
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    float m[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f};  // of this lane's columns, m in units of log2
    const float sc = a.scale2;

    // 32 slots from t0 on, as fragments at `tile`; `whole`: seen by every row
    auto step = [&](const uint4 *tile, int t0, auto whole) {
        float c[4][4];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            uint4 u[kP], v[kP];
#pragma unroll
            for (int x = 0; x < kP; ++x) {
                u[x] = kP == 1 ? q[kP == 1 ? j : 0][0] : own[(j * kP + x) * 64];
                v[x] = kP == 1 ? q[kP == 1 ? j : 0][1] : own[(j * kP + x) * 64 + 32];
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                uint4 raw[kRaw], w[kP];
#pragma unroll
                for (int x = 0; x < kRaw; ++x) raw[x] = tile[((n * NB + j) * kRaw + x) * 32];
                Parts<Tag>::split(raw, w);
                if (j == 0) tile_products<Tag, true>(c[n], u, v, w);
                else tile_products<Tag, false>(c[n], u, v, w);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // the scaled products are rounded here and in k_score_slots
            // alike: fused, they would differ from m's by half a step of s
            float x[8];
#pragma unroll
            for (int n = 0; n < 4; ++n)
                x[2 * n] = __fmul_rn(c[n][2 * half], sc), x[2 * n + 1] = __fmul_rn(c[n][2 * half + 1], sc);
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int slot = t0 + (e >> 1) * 8 + 2 * t + (e & 1);
                    if (!(slot < t_end && slot <= last[half])) x[e] = -INFINITY;
                }
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
            if (top > m[half]) {
                l[half] *= ex2_approx(m[half] - top);
                m[half] = top;
            }
            const unsigned long long nm = f2_pack(-m[half], -m[half]);
            unsigned long long e01 = f2_ex2(f2_add(f2_pack(x[0], x[1]), nm));
#pragma unroll
            for (int n = 1; n < 4; ++n) e01 = f2_add(e01, f2_ex2(f2_add(f2_pack(x[2 * n], x[2 * n + 1]), nm)));
            float e0, e1;
            f2_unpack(e01, e0, e1);
            l[half] += e0 + e1;
        }
    };
    for (int s = 0; s < stages; ++s) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kRowStages - 2) : "memory");
        __syncthreads();
        {
            const int next = s + kRowStages - 1;
            if (next < stages)
                copy_slots<Tag, NB>(a, keys, t_begin + next * stage_slots, stage_slots, t_end, ring + next % kRowStages * stage);
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        }
        const int t0 = t_begin + s * stage_slots + sg * row_slots;
        const uint4 *tile = ring + s % kRowStages * stage + sg * (row_slots / 8) * NB * 32 * kRaw + lane;
        if (rw >= nr || t0 >= t_end) continue;
        if (t0 + row_slots <= min(t_end, sp.begin + 1)) {
#pragma unroll 1
            for (int n0 = 0; n0 < row_slots; n0 += 32) step(tile + n0 / 8 * NB * 32 * kRaw, t0 + n0, std::true_type{});
        } else {
#pragma unroll 1
            for (int n0 = 0; n0 < row_slots; n0 += 32) step(tile + n0 / 8 * NB * 32 * kRaw, t0 + n0, std::false_type{});
        }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float mm = m[half], ll = l[half];
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            const float om = __shfl_xor_sync(kFull, mm, o), ol = __shfl_xor_sync(kFull, ll, o);
            merge(mm, ll, om, ol);
            if (ol != ol) ll = ol;
        }
        if (t == 0) stat[warp][g + 8 * half] = make_float2(mm, ll);
    }
    __syncthreads();
    bool again = false;
    for (int r = threadIdx.x; r < nr; r += blockDim.x) {
        float mm = -INFINITY, ll = 0.f;
        for (int x = 0; x < groups; ++x) {
            const float2 y = stat[x * wr + r / 16][r % 16];
            merge(mm, ll, y.x, y.y);
            if (y.y != y.y) ll = y.y;
        }
        if (kSplit<Tag> && ll != ll) {
            again = true;
            stat[r / 16][r % 16].y = NAN;
        }
        __stcg(a.stats + (head * a.R + r0 + r) * a.chunks + blockIdx.x, make_float2(mm, ll));
    }
    if constexpr (kSplit<Tag>) {
        if (!__syncthreads_or(again)) return;
        for (int x = warp; x < nr; x += blockDim.x >> 5) {
            if (stat[x / 16][x % 16].y == stat[x / 16][x % 16].y) continue;
            const float2 y = plain_row<Tag>(a, b, h, r0 + x, t_begin, min(t_end, sp.begin + (r0 + x) / a.G + 1), nullptr);
            if (lane == 0) __stcg(a.stats + (head * a.R + r0 + x) * a.chunks + blockIdx.x, y);
        }
    }
}

// -m and 1 / l of every row from its chunks' statistics: a warp a row (6 us
// cold, of which the launch hides all but the chain of reads).
__global__ void __launch_bounds__(kScoreThreads) k_score_merge(const __grid_constant__ ScoreArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * kScoreThreads + threadIdx.x) >> 5;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (row >= static_cast<int64_t>(a.B) * a.H * a.R) return;
    const Span sp = span_of(a, static_cast<int>(row / (static_cast<int64_t>(a.H) * a.R)));
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (!sp.ok || row % a.R >= (sp.end - sp.begin) * a.G) return;
    const int chunks = (sp.end + a.part - 1) / a.part;
    float m = -INFINITY, l = 0.f;
#pragma unroll 2
    for (int c = lane; c < chunks; c += 32) {
        const float2 y = __ldcg(a.stats + row * a.chunks + c);
        merge(m, l, y.x, y.y);
        if (y.y != y.y) l = y.y;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float om = __shfl_xor_sync(kFull, m, o), ol = __shfl_xor_sync(kFull, l, o);
        merge(m, l, om, ol);
        if (ol != ol) l = ol;
    }
    const float2 norm = norm_of(m, l);
    if (lane == 0) __stcg(a.norm + row, make_float2(-norm.x, norm.y));
}

// The weights of one chunk of slots: grid (chunk, request and head).
template <class Tag, int NB>
__global__ void __launch_bounds__(kScoreThreads, Many<Tag>::kBlocks) k_score_slots(const __grid_constant__ ScoreArgs a)
{
    constexpr int kP = Parts<Tag>::kParts, kRaw = Parts<Tag>::kRaw, kRows = Many<Tag>::kRows;
    constexpr int kN = Many<Tag>::template kTiles<NB>;  // tiles of 8 slots a warp
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *sq = reinterpret_cast<uint4 *>(smem);
    __shared__ float2 norm[kRows];
    const int64_t head = blockIdx.y;
    const int b = static_cast<int>(head / a.H), h = static_cast<int>(head % a.H);
    const Span sp = span_of(a, b);
    if (!sp.ok) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0 && a.status) atomicOr(a.status, SPEC_STATUS_CAPACITY);
        return;
    }
    const int rows = (sp.end - sp.begin) * a.G;
    const int t_begin = blockIdx.x * a.slots, t_end = min(sp.end, t_begin + a.slots);
    if (t_begin >= t_end) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const auto *keys = static_cast<const typename Tag::elem *>(a.k) + b * a.k_req + h * a.k_head;
    const float *in = a.in + head * a.C;
    float *out = a.out + head * a.C;
    const float sc = a.scale2;
    for (int r0 = 0; r0 < max(rows, 1); r0 += kRows) {
        const int nr = min(rows - r0, kRows), tiles = (nr + 15) / 16;
        __syncthreads();
        stage_rows<Tag>(a, b, h, r0, rows, tiles, NB, sq);
        if (r0 == 0) asm volatile("griddepcontrol.wait;\n" ::: "memory");
        // a row that is none weighs nothing
        for (int r = threadIdx.x; r < tiles * 16; r += kScoreThreads) {
            norm[r] = __ldcg(a.norm + head * a.R + r0 + min(r, nr - 1));
            if (r >= nr) norm[r].y = 0.f;
        }
        __syncthreads();
        for (int t0 = t_begin + warp * 8 * kN; t0 < t_end; t0 += kScoreWarps * 8 * kN) {
            uint4 k[kN][NB][kRaw];  // lane (g, t): elements 32 j + 8 t .. + 7 of slot g of each 8
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const int slot = t0 + 8 * n + g;
                const auto *row = keys + slot * a.k_slot;
#pragma unroll
                for (int j = 0; j < NB; ++j) load8<Tag>(row, slot < t_end ? 32 * j + 8 * t : a.D, a.D, k[n][j]);
            }
            // lane (g, t) writes slots 2 t, 2 t + 1 of tile g
            const int mine = t0 + 8 * g + 2 * t;
            float old[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                old[e] = g >= kN || mine + e >= t_end ? 0.f : r0 > 0 ? out[mine + e] : mine + e < sp.begin ? in[mine + e] : 0.f;
            unsigned long long sum[kN];  // slots 2 t, 2 t + 1 of each tile, this lane's rows
#pragma unroll
            for (int n = 0; n < kN; ++n) sum[n] = f2_pack(0.f, 0.f);
            // rows 16 x .. 16 x + 15; `whole`: the slots are seen by every row
            auto step = [&](int x, auto whole) {
                float c[kN][4];
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    uint4 u[kP], v[kP];
#pragma unroll
                    for (int y = 0; y < kP; ++y) {
                        u[y] = sq[((x * NB + j) * kP + y) * 64 + lane];
                        v[y] = sq[((x * NB + j) * kP + y) * 64 + 32 + lane];
                    }
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        uint4 w[kP];
                        Parts<Tag>::split(k[n][j], w);
                        if (j == 0) tile_products<Tag, true>(c[n], u, v, w);
                        else tile_products<Tag, false>(c[n], u, v, w);
                    }
                }
#pragma unroll
                for (int low = 0; low < 2; ++low) {
                    const int r = 16 * x + g + 8 * low;
                    const float2 y = norm[r];
                    const unsigned long long y2 = f2_pack(y.x, y.x), l2 = f2_pack(y.y, y.y);
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        unsigned long long z =
                            f2_add(f2_pack(__fmul_rn(c[n][2 * low], sc), __fmul_rn(c[n][2 * low + 1], sc)), y2);
                        unsigned long long f2 = l2;
                        if (!whole) {  // the first row that sees a slot; others neither weigh nor pass on a NaN
                            float z0, z1, l0 = y.y, l1 = y.y;
                            f2_unpack(z, z0, z1);
                            const int first = (t0 + 8 * n + 2 * t - sp.begin) * a.G - r0;
                            if (r < first) z0 = -INFINITY, l0 = 0.f;
                            if (r < first + a.G) z1 = -INFINITY, l1 = 0.f;
                            z = f2_pack(z0, z1);
                            f2 = f2_pack(l0, l1);
                        }
                        sum[n] = f2_fma(f2_ex2(z), f2, sum[n]);
                    }
                }
            };
            if (t0 + 8 * kN <= sp.begin + 1) {
#pragma unroll 1
                for (int x = 0; x < tiles; ++x) step(x, std::true_type{});
            } else {
#pragma unroll 1
                for (int x = 0; x < tiles; ++x) step(x, std::false_type{});
            }
            float add[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                float x0, x1;
                f2_unpack(sum[n], x0, x1);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    x0 += __shfl_xor_sync(kFull, x0, o);
                    x1 += __shfl_xor_sync(kFull, x1, o);
                }
                if (g == n) add[0] = x0, add[1] = x1;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (g < kN && mine + e < t_end) {
                    if (kSplit<Tag> && add[e] != add[e])
                        add[e] = plain_slot<Tag>(a, b, h, r0, max(0, (mine + e - sp.begin) * a.G - r0), nr, mine + e, norm);
                    out[mine + e] = old[e] + add[e];
                }
        }
    }
}

constexpr size_t kScoreAlign = 256;
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t align_up(size_t x) { return (x + kScoreAlign - 1) / kScoreAlign * kScoreAlign; }

std::mutex g_score_mu;
// Few rows, for the form that stores its products: while that moves no more
// (8 bytes a product, there and back) than a second read of the keys.  (bf16,
// stored / swept twice, us.  512 K slots in 32 heads, D = 64, 128, 256: R = 16
// 26 / 36, 34 / 63, 70 / 152; R = 32 36 / 44, 46 / 68, 83 / 135.)  The second
// kernel merges every chunk's statistics in each of its blocks, which tells with
// rows and with long heads where the slots are few: below a quarter million
// half as many rows pay.  (64 K slots, R = 16: D = 64 9.9 / 10.6 in 32 heads, 12.1 /
// 10.5 in 8, 17.2 / 11.8 in one; D = 128 11.0 / 13.7, 13.1 / 14.2, 18.1 / 15.3.  R =
// 32, D = 128: 14.9 / 15.9, 18.7 / 15.6, 23.9 / 16.9; D = 256 22.4 / 25.1, 26.5 /
// 25.1, 31.3 / 26.4.)  In fp32 the products cost six times as much and are not
// formed twice (128 K slots: R = 32, D = 128 45 / 85 us).
bool few_rows(bool f32, int R, int D, int64_t slots)
{
    if (f32) return R <= kFewRows && 2 * R <= D;
    return slots >= 1 << 18 ? R <= kFewRows && 4 * R <= D : R <= 16 && 8 * R <= D;
}

// What the stored products may take: the heads go in groups that fit, and the
// next group's products overwrite the last one's.  (Two groups / one, D = 128
// bf16: 128 heads of 262144 slots, 4 rows 1372 / 1325 us; 64 of 131072, 16 rows
// 397 / 390; 64 of 65536, 32 rows 266 / 266.  Swept twice the keys would be read
// once more.)
constexpr size_t kHeldMost = size_t(256) << 20;

struct FewPlan {
    int heads;  // of a group; 0: not even one fits
    int part, chunks, pitch;
    size_t stats_bytes, held_bytes;
};
// Chunks of up to 1024 slots, halved while that leaves less than four blocks
// a SM.
FewPlan few_plan(int B, int H, int R, int C)
{
    FewPlan p;
    const int64_t pitch = ceil_div(C, 32) * 32;
    p.pitch = static_cast<int>(pitch);
    const size_t one = sizeof(float) * static_cast<size_t>(R) * static_cast<size_t>(pitch);
    p.heads = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(B) * H, static_cast<int64_t>(kHeldMost / one)));
    p.part = 1024;
    while (p.part > kPartSlots && p.heads * ceil_div(C, p.part) < 4 * 148) p.part /= 2;
    p.chunks = static_cast<int>(ceil_div(C, p.part));
    p.stats_bytes = align_up(sizeof(float2) * static_cast<size_t>(p.heads) * R * p.chunks);
    p.held_bytes = align_up(one * p.heads);
    return p;
}

bool g_few_attr[64][2][3][2];

template <class Tag, int NB, int MT>
int launch_few(ScoreArgs a, int group, int dtype_index, int nb_index, int mt_index, cudaStream_t st)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ECUDA;
    const int nb = (a.D + 31) / 32;
    const size_t smem = static_cast<size_t>(ceil_div(a.R, 16)) * nb * 1024 * Parts<Tag>::kParts;
    {
        std::lock_guard<std::mutex> lock(g_score_mu);
        if (!g_few_attr[dev][dtype_index][nb_index][mt_index]) {
            if (cudaFuncSetAttribute(k_score_few<Tag, NB, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     MT * NB * 1024 * Parts<Tag>::kParts) != cudaSuccess)
                return SPEC_ECUDA;
            g_few_attr[dev][dtype_index][nb_index][mt_index] = true;
        }
    }
    for (; a.head0 < a.B * a.H; a.head0 += group) {
        const unsigned heads = static_cast<unsigned>(std::min(group, a.B * a.H - a.head0));
        k_score_few<Tag, NB, MT><<<dim3(static_cast<unsigned>(a.chunks), heads), kScoreThreads, smem, st>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SPEC_ECUDA;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(a.C, kSumSlots)), heads);
        cfg.blockDim = dim3(kScoreThreads);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, k_score_sum, a) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
    }
    return SPEC_OK;
}
template <class Tag, int NB>
int launch_few(const ScoreArgs &a, int group, int dtype_index, int nb_index, cudaStream_t st)
{
    return a.R <= 16 ? launch_few<Tag, NB, 1>(a, group, dtype_index, nb_index, 0, st)
                     : launch_few<Tag, NB, 2>(a, group, dtype_index, nb_index, 1, st);
}
template <class Tag>
int launch_few(const ScoreArgs &a, int group, int dtype_index, cudaStream_t st)
{
    if (a.D <= 64) return launch_few<Tag, 2>(a, group, dtype_index, 0, st);
    if (a.D <= 128) return launch_few<Tag, 4>(a, group, dtype_index, 1, st);
    return launch_few<Tag, 8>(a, group, dtype_index, 2, st);
}

// Chunks of slots of the statistics step and slots of a block of the weights
// step: about two blocks a SM for each, in whole stages.
struct ManyPlan {
    int part, chunks, slots;
    size_t stats_bytes, norm_bytes;
};
template <class Tag>
ManyPlan many_plan(int B, int H, int R, int C)
{
    constexpr int64_t kWave = Many<Tag>::kBlocks * 148;
    ManyPlan p;
    const int64_t heads = static_cast<int64_t>(B) * H, tiles = ceil_div(R, Many<Tag>::kRows);
    const int64_t want = std::max<int64_t>(1, kWave / (heads * tiles));
    p.part = static_cast<int>(ceil_div(ceil_div(C, want), 128) * 128);
    p.chunks = static_cast<int>(ceil_div(C, p.part));
    const int64_t blocks = std::max<int64_t>(1, kWave / heads);
    p.slots = static_cast<int>(ceil_div(ceil_div(C, blocks), 256) * 256);
    p.stats_bytes = align_up(sizeof(float2) * static_cast<size_t>(heads) * R * p.chunks);
    p.norm_bytes = align_up(sizeof(float2) * static_cast<size_t>(heads) * R);
    return p;
}

bool g_many_attr[64][2][3];

template <class Tag, int NB>
int launch_many(ScoreArgs a, int dtype_index, int nb_index, cudaStream_t st)
{
    constexpr int kRows = Many<Tag>::kRows;
    constexpr size_t kFrag = static_cast<size_t>(NB) * 1024 * Parts<Tag>::kParts;  // of 16 rows
    constexpr size_t kSlotBytes = static_cast<size_t>(NB) * 64 * Parts<Tag>::kRaw;
    // bf16: two blocks a SM, the rows in registers; fp32: one, the rows behind
    // the ring
    constexpr size_t kRing = Parts<Tag>::kParts == 1 ? 110 * 1024 : 220 * 1024 - kRows / 16 * kFrag;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ECUDA;
    {
        std::lock_guard<std::mutex> lock(g_score_mu);
        if (!g_many_attr[dev][dtype_index][nb_index]) {
            if (cudaFuncSetAttribute(k_score_rows<Tag, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) !=
                    cudaSuccess ||
                cudaFuncSetAttribute(k_score_slots<Tag, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(kRows / 16 * kFrag)) != cudaSuccess)
                return SPEC_ECUDA;
            g_many_attr[dev][dtype_index][nb_index] = true;
        }
    }
    const int top = std::min(a.R, kRows);
    // warps beyond the rows' take slots of their own, as far as the ring has
    // room: 64 slots a stage each while it fits, else 32
    const int wr = static_cast<int>(ceil_div(top, 16));
    const int fit = static_cast<int>(kRing / (kRowStages * 32 * kSlotBytes));
    static_assert(kRing >= kRowStages * 32 * kSlotBytes, "one group fits");
    const int groups = std::max(1, std::min(kScoreWarps / wr, fit));
    const int row_slots = groups > fit / 2 ? 32 : 64;
    const size_t ring = static_cast<size_t>(kRowStages) * row_slots * groups * kSlotBytes +
                        (Parts<Tag>::kParts == 1 ? 0 : ceil_div(top, 16) * kFrag);
    const int slots = a.slots;
    a.slots = row_slots;
    const unsigned heads = static_cast<unsigned>(a.B * a.H);
    k_score_rows<Tag, NB><<<dim3(static_cast<unsigned>(a.chunks), static_cast<unsigned>(ceil_div(a.R, kRows)), heads),
                            32 * wr * groups, ring, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SPEC_ECUDA;
    a.slots = slots;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(heads) * a.R, kScoreWarps)));
    cfg.blockDim = dim3(kScoreThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_score_merge, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(a.C, a.slots)), heads);
    cfg.blockDim = dim3(kScoreThreads);
    cfg.dynamicSmemBytes = ceil_div(top, 16) * kFrag;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_score_slots<Tag, NB>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

template <class Tag>
int launch_many(ScoreArgs a, void *workspace, int dtype_index, cudaStream_t st)
{
    const ManyPlan p = many_plan<Tag>(a.B, a.H, a.R, a.C);
    a.part = p.part;
    a.chunks = p.chunks;
    a.slots = p.slots;
    a.norm = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + p.stats_bytes);
    if (a.D <= 64) return launch_many<Tag, 2>(a, dtype_index, 0, st);
    if (a.D <= 128) return launch_many<Tag, 4>(a, dtype_index, 1, st);
    return launch_many<Tag, 8>(a, dtype_index, 2, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

namespace {
// The form of a call and what it needs.
struct ScorePlan {
    bool few;
    FewPlan f;
    size_t bytes;
};
ScorePlan score_plan(bool f32, int D, int B, int H, int R, int C)
{
    ScorePlan p;
    p.f = few_plan(B, H, R, C);
    p.few = p.f.heads > 0 && few_rows(f32, R, D, static_cast<int64_t>(B) * H * C);
    if (p.few) {
        p.bytes = p.f.stats_bytes + p.f.held_bytes;
    } else {
        const ManyPlan m = f32 ? many_plan<F32>(B, H, R, C) : many_plan<Bf16>(B, H, R, C);
        p.bytes = m.stats_bytes + m.norm_bytes;
    }
    return p;
}

bool score_sizes(int batch, int queries, int q_heads, int kv_heads, int capacity)
{
    return batch >= 0 && queries >= 1 && kv_heads >= 1 && q_heads >= kv_heads && q_heads % kv_heads == 0 && capacity >= 1 &&
           static_cast<int64_t>(queries) * (q_heads / kv_heads) <= INT_MAX;
}
}  // namespace

extern "C" size_t spec_score_workspace_size_for(spec_dtype_t dtype, int head_dim, int batch, int queries, int q_heads,
                                                int kv_heads, int capacity)
{
    if ((dtype != SPEC_F32 && dtype != SPEC_BF16) || head_dim < 1 || !score_sizes(batch, queries, q_heads, kv_heads, capacity))
        return 0;
    return score_plan(dtype == SPEC_F32, head_dim, std::max(batch, 1), kv_heads, queries * (q_heads / kv_heads), capacity).bytes;
}

// Whichever form a type and head dimension takes: the rules turn to stored
// products as D grows, so the most is that of one of their ends.
extern "C" size_t spec_score_workspace_size(int batch, int queries, int q_heads, int kv_heads, int capacity)
{
    size_t most = 0;
    for (const spec_dtype_t dtype : {SPEC_F32, SPEC_BF16})
        for (const int dim : {8, SPEC_MAX_HEAD_DIM})
            most = std::max(most, spec_score_workspace_size_for(dtype, dim, batch, queries, q_heads, kv_heads, capacity));
    return most;
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
    const float scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    if (!std::isfinite(scale2)) return SPEC_EINVAL;
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
    const bool f32 = dtype == SPEC_F32;
    const ScorePlan plan = score_plan(f32, head_dim, batch, kv_heads, queries * (q_heads / kv_heads), capacity);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kScoreAlign) != 0 || workspace_bytes < plan.bytes)
        return SPEC_EWORKSPACE;
    if (static_cast<int64_t>(batch) * kv_heads > 65535) return SPEC_EUNSUPPORTED;
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
    a.scale2 = scale2;
    a.in = scores;
    a.out = out_scores;
    a.status = status;
    a.stats = static_cast<float2 *>(workspace);
    if (plan.few) {
        a.part = plan.f.part;
        a.chunks = plan.f.chunks;
        a.pitch = plan.f.pitch;
        a.held = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.f.stats_bytes);
        return f32 ? launch_few<F32>(a, plan.f.heads, 0, stream) : launch_few<Bf16>(a, plan.f.heads, 1, stream);
    }
    return f32 ? launch_many<F32>(a, workspace, 0, stream) : launch_many<Bf16>(a, workspace, 1, stream);
}
