// beam.cu -- spec_beam_select: the best continuations over (beam, vocabulary).
//
// "Accelerating Sonar through speculation", section "EAGLE": a draft tree
// takes top-K candidates and scores their sequences; one call per level
// grows the tree that spec_verify_tree verifies.
//
// Mathematics.  The score of (w, v) is base_w + (l_v - m_w)/T with
// base_w = scores_w - ln sum_u exp((l_u - m_w)/T), so
//  (1) inside a row candidates are ordered by their logits alone, exactly;
//  (2) a candidate among the K best lies in one of the at most K items (2048
//      bf16 or 1024 fp32 entries of a row) whose maxima are the best: an item
//      that comes before its own item's maximum holds a better candidate.
// Pass 1 (the streaming loop of sv_verify.cuh) therefore reads every logit once for
// (max, sum exp) per item, and the select step re-reads about K items per
// request, whatever W is.
//
// Order.  The scores are compared as exact numbers.  Pass 1 leaves base_w
// with an error below BeamArgs::err; two candidates of different rows that lie
// within the sum of their rows' errors are told apart by recomputing those
// rows' sums in fp64 (one block, rarely: with K = 16 about one request in a
// thousand), after which the order holds to fp64 rounding.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/specverify.h"
#include "sv_common.cuh"
#include "sv_verify.cuh"

namespace sv {

// Beam selection as a mode of pass 1: R = W rows a request, and what its
// items need beside the shared parameters.
constexpr int kBeam = 3;
struct BeamParams : Params {
    const float *beam_scores;   // [B][W]
    const int32_t *beam_done;   // [B][W], nullable
};

// An item of row r of request b; the rows of beams that are not in use or
// have ended are not read.
template <class Tag>
__device__ __forceinline__ Item1 beam_item(const Params &p, unsigned item)
{
    const auto &q = static_cast<const BeamParams &>(p);
    Item1 it;
    it.b = static_cast<int>(fdiv(item, p.div_req));
    const unsigned rem = item - static_cast<unsigned>(it.b) * p.div_req.d;
    it.r = static_cast<int>(fdiv(rem, p.div_s));
    it.s = static_cast<int>(rem - static_cast<unsigned>(it.r) * p.div_s.d);
    it.e_begin = it.s * Pass1Shape<Tag>::kItem;
    it.e_end = min(p.V, it.e_begin + Pass1Shape<Tag>::kItem);
    const int64_t row = static_cast<int64_t>(it.b) * p.R + it.r;
    it.active = __ldg(q.beam_scores + row) != -INFINITY && !(q.beam_done && __ldg(q.beam_done + row));
    it.row = static_cast<const char *>(p.tl) + row * p.stride * static_cast<int64_t>(sizeof(typename Tag::elem));
    return it;
}
template <>
__device__ __forceinline__ Item1 item1<Bf16, kBeam>(const Params &p, unsigned item, bool)
{
    return beam_item<Bf16>(p, item);
}
template <>
__device__ __forceinline__ Item1 item1<F32, kBeam>(const Params &p, unsigned item, bool)
{
    return beam_item<F32>(p, item);
}

// Up to this |m c| the rounding of m c (2^-12 here) is made good by its
// first-order term, to 2e-8; past it (small temperatures; a lane of nothing
// but mask values near the type's lowest) the differences are formed first.
constexpr float kDirectProduct = 8192.f;

// (max, sum 2^((l - max) c)) of a staged item: one FMA and one
// special-function exponential per entry against the lane's own maximum,
// four sums, the lanes brought to the warp's maximum.
template <class Tag>
__device__ __forceinline__ void reduce_beam_item(const Params &p, unsigned item, int s, const uint4 *slot)
{
    constexpr int kVec = Tag::kVec;
    constexpr int kV = Pass1Shape<Tag>::kVecL;
    const int lane = threadIdx.x & 31;
    const int e_begin = s * Pass1Shape<Tag>::kItem;
    uint4 raw[kV];
    if (e_begin + Pass1Shape<Tag>::kItem <= p.V) {
#pragma unroll
        for (int v = 0; v < kV; ++v) raw[v] = slot[v * 32 + lane];
    } else {  // the ragged end of a row
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int e0 = e_begin + (v * 32 + lane) * kVec;
            raw[v] = e0 < p.V ? mask_tail<Tag>(slot[v * 32 + lane], p.V - e0)
                              : make_uint4(Tag::kNegInfWord, Tag::kNegInfWord, Tag::kNegInfWord, Tag::kNegInfWord);
        }
    }
    const float c = p.c;
    const float m = lane_max<Tag>(raw);
    const float mc = m == -INFINITY ? 0.f : m * c;  // all -inf: every term is 0
    const bool direct = fabsf(mc) > kDirectProduct && fabsf(m) < INFINITY;
    float lsum;
    if (!direct) {
        const unsigned long long c2 = f2_pack(c, c), n2 = f2_pack(-mc, -mc);
        unsigned long long acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            float x[kVec];
            unpack<Tag>(raw[v], x);
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
                float z0, z1;
                f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), c2, n2), z0, z1);
                acc[(e >> 1) & 1] = f2_add(acc[(e >> 1) & 1], f2_pack(ex2_approx(z0), ex2_approx(z1)));
            }
        }
        float a0, a1, a2, a3;
        f2_unpack(acc[0], a0, a1);
        f2_unpack(acc[1], a2, a3);
        // fl(m c) - m c, exactly, as a factor
        lsum = ((a0 + a1) + (a2 + a3)) * fmaf(-fmaf(m == -INFINITY ? 0.f : m, c, -mc), 0.693147180559945309f, 1.0f);
    } else {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            float x[kVec];
            unpack<Tag>(raw[v], x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) a[e & 3] += ex2_approx((x[e] - m) * c);
        }
        lsum = (a[0] + a[1]) + (a[2] + a[3]);
    }
    const float M = warp_max_nan(m);
    const float sum = warp_sum(m == -INFINITY ? 0.f : lsum * ex2_approx((m - M) * c));
    if (lane == 0) __stcg(p.rowpart + item, make_float2(M, sum));
}
template <>
__device__ __forceinline__ void reduce_item1<Bf16, kBeam>(const Params &p, unsigned item, int s, const uint4 *slot)
{
    reduce_beam_item<Bf16>(p, item, s, slot);
}
template <>
__device__ __forceinline__ void reduce_item1<F32, kBeam>(const Params &p, unsigned item, int s, const uint4 *slot)
{
    reduce_beam_item<F32>(p, item, s, slot);
}

namespace {

// Pass 1 over the beams' rows: the streaming loop of the other calls.  (512
// rows of 128256 bf16, 131 MB: 28 us, 4.7 TB/s with a cold start; one
// exponential a logit keeps the special-function unit 59 % busy.)
template <class Tag>
__global__ void __launch_bounds__(kThreads, 2) k_beam_pass1(const __grid_constant__ BeamParams p)
{
    extern __shared__ uint4 rings[];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int warp = threadIdx.x >> 5;
    pass1_stream<Tag, kBeam>(p, rings + warp * kRing1 * Pass1Shape<Tag>::kSlot, blockIdx.x * kWarps + warp,
                             gridDim.x * kWarps);
}

constexpr int kBeamThreads = 512;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kListMax = 256;  // items kept on the fast path
constexpr int kHeldItems = 4096;     // item maxima kept in shared memory
constexpr int kGroups = 128;   // maxima the threshold is taken from (SPEC_MAX_BEAMS at least)
constexpr int kLaneItems = 4;        // a lane's items kept in registers (rows of up to 128 items)
// Bound on |ln S - ln S_exact| for a row sum merged from pass-1 partials.  A
// term's exponent z = (l - m) log2(e)/T comes in three parts (to the lane's, the
// item's, the row's maximum), each with at most three roundings of half a step
// (the difference, log2(e)/T, the product): 3 |z| 2^-24 ln 2, whose weighted
// mean is at most log2 V bits (entropy), 3.1e-6 for V = 2^25.  The exponential
// itself 2^-22; the sum of an item, 23 additions deep, 1.4e-6; two rescalings
// by fp32 exponentials 6e-7; the sum over the items 5e-7 whatever their number
// (two additions in fp32, the rest in fp64, one rounding and the warp's five); the
// logarithm 1e-7.  Together 5.9e-6, and 6.7e-6 for the longest rows (2^31).
constexpr double kBaseErr = 6e-6, kBaseErrLong = 7e-6;
constexpr int kLongRow = 1 << 25;

struct BeamArgs {
    int end_token, keep, cap;  // cap: candidates the shared list holds
    double err;                // bound on the error of a row's base
    float *out_s;
    int32_t *out_p, *out_t, *out_f;
};

struct Cand {
    double s;
    int w, v;
};

// The documented order: score, then lower beam, then lower token.
__device__ __forceinline__ bool better(const Cand &a, const Cand &b)
{
    return a.s > b.s || (a.s == b.s && (a.w < b.w || (a.w == b.w && a.v < b.v)));
}

// fp32 to an unsigned integer of the same order (and back).
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// ln s for a normal s > 0: exponent and fp32 logarithm of the mantissa in [1, 2),
// within 1e-7 (an eighth of the fp64 logarithm's time on the critical path).
__device__ __forceinline__ double log_fast(float s)
{
    const int u = __float_as_int(s);
    const float m = __int_as_float((u & 0x7FFFFF) | 0x3F800000);
    return static_cast<double>((u >> 23) - 127) * kLn2 + static_cast<double>(logf(m));
}

enum : int { kRowNone = 0, kRowLive = 1, kRowDone = 2 };

struct BeamRows {
    double base[SPEC_MAX_BEAMS];  // scores - ln S
    double err[SPEC_MAX_BEAMS];   // bound on base's error
    float base32[SPEC_MAX_BEAMS];
    float m[SPEC_MAX_BEAMS];
    float score[SPEC_MAX_BEAMS];
    int kind[SPEC_MAX_BEAMS];
    int exact[SPEC_MAX_BEAMS];    // 1: recompute wanted, 2: done
};

// This lane's vector v of item s of row w, -inf past the vocabulary.
template <class Tag>
__device__ __forceinline__ uint4 item_vector(const Params &p, int b, int w, int s, int v)
{
    constexpr int kVec = Tag::kVec;
    constexpr int kEsz = sizeof(typename Tag::elem);
    const int e = s * Pass1Shape<Tag>::kItem + (v * 32 + static_cast<int>(threadIdx.x & 31)) * kVec;
    const char *row = static_cast<const char *>(p.tl) + (static_cast<int64_t>(b) * p.R + w) * p.stride * kEsz;
    return e < p.V ? mask_tail<Tag>(ldg_vec(row + static_cast<int64_t>(e) * kEsz), p.V - e)
                   : make_uint4(Tag::kNegInfWord, Tag::kNegInfWord, Tag::kNegInfWord, Tag::kNegInfWord);
}

// Append the candidates of one item (row w, segment s) that reach lthr to
// the list.  One warp.  *count is the list's new length, which may pass cap
// (entries beyond it are not stored).  A vector's packed maximum decides
// whether it is looked into; the few that are, are read again (L1), so that
// the entries' code exists once: unrolled over the item it spent four times
// as long, on instruction fetches.
template <class Tag>
__device__ __forceinline__ void gather_item(const Params &p, int b, int w, int s, float lthr, double base,
                                            float m, Cand *cand, int cap, int *count)
{
    constexpr int kVec = Tag::kVec;
    constexpr int kV = Pass1Shape<Tag>::kVecL;
    constexpr int kEsz = sizeof(typename Tag::elem);
    const int lane = threadIdx.x & 31;
    const int e0 = s * Pass1Shape<Tag>::kItem + lane * kVec;
    const char *row = static_cast<const char *>(p.tl) + (static_cast<int64_t>(b) * p.R + w) * p.stride * kEsz;
    auto vector = [&](int v) { return item_vector<Tag>(p, b, w, s, v); };
    auto reaches = [&](uint4 raw) {
        const float top = vec_max<Tag>(raw);
        return top >= lthr && top > -INFINITY;
    };
    unsigned hit = 0;
    if (s * Pass1Shape<Tag>::kItem + Pass1Shape<Tag>::kItem <= p.V) {
        uint4 raw[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) raw[v] = ldg_vec(row + static_cast<int64_t>(e0 + v * 32 * kVec) * kEsz);
#pragma unroll
        for (int v = 0; v < kV; ++v) hit |= reaches(raw[v]) ? 1u << v : 0u;
    } else {
#pragma unroll 1
        for (int v = 0; v < kV; ++v) hit |= reaches(vector(v)) ? 1u << v : 0u;
    }
    for (unsigned todo = __reduce_or_sync(kFull, hit); todo; todo &= todo - 1) {
        const int v = __ffs(todo) - 1;
        float x[kVec];
        unpack<Tag>(vector(v), x);
        unsigned in = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) in |= x[e] >= lthr && x[e] > -INFINITY ? 1u << e : 0u;
        int incl = __popc(in);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        int at = 0;
        if (lane == 31) at = atomicAdd(count, incl);
        at = __shfl_sync(kFull, at, 31) + incl - __popc(in);
        for (; in; in &= in - 1, ++at) {
            const int e = e0 + v * 32 * kVec + __ffs(in) - 1;
            const float l = load_logit<Tag>(row, e);
            if (at < cap) cand[at] = {base + (static_cast<double>(l) - static_cast<double>(m)) * p.inv_t, w, e};
        }
    }
}

// The `keep` best entries of one item, appended: those above the largest
// value that `keep` entries reach, and of those equal to it the first in
// index order.  One warp; for rows of many equal values.
template <class Tag>
__device__ __noinline__ void gather_best(const Params &p, int b, int w, int s, double base, float m, int keep,
                                         Cand *cand, int cap, int *count)
{
    constexpr int kEsz = sizeof(typename Tag::elem);
    const int lane = threadIdx.x & 31;
    const int e0 = s * Pass1Shape<Tag>::kItem, n = min(p.V - e0, Pass1Shape<Tag>::kItem);
    const int64_t row = (static_cast<int64_t>(b) * p.R + w) * p.stride + e0;
    static_assert(kEsz == 2 || kEsz == 4, "bf16 or fp32");
    auto reaching = [&](float t) {
        int c = 0;
        for (int i = lane; i < n; i += 32) {
            const float x = load_logit<Tag>(p.tl, row + i);
            c += x >= t && x > -INFINITY ? 1 : 0;
        }
        return __reduce_add_sync(kFull, c);
    };
    uint32_t lo = order_key(-INFINITY), hi = order_key(INFINITY);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (reaching(order_value(mid)) >= keep) lo = mid;
        else hi = mid - 1;
    }
    const float t = order_value(lo);
    const int all = reaching(t);
    int above = 0;
    for (int i = lane; i < n; i += 32) above += load_logit<Tag>(p.tl, row + i) > t ? 1 : 0;
    int ties = min(all, keep) - __reduce_add_sync(kFull, above);  // entries equal to t to take
    int at = 0;
    if (lane == 0) at = atomicAdd(count, min(all, keep));
    at = __shfl_sync(kFull, at, 0);
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const float x = i < n ? load_logit<Tag>(p.tl, row + i) : -INFINITY;
        const unsigned eq = __ballot_sync(kFull, x == t && x > -INFINITY);
        const bool take = x > t || (x == t && x > -INFINITY && __popc(eq & ((1u << lane) - 1)) < ties);
        const unsigned taken = __ballot_sync(kFull, take);
        const int slot = at + __popc(taken & ((1u << lane) - 1));
        if (take && slot < cap)
            cand[slot] = {base + (static_cast<double>(x) - static_cast<double>(m)) * p.inv_t, w, e0 + i};
        at += __popc(taken);
        ties -= min(ties, __popc(eq));
    }
}

// The fp64 sum of exp((l - m)/T) over row w of request b, the same order
// of additions for every row (equal rows give equal sums).  Whole block.
template <class Tag>
__device__ __forceinline__ double exact_sum(const Params &p, int b, int w, float m, const double *tab,
                                            double *scratch)
{
    constexpr int kVec = Tag::kVec;
    constexpr int kEsz = sizeof(typename Tag::elem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const char *row = static_cast<const char *>(p.tl) + (static_cast<int64_t>(b) * p.R + w) * p.stride * kEsz;
    double acc = 0.0;
    for (int e0 = tid * kVec; e0 < p.V; e0 += kBeamThreads * kVec) {
        float x[kVec];
        unpack<Tag>(mask_tail<Tag>(ldg_vec(row + static_cast<int64_t>(e0) * kEsz), p.V - e0), x);
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            acc += exp2_fp64((static_cast<double>(x[e]) - static_cast<double>(m)) * p.c64, tab);
    }
    acc = warp_sum(acc);
    __syncthreads();
    if (lane == 0) scratch[warp] = acc;
    __syncthreads();
    double sum = 0.0;
    for (int i = 0; i < kBeamWarps; ++i) sum += scratch[i];
    return sum;
}

// Select: one block per request, after pass 1.  A chain of block-wide steps
// bounds it, not bytes: 6 us after pass 1's end for one request with K = 4, 9
// for 32 with K = 16.  Where rows' sums are recomputed each of 128256 entries
// takes some 20 us more, one after the other: a call with 4 equal beams, which
// are all recomputed, takes 100 us, one with 64 1.4 ms (distinct beams 9 us, and
// 30 to 90 as near ties come).
template <class Tag>
__global__ void __launch_bounds__(kBeamThreads)
    k_beam_select(const __grid_constant__ BeamParams p, const __grid_constant__ BeamArgs a)
{
    extern __shared__ Cand cand[];
    __shared__ BeamRows rw;
    __shared__ double tab[kExp2Tab];
    __shared__ double scratch[kBeamWarps];
    __shared__ Cand best[SPEC_MAX_BEAMS];
    __shared__ int list[kListMax];
    __shared__ int nlist, ncand, bad, again;
    __shared__ Cand warp_best[kBeamWarps];
    __shared__ float thread_max[kBeamThreads];
    __shared__ __align__(16) float group_max[kGroups];
    __shared__ float held[kHeldItems];
    __shared__ unsigned bound;

    const int b = blockIdx.x, W = p.R, S = p.S, K = a.keep;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = 0;
    __syncthreads();
    if (tid < W) {
        const float sc = __ldg(p.beam_scores + static_cast<int64_t>(b) * W + tid);
        const bool done = p.beam_done && __ldg(p.beam_done + static_cast<int64_t>(b) * W + tid) != 0;
        rw.score[tid] = sc;
        rw.kind[tid] = sc == -INFINITY ? kRowNone : done ? kRowDone : kRowLive;
        rw.exact[tid] = 0;
        if (!(sc < INFINITY)) bad = 1;  // NaN or +inf
    }
    const float2 *part = p.rowpart + static_cast<int64_t>(b) * W * S;
    const int items = W * S;
    const float inv_t = static_cast<float>(p.inv_t);
    auto row_of = [&](int i) { return static_cast<int>(fdiv(static_cast<unsigned>(i), p.div_s)); };
    // score of row w's logit l (-inf: no candidate), in fp32.  A candidate past
    // fp32's range (the type's lowest value as a mask, at T < 1) gets the lowest
    // key, so that it stays one: equal keys are told apart in fp64.
    auto key_of = [&](int w, float l) -> float {
        return rw.kind[w] != kRowLive || l == -INFINITY ? -INFINITY
                                                        : fmaxf(fmaf(l - rw.m[w], inv_t, rw.base32[w]), -FLT_MAX);
    };
    // score of the best candidate of item i (item s of row w: w S + s)
    auto item_key = [&](int i) -> float { return key_of(row_of(i), i < kHeldItems ? held[i] : __ldcg(&part[i].x)); };
    // and in fp64
    auto item_score = [&](int i) -> double {
        const int w = row_of(i);
        if (rw.kind[w] != kRowLive) return -INFINITY;
        const float m = i < kHeldItems ? held[i] : __ldcg(&part[i].x);
        return m == -INFINITY ? -INFINITY
                              : rw.base[w] + (static_cast<double>(m) - static_cast<double>(rw.m[w])) * p.inv_t;
    };
    const int64_t o = static_cast<int64_t>(b) * K;
    int found = 0;
    // (Running the steps once before this, on the workspace's old contents, to have
    // their instructions at hand, took 2.7 us more than the 8.8 of one request: the
    // block starts when the first of pass 1 leave, so that run is waited for too.
    // On contents other than a last call's partials it took 10 us more.)
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    __syncthreads();
    // merge the rows, a warp each
    for (int w = warp; w < W; w += kBeamWarps) {
        if (rw.kind[w] != kRowLive) continue;
        // the items' maxima (kept for the steps below) and the row's, then
        // the sum of the items' sums brought to it, each by one factor
        float2 x[kLaneItems];
        float m = -INFINITY;
        auto item = [&](int i) {
            const float2 y = __ldcg(&part[w * S + i]);
            if (w * S + i < kHeldItems) held[w * S + i] = y.x;
            m = max_nan(m, y.x);
            return y;
        };
#pragma unroll
        for (int j = 0; j < kLaneItems; ++j) x[j] = lane + 32 * j < S ? item(lane + 32 * j) : make_float2(-INFINITY, 0.f);
        for (int i = lane + 32 * kLaneItems; i < S; i += 32) item(i);
        const float top = warp_max_nan(m);
        auto brought = [&](float2 y) { return y.x == -INFINITY ? 0.f : y.y * ex2_approx((y.x - top) * p.c); };
        static_assert(kLaneItems == 4, "two additions deep");
        float sum = (brought(x[0]) + brought(x[1])) + (brought(x[2]) + brought(x[3]));
        if (S > 32 * kLaneItems) {
            double rest = sum;
            for (int i = lane + 32 * kLaneItems; i < S; i += 32) rest += static_cast<double>(brought(__ldcg(&part[w * S + i])));
            sum = static_cast<float>(rest);
        }
        sum = warp_sum(sum);
        if (lane == 0) {
            rw.m[w] = top;
            if (top == -INFINITY) {
                rw.kind[w] = kRowNone;  // nothing to go on with
            } else if (!stoch_row_ok(top, sum)) {
                bad = 1;
            } else {
                rw.base[w] = static_cast<double>(rw.score[w]) - log_fast(sum);
                rw.err[w] = a.err;
                rw.base32[w] = static_cast<float>(rw.base[w]);
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (bad) {
        if (tid < K) {
            a.out_s[o + tid] = -INFINITY;
            a.out_p[o + tid] = -1;
            a.out_t[o + tid] = -1;
            if (a.out_f) a.out_f[o + tid] = 0;
        }
        if (tid == 0) report(p.status, kStLogit);
        return;
    }

    for (;;) {
        // a lower bound t0 of the K-th best candidate: the K-th largest of
        // kGroups maxima of distinct items (each a candidate's score)
        float mine = -INFINITY;
        for (int i = tid; i < items; i += kBeamThreads) mine = fmaxf(mine, item_key(i));
        thread_max[tid] = mine;
        if (tid == 0) {
            nlist = 0;
            ncand = 0;
            again = 0;
            bound = 0xFFFFFFFFu;
        }
        __syncthreads();
        // every kGroups-th item to a group: as many groups as items, up to
        // kGroups, and the best row's best items in different ones
        if (tid < kGroups) {
#pragma unroll
            for (int x = kGroups; x < kBeamThreads; x += kGroups) mine = fmaxf(mine, thread_max[tid + x]);
            group_max[tid] = mine;
        }
        __syncthreads();
        {
            // how many of the groups' maxima are larger, four threads a group:
            // the least of those with fewer than K is the K-th largest
            constexpr int kShare = kBeamThreads / kGroups;
            const int j0 = tid % kShare * (kGroups / kShare);
            const float x = group_max[tid / kShare];
            int above = 0;
#pragma unroll
            for (int j = j0; j < j0 + kGroups / kShare; j += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(&group_max[j]);
                above += (y.x > x ? 1 : 0) + (y.y > x ? 1 : 0) + (y.z > x ? 1 : 0) + (y.w > x ? 1 : 0);
            }
#pragma unroll
            for (int o = 1; o < kShare; o <<= 1) above += __shfl_xor_sync(kFull, above, o);
            const uint32_t least = __reduce_min_sync(kFull, above < K ? order_key(x) : 0xFFFFFFFFu);
            if (lane == 0) atomicMin(&bound, least);
        }
        __syncthreads();
        float t0f = order_value(bound);
        if (t0f <= -FLT_MAX) {
            // fewer than K items (with keys above the lowest): the K-th largest
            // of the maxima of their parts, 32 bf16 (16 fp32) entries a lane
            // and half
            float sub[2] = {-INFINITY, -INFINITY};
            for (int i = warp; i < items; i += kBeamWarps) {
                const int w = row_of(i);
                if (rw.kind[w] != kRowLive) continue;
#pragma unroll 1
                for (int v = 0; v < Pass1Shape<Tag>::kVecL; ++v) {
                    const float key = key_of(w, vec_max<Tag>(item_vector<Tag>(p, b, w, i - w * S, v)));
                    if (v < Pass1Shape<Tag>::kVecL / 2) sub[0] = fmaxf(sub[0], key);
                    else sub[1] = fmaxf(sub[1], key);
                }
            }
            const uint32_t k0 = order_key(sub[0]), k1 = order_key(sub[1]);
            uint32_t lo = order_key(-INFINITY), hi = order_key(INFINITY);
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                if (__syncthreads_count(k0 >= mid) + __syncthreads_count(k1 >= mid) >= K) lo = mid;
                else hi = mid - 1;
            }
            t0f = order_value(lo);
        }
        // the lowest key stands for scores of any size: no bound
        if (t0f <= -FLT_MAX) t0f = -INFINITY;
        // below t0 by the rows' errors, so that what the check below
        // compares is in the list too; and by the keys' rounding, at most
        // 4 steps of what adds up to a key
        const double t0 = t0f == -INFINITY ? -INFINITY : static_cast<double>(t0f) - 4.0 * a.err;
        auto slack = [&](int w) { return 4.8e-7f * (fabsf(t0f) + fabsf(rw.base32[w])); };
        const float least = t0f == -INFINITY ? -INFINITY : static_cast<float>(t0);
        for (int i = tid; i < items; i += kBeamThreads) {
            const float key = item_key(i);
            if (key > -INFINITY && key >= least - 2.f * slack(row_of(i))) {
                const int at = atomicAdd(&nlist, 1);
                if (at < kListMax) list[at] = i;
            }
        }
        auto add_done = [&]() {
            if (tid < W && rw.kind[tid] == kRowDone)
                cand[atomicAdd(&ncand, 1)] = {static_cast<double>(rw.score[tid]), tid, a.end_token};
        };
        add_done();
        __syncthreads();
        bool whole = nlist <= kListMax;
        if (whole) {
            for (int j = warp; j < nlist; j += kBeamWarps) {
                const int w = row_of(list[j]);
                // the row's logits that may reach t0, rounded down
                float lthr = -INFINITY;
                if (t0 != -INFINITY) {
                    const double l = static_cast<double>(rw.m[w]) + (t0 - 2.f * slack(w) - rw.base[w]) / p.inv_t;
                    lthr = static_cast<float>(l - fabs(l) * 1.2e-7);
                }
                gather_item<Tag>(p, b, w, list[j] - w * S, lthr, rw.base[w], rw.m[w], cand, a.cap, &ncand);
            }
            __syncthreads();
            whole = ncand <= a.cap;
        }
        if (!whole) {
            // many equal maxima: exactly the K best items, one by one, and of
            // each its K best entries (K * K fit the list)
            int n = 0;
            Cand last = {INFINITY, -1, -1};
            __syncthreads();
            if (tid == 0) ncand = 0;
            __syncthreads();
            add_done();
            for (; n < K; ++n) {
                Cand top = {-INFINITY, INT_MAX, INT_MAX};
                for (int i = tid; i < items; i += kBeamThreads) {
                    const int w = row_of(i);
                    const Cand c = {item_score(i), w, i - w * S};
                    if (c.s > -INFINITY && better(last, c) && better(c, top)) top = c;
                }
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) {
                    const Cand c = {__shfl_xor_sync(kFull, top.s, x), __shfl_xor_sync(kFull, top.w, x),
                                    __shfl_xor_sync(kFull, top.v, x)};
                    if (better(c, top)) top = c;
                }
                if (lane == 0) warp_best[warp] = top;
                __syncthreads();
                top = warp_best[0];
                for (int i = 1; i < kBeamWarps; ++i)
                    if (better(warp_best[i], top)) top = warp_best[i];
                __syncthreads();
                if (top.s == -INFINITY) break;
                if (tid == 0) list[n] = top.w * S + top.v;
                last = top;
            }
            __syncthreads();
            for (int j = warp; j < n; j += kBeamWarps) {
                const int w = row_of(list[j]);
                gather_best<Tag>(p, b, w, list[j] - w * S, rw.base[w], rw.m[w], K, cand, a.cap, &ncand);
            }
            if (tid == 0) nlist = n;
        }
        __syncthreads();

        // rank every candidate, a warp each; the first K are the selection
        const int n = ncand;
        found = min(n, K);
        for (int i = warp; i < n; i += kBeamWarps) {
            const Cand c = cand[i];
            int rank = 0;
            for (int j = lane; j < n; j += 32) rank += better(cand[j], c) ? 1 : 0;
            rank = __reduce_add_sync(kFull, rank);
            if (lane == 0 && rank < K) best[rank] = c;
        }
        __syncthreads();
        // rows whose errors could change it
        auto err = [&](int w) { return rw.kind[w] == kRowLive ? rw.err[w] : 0.0; };
        auto close = [&](const Cand &x, double s, int w) {
            const double e = err(x.w) + err(w);
            return w != x.w && e > 0.0 && fabs(x.s - s) <= e;
        };
        auto want = [&](int w) {
            if (rw.kind[w] == kRowLive && rw.err[w] > 0.0) {
                rw.exact[w] = 1;
                again = 1;
            }
        };
        if (tid + 1 < found && close(best[tid], best[tid + 1].s, best[tid + 1].w)) {
            want(best[tid].w);
            want(best[tid + 1].w);
        }
        if (found == K) {
            const Cand kth = best[K - 1];
            for (int i = tid; i < n; i += kBeamThreads) {
                const Cand c = cand[i];
                if (better(kth, c) && close(kth, c.s, c.w)) {
                    want(kth.w);
                    want(c.w);
                }
            }
            // items that are not in the list, by their maxima (a whole list
            // leaves out only what lies further below)
            if (!whole)
                for (int i = tid; i < items; i += kBeamThreads) {
                    const int w = row_of(i);
                    const double s = item_score(i);
                    if (s == -INFINITY || !close(kth, s, w)) continue;
                    bool in = false;
                    for (int j = 0; j < nlist && !in; ++j) in = list[j] == i;
                    if (!in) {
                        want(kth.w);
                        want(w);
                    }
                }
        }
        __syncthreads();
        if (!again) break;
        for (int j = tid; j < kExp2Tab; j += kBeamThreads) tab[j] = p.exp2tab[j];
        __syncthreads();
        for (int w = 0; w < W; ++w) {
            if (rw.exact[w] != 1) continue;
            const double sum = exact_sum<Tag>(p, b, w, rw.m[w], tab, scratch);
            if (tid == 0) {
                rw.base[w] = static_cast<double>(rw.score[w]) - log(sum);
                rw.base32[w] = static_cast<float>(rw.base[w]);
                rw.err[w] = 0.0;
                rw.exact[w] = 2;
            }
        }
        __syncthreads();
    }
    if (tid < K) {
        const bool in = tid < found;
        a.out_s[o + tid] = in ? static_cast<float>(best[tid].s) : -INFINITY;
        a.out_p[o + tid] = in ? best[tid].w : -1;
        a.out_t[o + tid] = in ? best[tid].v : -1;
        if (a.out_f) a.out_f[o + tid] = in && best[tid].v == a.end_token ? 1 : 0;
    }
}

constexpr size_t kBeamAlign = 256;
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

// pass 1's claim counter (touched, not used), then the pass-1 partials
// [B][W][S] (S of the shorter fp32 items, so that both dtypes fit)
size_t beam_bytes(int B, int W, int V)
{
    if (B < 0 || W < 1 || W > SPEC_MAX_BEAMS || V < 1) return 0;
    const size_t s = static_cast<size_t>(ceil_div(V, Pass1Shape<F32>::kItem));
    const size_t n = sizeof(float2) * static_cast<size_t>(B) * W * s;
    return kBeamAlign + (n + kBeamAlign - 1) / kBeamAlign * kBeamAlign;
}

std::mutex g_beam_mu;
int g_beam_blocks[64][2];
int g_beam_sms[64];
bool g_beam_attr[64][2];
constexpr int kCandMin = 1024;
size_t cand_count(int K) { return std::max(kCandMin, K * K) + SPEC_MAX_BEAMS; }

template <class Tag>
int launch_beam(BeamParams &p, BeamArgs &a, int dtype_index, cudaStream_t st)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ECUDA;
    int per_sm, sms;
    {
        std::lock_guard<std::mutex> lock(g_beam_mu);
        if (g_beam_blocks[dev][dtype_index] < 1) {
            int n = 0;
            if (cudaFuncSetAttribute(k_beam_pass1<Tag>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(kRingBytes)) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_beam_pass1<Tag>, kThreads, kRingBytes) !=
                    cudaSuccess ||
                n < 1)
                return SPEC_ECUDA;
            g_beam_blocks[dev][dtype_index] = n;
        }
        if (g_beam_sms[dev] < 1 &&
            (cudaDeviceGetAttribute(&g_beam_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
             g_beam_sms[dev] < 1))
            return SPEC_ECUDA;
        if (!g_beam_attr[dev][dtype_index]) {
            if (cudaFuncSetAttribute(k_beam_select<Tag>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(sizeof(Cand) * cand_count(SPEC_MAX_BEAMS))) != cudaSuccess)
                return SPEC_ECUDA;
            g_beam_attr[dev][dtype_index] = true;
        }
        per_sm = g_beam_blocks[dev][dtype_index];
        sms = g_beam_sms[dev];
    }
    const int64_t blocks =
        std::max<int64_t>(1, std::min<int64_t>(static_cast<int64_t>(per_sm) * sms, ceil_div(p.nA, kWarps)));
    // All items are static: the claimed tail of the other calls comes in
    // chunks of four items and clearing its counter is a launch of its own
    // (rows of 128256 bf16: a claimed tail takes 6.0 us more for 32 x 16, 3.6 for
    // 128 x 16, 4.7 for 256 x 4)
    p.nAs = p.nA;
    k_beam_pass1<Tag><<<static_cast<unsigned>(blocks), kThreads, kRingBytes, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SPEC_ECUDA;
    a.cap = static_cast<int>(cand_count(a.keep));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(p.B));
    cfg.blockDim = dim3(kBeamThreads);
    cfg.dynamicSmemBytes = sizeof(Cand) * static_cast<size_t>(a.cap);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_beam_select<Tag>, p, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

namespace {
struct Exp2Table {
    double at[kExp2Tab];
    Exp2Table()
    {
        for (int j = 0; j < kExp2Tab; ++j) at[j] = std::exp2(static_cast<double>(j) / kExp2Tab);
    }
};
}  // namespace

extern "C" size_t spec_beam_workspace_size(int batch, int beams, int vocab)
{
    return beam_bytes(batch, beams, vocab);
}

extern "C" int spec_beam_select(const void *logits, spec_dtype_t dtype, int64_t row_stride,
                                const float *scores, const int32_t *finished, int end_token,
                                int batch, int beams, int vocab, float temperature, int keep,
                                float *out_scores, int32_t *out_parents, int32_t *out_tokens,
                                int32_t *out_finished, int32_t *status, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream)
{
    if (batch < 0 || beams < 1 || keep < 1) return SPEC_EINVAL;
    if (beams > SPEC_MAX_BEAMS || keep > SPEC_MAX_BEAMS) return SPEC_EUNSUPPORTED;
    if (!(temperature > 0.f) || !(temperature < INFINITY)) return SPEC_EINVAL;
    if (!(static_cast<float>(1.4426950408889634074 / temperature) < INFINITY)) return SPEC_EINVAL;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EINVAL;
    if (vocab < 1 || row_stride < vocab) return SPEC_EINVAL;
    if (end_token < -1 || end_token >= vocab || (finished && end_token < 0)) return SPEC_EINVAL;
    const int esz = dtype == SPEC_BF16 ? 2 : 4;
    if ((row_stride * esz) % 16 != 0) return SPEC_EALIGN;
    if (batch == 0) return SPEC_OK;
    if (!logits || !scores || !out_scores || !out_parents || !out_tokens) return SPEC_EINVAL;
    // in place only where a request's outputs lie on its own inputs
    if (keep != beams && (out_scores == scores || (finished && out_finished == finished))) return SPEC_EINVAL;
    if ((reinterpret_cast<uintptr_t>(logits) & 15u) != 0) return SPEC_EALIGN;
    const size_t need = beam_bytes(batch, beams, vocab);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kBeamAlign) != 0 || workspace_bytes < need)
        return SPEC_EWORKSPACE;
    const int S = static_cast<int>(
        ceil_div(vocab, dtype == SPEC_BF16 ? Pass1Shape<Bf16>::kItem : Pass1Shape<F32>::kItem));
    const int64_t nA = static_cast<int64_t>(batch) * beams * S;
    if (nA >= (int64_t(1) << 31) || static_cast<int64_t>(batch) * keep > INT_MAX) return SPEC_EUNSUPPORTED;

    BeamParams p;
    std::memset(static_cast<void *>(&p), 0, sizeof p);
    p.tl = logits;
    p.stride = row_stride;
    p.B = batch;
    p.V = vocab;
    p.R = beams;
    p.S = S;
    p.nA = static_cast<unsigned>(nA);
    p.div_req = make_fastdiv(static_cast<uint32_t>(beams) * static_cast<uint32_t>(S));
    p.div_s = make_fastdiv(static_cast<uint32_t>(S));
    const double t = static_cast<double>(temperature);
    p.inv_t = 1.0 / t;
    p.c64 = 1.4426950408889634074 / t;
    p.c = static_cast<float>(p.c64);
    p.beam_scores = scores;
    p.beam_done = finished;
    p.status = status;
    p.a_claim = static_cast<unsigned *>(workspace);
    p.rowpart = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + kBeamAlign);
    static const Exp2Table table;  // 2 us of a call that takes 15
    std::memcpy(p.exp2tab, table.at, sizeof p.exp2tab);
    BeamArgs a{end_token,  keep,        0,          vocab <= kLongRow ? kBaseErr : kBaseErrLong,
               out_scores, out_parents, out_tokens, out_finished};
    return dtype == SPEC_BF16 ? launch_beam<Bf16>(p, a, 1, stream) : launch_beam<F32>(p, a, 0, stream);
}
