// spec_filter and spec_sample (include/specsample.h): temperature, top-k, top-p and min-p on rows of logits.
//
// Mathematics. The kept tokens are the first n of the ranking by logit, so a row's filter is a threshold: the logits above
// it are kept, and of those equal to it the first r by index. A weight is w = 2^((l - m) K), K = log2(e) / T, held as an
// integer W = round(2^44 w); sums of them are exact, and so is every comparison of sums (top-p's crossing, the inverse
// CDF's): the order in which threads add does not matter, and a draw differs from one in real numbers only where its
// target lies within the weights' own errors, some 2^-31 of each, of a border.
//
// Two ways to the threshold. A bfloat16 logit has few values: between 2^-26 and 2^10 each has a bin of its own (one
// more is zero's), a row's histogram of counts says it all, and weights are needed for the bins that hold something
// only. Where a logit lies outside those bins, and for float, the threshold's 32-bit key is found 12, 12 and 8 bits at a
// time, each from a histogram of the counts (top-k) or weights (top-p) of the elements still in question.
//
// Shape. A row is a cluster's of up to 8 CTAs, each of which holds its slice of the row in shared memory (one read
// from memory, however many passes follow), a warp a contiguous segment of it. Histograms are summed by slices of
// the bins through distributed shared memory into the first CTA's, which finds the threshold.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/specsample.h"
#include "sv_device.cuh"

namespace cg = cooperative_groups;

namespace sv {
namespace sample {

struct Args {
    const void* logits;
    int64_t stride;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const int32_t* request;
    int32_t requests, rows, V;
    const float* uniforms;  // spec_sample
    int32_t* tokens;
    float* logprob;
    void* out;  // spec_filter
    int64_t out_stride;
    int32_t* kept;
    uint32_t* status;
    float2 exp2_tab[128];
};

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCtas = 8;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kBits = 44;  // of a weight's fraction; 2^18 weights of 1 sum to 2^62
constexpr float kLowest = -3.402823466e38f;

// The bins of the quick way, one for each bfloat16 magnitude code in [kCodeLo, kCodeHi] of either sign, one in the middle for
// zero, and one at either end that stays empty.
constexpr uint32_t kCodeLo = 0x3280u, kCodeHi = 0x447fu;  // 2^-26, 1020
constexpr uint32_t kCodes = kCodeHi - kCodeLo + 1;
constexpr int kMid = kCodes + 1, kBins = 2 * kMid + 1;
constexpr int kGroupBins = 64, kGroups = (kBins + kGroupBins - 1) / kGroupBins;
constexpr int kHist = kGroups * kGroupBins;  // words
constexpr int kDigits = 4096;                // bins of the other way: two words each
static_assert(2 * kDigits <= kHist, "the histogram's words serve both ways");
static_assert(kGroups <= 160, "five groups a lane");

typedef unsigned long long u64;

struct RowPar {
    ExpConst E;
    float T, p, u;
    int32_t k;      // 0: none
    u64 least;      // of a kept weight, 0: none
    uint32_t err;
};

struct Result {
    float thr;      // logits above it are kept
    uint32_t r;     // and so many equal to it, in index order
    int32_t partial;  // these are not all of them (or may not be)
    int32_t n;      // kept, -1: not known yet
    float m;        // the largest logit
    uint32_t err;
    int32_t slow;   // the quick way could not tell
};

struct Found {  // a level of the slow way
    int32_t bin;    // -1: the target lies past all bins
    u64 rest;       // what is left of the target within the bin, or past all
    u64 value;      // of the bin
    u64 total;      // of the first level
};

struct alignas(16) Shared {
    uint32_t hist[kHist];
    float tab[2 * kExpTab];
    u64 group_mass[kGroups + 1];
    uint32_t group_count[kGroups + 1];
    u64 scan[kWarps];
    u64 warp_mass[kWarps];
    uint32_t warp_ties[kWarps], warp_above[kWarps];
    uint32_t warp_max[kWarps];
    uint32_t flags;
    uint32_t max_key;
    float floor;
    RowPar par;
    Result res;
    Found found;
    // of this CTA's warps, after all have counted
    int32_t ties_kept[kWarps];
    int32_t hit_warp;  // the warp (of the cluster) that holds the drawn token
    u64 hit_rest, total;
    uint32_t above;
};

enum : uint32_t { kNonfinite = 1, kOutside = 2 };

// A float's place in the order of all floats, zeros of both signs alike; the least of a finite one is above that of -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x) == 0x80000000u ? 0u : __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
constexpr uint32_t kKeyMinusInf = 0x007fffffu, kKeyInf = 0xff800000u;

// Fixed-point parts of two weights: W = (a << 22) + b. The first rounds to 2^-22 (the unit in the last place of 3 + w), the
// second what that leaves, and the low part of the weight, to 2^-44.
struct Fixed2 {
    int32_t ax, ay, bx, by;
};
__device__ __forceinline__ Fixed2 fixed2(ff2 w) {
    const float2 t = add2(w.hi, f2(3.f));
    const float2 rest = add2(sub2(w.hi, add2(t, f2(-3.f))), w.lo);
    const float2 s = add2(rest, f2(7.152557373046875e-07f));  // 1.5 2^-21
    return {(int32_t)(__float_as_uint(t.x) - 0x40400000u), (int32_t)(__float_as_uint(t.y) - 0x40400000u),
            (int32_t)(__float_as_uint(s.x) - 0x35400000u), (int32_t)(__float_as_uint(s.y) - 0x35400000u)};
}
__device__ __forceinline__ Fixed2 weights2(float x, float y, float m, const ExpConst& E, const float* tab) {
    return fixed2(exp2_ff2<true>(make_float2(x, y), f2(m), E, tab));
}
__device__ __forceinline__ u64 join(int32_t a, int32_t b) { return (u64)(((long long)a << 22) + b); }
__device__ __forceinline__ u64 weight(float x, float m, const ExpConst& E, const float* tab) {
    const Fixed2 f = weights2(x, x, m, E, tab);
    return join(f.ax, f.bx);
}

__device__ __forceinline__ u64 shfl_up64(u64 v, int o) { return __shfl_up_sync(kAll, v, o); }
__device__ __forceinline__ u64 warp_inscan(u64 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = shfl_up64(v, o);
        if (lane >= o) v += x;
    }
    return v;
}
// Sums of up to 2^62.
__device__ __forceinline__ u64 warp_sum(u64 v) {
    const u64 a = __reduce_add_sync(kAll, (uint32_t)v & 0x7ffffffu), b = __reduce_add_sync(kAll, (uint32_t)(v >> 27) & 0x7ffffffu),
              c = __reduce_add_sync(kAll, (uint32_t)(v >> 54));
    return a + (b << 27) + (c << 54);
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int N = 4;  // of 16 bytes
    static constexpr uint32_t kMinusInf = 0xff800000u;
    static __device__ __forceinline__ void unpack(const uint4& q, float* x) {
        x[0] = __uint_as_float(q.x);
        x[1] = __uint_as_float(q.y);
        x[2] = __uint_as_float(q.z);
        x[3] = __uint_as_float(q.w);
    }
    // a chunk with the elements of `mask` as they are and the others -inf
    static __device__ __forceinline__ uint4 masked(const uint4& q, uint32_t mask) {
        return make_uint4(mask & 1 ? q.x : kMinusInf, mask & 2 ? q.y : kMinusInf, mask & 4 ? q.z : kMinusInf, mask & 8 ? q.w : kMinusInf);
    }
    static constexpr uint32_t bits_minus_inf = kMinusInf;
    typedef uint32_t Bits;
    static __device__ __forceinline__ float value(Bits b) { return __uint_as_float(b); }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4& q, float* x) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16lo_to_f32(w[i]);
            x[2 * i + 1] = bf16hi_to_f32(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 masked(const uint4& q, uint32_t mask) {
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!(mask >> (2 * i) & 1u)) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
            if (!(mask >> (2 * i + 1) & 1u)) w[i] = (w[i] & 0xffffu) | 0xff800000u;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static constexpr uint16_t bits_minus_inf = 0xff80u;
    typedef uint16_t Bits;
    static __device__ __forceinline__ float value(Bits b) { return __uint_as_float((uint32_t)b << 16); }
};

// A cluster's barrier; a block's where a row has one CTA.
struct Team {
    int rank, size;
    __device__ __forceinline__ void arrive() const { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
    __device__ __forceinline__ void wait() const { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
    __device__ __forceinline__ void sync() const {
        if (size == 1) {
            __syncthreads();
        } else {
            arrive();
            wait();
        }
    }
    // the same object of another CTA
    template <typename P>
    __device__ __forceinline__ P* of(P* p, int who) const {
        return size == 1 ? p : cg::this_cluster().map_shared_rank(p, who);
    }
};

// A warp's segment of the row: chunks of 16 bytes, as memory is aligned, numbered from the one that holds the row's first
// element. Elements of a chunk that are not the row's are held as -inf.
struct Segment {
    const uint4* data;  // chunk c at data[c]
    int32_t c0, c1;
    int32_t off;  // elements before the row's first in chunk 0
};

template <typename T>
struct Work {
    typedef Elem<T> E;
    const Args& A;
    Shared& sh;
    const Team& team;
    Segment s;
    int lane, warp;

    // ------------------------------------------------------------------------------------------------
    // the quick way (bfloat16)
    // ------------------------------------------------------------------------------------------------
    __device__ __forceinline__ void count_one(uint32_t bits, uint32_t o, uint32_t& flags) {
        if (o - 1u < kCodes) {
            const int s = -(int)(bits >> 15 & 1u);
            atomicAdd(&sh.hist[kMid + (((int)o ^ s) - s)], 1u);
            return;
        }
        const uint32_t a = bits & 0x7fffu;
        if (a == 0) atomicAdd(&sh.hist[kMid], 1u);
        else if ((bits & 0xffffu) == 0xff80u) return;  // -inf: not ranked
        else flags |= a >= 0x7f80u ? kNonfinite : kOutside;
    }
    __device__ __forceinline__ void count_values() {
        uint32_t flags = 0;
#pragma unroll 2
        for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
            const uint4 q = s.data[c];
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr uint32_t lo = (kCodeLo - 1) * 0x10001u, hi = (kCodeHi + 1) * 0x10001u;
                const uint32_t o = __vminu2(__vmaxu2(w[i] & 0x7fff7fffu, lo), hi) - lo;
                count_one(w[i], o & 0xffffu, flags);
                count_one(w[i] >> 16, o >> 16, flags);
            }
        }
        flags = __reduce_or_sync(kAll, flags);
        if (lane == 0 && flags) atomicOr(&sh.flags, flags);
    }
    // Value of bin kBins - 1 - d, d in the ranking's order.
    static __device__ __forceinline__ float value_at(int d) {
        const int o = kMid - d;
        const uint32_t a = (uint32_t)(o < 0 ? -o : o);
        return __uint_as_float(a == 0 ? 0u : (o < 0 ? 0x80000000u : 0u) | (kCodeLo - 1 + a) << 16);
    }
    // Of group g of 64 bins, a lane's two: counts and weights.
    __device__ __forceinline__ void pair_at(int g, float m, uint32_t* c, u64* w) {
        const int d = g * kGroupBins + 2 * lane;
        c[0] = d < kBins ? sh.hist[kBins - 1 - d] : 0u;
        c[1] = d + 1 < kBins ? sh.hist[kBins - 2 - d] : 0u;
        w[0] = w[1] = 0;
        if (c[0] | c[1]) {
            const Fixed2 f = weights2(value_at(d), value_at(d + 1), m, sh.par.E, sh.tab);
            w[0] = join(f.ax, f.bx);
            w[1] = join(f.ay, f.by);
        }
    }
    struct Crossing {
        uint32_t n, r, ties;  // tokens up to it, of them in its bin, and the bin's
        u64 sum;              // of the weights up to it
        float thr;
    };
    // The bin in which the count or the sum of the ranking's weights reaches a target that it does reach. Warp 0; `before`:
    // count and sum before the lane's five groups, which hold cl and ml.
    template <bool kMass>
    __device__ __forceinline__ Crossing cross(u64 target, float m, uint32_t c_before, u64 m_before, uint32_t cl, u64 ml) {
        const bool mine = kMass ? m_before < target && target <= m_before + ml : c_before < target && target <= c_before + cl;
        int g = 5 * lane;
        uint32_t pc = c_before;
        u64 pm = m_before;
        if (mine)
#pragma unroll 1
            for (; g < 5 * lane + 4 && (kMass ? pm + sh.group_mass[g] : pc + sh.group_count[g]) < target; ++g) {
                pm += sh.group_mass[g];
                pc += sh.group_count[g];
            }
        const int src = __ffs(__ballot_sync(kAll, mine)) - 1;
        g = __shfl_sync(kAll, g, src);
        pc = __shfl_sync(kAll, pc, src);
        pm = __shfl_sync(kAll, pm, src);
        uint32_t c[2];
        u64 w[2];
        pair_at(g, m, c, w);
        const u64 mass = c[0] * w[0] + c[1] * w[1];
        uint32_t cc = c[0] + c[1];
        const u64 upto = warp_inscan(mass, lane);
        const uint32_t c_upto = (uint32_t)warp_inscan(cc, lane);
        pc += c_upto - cc;
        pm += upto - mass;
        const bool here = kMass ? pm < target && target <= pm + mass : pc < target && target <= pc + cc;
        int i = 0;
        if (kMass ? pm + c[0] * w[0] < target : pc + c[0] < target) {
            i = 1;
            pm += c[0] * w[0];
            pc += c[0];
        }
        const uint32_t ties = i ? c[1] : c[0];
        const u64 wt = i ? w[1] : w[0];
        Crossing x;
        x.r = kMass ? (uint32_t)((target - pm + wt - 1) / (wt ? wt : 1)) : (uint32_t)(target - pc);
        x.ties = ties;
        x.n = pc + x.r;
        x.sum = pm + x.r * wt;
        x.thr = value_at(g * kGroupBins + 2 * lane + i);
        const int at = __ffs(__ballot_sync(kAll, here)) - 1;
        x.r = __shfl_sync(kAll, x.r, at);
        x.ties = __shfl_sync(kAll, x.ties, at);
        x.n = __shfl_sync(kAll, x.n, at);
        x.sum = __shfl_sync(kAll, x.sum, at);
        x.thr = __shfl_sync(kAll, x.thr, at);
        return x;
    }
    // By the first CTA, whose histogram is the row's.
    __device__ __forceinline__ void choose(uint32_t flags) {
        // the largest
        int d_max = kBins;
        for (int d = threadIdx.x; d < kBins; d += kThreads)
            if (sh.hist[kBins - 1 - d]) {
                d_max = d;
                break;
            }
        d_max = __reduce_min_sync(kAll, d_max);
        if (lane == 0) sh.warp_max[warp] = (uint32_t)d_max;
        __syncthreads();
        d_max = (int)__reduce_min_sync(kAll, sh.warp_max[lane % kWarps]);
        const bool any = d_max < kBins;
        const float m = any ? value_at(d_max) : 0.f;
        // groups; and the weights of at least par.least, which are the ranking's first
        const u64 least = sh.par.least;
        uint32_t many = 0;
        int last = -1;
#pragma unroll 1
        for (int g = warp; g < kGroups; g += kWarps) {
            uint32_t c[2];
            u64 w[2];
            pair_at(g, m, c, w);
            uint32_t cc = c[0] + c[1];
            u64 mass = 0;
            if (__any_sync(kAll, cc)) {
                mass = warp_sum(c[0] * w[0] + c[1] * w[1]);
                if (least) {
                    const int d = g * kGroupBins + 2 * lane;
                    if (c[0] && w[0] >= least) many += c[0], last = d;
                    if (c[1] && w[1] >= least) many += c[1], last = d + 1;
                }
                cc = __reduce_add_sync(kAll, cc);
            }
            if (lane == 0) {
                sh.group_count[g] = cc;
                sh.group_mass[g] = mass;
            }
        }
        if (least) {
            many = __reduce_add_sync(kAll, many);
            last = __reduce_max_sync(kAll, last);
        }
        if (lane == 0) {
            sh.warp_above[warp] = many;
            sh.warp_ties[warp] = (uint32_t)(last + 1);
        }
        __syncthreads();
        if (warp > 0) return;
        uint32_t cl = 0;
        u64 ml = 0;
        for (int g = 5 * lane; g < 5 * lane + 5 && g < kGroups; ++g) {
            cl += sh.group_count[g];
            ml += sh.group_mass[g];
        }
        const uint32_t c_upto = (uint32_t)warp_inscan(cl, lane), all = __shfl_sync(kAll, c_upto, 31);
        const u64 m_upto = warp_inscan(ml, lane);
        u64 sum = __shfl_sync(kAll, m_upto, 31);
        const RowPar& R = sh.par;
        Result res{};
        res.m = m;
        res.n = (int32_t)all;
        res.thr = kLowest;  // all that are ranked, unless something says otherwise
        if (R.k > 0 && (uint32_t)R.k < all) {
            const Crossing x = cross<false>((u64)R.k, m, c_upto - cl, m_upto - ml, cl, ml);
            res.thr = x.thr;
            res.r = x.r;
            res.partial = x.r < x.ties;
            res.n = (int32_t)x.n;
            sum = x.sum;
        }
        if (R.p < 1.f && any) {
            const u64 target = max((u64)ceil((double)R.p * (double)sum), (u64)1);
            const Crossing x = cross<true>(min(target, sum), m, c_upto - cl, m_upto - ml, cl, ml);
            if ((int32_t)x.n < res.n) {
                res.thr = x.thr;
                res.r = x.r;
                res.partial = x.r < x.ties;
                res.n = (int32_t)x.n;
            }
        }
        if (least) {
            many = __reduce_add_sync(kAll, lane < kWarps ? sh.warp_above[lane] : 0u);
            last = (int)__reduce_max_sync(kAll, lane < kWarps ? sh.warp_ties[lane] : 0u) - 1;
            if ((int32_t)many < res.n) {
                res.thr = value_at(last);
                res.partial = 0;
                res.n = (int32_t)many;
            }
        }
        if (R.T == 0.f) {
            res.thr = m;
            res.r = 1;
            res.partial = sh.hist[kBins - 1 - min(d_max, kBins - 1)] > 1;
            res.n = 1;
        }
        res.err = R.err | (flags & kNonfinite ? 1u << SV_ERR_NONFINITE : 0u);
        res.slow = (flags & kOutside) != 0;
        if (!any && !res.slow && !(flags & kNonfinite)) res.err |= 1u << SV_ERR_EMPTY_ROW;
        if (lane == 0) sh.res = res;
    }
    // Histograms of the cluster, summed into the first CTA's, a share of the bins by each.
    __device__ __forceinline__ void merge_counts() {
        if (team.size == 1) return;
        const int per = (kHist / 4 + team.size - 1) / team.size, v0 = team.rank * per, v1 = min(v0 + per, kHist / 4);
        for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
            uint4 t = make_uint4(0, 0, 0, 0);
            for (int q = 0; q < team.size; ++q) {
                const uint4 x = reinterpret_cast<const uint4*>(team.of(sh.hist, q))[v];
                t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
            }
            reinterpret_cast<uint4*>(team.of(sh.hist, 0))[v] = t;
        }
        team.sync();
    }
    __device__ __forceinline__ void zero_hist() {
        for (int i = threadIdx.x; i < kHist / 4; i += kThreads) reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
    }

    // ------------------------------------------------------------------------------------------------
    // the slow way
    // ------------------------------------------------------------------------------------------------
    __device__ __forceinline__ uint32_t largest(uint32_t& flags) {
        uint32_t top = 0;
        flags = 0;
#pragma unroll 2
        for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
            float x[E::N];
            E::unpack(s.data[c], x);
#pragma unroll
            for (int e = 0; e < E::N; ++e) {
                const uint32_t k = key_of(x[e]);
                if (k >= kKeyInf || k < kKeyMinusInf) flags = kNonfinite;
                else top = max(top, k);
            }
        }
        flags = __reduce_or_sync(kAll, flags);
        return __reduce_max_sync(kAll, top);
    }
    // One level: the elements whose keys lie in [lo, lo + (bins << shift)), above `floor` and above -inf's, by digit, and
    // the digit at which their counts (or weights, in the ranking's order) reach the target. first: the target is top_p
    // of all weights and `extra`.
    template <bool kMass>
    __device__ __noinline__ Found level(uint32_t lo, int shift, int bins, uint32_t floor, float m, u64 target, bool first, u64 extra) {
        __syncthreads();
        for (int i = threadIdx.x; i < kDigits; i += kThreads) sh.hist[i] = sh.hist[kDigits + i] = 0;
        __syncthreads();
#pragma unroll 1
        for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
            float x[E::N];
            E::unpack(s.data[c], x);
#pragma unroll
            for (int e = 0; e < E::N; e += 2) {
                const uint32_t k[2] = {key_of(x[e]), key_of(x[e + 1])};
                bool in[2];
                uint32_t at[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    at[i] = (k[i] - lo) >> shift;
                    in[i] = k[i] >= lo && at[i] < (uint32_t)bins && k[i] > floor && k[i] > kKeyMinusInf;
                }
                if (!(in[0] || in[1])) continue;
                if (!kMass) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (in[i]) atomicAdd(&sh.hist[at[i]], 1u);
                    continue;
                }
                const Fixed2 f = weights2(x[e], x[e + 1], m, sh.par.E, sh.tab);
                const u64 w[2] = {join(f.ax, f.bx), join(f.ay, f.by)};
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (in[i] && w[i]) {
                        const uint32_t low = (uint32_t)w[i], old = atomicAdd(&sh.hist[at[i]], low);
                        const uint32_t high = (uint32_t)(w[i] >> 32) + (old + low < old);
                        if (high) atomicAdd(&sh.hist[kDigits + at[i]], high);
                    }
            }
        }
        team.sync();
        if (team.size > 1) {
            const int per = (bins + team.size - 1) / team.size, b0 = team.rank * per, b1 = min(b0 + per, bins);
            for (int b = b0 + threadIdx.x; b < b1; b += kThreads) {
                u64 t = 0;
                for (int q = 0; q < team.size; ++q) {
                    const uint32_t* h = team.of(sh.hist, q);
                    t += h[b] + ((u64)h[kDigits + b] << 32);
                }
                uint32_t* h = team.of(sh.hist, 0);
                h[b] = (uint32_t)t;
                h[kDigits + b] = (uint32_t)(t >> 32);
            }
            team.sync();
        }
        if (team.rank == 0) {
            const int per = (bins + kThreads - 1) / kThreads;
            u64 mine = 0;
            for (int i = 0; i < per; ++i) {
                const int b = bins - 1 - (per * (int)threadIdx.x + i);
                if (b >= 0) mine += sh.hist[b] + ((u64)sh.hist[kDigits + b] << 32);
            }
            const u64 upto = warp_inscan(mine, lane);
            if (lane == 31) sh.scan[warp] = upto;
            __syncthreads();
            u64 before = upto - mine, total = 0;
            for (int i = 0; i < kWarps; ++i) {
                if (i < warp) before += sh.scan[i];
                total += sh.scan[i];
            }
            if (first && kMass) {
                const u64 sum = total + extra;
                target = min(max((u64)ceil((double)sh.par.p * (double)sum), (u64)1), sum);
            }
            if (threadIdx.x == 0 && target > total) sh.found = {-1, target - total, 0, total};
            if (before < target && target <= before + mine) {
                int b = bins - 1 - per * (int)threadIdx.x;
                u64 v;
                for (;; --b) {
                    v = sh.hist[b] + ((u64)sh.hist[kDigits + b] << 32);
                    if (target <= before + v) break;
                    before += v;
                }
                sh.found = {b, target - before, v, total};
            }
        }
        team.sync();
        return *team.of(&sh.found, 0);
    }
    // The key at which the counts or weights of the elements above `floor` reach the target; rest: what is left of the
    // target there, value: what its elements come to. False: they do not reach it (rest: by how much).
    template <bool kMass>
    __device__ __forceinline__ bool seek(uint32_t floor, float m, u64 target, u64 extra, uint32_t& key, u64& rest, u64& value) {
        Found f = level<kMass>(0u, 20, kDigits, floor, m, target, true, extra);
        rest = f.rest;
        if (f.bin < 0) return false;
        key = (uint32_t)f.bin << 20;
        f = level<kMass>(key, 8, kDigits, floor, m, f.rest, false, 0);
        key += (uint32_t)f.bin << 8;
        f = level<kMass>(key, 0, 256, floor, m, f.rest, false, 0);
        key += (uint32_t)f.bin;
        rest = f.rest;
        value = f.value;
        return true;
    }
    __device__ __forceinline__ Result choose_slow() {
        const RowPar& R = sh.par;
        uint32_t flags, top = largest(flags);
        __syncthreads();
        if (threadIdx.x == 0) sh.flags = 0, sh.max_key = 0;
        __syncthreads();
        if (lane == 0) {
            if (flags) atomicOr(&sh.flags, flags);
            atomicMax(&sh.max_key, top);
        }
        team.sync();
        flags = top = 0;
        for (int q = 0; q < team.size; ++q) {
            flags |= *team.of(&sh.flags, q);
            top = max(top, *team.of(&sh.max_key, q));
        }
        Result res{};
        res.err = R.err | (flags ? 1u << SV_ERR_NONFINITE : 0u);
        if (!flags && top <= kKeyMinusInf) res.err |= 1u << SV_ERR_EMPTY_ROW;
        res.n = -1;
        if (res.err) return res;
        const float m = res.m = float_of(top);
        res.thr = kLowest;
        if (R.T == 0.f) {
            res.thr = m;
            res.r = 1;
            res.partial = 1;
            return res;
        }
        uint32_t floor = 0;  // keys above it, and r of its own
        u64 ties = 0, r = 0, rest, value;
        if (R.k > 0 && R.k < A.V && seek<false>(0u, m, (u64)R.k, 0, floor, rest, value)) {
            r = rest;
            ties = value;
        }
        if (R.p < 1.f) {
            const u64 w = r ? weight(float_of(floor), m, R.E, sh.tab) : 0;
            uint32_t key;
            if (seek<true>(floor, m, 0, r * w, key, rest, value)) {
                const u64 wk = weight(float_of(key), m, R.E, sh.tab);
                floor = key;
                r = (rest + wk - 1) / wk;
                ties = value / wk;
            } else {
                r = (rest + w - 1) / w;
            }
        }
        if (r) {
            res.thr = float_of(floor);
            res.r = (uint32_t)r;
            res.partial = r < ties;
        }
        if (R.least) {  // the least logit of a weight that is large enough
            __syncthreads();
            if (warp == 0) {
                uint32_t lo = kKeyMinusInf, hi = top;  // lo's weight is too small, hi's is not
                while (hi - lo > 1) {
                    const uint32_t step = (hi - lo + 32) / 33, k = lo + step * (lane + 1);
                    const bool enough = k >= hi || k < lo || weight(float_of(k), m, R.E, sh.tab) >= R.least;
                    const int i = __ffs(__ballot_sync(kAll, enough)) - 1;  // -1: none
                    const uint32_t at = i < 0 ? hi : min(hi, lo + step * (i + 1));
                    lo += step * (i < 0 ? 32 : i);
                    hi = at;
                }
                if (lane == 0) sh.floor = float_of(hi);
            }
            __syncthreads();
            if (sh.floor > res.thr) {
                res.thr = sh.floor;
                res.partial = 0;
            }
        }
        return res;
    }

    // ------------------------------------------------------------------------------------------------
    // with the threshold
    // ------------------------------------------------------------------------------------------------
    // What a warp has of kept tokens: those above the threshold (or at it, where all of these are kept), their weights, and
    // how many are at it.
    template <bool kMass>
    __device__ __forceinline__ void tally(const Result& res) {
        uint32_t above = 0, ties = 0;
        u64 mass = 0;
        int32_t sa = 0, sb = 0;  // of at most 192 weights
        const ExpConst C = sh.par.E;
        const bool whole = !res.partial;
#pragma unroll 1
        for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
            float x[E::N];
            E::unpack(s.data[c], x);
#pragma unroll
            for (int e = 0; e < E::N; e += 2) {
                const bool in0 = x[e] > res.thr || (whole && x[e] == res.thr), in1 = x[e + 1] > res.thr || (whole && x[e + 1] == res.thr);
                if (!whole) ties += (x[e] == res.thr) + (x[e + 1] == res.thr);
                if (!(in0 || in1)) continue;
                above += in0 + in1;
                if (!kMass) continue;
                const Fixed2 f = weights2(x[e], x[e + 1], res.m, C, sh.tab);
                sa += (in0 ? f.ax : 0) + (in1 ? f.ay : 0);
                sb += (in0 ? f.bx : 0) + (in1 ? f.by : 0);
            }
        }
        if (kMass) mass = warp_sum(join(sa, sb));
        above = __reduce_add_sync(kAll, above);
        ties = __reduce_add_sync(kAll, ties);
        if (lane == 0) {
            sh.warp_above[warp] = above;
            sh.warp_ties[warp] = ties;
            sh.warp_mass[warp] = mass;
        }
    }
    // The cluster's tallies in index order, by the first warp of each CTA: how many ties each of its own warps keeps, the
    // count, and the warp that holds the draw.
    template <bool kMass>
    __device__ __forceinline__ void settle(const Result& res) {
        if (warp > 0) return;
        const int all = team.size * kWarps;
        const u64 w = kMass && res.partial && sh.par.T > 0.f ? weight(res.thr, res.m, sh.par.E, sh.tab) : (u64)1 << kBits;
        uint32_t tie_base = 0, above_base = 0;
        u64 mass_base = 0;
        u64 upto[kMaxCtas * kWarps / 32], own[kMaxCtas * kWarps / 32];
#pragma unroll
        for (int i = 0; i < kMaxCtas * kWarps / 32; ++i) {
            const int g = 32 * i + lane;
            if (32 * i >= all) break;
            uint32_t ties = 0, above = 0;
            u64 mass = 0;
            if (g < all) {
                const Shared* o = team.of(&sh, g / kWarps);
                ties = o->warp_ties[g % kWarps];
                above = o->warp_above[g % kWarps];
                if (kMass) mass = o->warp_mass[g % kWarps];
            }
            const uint32_t t = (uint32_t)warp_inscan(ties, lane);
            const int64_t left = (int64_t)res.r - (tie_base + t - ties);
            const uint32_t keeps = !res.partial || left <= 0 ? 0u : (uint32_t)min((int64_t)ties, left);
            if (g < all && g / kWarps == team.rank) sh.ties_kept[g % kWarps] = (int32_t)keeps;
            tie_base += __shfl_sync(kAll, t, 31);
            above_base += __reduce_add_sync(kAll, above + keeps);
            if (kMass) {
                own[i] = mass + keeps * w;
                upto[i] = mass_base + warp_inscan(own[i], lane);
                mass_base = __shfl_sync(kAll, upto[i], 31);
            }
        }
        if (lane == 0) {
            sh.above = above_base;
            sh.total = mass_base;
        }
        if (!kMass) return;
        const u64 target = (u64)((double)sh.par.u * (double)mass_base);  // the running weight must exceed it
#pragma unroll
        for (int i = 0; i < kMaxCtas * kWarps / 32; ++i) {
            if (32 * i >= all) break;
            if (target < upto[i] && target >= upto[i] - own[i]) {
                sh.hit_warp = 32 * i + lane;
                sh.hit_rest = target - (upto[i] - own[i]);
            }
        }
    }
    // The index of the n-th tie of the segment (n >= 1).
    __device__ __forceinline__ int32_t nth_tie(float thr, int32_t n) {
#pragma unroll 1
        for (int32_t c0 = s.c0; c0 < s.c1; c0 += 32) {
            const int32_t c = c0 + lane;
            uint32_t eq = 0;
            if (c < s.c1) {
                float x[E::N];
                E::unpack(s.data[c], x);
#pragma unroll
                for (int e = 0; e < E::N; ++e) eq |= (uint32_t)(x[e] == thr) << e;
            }
            const int32_t upto = (int32_t)warp_inscan((u64)__popc(eq), lane);
            int32_t at = -1;
            if (upto >= n && upto - __popc(eq) < n) {
                for (int32_t i = n - (upto - __popc(eq)); i > 1; --i) eq &= eq - 1;
                at = c * E::N + __ffs(eq) - 1 - s.off;
            }
            at = __reduce_max_sync(kAll, at);
            if (at >= 0) return at;
            n -= __shfl_sync(kAll, upto, 31);
        }
        return A.V;
    }
    // Ties up to this index are kept.
    __device__ __forceinline__ int32_t cut_of(const Result& res) {
        if (!res.partial) return 0x7fffffff;
        const int32_t keeps = sh.ties_kept[warp], ties = (int32_t)sh.warp_ties[warp];
        if (keeps == ties) return 0x7fffffff;
        return keeps == 0 ? -1 : nth_tie(res.thr, keeps);
    }
    __device__ __forceinline__ uint32_t kept_of(const float* x, int32_t i0, const Result& res, int32_t cut) {
        uint32_t k = 0;
#pragma unroll
        for (int e = 0; e < E::N; ++e) k |= (uint32_t)(x[e] > res.thr || (x[e] == res.thr && i0 + e <= cut)) << e;
        return k;
    }
    // The draw, by the warp that holds it: the first kept token whose running weight exceeds `target`.
    __device__ __forceinline__ void pick(const Result& res, int32_t row, u64 target) {
        const int32_t cut = cut_of(res);
        const RowPar& R = sh.par;
        u64 base = 0;
#pragma unroll 1
        for (int32_t c0 = s.c0; c0 < s.c1; c0 += 32) {
            const int32_t c = c0 + lane;
            u64 w[E::N], sum = 0;
            float x[E::N];
#pragma unroll
            for (int e = 0; e < E::N; ++e) w[e] = 0;
            if (c < s.c1) {
                E::unpack(s.data[c], x);
                const uint32_t k = kept_of(x, c * E::N - s.off, res, cut);
#pragma unroll
                for (int e = 0; e < E::N; e += 2)
                    if (k >> e & 3u) {
                        Fixed2 f{1 << 22, 1 << 22, 0, 0};
                        if (R.T > 0.f) f = weights2(x[e], x[e + 1], res.m, R.E, sh.tab);
                        w[e] = k >> e & 1u ? join(f.ax, f.bx) : 0;
                        w[e + 1] = k >> e & 2u ? join(f.ay, f.by) : 0;
                    }
#pragma unroll
                for (int e = 0; e < E::N; ++e) sum += w[e];
            }
            const u64 upto = base + warp_inscan(sum, lane);
            if (target < upto && target >= upto - sum) {
                u64 run = upto - sum;
                int at = -1;
#pragma unroll
                for (int e = 0; e < E::N; ++e) {
                    run += w[e];
                    if (at < 0 && run > target) at = e;
                }
                float l = x[0];
#pragma unroll
                for (int e = 1; e < E::N; ++e) l = e == at ? x[e] : l;
                A.tokens[row] = c * E::N + at - s.off;
                // l - m in float is exact or far below the result's rounding
                if (A.logprob)
                    A.logprob[row] = R.T > 0.f ? (float)(((double)l - res.m) / R.T - (log((double)sh.total) - kBits * 0.6931471805599453)) : 0.f;
            }
            base = __shfl_sync(kAll, upto, 31);
            if (target < base) return;
        }
    }
    // The segment with -inf where a token is not kept (copy: as it is).
    __device__ __forceinline__ void write(const Result& res, int32_t row, bool copy) {
        typedef typename E::Bits Bits;
        const int32_t cut = copy ? 0 : cut_of(res);
        Bits* out = (Bits*)A.out + (int64_t)row * A.out_stride;
        const int32_t o_off = (int32_t)((uintptr_t)out % 16 / sizeof(Bits));
        if (o_off == s.off) {
#pragma unroll 2
            for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
                const uint4 q = s.data[c];
                float x[E::N];
                E::unpack(q, x);
                const int32_t i0 = c * E::N - s.off;
                const uint32_t k = copy ? ~0u : kept_of(x, i0, res, cut);
                const uint4 y = E::masked(q, k);
                if (i0 >= 0 && i0 + E::N <= A.V) {
                    *reinterpret_cast<uint4*>(out + i0) = y;
                } else {
                    const Bits* b = reinterpret_cast<const Bits*>(&y);
#pragma unroll
                    for (int e = 0; e < E::N; ++e)
                        if (i0 + e >= 0 && i0 + e < A.V) out[i0 + e] = b[e];
                }
            }
            return;
        }
        // chunks of the output, which begin elsewhere
        const Bits* in = reinterpret_cast<const Bits*>(s.data) + s.off;  // element i at in[i]
        const int32_t e0 = max(0, s.c0 * E::N - s.off), e1 = min(A.V, s.c1 * E::N - s.off);
#pragma unroll 1
        for (int32_t c = (e0 + o_off) / E::N + lane; c * E::N - o_off < e1; c += 32) {
            const int32_t i0 = c * E::N - o_off;
            Bits b[E::N];
#pragma unroll
            for (int e = 0; e < E::N; ++e) {
                const int32_t i = i0 + e;
                b[e] = E::bits_minus_inf;
                if (i >= e0 && i < e1) {
                    const float x = E::value(in[i]);
                    if (copy || x > res.thr || (x == res.thr && i <= cut)) b[e] = in[i];
                }
            }
            if (i0 >= e0 && i0 + E::N <= e1) {
                uint4 y;
                memcpy(&y, b, 16);
                *reinterpret_cast<uint4*>(out + i0) = y;
            } else {
#pragma unroll
                for (int e = 0; e < E::N; ++e)
                    if (i0 + e >= e0 && i0 + e < e1) out[i0 + e] = b[e];
            }
        }
    }
};

// What the row's request asks for, by one thread.
__device__ __forceinline__ void read_par(const Args& A, RowPar& R, int32_t row, bool draws) {
    R = RowPar{};
    R.T = 1.f;
    R.p = 1.f;
    int32_t q = row;
    if (A.request) q = A.request[row];
    bool ok = q >= 0 && q < A.requests;
    if (ok) {
        if (A.temperature) R.T = A.temperature[q];
        if (A.top_k) R.k = max(A.top_k[q], 0);
        if (A.top_p) R.p = A.top_p[q];
        float mp = A.min_p ? A.min_p[q] : 0.f;
        if (draws) R.u = A.uniforms[row];
        ok = R.T >= 0.f && R.T < INFINITY && R.p == R.p && mp == mp && R.u >= 0.f && R.u < 1.f;
        if (mp > 0.f) R.least = max((u64)ceil((double)fminf(mp, 1.f) * (double)((u64)1 << kBits)), (u64)1);
    }
    if (ok && R.T > 0.f) {
        const double K = 1.4426950408889634074 / (double)R.T;
        R.E.K_hi = (float)K;
        R.E.K_lo = (float)(K - (double)R.E.K_hi);
        R.E.d_min = (float)(-126.5 / (double)R.E.K_hi);
        ok = R.E.K_hi < INFINITY;
    }
    if (!ok) R.err = 1u << SV_ERR_INVALID_ARG;
    if (R.T == 0.f) R.least = 0;  // the first alone, whatever its weight
}

template <typename T, bool kDraws>
__global__ void __launch_bounds__(kThreads, 2) k_rows(const __grid_constant__ Args A, int32_t C) {
    typedef Elem<T> E;
    extern __shared__ __align__(16) char raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    uint4* held = reinterpret_cast<uint4*>(raw + sizeof(Shared));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Team team{(int)(blockIdx.x % (unsigned)C), C};
    const int32_t row = (int32_t)(blockIdx.x / (unsigned)C);
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the segment on its way
    const T* base = (const T*)A.logits + (int64_t)row * A.stride;
    Segment s;
    s.off = (int32_t)((uintptr_t)base % 16 / sizeof(T));
    const int32_t chunks = (s.off + A.V + E::N - 1) / E::N;
    const int parts = C * kWarps, part = team.rank * kWarps + warp;
    s.c0 = (int32_t)((int64_t)chunks * part / parts);
    s.c1 = (int32_t)((int64_t)chunks * (part + 1) / parts);
    const int32_t first = (int32_t)((int64_t)chunks * (team.rank * kWarps) / parts);  // of the CTA
    s.data = held - first;
    for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
        const int32_t i0 = c * E::N - s.off;
        if (i0 >= 0 && i0 + E::N <= A.V) {
            cp_async16(held + (c - first), base + i0);
        } else {
            typename E::Bits b[E::N];
#pragma unroll
            for (int e = 0; e < E::N; ++e)
                b[e] = i0 + e >= 0 && i0 + e < A.V ? reinterpret_cast<const typename E::Bits*>(base)[i0 + e] : E::bits_minus_inf;
            memcpy(held + (c - first), b, 16);
        }
    }
    cp_async_commit();
    if (tid < 128) {
        sh.tab[tid] = A.exp2_tab[tid].x;
        sh.tab[kExpTab + tid] = A.exp2_tab[tid].y;
    }
    if (tid == kThreads - 1) {
        sh.flags = 0;
        sh.hit_warp = -1;
        read_par(A, sh.par, row, kDraws);
    }
    Work<T> work{A, sh, team, s, lane, warp};
    constexpr bool kQuick = sizeof(T) == 2;
    if (kQuick) work.zero_hist();
    __syncthreads();
    cp_async_wait<0>();
    __syncwarp();

    Result res{};
    res.slow = 1;
    if (kQuick) {
        work.count_values();
        team.sync();
        work.merge_counts();
        if (team.rank == 0) {
            uint32_t flags = 0;
            for (int q = 0; q < C; ++q) flags |= *team.of(&sh.flags, q);
            work.choose(flags);
        }
        team.sync();
        res = *team.of(&sh.res, 0);
    }
    if (res.slow) res = work.choose_slow();

    const bool ok = !res.err;
    bool told = false;  // the row's count is known
    if (ok && (kDraws || res.partial || res.n < 0)) {
        __syncthreads();
        work.template tally<kDraws>(res);
        team.sync();
        work.template settle<kDraws>(res);
        told = true;
        __syncthreads();
    }
    if (C > 1) team.arrive();  // nothing of another CTA is read from here on
    if (ok && kDraws) {
        if (sh.hit_warp == part) work.pick(res, row, sh.hit_rest);
    } else if (!kDraws) {
        work.write(res, row, !ok);
    }
    if (team.rank == 0 && tid == 0) {
        if (A.kept) A.kept[row] = !ok ? -1 : told ? (int32_t)sh.above : res.n;
        if (!ok) {
            if (kDraws) {
                A.tokens[row] = -1;
                if (A.logprob) A.logprob[row] = NAN;
            }
            if (A.status) atomicOr(A.status, res.err);
        }
    }
    if (C > 1) team.wait();
}

// CTAs of a row: as few as hold it, then more while the launch leaves SMs idle and a slice is worth a CTA.
constexpr int kSmem2 = 113 * 1024, kSmem1 = 227 * 1024;  // of a CTA, two and one an SM
constexpr int kLeast = 2048;                             // elements of a slice

template <typename T, bool kDraws>
cudaError_t launch(const Args& A, cudaStream_t st) {
    int dev, sms;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t chunks = (A.V + Elem<T>::N - 1) / Elem<T>::N + 1;
    auto bytes = [&](int c) { return (int64_t)sizeof(Shared) + ((chunks + c - 1) / c + 1) * 16; };
    int C = 1;
    while (C < kMaxCtas && bytes(C) > kSmem2) C *= 2;
    while (C < kMaxCtas && (int64_t)A.rows * C <= sms && A.V / (2 * C) >= kLeast) C *= 2;
    auto kernel = k_rows<T, kDraws>;
    if (bytes(C) > kSmem1 || (int64_t)A.rows * C > 0x7fffffff) return cudaErrorInvalidValue;
    // the devices on which the kernel may use an SM's shared memory: setting that twice does no harm
    static std::atomic<unsigned long long> allowed{0};
    if (dev >= 64 || !(allowed.load() >> dev & 1u)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem1);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed.fetch_or(1ull << dev);
    }
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)A.rows * (unsigned)C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)bytes(C);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, A, (int32_t)C);
}

struct ExpTable {  // 2^(j / 128) as two floats each
    float2 v[128];
    ExpTable() {
        for (int j = 0; j < 128; ++j) {
            const double x = std::exp2(j / 128.0);
            v[j].x = (float)x;
            v[j].y = (float)(x - (double)v[j].x);
        }
    }
};

// Whether a call is valid, and its common arguments. rows == 0 leaves nothing to do.
bool common(Args& A, const void* logits, int dtype, int32_t rows, int32_t V, int64_t stride, const sv_filter* f, int32_t* kept,
            uint32_t* status) {
    if (dtype != SV_F32 && dtype != SV_BF16) return false;
    if (rows < 0 || V < 1 || V > SV_MAX_FILTER_V || !f || f->reserved != 0) return false;
    if (stride < V || stride >= (int64_t)1 << 38) return false;
    for (const void* p : {(const void*)f->temperature, (const void*)f->top_k, (const void*)f->top_p, (const void*)f->min_p,
                          (const void*)f->request, (const void*)kept, (const void*)status})
        if ((uintptr_t)p % 4) return false;
    if (f->requests < (f->request ? 1 : rows)) return false;
    if (rows > 0 && (!logits || (uintptr_t)logits % (dtype == SV_BF16 ? 2 : 4))) return false;
    A.logits = logits;
    A.stride = stride;
    A.temperature = f->temperature;
    A.top_k = f->top_k;
    A.top_p = f->top_p;
    A.min_p = f->min_p;
    A.request = f->request;
    A.requests = f->requests;
    A.rows = rows;
    A.V = V;
    A.kept = kept;
    A.status = status;
    static const ExpTable table;
    memcpy(A.exp2_tab, table.v, sizeof table.v);
    return true;
}

int result(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

}  // namespace
}  // namespace sample
}  // namespace sv

using namespace sv::sample;

extern "C" {

int spec_filter(const void* logits, sv_dtype dtype, int32_t rows, int32_t V, int64_t stride, const sv_filter* filter, void* out,
                int64_t out_stride, int32_t* out_kept, uint32_t* device_status, void* cuda_stream) {
    Args A{};
    if (!common(A, logits, dtype, rows, V, stride, filter, out_kept, device_status)) return SV_ERR_INVALID_ARG;
    if (out_stride < V || out_stride >= (int64_t)1 << 38) return SV_ERR_INVALID_ARG;
    if (rows == 0) return SV_OK;
    if (!out || (uintptr_t)out % (dtype == SV_BF16 ? 2 : 4)) return SV_ERR_INVALID_ARG;
    if (out == logits && out_stride != stride) return SV_ERR_INVALID_ARG;
    A.out = out;
    A.out_stride = out_stride;
    const auto st = (cudaStream_t)cuda_stream;
    return result(dtype == SV_BF16 ? launch<__nv_bfloat16, false>(A, st) : launch<float, false>(A, st));
}

int spec_sample(const void* logits, sv_dtype dtype, int32_t rows, int32_t V, int64_t stride, const sv_filter* filter,
                const float* uniforms, int32_t* out_tokens, float* out_logprob, int32_t* out_kept, uint32_t* device_status,
                void* cuda_stream) {
    Args A{};
    if (!common(A, logits, dtype, rows, V, stride, filter, out_kept, device_status)) return SV_ERR_INVALID_ARG;
    if ((uintptr_t)out_logprob % 4) return SV_ERR_INVALID_ARG;
    if (rows == 0) return SV_OK;
    if (!uniforms || (uintptr_t)uniforms % 4 || !out_tokens || (uintptr_t)out_tokens % 4) return SV_ERR_INVALID_ARG;
    A.uniforms = uniforms;
    A.tokens = out_tokens;
    A.logprob = out_logprob;
    const auto st = (cudaStream_t)cuda_stream;
    return result(dtype == SV_BF16 ? launch<__nv_bfloat16, true>(A, st) : launch<float, true>(A, st));
}

}  // extern "C"
