// spec_filter and spec_sample (include/specsample.h): temperature, top-k, top-p and min-p on rows of logits.
//
// Mathematics. The kept tokens are the first n of the ranking by logit, so a row's filter is a threshold: the logits above
// it are kept, and of those equal to it the first r by index. A weight is w = 2^((l - m) K), K = log2(e) / T, held as an
// integer W = round(2^44 w); sums of them are exact, and so is every comparison of sums (top-p's crossing, the inverse
// CDF's): the order in which threads add does not matter, and a draw differs from one in real numbers only where its
// target lies within the weights' own errors, some 2^-31 of each, of a border. min-p compares logits.
//
// Three ways to the threshold.
// - Few candidates. With top-k (up to a CTA's threads), with min-p alone and for T = 0 most logits are known to be too low
//   from the threads' largest ones. The others, some hundred, are gathered in a list and sorted, one a thread: what is kept
//   and what is drawn follows from prefix sums of their weights.
// - Quick bins. A bfloat16 logit has few values: between 2^-26 and 2^10 each has a bin of its own (one more is zero's), a
//   row's histogram of counts says it all, and weights are needed for the bins that hold something only. The draw's
//   place is then found from the CTAs' histograms, from shares of one CTA's slice, and in one share.
// - The slow way, for float and where a logit lies outside the quick bins: top-p's crossing from a histogram of the weights
//   over bins that are even in their logarithms, and the list for the one bin it lies in; where that has too many logits, and for
//   larger top-k, the threshold's 32-bit key 12, 12 and 8 bits at a time from histograms of what is still in question.
//
// Shape. A row is a cluster's of up to 8 CTAs, a warp of which has a contiguous segment of it. Where the rows fit the GPU at
// once, they are held in shared memory: one read from memory, however many passes follow. Else one CTA of 1024 threads an
// SM takes a row where it lies, each pass from the end at which the last one stopped, so that L2 has most of it (704 rows
// of 128256: 188 MB read from memory, about the rows once), and brings the next one's first bytes there before it writes.
//
// What bounds it: small batches a chain of short steps (load, survey, gather, sort, sums: a block or cluster barrier and one to
// three us each; one row of 32000 14.5 to 15.5 us), many rows the same steps with nothing else on the SM meanwhile, though a row
// is read from memory once (704 rows filtered, a filter for each sequence: 141 to 146 us, 0.37 of the copy rate; before
// the next row was brought, 153, and 163 and 246 with 2 and 4 CTAs an SM). 64 rows of 128256, nucleus alone: 33 us, 12 of them counting and finding the threshold, 9 drawing.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/specsample.h"
#include "sv_device.cuh"
#include "sv_sample_words.h"

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

constexpr int kMostThreads = 1024, kMostWarps = kMostThreads / 32, kMaxCtas = 8;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kBits = 44;  // of a weight's fraction; 2^18 weights of 1 sum to 2^62
constexpr float kLowest = -3.402823466e38f;
// l - m in float may be minus infinity, which is a weight of 0; up to this temperature it is one (2^-490 and less)
constexpr float kMostTemperature = 1e36f;

// The bins of the quick way, in the ranking's order: one for each bfloat16 magnitude code in [kCodeLo, kCodeHi] of either sign, one
// in the middle for zero, and one at either end that counts for nothing (the last has -inf). Their words lie in the order
// of the magnitudes: zero and the positive ones, from kNegative on zero (-0.0) and the negative ones.
constexpr uint32_t kCodeLo = 0x3280u, kCodeHi = 0x447fu;  // 2^-26, 1020
constexpr uint32_t kCodes = kCodeHi - kCodeLo + 1;
constexpr int kMid = kCodes + 1, kBins = 2 * kMid + 1, kNegative = kMid + 1;
constexpr int kGroupBins = 64, kGroups = (kBins + kGroupBins - 1) / kGroupBins;
constexpr int kHist = kGroups * kGroupBins;  // words
constexpr int kDigits = 4608;                // bins of the other way: two words each
static_assert(2 * kDigits <= kHist, "the histogram's words serve both ways");
static_assert(kGroups <= 160, "five groups a lane");

typedef unsigned long long u64;

struct RowPar {
    ExpConst E;
    float T, p, u;
    double per;     // 1 / T
    double drop;    // T ln min_p: a kept logit is this far below the largest at most
    int32_t k;      // 0: none
    int32_t drops;  // whether there is such a bound
    uint32_t err;
};

struct Result {
    float thr;        // logits above it are kept; and those equal to it, all or (partial) the first r by index
    uint32_t r;
    int32_t partial;
    int32_t n;        // kept, -1: not known yet
    float m;          // the largest logit
    uint32_t err;
    int32_t slow;     // the quick way could not tell
    int32_t listed;   // ranked from a list: a tie is kept up to index `cut`
    int32_t cut;
    int32_t at;       // quick: the threshold's place among the bins
    uint32_t ties;    // quick: logits equal to it
    u64 mass;         // quick: of those above the threshold (and equal to it, where all are kept)
};

// A row whose kept tokens lie among few: those candidates, in the first CTA's shared memory (the histogram's place).
struct List {
    u64 order[kMostThreads];      // key << 32 | ~index: larger is earlier in the ranking
    u64 trade[2][kMostThreads];   // for the sort
};

struct Found {  // a level of the slow way
    int32_t bin;    // -1: the target lies past all bins
    u64 rest;       // what is left of the target within the bin, or past all
    u64 value;      // of the bin
};

// What a CTA, or a warp, has: the weights and the number of its logits above the threshold (or at it, where all of those are
// kept), and how many are at it, where some are.
struct Part {
    u64 mass;
    uint32_t above, ties;
};

struct alignas(16) Shared {
    uint32_t hist[kHist];
    float tab[2 * kExpTab];
    u64 group_mass[kGroups + 1];
    uint32_t group_count[kGroups + 1];
    u64 scan[kMostWarps];
    Part warp_part[kMostWarps], part;  // part: the CTA's
    uint32_t tops[kMostThreads], warp_max[kMostWarps], warp_min[kMostWarps];  // keys of the threads' largest
    uint32_t max_key, low_key, share_key;  // the CTA's largest logit, the least that it counts, and the least of its share of k
    uint32_t listed;                       // candidates
    uint32_t flags;
    RowPar par;
    Result res;
    Found found;
    int32_t hit;      // the CTA, then the warp of the cluster, that holds the drawn token
    u64 hit_rest, total;
    uint32_t keeps;   // of the ties of the CTA (filter) or of the CTA that holds the draw
    int32_t warp_keeps[kMostWarps], n;
    int32_t token;
    float logit;
    double log_total;
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
constexpr uint32_t kKeyMinusInf = 0x007fffffu;

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
    // a chunk with the elements from `least` on as they are and the others -inf
    static __device__ __forceinline__ uint4 keep(const uint4& q, float least) {
        return make_uint4(__uint_as_float(q.x) >= least ? q.x : kMinusInf, __uint_as_float(q.y) >= least ? q.y : kMinusInf,
                          __uint_as_float(q.z) >= least ? q.z : kMinusInf, __uint_as_float(q.w) >= least ? q.w : kMinusInf);
    }
    // which of them are from `least` on
    static __device__ __forceinline__ uint32_t from(const uint4& q, float least) {
        return (uint32_t)(__uint_as_float(q.x) >= least) | (uint32_t)(__uint_as_float(q.y) >= least) << 1 |
               (uint32_t)(__uint_as_float(q.z) >= least) << 2 | (uint32_t)(__uint_as_float(q.w) >= least) << 3;
    }
    static __device__ __forceinline__ float next(float x) { return float_of(key_of(x) + 1u); }
    // the least value of the type from x on
    static __device__ __forceinline__ float up(float x) { return x; }
    // how many are x
    static __device__ __forceinline__ uint32_t equal(const uint4& q, float x) {
        return (uint32_t)(__uint_as_float(q.x) == x) + (uint32_t)(__uint_as_float(q.y) == x) + (uint32_t)(__uint_as_float(q.z) == x) +
               (uint32_t)(__uint_as_float(q.w) == x);
    }
    // the largest so far, NaN from the first NaN on
    static __device__ __forceinline__ void larger(uint32_t& top, const uint4& q) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+r"(top) : "r"(w[i]));
    }
    static __device__ __forceinline__ float largest(uint32_t top) { return __uint_as_float(top); }
    static constexpr uint32_t kNone = kMinusInf;
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
    static __device__ __forceinline__ uint32_t from2(uint32_t w, __nv_bfloat162 least) {
        return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w), least);
    }
    static __device__ __forceinline__ uint4 keep(const uint4& q, float least) {
        const __nv_bfloat162 l = __float2bfloat162_rn(least);
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = from2(w[i], l);
            w[i] = (w[i] & m) | (0xff80ff80u & ~m);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ uint32_t from(const uint4& q, float least) {
        const __nv_bfloat162 l = __float2bfloat162_rn(least);
        const uint32_t m[4] = {from2(q.x, l), from2(q.y, l), from2(q.z, l), from2(q.w, l)};
        if (!(m[0] | m[1] | m[2] | m[3])) return 0;
        uint32_t k = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) k |= ((m[i] & 1u) | (m[i] >> 15 & 2u)) << 2 * i;
        return k;
    }
    static __device__ __forceinline__ float next(float x) { return float_of(key_of(x) + 0x10000u); }
    static __device__ __forceinline__ float up(float x) { return __bfloat162float(__float2bfloat16_ru(x)); }
    static __device__ __forceinline__ uint32_t equal(const uint4& q, float x) {
        const __nv_bfloat162 v = __float2bfloat162_rn(x);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n += (uint32_t)__popc(__heq2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), v));
        return n / 16;
    }
    static __device__ __forceinline__ void larger(uint32_t& top, const uint4& q) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w[i]));
    }
    static __device__ __forceinline__ float largest(uint32_t top) {
        const float a = bf16lo_to_f32(top), b = bf16hi_to_f32(top);
        return a != a ? a : b != b ? b : fmaxf(a, b);
    }
    static constexpr uint32_t kNone = 0xff80ff80u;
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

// Chunks of 16 bytes of the row, as memory is aligned, numbered from the one that holds the row's first element. Elements of
// a chunk that are not the row's are held as -inf. (Of a warp's own slice, or in another CTA.)
struct Segment {
    const uint4* data;  // chunk c at data[c]
    int32_t c0, c1;
};

// ceil(f x) or floor(f x) for f in [0, 1), exactly: f is 24 bits and an exponent.
__device__ __forceinline__ u64 scaled(u64 x, float f, bool up) {
    if (!(f > 0.f)) return 0;
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const u64 m = e ? (b & 0x7fffffu) | 0x800000u : b;
    const int shift = 150 - (int)max(e, 1u);  // f = m 2^-shift, shift >= 24
    const u64 hi = __umul64hi(x, m), lo = x * m;
    u64 q, rest;
    if (shift < 64) {
        q = hi << (64 - shift) | lo >> shift;
        rest = lo & (((u64)1 << shift) - 1);
    } else {
        q = shift < 128 ? hi >> (shift - 64) : 0;
        rest = 1;  // of no matter below 1, and never exactly none: x m < 2^86
        if (shift < 128) rest = lo | (hi & (((u64)1 << (shift - 64)) - 1));
        else rest = x;
    }
    return q + (up && rest);
}
// ceil(a / b) where it is at most 2^18 (or so): the quotient in float is off by less than one, and one is taken off it, so that
// four steps are enough. (And no more are made, for a row that someone writes to while it is read where it lies may say
// anything.)
__device__ __forceinline__ uint32_t div_up(u64 a, u64 b) {
    if (b == 0) return 1;
    uint32_t q = (uint32_t)__fdividef((float)a, (float)b);
    if (q > 0) --q;
#pragma unroll 1
    for (int i = 0; i < 4 && q * b < a; ++i) ++q;
    return q;
}

// kHeld: the slice lies in shared memory; else it is read where the logits are, again in every pass (from L2, mostly).
template <typename T, bool kHeld>
struct Work {
    typedef Elem<T> E;
    // held rows: two CTAs an SM; others: one, as fewer rows at a time leave more of each in L2 (704 rows of 128256 bf16, the next not brought yet: 153 us,
    // with two of 512 threads 163, with four of 256 246)
    static constexpr int kThreads = kHeld ? 512 : 1024, kWarps = kThreads / 32;
    static constexpr int kList = kThreads;  // candidates that the first CTA ranks, a thread each
    const Args& A;
    Shared& sh;
    const Team& team;
    Segment s;    // the warp's
    int32_t off;  // elements before the row's first in chunk 0
    int32_t full0;   // the first chunk that is all the row's, and how many there are
    uint32_t fulls;
    int lane, warp;
    float low;    // logits below it decide nothing

    // A chunk that is not all the row's.
    __device__ __noinline__ uint4 edge(const Segment& g, int32_t c) const {
        typedef typename E::Bits Bits;
        const Bits* p = reinterpret_cast<const Bits*>(g.data) + off;
        const int32_t i0 = c * E::N - off;
        Bits b[E::N];
#pragma unroll
        for (int e = 0; e < E::N; ++e) b[e] = i0 + e >= 0 && i0 + e < A.V ? p[i0 + e] : (Bits)E::bits_minus_inf;
        uint4 q;
        memcpy(&q, b, 16);
        return q;
    }
    __device__ __forceinline__ uint4 chunk(const Segment& g, int32_t c) const {
        if (kHeld || (uint32_t)(c - full0) < fulls) return g.data[c];
        return edge(g, c);
    }
    // All chunks of the warp's segment, four reads at a time. back: from the end on, as the pass after one from the beginning
    // does: what that one read last is still in L2.
    template <typename F>
    __device__ __forceinline__ void each(F&& f, bool back = false) const {
        const int32_t n = (s.c1 - s.c0 + 127) / 128;
#pragma unroll 1
        for (int32_t i = 0; i < n; ++i) {
            const int32_t c0 = s.c0 + lane + 128 * (back ? n - 1 - i : i);
            uint4 q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + 32 * k < s.c1) q[k] = chunk(s, c0 + 32 * k);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + 32 * k < s.c1) f(c0 + 32 * k, q[k]);
        }
    }

    __device__ __forceinline__ List& list() const { return reinterpret_cast<List&>(sh.hist); }
    // The logits that f tells (by a bit each) of a chunk, into the first CTA's list, in any order.
    template <typename F>
    __device__ __forceinline__ void collect(F&& f) const {
        typedef typename E::Bits Bits;
        List* to = team.of(&list(), 0);
        uint32_t* count = team.of(&sh.listed, 0);
        const Bits* p = reinterpret_cast<const Bits*>(s.data);
        const int32_t turns = (s.c1 - s.c0 + 127) / 128;
#pragma unroll 1
        for (int32_t t = turns - 1; t >= 0; --t) {
            const int32_t c0 = s.c0 + 128 * t;
            uint4 q[4];
            uint32_t in = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + 32 * k + lane < s.c1) q[k] = chunk(s, c0 + 32 * k + lane);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + 32 * k + lane < s.c1) in |= f(q[k]) << k * E::N;
            if (!__any_sync(kAll, in)) continue;
            // one count for the warp's
            const uint32_t n = (uint32_t)__popc(in), upto = (uint32_t)warp_inscan(n, lane);
            uint32_t at = 0;
            if (lane == 31) at = atomicAdd(count, upto);
            at = __shfl_sync(kAll, at, 31) + upto - n;
#pragma unroll 1
            for (; in; in &= in - 1, ++at) {
                const int bit = __ffs(in) - 1;
                const int32_t i = (c0 + 32 * (bit / E::N) + lane) * E::N + bit % E::N;  // from chunk 0 on
                if (at < kList) to->order[at] = (u64)key_of(E::value(p[i])) << 32 | (uint32_t)~(i - off);
            }
        }
    }

    // The same part of the row `ahead` rows on, which this SM takes next or nearly, into L2: whole chunks, in its bounds. Measured,
    // in turn: 704 rows filtered 152.6 us without, 147.4 with it once the threshold is known, 148.1 before the candidates are
    // sorted, 150.3 before they are gathered; 128 float rows 121.8 and 122.2.
    __device__ __forceinline__ void bring(const T* base, int32_t row, int32_t ahead) const {
        if (ahead <= 0 || row >= A.rows - ahead || lane > 0) return;
        const T* next = base + (int64_t)ahead * A.stride;
        const int32_t o = (int32_t)((uintptr_t)next % 16 / sizeof(T));
        const int32_t c0 = max(s.c0, (int32_t)(o > 0)), c1 = min(s.c1, (o + A.V) / E::N);
        if (c0 < c1)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(next - o + (int64_t)c0 * E::N)),
                         "r"((uint32_t)(c1 - c0) * 16u)
                         : "memory");
    }

    // ------------------------------------------------------------------------------------------------
    // the largest, and what lies too low to matter
    // ------------------------------------------------------------------------------------------------
    // The key of a thread's largest, and whether it met a NaN or +inf.
    __device__ __forceinline__ uint32_t largest(uint32_t& flags) const {
        uint32_t top = E::kNone;
        each([&](int32_t, const uint4& q) { E::larger(top, q); });
        const float x = E::largest(top);
        flags = x < INFINITY ? 0u : (uint32_t)kNonfinite;
        return x < INFINITY ? key_of(x) : kKeyMinusInf;
    }
    // Of the threads' largest logits, whose keys are in `tops`: a logit that `many` of them reach, the largest such or nearly.
    // By a warp; the CTA's largest is `high`, the least of the threads' `low`.
    static __device__ __forceinline__ uint32_t reached(const uint32_t* tops, int many, uint32_t low_key, uint32_t high_key) {
        uint32_t x[kThreads / 32];
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) x[i] = tops[32 * i + (threadIdx.x & 31)];
        float low = low_key <= kKeyMinusInf ? -INFINITY : float_of(low_key), high = float_of(high_key), step = 4.f;
#pragma unroll 1
        for (int i = 0; i < 9; ++i) {  // low: `many` threads at least reach it
            const float mid = low > -INFINITY ? 0.5f * low + 0.5f * high : high - step;
            if (!(mid > low && mid < high)) break;
            const uint32_t key = key_of(mid);
            int n = 0;
#pragma unroll
            for (int k = 0; k < kThreads / 32; ++k) n += x[k] >= key;
            if (__reduce_add_sync(kAll, n) >= many) low = mid;
            else high = mid;
            step *= 4.f;
        }
        return low > -INFINITY ? key_of(low) : kKeyMinusInf;
    }
    // The CTA's largest, and the least logit that decides anything, with a block barrier at the end. With top-k, k up to the
    // threads of a CTA: if k threads have a logit of x or more, what is below x is not among the first k of the ranking;
    // and if in every CTA of the row k / C of them have x or more, neither. With min-p alone: those that it does not keep of
    // the CTA's.
    __device__ __forceinline__ void survey() {
        uint32_t flags;
        const uint32_t top = largest(flags);
        flags = __reduce_or_sync(kAll, flags);
        const uint32_t hi = __reduce_max_sync(kAll, top), lo = __reduce_min_sync(kAll, top);
        sh.tops[threadIdx.x] = top;
        if (lane == 0) {
            sh.warp_max[warp] = hi;
            sh.warp_min[warp] = lo;
            if (flags) atomicOr(&sh.flags, flags);
        }
        __syncthreads();
        const uint32_t high = __reduce_max_sync(kAll, sh.warp_max[lane % kWarps]);
        uint32_t low = kKeyMinusInf, share = kKeyMinusInf;
        const RowPar& R = sh.par;
        if (R.T == 0.f) {
            low = high;
        } else if (R.k > 0 && R.k <= kThreads) {
            low = __reduce_min_sync(kAll, sh.warp_min[lane % kWarps]);
            if (warp == 0) low = reached(sh.tops, R.k, low, high);
            if (warp == 1) share = reached(sh.tops, (R.k + team.size - 1) / team.size, low, high);
        } else if (R.drops && !(R.p < 1.f)) {
            low = key_of(floor_of(float_of(high)));
        }
        if (threadIdx.x == 0) {
            sh.max_key = high;
            sh.low_key = low;
        }
        if (threadIdx.x == 32) sh.share_key = share;
        __syncthreads();
    }
    // The least logit of the row that decides anything, from all CTAs' surveys.
    __device__ __forceinline__ float row_low() const {
        const RowPar& R = sh.par;
        uint32_t low = 0, share = ~0u;
        if (lane < team.size) {
            low = *team.of(&sh.low_key, lane);
            share = *team.of(&sh.share_key, lane);
        }
        low = __reduce_max_sync(kAll, low);  // (of top-k any CTA's will do, of the others the largest logit's)
        share = __reduce_min_sync(kAll, share);
        if (R.T > 0.f && R.k > 0) low = max(low, share);
        float f = low <= kKeyMinusInf ? -INFINITY : float_of(low);
        if (sizeof(T) == 2) f = __bfloat162float(__float2bfloat16_rd(f));
        return f;
    }
    // The least logit that min-p keeps of a row whose largest is m. By logits and not by their weights: those are within 2^-31 of
    // themselves only, and of two logits nearer to each other the lesser one's can be the larger one's by a step, but what is
    // kept has to be the ranking's first, and the same in every way to the threshold.
    __device__ __forceinline__ float floor_of(float m) const {
        const RowPar& R = sh.par;
        return R.drops ? E::up(__double2float_ru((double)m + R.drop)) : -INFINITY;
    }
    __device__ __forceinline__ uint32_t cluster_max() const {
        uint32_t k = 0;
        if (lane < team.size) k = *team.of(&sh.max_key, lane);
        return __reduce_max_sync(kAll, k);
    }
    __device__ __forceinline__ uint32_t cluster_flags() const {
        uint32_t f = 0;
        if (lane < team.size) f = *team.of(&sh.flags, lane);
        return __reduce_or_sync(kAll, f);
    }

    // ------------------------------------------------------------------------------------------------
    // few candidates
    // ------------------------------------------------------------------------------------------------
    // The segment's logits from `low` on, into the first CTA's list, in any order.
    __device__ __forceinline__ void gather() const {
        const float low = fmaxf(this->low, sizeof(T) == 2 ? -3.3895314e38f : kLowest);  // -inf is not ranked
        collect([&](const uint4& q) { return E::from(q, low); });
    }
    // The CTA's values, one a thread and no two alike (those of threads from n on are 0), sorted: the largest first. Every warp
    // sorts its own, by a bitonic network of shuffles; a value's place is then its place in its warp and those that it would
    // have in the others' lists, each found by halving.
    __device__ __noinline__ u64 sorted(u64 x, int n) const {
        const int tid = threadIdx.x, lists = (n + 31) / 32;
        List& L = list();
        int place = 0;
        if (warp < lists) {
#pragma unroll 1
            for (int k = 2; k <= 32; k *= 2)
#pragma unroll 1
                for (int j = k / 2; j > 0; j /= 2) {
                    const u64 y = __shfl_xor_sync(kAll, x, j);
                    // the larger one stays where the block of k runs down (the first of two, and the last of all)
                    const bool larger = ((lane & k) == 0) == ((lane & j) == 0);
                    if ((y > x) == larger) x = y;
                }
            L.trade[0][tid] = x;
        }
        __syncthreads();
        if (warp < lists) {
            place = lane;
#pragma unroll 4
            for (int l = 0; l < lists; ++l) {
                const u64* v = L.trade[0] + 32 * l;
                int at = 0;  // values of the list that are larger
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    if (v[at + o - 1] > x) at += o;
                at += v[31] > x;
                if (l != warp) place += at;
            }
            L.trade[1][x ? place : tid] = x;  // (zeros are the last, wherever)
        }
        __syncthreads();
        return tid < n ? L.trade[1][tid] : 0;
    }
    // Sums of the CTA's values up to a thread's.
    __device__ __noinline__ u64 block_inscan(u64 x) const {
        const u64 upto = warp_inscan(x, lane);
        __syncthreads();  // sh.scan is free
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        const u64 mine = lane < kWarps ? sh.scan[lane] : 0, before = warp_inscan(mine, lane) - mine;
        return upto + __shfl_sync(kAll, before, warp);
    }
    // By the first CTA: the candidates sorted, one a thread, and the sums of their weights; with them what is kept. The draw
    // is the same once more, with the kept ones by index.
    template <bool kDraws>
    __device__ __forceinline__ void rank(int32_t row) {
        List& L = list();
        const RowPar& R = sh.par;
        const int n = (int)sh.listed, tid = threadIdx.x;
        const uint32_t flags = cluster_flags() & kNonfinite, top = cluster_max();
        Result res{};
        res.m = float_of(top);
        res.listed = 1;
        res.err = R.err | (flags ? 1u << SV_ERR_NONFINITE : 0u);
        if (!flags && top <= kKeyMinusInf) res.err |= 1u << SV_ERR_EMPTY_ROW;
        res.slow = n > kList;
        if (res.err || res.slow) {
            if (tid == 0) sh.res = res;
            return;
        }
        const u64 x = sorted(tid < n ? L.order[tid] : 0, n);
        const u64 w = tid < n ? weight(float_of((uint32_t)(x >> 32)), res.m, R.E, sh.tab) : 0;
        const u64 upto = block_inscan(w);
        // the first k, then as many as sum to top_p of their weights
        const int first = R.T == 0.f ? 1 : R.k > 0 ? min(R.k, n) : n;
        if (tid == first - 1) sh.total = upto;
        __syncthreads();
        u64 enough = ~0ull;
        if (R.p < 1.f) enough = max(scaled(sh.total, R.p, true), (u64)1);
        const bool kept = tid < first && upto - w < enough && float_of((uint32_t)(x >> 32)) >= floor_of(res.m);
        res.n = __syncthreads_count(kept);
        if (tid == res.n - 1) {
            sh.total = upto;
            sh.hit_rest = x;
        }
        __syncthreads();
        const u64 total = sh.total, border = sh.hit_rest;  // the last that is kept
        res.thr = float_of((uint32_t)(border >> 32));
        res.partial = 1;
        res.cut = (int32_t)~(uint32_t)border;
        if (tid == 0) sh.res = res;
        if (!kDraws) return;
        if (warp == kWarps - 1 && A.logprob && lane == 0 && R.T > 0.f) sh.log_total = log((double)total) - kBits * 0.6931471805599453;
        const u64 target = scaled(total, R.u, false);
        const u64 y = ~sorted(kept ? (u64)(uint32_t)x << 32 | (uint32_t)~(uint32_t)(x >> 32) : 0, res.n);
        const u64 wy = tid < res.n ? weight(float_of((uint32_t)y), res.m, R.E, sh.tab) : 0;
        const u64 run = block_inscan(wy);
        if (run - wy <= target && target < run) {
            A.tokens[row] = (int32_t)(y >> 32);
            if (A.logprob) A.logprob[row] = R.T > 0.f ? (float)(((double)float_of((uint32_t)y) - res.m) * R.per - sh.log_total) : 0.f;
        }
    }

    // ------------------------------------------------------------------------------------------------
    // the quick way (bfloat16)
    // ------------------------------------------------------------------------------------------------
    // Of a pair of logits, the words of their bins.
    static __device__ __forceinline__ uint32_t bins_of(uint32_t w) {
        constexpr uint32_t lo = (kCodeLo - 1) * 0x10001u, hi = (kCodeHi + 1) * 0x10001u;
        return __vminu2(__vmaxu2(w & 0x7fff7fffu, lo), hi) - lo + (w >> 15 & 0x10001u) * kNegative;
    }
    // Whether one of them has no bin: 0 < |x| < 2^-26, or |x| >= 1024 but for -inf.
    static __device__ __forceinline__ bool outside(uint32_t w, uint32_t in) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t b = w >> 16 * i & 0xffffu, a = b & 0x7fffu;
            any |= (in >> 16 * i & 1u) && (a - 1u < kCodeLo - 1u || (a > kCodeHi && b != 0xff80u));
        }
        return any;
    }
    // Counts the logits from `low` on.
    __device__ __forceinline__ void count_values() {
        bool odd = false;
        if (low > -INFINITY) {  // few: most chunks have none
            const __nv_bfloat162 low2 = __float2bfloat162_rn(low);
            each([&](int32_t, const uint4& q) {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
                uint32_t in[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) in[i] = __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), low2);
                if (!(in[0] | in[1] | in[2] | in[3])) return;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!in[i]) continue;
                    const uint32_t at = bins_of(w[i]);
                    odd |= outside(w[i], in[i]);
                    if (in[i] & 1u) atomicAdd(&sh.hist[at & 0xffffu], 1u);
                    if (in[i] >> 16) atomicAdd(&sh.hist[at >> 16], 1u);
                }
            }, true);
        } else {
            uint32_t least = ~0u, most = 0;  // of |x| - 1, of |x| but for -inf
            each([&](int32_t, const uint4& q) {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t at = bins_of(w[i]), a = w[i] & 0x7fff7fffu;
                    least = __vminu2(least, __vsub2(a, 0x00010001u));
                    most = __vmaxu2(most, a & ~__vcmpeq2(w[i], 0xff80ff80u));
                    atomicAdd(&sh.hist[at & 0xffffu], 1u);
                    atomicAdd(&sh.hist[at >> 16], 1u);
                }
            }, true);
            odd = (least & 0xffffu) < kCodeLo - 1 || least >> 16 < kCodeLo - 1 || (most & 0xffffu) > kCodeHi || most >> 16 > kCodeHi;
        }
        if (__any_sync(kAll, odd) && lane == 0) atomicOr(&sh.flags, (uint32_t)kOutside);
    }
    // Value of bin d.
    static __device__ __forceinline__ float value_at(int d) {
        const int o = kMid - d;
        const uint32_t a = (uint32_t)(o < 0 ? -o : o);
        return __uint_as_float(a == 0 ? 0u : (o < 0 ? 0x80000000u : 0u) | (kCodeLo - 1 + a) << 16);
    }
    // Bin of a value.
    static __device__ __forceinline__ int bin_of(float x) {
        const uint32_t b = __float_as_uint(x) >> 16;
        const int a = (int)min(max(b & 0x7fffu, kCodeLo - 1), kCodeHi + 1) - (int)(kCodeLo - 1);
        return kMid + (b & 0x8000u ? a : -a);
    }
    __device__ __forceinline__ uint32_t count_at(int d) const {
        const int o = kMid - d;
        if (o >= kMid || o <= -kMid) return 0;
        if (o > 0) return sh.hist[o];
        return sh.hist[kNegative - o] + (o == 0 ? sh.hist[0] : 0u);
    }
    // Of group g of 64 bins, a lane's two: counts and weights. False, for the warp, if there is nothing.
    __device__ __forceinline__ bool pair_at(int g, float m, uint32_t* c, u64* w) const {
        const int d = g * kGroupBins + 2 * lane;
        c[0] = count_at(d);
        c[1] = count_at(d + 1);
        w[0] = w[1] = 0;
        if (!__any_sync(kAll, c[0] | c[1])) return false;
        const Fixed2 f = weights2(value_at(d), value_at(d + 1), m, sh.par.E, sh.tab);
        w[0] = join(f.ax, f.bx);
        w[1] = join(f.ay, f.by);
        return true;
    }
    // By the first CTA, whose histogram is the row's.
    __device__ __forceinline__ void choose() {
        const uint32_t flags = cluster_flags(), top = cluster_max();
        const RowPar& R = sh.par;
        const float m = float_of(top), floor = floor_of(m);
        const int g0 = bin_of(m) / kGroupBins, g1 = bin_of(low) / kGroupBins;  // groups that hold something
        uint32_t many = 0;  // of logits from `floor` on, which are the ranking's first
        u64 heavy = 0;
        int last = -1;
#pragma unroll 3
        for (int g = warp; g < kGroups; g += kWarps) {
            uint32_t c[2], cc = 0;
            u64 w[2], mass = 0;
            if (g >= g0 && g <= g1 && pair_at(g, m, c, w)) {
                mass = c[0] * w[0] + c[1] * w[1];
                const int d = g * kGroupBins + 2 * lane;
                if (R.drops && c[0] && value_at(d) >= floor) many += c[0], heavy += c[0] * w[0], last = d;
                if (R.drops && c[1] && value_at(d + 1) >= floor) many += c[1], heavy += c[1] * w[1], last = d + 1;
                mass = warp_sum(mass);
                cc = __reduce_add_sync(kAll, c[0] + c[1]);
            }
            if (lane == 0) {
                sh.group_count[g] = cc;
                sh.group_mass[g] = mass;
            }
        }
        many = __reduce_add_sync(kAll, many);
        last = __reduce_max_sync(kAll, last);
        heavy = warp_sum(heavy);
        if (lane == 0) {
            sh.warp_part[warp] = Part{heavy, many, (uint32_t)(last + 1)};
        }
        __syncthreads();
        if (warp > 0) return;
        uint32_t cl = 0;
        u64 ml = 0;
#pragma unroll 1
        for (int g = 5 * lane; g < 5 * lane + 5 && g < kGroups; ++g) {
            cl += sh.group_count[g];
            ml += sh.group_mass[g];
        }
        const u64 c_upto = warp_inscan(cl, lane), m_upto = warp_inscan(ml, lane);
        const uint32_t all = (uint32_t)__shfl_sync(kAll, c_upto, 31);
        u64 sum = __shfl_sync(kAll, m_upto, 31);
        Result res{};
        res.m = m;
        res.n = (int32_t)all;
        res.thr = kLowest;  // all that are ranked, unless something says otherwise
        res.at = kBins - 1;
        res.mass = sum;
        const bool found = top > kKeyMinusInf && R.T > 0.f;
#pragma unroll 1
        for (int step = 0; step < 2 && found; ++step) {  // the first k, then as many as sum to top_p of their weights
            u64 target = (u64)R.k;
            if (step == 0 && (R.k <= 0 || (uint32_t)R.k > all)) continue;
            if (step == 1) {
                if (!(R.p < 1.f)) continue;
                target = max(scaled(sum, R.p, true), (u64)1);
            }
            // the lane, the group and the bin in which the counts or weights reach the target
            const u64 before = step ? m_upto - ml : c_upto - cl, own = step ? ml : cl;
            const bool mine = before < target && target <= before + own;
            int g = 5 * lane;
            u64 pc = c_upto - cl, pm = m_upto - ml;
            if (mine)
#pragma unroll 1
                for (; (step ? pm + sh.group_mass[g] : pc + sh.group_count[g]) < target; ++g) {
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
            const u64 mass = c[0] * w[0] + c[1] * w[1], cc = c[0] + c[1];
            pm += warp_inscan(mass, lane) - mass;
            pc += warp_inscan(cc, lane) - cc;
            const bool here = step ? pm < target && target <= pm + mass : pc < target && target <= pc + cc;
            int i = 0;
            if ((step ? pm + c[0] * w[0] : pc + c[0]) < target) {
                i = 1;
                pm += c[0] * w[0];
                pc += c[0];
            }
            const uint32_t ties = i ? c[1] : c[0];
            const u64 wt = i ? w[1] : w[0];
            uint32_t r = 0;
            if (here) r = step ? div_up(target - pm, wt) : (uint32_t)(target - pc);
            const int at = __ffs(__ballot_sync(kAll, here)) - 1;
            const uint32_t n = (uint32_t)__shfl_sync(kAll, pc + r, at);
            if (step == 0) sum = __shfl_sync(kAll, pm + r * wt, at);
            if ((int32_t)n <= res.n) {  // (equal, too: logits that were too low to count are not kept)
                res.n = (int32_t)n;
                res.r = __shfl_sync(kAll, r, at);
                res.ties = __shfl_sync(kAll, ties, at);
                res.partial = res.r < res.ties;
                res.at = __shfl_sync(kAll, g * kGroupBins + 2 * lane + i, at);
                res.mass = __shfl_sync(kAll, pm + (r < ties ? 0 : r * wt), at);
            }
        }
        if (R.drops && found) {
            const Part x = lane < kWarps ? sh.warp_part[lane] : Part{0, 0, 0};
            many = __reduce_add_sync(kAll, x.above);
            last = (int)__reduce_max_sync(kAll, x.ties) - 1;
            heavy = warp_sum(x.mass);
            if ((int32_t)many <= res.n) {
                res.n = (int32_t)many;
                res.partial = 0;
                res.at = last;
                res.mass = heavy;
            }
        }
        if (R.T == 0.f && top > kKeyMinusInf) {  // the bins hold what equals the largest of a CTA, the first of them that of all
            res.at = bin_of(m);
            res.ties = count_at(res.at);
            res.r = 1;
            res.partial = res.ties > 1;
            res.n = 1;
            res.mass = res.partial ? 0 : (u64)1 << kBits;
        }
        if (res.at < kBins - 1) res.thr = value_at(res.at);
        res.err = R.err | (flags & kNonfinite ? 1u << SV_ERR_NONFINITE : 0u);
        if (!(flags & kNonfinite) && top <= kKeyMinusInf) res.err |= 1u << SV_ERR_EMPTY_ROW;
        res.slow = !res.err && (flags & kOutside);
        if (lane == 0) sh.res = res;
    }
    // Histograms of the cluster, summed into the first CTA's, a share of the bins by each.
    __device__ __forceinline__ void merge_counts() {
        if (team.size == 1) return;
        // 16 bytes of the words from the least to the largest logit that is counted: of the positive ones, and of the negative
        const int o1 = kMid - bin_of(float_of(cluster_max())), o0 = kMid - bin_of(low);
        const int a0 = max(o0, 0) / 4, na = o1 >= 0 ? o1 / 4 - a0 + 1 : 0;
        const int b0 = (kNegative + max(-o1, 0)) / 4, nb = o0 <= 0 ? (kNegative - o0) / 4 - b0 + 1 : 0;
#pragma unroll 1
        for (int i = team.rank * kThreads + threadIdx.x; i < na + nb; i += team.size * kThreads) {
            const int v = i < na ? a0 + i : b0 + i - na;
            if (i >= na && na > 0 && v < a0 + na) continue;  // the word of both
            uint4 x[kMaxCtas];
#pragma unroll
            for (int q = 0; q < kMaxCtas; ++q) {
                x[q] = make_uint4(0, 0, 0, 0);
                if (q < team.size) x[q] = reinterpret_cast<const uint4*>(team.of(sh.hist, q))[v];
            }
            uint4 t = x[0];
#pragma unroll
            for (int q = 1; q < kMaxCtas; ++q) t.x += x[q].x, t.y += x[q].y, t.z += x[q].z, t.w += x[q].w;
            reinterpret_cast<uint4*>(team.of(sh.hist, 0))[v] = t;
        }
        team.sync();
    }
    __device__ __forceinline__ void zero_hist() {
#pragma unroll 1
        for (int i = threadIdx.x; i < kHist / 4; i += kThreads) reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
    }
    // What a CTA has of the kept, from its histogram. (The first one's is the row's by now: it has what the others have not.)
    template <bool kMass>
    __device__ __forceinline__ void part_of_counts(const Result& res) {
        if (!kMass) {
            if (threadIdx.x == 0) sh.part = Part{0, 0, team.rank > 0 && res.partial ? count_at(res.at) : 0};
            return;
        }
        const int end = res.partial ? res.at : res.at + 1;
        u64 mass = 0;
        uint32_t ties = 0, above = 0;
#pragma unroll 1
        for (int g = bin_of(res.m) / kGroupBins + warp; g * kGroupBins <= res.at && team.rank > 0; g += kWarps) {
            uint32_t c[2];
            u64 w[2];
            if (!pair_at(g, res.m, c, w)) continue;
            const int d = g * kGroupBins + 2 * lane;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (d + i < end) mass += c[i] * w[i], above += c[i];
                else if (d + i == res.at) ties += c[i];
            }
        }
        sum_up(mass, above, ties);
    }
    // The CTA's part, from its warps'.
    __device__ __forceinline__ void sum_up(u64 mass, uint32_t above, uint32_t ties) {
        mass = warp_sum(mass);
        above = __reduce_add_sync(kAll, above);
        ties = __reduce_add_sync(kAll, ties);
        if (lane == 0) sh.warp_part[warp] = Part{mass, above, ties};
        __syncthreads();
        if (warp == 0) {
            const Part x = lane < kWarps ? sh.warp_part[lane] : Part{0, 0, 0};
            mass = warp_sum(x.mass);
            above = __reduce_add_sync(kAll, x.above);
            ties = __reduce_add_sync(kAll, x.ties);
            if (lane == 0) sh.part = Part{mass, above, ties};
        }
    }

    // ------------------------------------------------------------------------------------------------
    // the slow way
    // ------------------------------------------------------------------------------------------------
    // One level: the logits for which `index` gives a bin below `bins`, the larger ones' higher, and the bin at which their
    // counts (or weights, in the ranking's order) reach the target. first: the target is top_p of all weights and `extra`.
    template <bool kMass, typename F>
    __device__ __forceinline__ Found level(int bins, F&& index, float m, u64 target, bool first, u64 extra) {
        __syncthreads();
        for (int i = threadIdx.x; i < kDigits; i += kThreads) sh.hist[i] = sh.hist[kDigits + i] = 0;
        if (threadIdx.x == 0) sh.listed = 0;
        __syncthreads();
#pragma unroll 1
        for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
            float x[E::N];
            E::unpack(chunk(s, c), x);
#pragma unroll
            for (int e = 0; e < E::N; e += 2) {
                const uint32_t at[2] = {index(x[e]), index(x[e + 1])};
                const bool in[2] = {at[0] < (uint32_t)bins, at[1] < (uint32_t)bins};
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
                target = max(scaled(sum, sh.par.p, true), (u64)1);
            }
            if (threadIdx.x == 0 && target > total) sh.found = {-1, target - total, 0};
            if (before < target && target <= before + mine) {
                int b = bins - 1 - per * (int)threadIdx.x;
                u64 v;
                for (;; --b) {
                    v = sh.hist[b] + ((u64)sh.hist[kDigits + b] << 32);
                    if (target <= before + v) break;
                    before += v;
                }
                sh.found = {b, target - before, v};
            }
        }
        team.sync();
        return *team.of(&sh.found, 0);
    }
    template <bool kMass>
    __device__ __noinline__ Found digit(uint32_t lo, int shift, int bins, uint32_t floor, float m, u64 target, bool first, u64 extra) {
        return level<kMass>(
            bins,
            [&](float x) {
                const uint32_t k = key_of(x);
                return k >= lo && k > floor && k > kKeyMinusInf ? (k - lo) >> shift : ~0u;
            },
            m, target, first, extra);
    }
    // The key at which the counts or weights of the elements above `floor` reach the target; r: of the elements with that key
    // so many are needed, of `ties`. False: they do not reach it (rest: by how much).
    template <bool kMass>
    __device__ __forceinline__ bool seek(uint32_t floor, float m, u64 target, u64 extra, uint32_t& key, uint32_t& r, uint32_t& ties, u64& rest) {
        Found f = digit<kMass>(0u, 20, 4096, floor, m, target, true, extra);
        rest = f.rest;
        if (f.bin < 0) return false;
        key = (uint32_t)f.bin << 20;
        f = digit<kMass>(key, 8, 4096, floor, m, f.rest, false, 0);
        key += (uint32_t)f.bin << 8;
        f = digit<kMass>(key, 0, 256, floor, m, f.rest, false, 0);
        key += (uint32_t)f.bin;
        const u64 w = kMass ? weight(float_of(key), m, sh.par.E, sh.tab) : 1;
        r = div_up(f.rest, w);
        ties = div_up(f.value, w);
        return true;
    }
    // The same for top_p of all weights, in fewer passes: the bins are even in the weights' logarithms, and so narrow that
    // the one with the crossing has few logits; those are sorted. False, for the cluster, if they are not so few.
    __device__ __noinline__ bool seek_even(float m, uint32_t& key, uint32_t& r, uint32_t& ties) {
        // (to 2^-46, past the last weight that is not rounded to nothing; finite, whatever the temperature: the largest logit is
        // 0 bins away)
        const float per = fminf(sh.par.E.K_hi * ((float)kDigits / (kBits + 2)), -kLowest);
        auto index = [&](float x) { return (uint32_t)(kDigits - 1) - (uint32_t)fminf((m - x) * per, 1e9f); };  // monotone in x
        const Found f = level<true>(kDigits, index, m, 0, true, 0);
        if (f.bin < 0) return false;
        collect([&](const uint4& q) {
                float x[E::N];
                E::unpack(q, x);
                uint32_t in = 0;
#pragma unroll
                for (int e = 0; e < E::N; ++e) in |= (uint32_t)(index(x[e]) == (uint32_t)f.bin) << e;
                return in;
            });
        team.sync();
        if (team.rank == 0) {
            const int n = (int)sh.listed;
            Found g{-1, 0, 0};
            if (n <= kList) {
                List& L = list();
                const int tid = threadIdx.x;
                const u64 x = sorted(tid < n ? L.order[tid] : 0, n);
                const u64 w = tid < n ? weight(float_of((uint32_t)(x >> 32)), m, sh.par.E, sh.tab) : 0;
                const u64 upto = block_inscan(w);
                // the last that is needed, and those like it
                if (upto - w < f.rest && f.rest <= upto) sh.hit_rest = x;
                __syncthreads();
                const uint32_t k = (uint32_t)(sh.hit_rest >> 32);
                const bool like = tid < n && (uint32_t)(x >> 32) == k;
                const int need = __syncthreads_count(like && x >= sh.hit_rest), all = __syncthreads_count(like);
                g = {0, (u64)k << 32 | (uint32_t)need, (u64)all};
            }
            if (threadIdx.x == 0) sh.found = g;
        }
        team.sync();
        const Found g = *team.of(&sh.found, 0);
        if (g.bin < 0) return false;
        key = (uint32_t)(g.rest >> 32);
        r = (uint32_t)g.rest;
        ties = (uint32_t)g.value;
        return true;
    }
    __device__ __forceinline__ Result choose_slow() {
        const RowPar& R = sh.par;
        const uint32_t flags = cluster_flags() & kNonfinite, top = cluster_max();
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
        uint32_t floor = 0, r = 0, ties = 0, key;  // keys above the floor are kept, and r of its own
        u64 rest;
        if (R.k > 0 && R.k < A.V) seek<false>(0u, m, (u64)R.k, 0, floor, r, ties, rest);
        if (R.p < 1.f) {
            const u64 w = r ? weight(float_of(floor), m, R.E, sh.tab) : 0;
            uint32_t q, all;
            if (!r && seek_even(m, key, q, all)) {
                floor = key, r = q, ties = all;
            } else if (seek<true>(floor, m, 0, r * w, key, q, all, rest)) {
                floor = key, r = q, ties = all;
            } else {
                r = div_up(rest, w);
            }
        }
        if (r) {
            res.thr = float_of(floor);
            res.r = r;
            res.partial = r < ties;
        }
        const float least = floor_of(m);
        if (least > res.thr) {
            res.thr = least;
            res.partial = 0;
        }
        return res;
    }

    // ------------------------------------------------------------------------------------------------
    // with the threshold
    // ------------------------------------------------------------------------------------------------
    // What a segment has of the kept.
    template <bool kMass>
    __device__ __forceinline__ void tally(const Result& res, const Segment& g, u64& mass, uint32_t& above, uint32_t& ties) const {
        above = ties = 0;
        int32_t sa = 0, sb = 0;  // of at most 256 weights (2^18 logits by 1024 threads): 2^30
        const bool whole = !res.partial;
#pragma unroll 1
        for (int32_t c = g.c0 + lane; c < g.c1; c += 32) {
            float x[E::N];
            E::unpack(chunk(g, c), x);
#pragma unroll
            for (int e = 0; e < E::N; e += 2) {
                const bool in0 = x[e] > res.thr || (whole && x[e] == res.thr), in1 = x[e + 1] > res.thr || (whole && x[e + 1] == res.thr);
                if (!whole) ties += (x[e] == res.thr) + (x[e + 1] == res.thr);
                if (!(in0 || in1)) continue;
                above += in0 + in1;
                if (!kMass) continue;
                const Fixed2 f = weights2(x[e], x[e + 1], res.m, sh.par.E, sh.tab);
                sa += (in0 ? f.ax : 0) + (in1 ? f.ay : 0);
                sb += (in0 ? f.bx : 0) + (in1 ? f.by : 0);
            }
        }
        mass = kMass ? join(sa, sb) : 0;
    }
    // Every CTA's part, by the first warp: lane q has CTA q's, and the ties that it keeps. known: the first CTA's is what the
    // others leave of the row's.
    __device__ __forceinline__ Part parts(const Result& res, bool known, uint32_t& keeps) const {
        Part p{0, 0, 0};
        if (lane < team.size) p = *team.of(&sh.part, lane);
        if (known) {
            const u64 mass = warp_sum(p.mass);
            const uint32_t ties = __reduce_add_sync(kAll, p.ties), above = __reduce_add_sync(kAll, p.above);
            if (lane == 0) {
                p.mass = res.mass - mass;
                p.ties = res.partial ? res.ties - ties : 0;
                p.above = (uint32_t)res.n - (res.partial ? res.r : 0) - above;
            }
        }
        const uint32_t upto = (uint32_t)warp_inscan(p.ties, lane);
        keeps = res.partial ? min(p.ties, res.r - min(res.r, upto - p.ties)) : 0;
        return p;
    }
    __device__ __forceinline__ u64 tie_weight(const Result& res) const {
        return res.partial ? weight(res.thr, res.m, sh.par.E, sh.tab) : 0;
    }
    // The index of the n-th tie of a segment (n >= 1).
    __device__ __forceinline__ int32_t nth_tie(float thr, const Segment& g, int32_t n) const {
#pragma unroll 1
        for (int32_t c0 = g.c0; c0 < g.c1; c0 += 32) {
            const int32_t c = c0 + lane;
            uint32_t eq = 0;
            if (c < g.c1) {
                float x[E::N];
                E::unpack(chunk(g, c), x);
#pragma unroll
                for (int e = 0; e < E::N; ++e) eq |= (uint32_t)(x[e] == thr) << e;
            }
            const int32_t upto = (int32_t)warp_inscan((u64)__popc(eq), lane);
            int32_t at = -1;
            if (upto >= n && upto - __popc(eq) < n) {
#pragma unroll 1
                for (int32_t i = n - (upto - __popc(eq)); i > 1; --i) eq &= eq - 1;
                at = c * E::N + __ffs(eq) - 1 - off;
            }
            at = __reduce_max_sync(kAll, at);
            if (at >= 0) return at;
            n -= __shfl_sync(kAll, upto, 31);
        }
        return A.V;
    }
    // Ties up to this index are kept, in a segment that has `ties` and keeps `keeps` of them.
    __device__ __forceinline__ int32_t cut_of(const Result& res, const Segment& g, uint32_t ties, uint32_t keeps) const {
        if (!res.partial || keeps == ties) return 0x7fffffff;
        return keeps == 0 ? -1 : nth_tie(res.thr, g, (int32_t)keeps);
    }
    __device__ __forceinline__ uint32_t kept_of(const float* x, int32_t i0, const Result& res, int32_t cut) const {
        uint32_t k = 0;
#pragma unroll
        for (int e = 0; e < E::N; ++e) k |= (uint32_t)(x[e] > res.thr || (x[e] == res.thr && i0 + e <= cut)) << e;
        return k;
    }

    // ------------------------------------------------------------------------------------------------
    // the draw
    // ------------------------------------------------------------------------------------------------
    // The CTA that holds it, from the CTAs' parts; then all warps of the cluster share out that CTA's slice, and the warp
    // whose share holds it finds it. `slices`: the first chunk of a CTA's slice.
    template <typename F>
    __device__ __forceinline__ void draw(const Result& res, bool known, int32_t row, F&& slices) {
        const RowPar& R = sh.par;
        const u64 w = tie_weight(res);
        if (warp == 0) {
            uint32_t keeps;
            const Part p = parts(res, known, keeps);
            const u64 own = p.mass + keeps * w, upto = warp_inscan(own, lane), all = __shfl_sync(kAll, upto, 31);
            const u64 target = scaled(all, R.u, false);  // the running weight must exceed it
            const uint32_t n = __reduce_add_sync(kAll, p.above + keeps);
            if (target < upto && target >= upto - own) {
                sh.hit = lane;
                sh.hit_rest = target - (upto - own);
                sh.keeps = keeps;
                sh.total = all;
                sh.n = (int32_t)n;
            }
        }
        __syncthreads();
        const int hit = sh.hit;
        // the shares
        const int32_t h0 = slices(hit), h1 = slices(hit + 1), n = team.size * kWarps, me = team.rank * kWarps + warp;
        auto share = [&](int i) { return h0 + (int32_t)((int64_t)(h1 - h0) * i / n); };
        const uint4* data = s.data;
        if (kHeld) data = team.of(const_cast<uint4*>(reinterpret_cast<const uint4*>(&sh + 1)), hit) - h0;
        const Segment g{data, share(me), share(me + 1)};
        u64 mass;
        uint32_t above, ties;
        tally<true>(res, g, mass, above, ties);
        mass = warp_sum(mass);
        ties = __reduce_add_sync(kAll, ties);
        if (lane == 0) sh.warp_part[warp] = Part{mass, 0, ties};
        team.sync();
        // lane i has shares 4 i .. 4 i + 3
        if (warp == 0) {
            Part p[4];
            uint32_t tl = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 4 * lane + i;
                p[i] = Part{0, 0, 0};
                if (at < n) p[i] = team.of(&sh, at / kWarps)->warp_part[at % kWarps];
                tl += p[i].ties;
            }
            uint32_t left = sh.keeps - min(sh.keeps, (uint32_t)warp_inscan(tl, lane) - tl);  // ties that the lane's shares may keep
            u64 ml = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t k = min(left, p[i].ties);
                left -= k;
                p[i].above = k;
                p[i].mass += k * w;
                ml += p[i].mass;
            }
            u64 at = warp_inscan(ml, lane) - ml;
            const u64 target = sh.hit_rest;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (target >= at && target < at + p[i].mass) {
                    sh.hit = 4 * lane + i;
                    sh.hit_rest = target - at;
                    sh.warp_keeps[0] = (int32_t)p[i].above;
                }
                at += p[i].mass;
            }
        }
        __syncthreads();
        if (sh.hit / kWarps == team.rank) {
            const int who = sh.hit % kWarps;
            if (warp == who) pick(res, g, cut_of(res, g, ties, (uint32_t)sh.warp_keeps[0]), sh.hit_rest);
            else if (warp == (who ^ 1) && lane == 0) sh.log_total = log((double)sh.total) - kBits * 0.6931471805599453;
            __syncthreads();
            if (threadIdx.x == 0) {
                A.tokens[row] = sh.token;
                if (A.logprob) A.logprob[row] = R.T > 0.f ? (float)(((double)sh.logit - res.m) * R.per - sh.log_total) : 0.f;
            }
        }
    }
    // The first kept token of a segment whose running weight exceeds `target`.
    __device__ __forceinline__ void pick(const Result& res, const Segment& g, int32_t cut, u64 target) {
        u64 base = 0;
#pragma unroll 1
        for (int32_t c0 = g.c0; c0 < g.c1; c0 += 32) {
            const int32_t c = c0 + lane;
            u64 w[E::N], sum = 0;
            float x[E::N];
#pragma unroll
            for (int e = 0; e < E::N; ++e) w[e] = 0;
            if (c < g.c1) {
                E::unpack(chunk(g, c), x);
                const uint32_t k = kept_of(x, c * E::N - off, res, cut);
#pragma unroll
                for (int e = 0; e < E::N; e += 2)
                    if (k >> e & 3u) {
                        const Fixed2 f = weights2(x[e], x[e + 1], res.m, sh.par.E, sh.tab);
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
                float l = 0.f;
#pragma unroll
                for (int e = 0; e < E::N; ++e) {
                    run += w[e];
                    if (at < 0 && run > target) {
                        at = e;
                        l = x[e];
                    }
                }
                sh.token = c * E::N + at - off;
                sh.logit = l;
            }
            base = __shfl_sync(kAll, upto, 31);
            if (target < base) return;
        }
    }

    // ------------------------------------------------------------------------------------------------
    // the filtered row
    // ------------------------------------------------------------------------------------------------
    // The ties that this CTA's warps keep, where they are not all kept; and the row's count where it is not known.
    __device__ __forceinline__ int32_t cut_here(const Result& res, bool known) {
        uint32_t ties = 0;
        if (warp == 0) {
            uint32_t keeps;
            const Part p = parts(res, known, keeps);
            const uint32_t n = __reduce_add_sync(kAll, p.above + keeps);
            if (lane == team.rank) {
                sh.keeps = keeps;
                sh.total = p.ties;
                sh.n = known ? res.n : (int32_t)n;
            }
        }
        __syncthreads();
        if (!res.partial || sh.keeps == (uint32_t)sh.total) return 0x7fffffff;
        if (sh.keeps == 0) return -1;
        each([&](int32_t, const uint4& q) { ties += E::equal(q, res.thr); });
        ties = __reduce_add_sync(kAll, ties);
        if (lane == 0) sh.warp_keeps[warp] = (int32_t)ties;
        __syncthreads();
        const uint32_t mine = lane < kWarps ? (uint32_t)sh.warp_keeps[lane] : 0u;
        const uint32_t before = (uint32_t)__shfl_sync(kAll, warp_inscan(mine, lane) - mine, warp);
        return cut_of(res, s, ties, min(ties, sh.keeps - min(sh.keeps, before)));
    }
    // The segment with -inf where a token is not kept (copy: as it is); of those equal to the threshold, the ones up to index
    // `cut` are kept.
    __device__ __forceinline__ void write(const Result& res, int32_t row, bool copy, int32_t cut) const {
        typedef typename E::Bits Bits;
        Bits* out = (Bits*)A.out + (int64_t)row * A.out_stride;
        const int32_t o_off = (int32_t)((uintptr_t)out % 16 / sizeof(Bits));
        const float at = res.thr, above = E::next(res.thr);
        const Bits* in = reinterpret_cast<const Bits*>(s.data) + off;  // element i at in[i]
        const int32_t e0 = max(0, s.c0 * E::N - off), e1 = min(A.V, s.c1 * E::N - off);
        const uint32_t* words = reinterpret_cast<const uint32_t*>(s.data);
        const bool same = o_off == off;
        const Apart apart{off, o_off, (int32_t)sizeof(Bits), E::N};
        const uint32_t shift = apart.shift();
        // by the output's chunks of 16 bytes, which lie as the logits' do, or between two of them: whole ones, and others, or the
        // one that the last tie lies in, by element
        const int32_t w0 = apart.c0(e0), w1 = apart.c1(e1, A.V);
        const int32_t last = copy || cut == 0x7fffffff ? 0x7fffffff : (cut + o_off + E::N) / E::N - 1;  // the chunk of `cut`
        const int32_t split = copy || cut == 0x7fffffff || (cut + o_off) % E::N == E::N - 1 || cut < 0 ? -1 : last;
        auto whole = [&](int32_t c) { return c >= w0 && c < w1 && c != split; };
        constexpr int kAtOnce = 4;
#pragma unroll 1
        for (int32_t c0 = (e0 + o_off) / E::N + lane; c0 * E::N - o_off < e1; c0 += 32 * kAtOnce) {
            uint4 q[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int32_t c = c0 + 32 * k;
                if (!whole(c)) continue;
                if (same) {
                    q[k] = kHeld ? s.data[c] : __ldcs(s.data + c);
                } else {
                    const uint32_t* w = words + apart.word(c);
                    uint32_t x[5];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = w[i];
                    x[4] = apart.words() > 4 ? w[4] : 0u;
                    q[k] = make_uint4(__funnelshift_r(x[0], x[1], shift), __funnelshift_r(x[1], x[2], shift),
                                      __funnelshift_r(x[2], x[3], shift), __funnelshift_r(x[3], x[4], shift));
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int32_t c = c0 + 32 * k, i0 = c * E::N - o_off;
                if (whole(c)) {
                    __stcs(reinterpret_cast<uint4*>(out + i0), copy ? q[k] : E::keep(q[k], c > last ? above : at));
                    continue;
                }
#pragma unroll 1
                for (int32_t i = max(i0, e0); i < min(i0 + E::N, e1); ++i) {
                    const float x = E::value(in[i]);
                    out[i] = copy || x > res.thr || (x == res.thr && i <= cut) ? in[i] : (Bits)E::bits_minus_inf;
                }
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
        const float mp = A.min_p ? A.min_p[q] : 0.f;
        if (draws) R.u = A.uniforms[row];
        ok = R.T >= 0.f && R.T <= kMostTemperature && R.p == R.p && mp == mp && R.u >= 0.f && R.u < 1.f;
        R.drops = mp > 0.f && R.T > 0.f;  // (a temperature of 0 keeps the first alone)
        if (ok && R.drops) R.drop = (double)R.T * log((double)fminf(mp, 1.f));
    }
    if (ok && R.T > 0.f) {
        R.per = 1.0 / (double)R.T;
        const double K = 1.4426950408889634074 / (double)R.T;
        R.E.K_hi = (float)K;
        R.E.K_lo = (float)(K - (double)R.E.K_hi);
        R.E.d_min = (float)(-126.5 / (double)R.E.K_hi);
        ok = R.E.K_hi < INFINITY;
    }
    if (!ok) R.err = 1u << SV_ERR_INVALID_ARG;
}

template <typename T, bool kDraws, bool kHeld>
__global__ void __launch_bounds__(Work<T, kHeld>::kThreads, kHeld ? 2 : 1) k_rows(const __grid_constant__ Args A, int32_t C, int32_t ahead) {
    typedef Elem<T> E;
    constexpr int kThreads = Work<T, kHeld>::kThreads, kWarps = kThreads / 32;
    extern __shared__ __align__(16) char raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    uint4* held = reinterpret_cast<uint4*>(raw + sizeof(Shared));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Team team{(int)(blockIdx.x % (unsigned)C), C};
    const int32_t row = (int32_t)(blockIdx.x / (unsigned)C);
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the slice on its way
    const T* base = (const T*)A.logits + (int64_t)row * A.stride;
    const int32_t off = (int32_t)((uintptr_t)base % 16 / sizeof(T));
    const int32_t chunks = (off + A.V + E::N - 1) / E::N;
    const int parts = C * kWarps, part = team.rank * kWarps + warp;
    auto begin = [&](int i) { return (int32_t)((int64_t)chunks * i / parts); };
    const int32_t first = begin(team.rank * kWarps);
    const Segment s{kHeld ? held - first : reinterpret_cast<const uint4*>(base - off), begin(part), begin(part + 1)};
    if (kHeld) {
        for (int32_t c = s.c0 + lane; c < s.c1; c += 32) {
            const int32_t i0 = c * E::N - off;
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
    }
    if (tid < 128) {
        sh.tab[tid] = A.exp2_tab[tid].x;
        sh.tab[kExpTab + tid] = A.exp2_tab[tid].y;
    }
    if (tid == kThreads - 1) {
        sh.flags = sh.listed = 0;
        sh.hit = 0;  // of a CTA and a warp that there are, whatever the row's passes see
        sh.token = -1;
        read_par(A, sh.par, row, kDraws);
    }
    const int32_t full0 = off > 0;
    Work<T, kHeld> work{A, sh, team, s, off, full0, (uint32_t)max(0, (off + A.V) / E::N - full0), lane, warp, -INFINITY};
    constexpr bool kQuick = sizeof(T) == 2;
    __syncthreads();
    if (kHeld) {
        cp_async_wait<0>();
        __syncwarp();
    }

    work.survey();
    team.sync();
    work.low = work.row_low();
    Result res{};
    res.slow = 1;
    if (work.low > -INFINITY || A.V <= Work<T, kHeld>::kList) {
        work.gather();
        team.sync();
        if (team.rank == 0) work.template rank<kDraws>(row);
        team.sync();
        res = *team.of(&sh.res, 0);
    }
    if (kQuick && res.slow) {
        work.zero_hist();
        __syncthreads();
        work.count_values();
        team.sync();
        work.merge_counts();
        if (team.rank == 0) work.choose();
        team.sync();
        res = *team.of(&sh.res, 0);
    }
    const bool known = !res.slow;
    if (res.slow) res = work.choose_slow();

    if (!kHeld) work.bring(base, row, ahead);
    const bool ok = !res.err;
    int32_t n = ok ? res.n : -1, cut = res.listed ? res.cut : 0x7fffffff;
    if (ok && !res.listed && (kDraws || res.partial || !known)) {
        if (known) {
            work.template part_of_counts<kDraws>(res);
        } else {
            u64 mass;
            uint32_t above, ties;
            work.template tally<kDraws>(res, s, mass, above, ties);
            __syncthreads();
            work.sum_up(mass, above, ties);
        }
        team.sync();
        if (kDraws) work.draw(res, known, row, [&](int q) { return begin(q * kWarps); });
        else cut = work.cut_here(res, known);
        n = sh.n;
    }
    if (C > 1) team.arrive();  // nothing of another CTA is read from here on
    if (!kDraws) work.write(res, row, !ok, cut);
    if (team.rank == 0 && tid == 0) {
        if (A.kept) A.kept[row] = n;
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

constexpr int kSmem = 113 * 1024, kSmemAlone = 227 * 1024;  // of a CTA, two an SM and one
constexpr int kLeast = 4096;       // logits of a slice that is worth a CTA
constexpr int kMostShares = 4;     // CTAs of a row that is not held: the draw's shares are 128

template <typename T, bool kDraws, bool kHeld>
cudaError_t launch(const Args& A, int dev, int C, int32_t ahead, int64_t smem, cudaStream_t st) {
    auto kernel = k_rows<T, kDraws, kHeld>;
    // the devices on which the kernel may use an SM's shared memory: setting that twice does no harm
    static std::atomic<unsigned long long> allowed{0};
    if (dev >= 64 || !(allowed.load() >> dev & 1u)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlone);
        if (e == cudaSuccess && kHeld) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
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
    cfg.blockDim = dim3(Work<T, kHeld>::kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, A, (int32_t)C, ahead);
}

// CTAs of a row, a power of two. Held rows take as few as hold them in shared memory, and more while that leaves SMs idle and a
// slice is worth a CTA; all CTAs that two an SM allow are hardly ever there at once, as a cluster wants its SMs together, so
// some are left over. Else the rows are read where they lie. A turn of the GPU's takes held rows about half as long, so they
// are held if that takes less than twice the turns: measured, held and not, 157 rows of 24559 floats 35 and 53 us (2 turns
// each), 198 of 59737 bf16 42 and 57 (2 and 2), 121 of 96499 60 and 48 (2 and 1), 704 of 128256 242 and 153 (10 and 5).
template <typename T, bool kDraws>
cudaError_t launch(const Args& A, cudaStream_t st) {
    int dev, sms;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t chunks = (A.V + Elem<T>::N - 1) / Elem<T>::N + 1, rows = A.rows, at_once = 15 * (int64_t)sms / 8;
    auto bytes = [&](int c) { return (int64_t)sizeof(Shared) + ((chunks + c - 1) / c + 1) * 16; };
    auto least = [&](int64_t smem) {
        int c = 1;
        while (c < kMaxCtas && bytes(c) > smem) c *= 2;
        return c;
    };
    int C = least(kSmem);
    const int64_t turns = (rows * C + at_once - 1) / at_once;
    // long rows that fit at once by one CTA an SM
    const bool alone = !(bytes(C) <= kSmem && turns == 1) && bytes(least(kSmemAlone)) <= kSmemAlone && rows * least(kSmemAlone) <= at_once / 2;
    const bool held = alone || (bytes(C) <= kSmem && turns < 2 * ((rows + sms - 1) / sms));
    if (held) {
        if (alone) C = least(kSmemAlone);
        while (C < kMaxCtas && rows * 2 * C <= (alone ? at_once / 2 : at_once) && A.V / (2 * C) >= kLeast) C *= 2;
    } else {  // measured: 128 rows of 129281 floats 166, 122 and 137 us with 1, 2 and 4; 704 of 128256 bf16 153, 216 and 343
        C = 1;
        while (C < kMostShares && 2 * rows * C < 3 * sms && A.V / (2 * C) >= kLeast) C *= 2;
    }
    if (rows * C > 0x7fffffff) return cudaErrorInvalidValue;
    return held ? launch<T, kDraws, true>(A, dev, C, 0, bytes(C), st) : launch<T, kDraws, false>(A, dev, C, sms / C, sizeof(Shared), st);
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
