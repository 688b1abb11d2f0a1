// spec_cache_attend for chunks of up to 64 rows (a row is a token and a query head of the group): plain decoding and
// drafts. The mathematics, the numbering of the work and its split over the CTAs are sv_cache_attend.cu's.
//
// Such a chunk is bound by the bytes of its keys and values: a tile of 128 slots takes an SM about 2800 cycles to
// bring in at the HBM rate (16 bits, D = 128), half of that with D = 64 or 8 bits, so whatever is done per tile has
// to fit beneath. With the rows as the first dimension of a product (128 lanes) most of a softmax is padding, and
// the few real rows sit in one warp, 128 scores each: 1300 to 3000 cycles a tile measured, more than the loads.
// The products are therefore turned around,
//     S^T = K Q^T  (128 slots x rows),   O^T += V^T P^T  (D x rows),
// with the slots on the lanes: every thread has one slot and as many scores as there are rows, all four warps of a
// group work, and rows are rounded up to 16, 32 or 64 columns only. The weights go to shared memory, the product's
// other operand; a row's sum stays spread over the lanes until the item ends. All threads hold their weights against
// the rows' references, and one word tells the four warps of a group when a reference has to move (a first tile, or
// a weight too large for its type), which costs three more barriers and a pass of maxima.
//
// Up to 32 rows a CTA has one softmax warpgroup, and two CTAs share an SM: one's beginnings and endings of items (a
// fifth of the time of an item of ten tiles) lie under the other's tiles. (Three an SM, where registers and shared
// memory allow it, measured the same: 62 against 63 us for the window below.) Above 32 rows two operand sets would leave
// an SM four tiles of 16 bits and D = 128, too few in flight, so there is one CTA, whose two warpgroups have half of the
// rows each.
//
// What bounds it beside the bytes is code: eight roles' instructions pass through one instruction cache, and what is
// not in it takes some 16 cycles an instruction. So waits are short, loops rolled where they need not be fast, rare
// paths put aside, and columns past an item's rows are branched over.
//
// Measured (one copy reads and writes 6.7 TB/s): bfloat16, D = 128, pages of 16, 8 key heads: 64 sequences of 6 tokens,
// 500 to 8000 cached, 4 heads a group, 129 us (0.87 of the copy rate; with the rows on the lanes 133 to 141); 2
// sequences of 8 tokens, 60000 to 131072 cached, 8 heads a group, 159 us (154 to 161, 0.92; two CTAs an SM 213, rows on
// the lanes 180). float16, D = 64, 16 heads of their own, 128 sequences of one token with a window of 1024: 58 us (0.45;
// rows on the lanes 128), of which some 10 are the launches and the first tiles' way; its 128-byte pieces lie 2 KB apart,
// and more than half of its items have one tile. e4m3, D = 128, 32 sequences of 4 tokens, 2000 to 16384 cached: 93 us
// (0.79; rows on the lanes 150). Of the nine kernels the one for e4m3 and 64 rows spills, 76 bytes a thread.
#include "sv_cache_attend.cuh"

#include <type_traits>

namespace sv {
namespace cache {
namespace {

// The weights' tile: a slot's weights lie side by side, NR of them. e4m3: NR bytes for what rounding gives, hi, and NR
// for what it leaves, 2^kLow lo; a product of twice the columns then has both, O = O_hi + 2^-kLow O_lo. A weight
// 2^-n of the largest, which is 2^kShift or more, is kept to 2^-8 of itself, from n = 13 on to 2^-18 of the largest.
template <int K, int NR>
struct Weights {
    static constexpr int kPitch = 2 * NR;  // 32, 64 or 128 bytes, the width of the swizzle
    static constexpr int kBytes = kTile * kPitch;
    static constexpr int kColumns = K == kE4m3 ? 2 * NR : NR;  // of O
    static constexpr int kLow = 4;
    static constexpr uint32_t kSwizzle = kPitch == 128 ? 2u : kPitch == 64 ? 4u : 6u;
    static constexpr uint32_t kHigh = (uint32_t)(8 * kPitch) >> 4 | 1u << 14 | kSwizzle << 29;
    // weights are 2^kShift at a new reference, which stays until one is above 2^kMost: e4m3 ends at 448, fp16 at 65504
    static constexpr float kShift = K == kBf16 ? 0.f : K == kFp16 ? 7.f : 4.f;
    static constexpr float kMost = K == kBf16 ? 64.f : K == kFp16 ? 15.f : 8.75f;
    static_assert(kPitch >= 32 && kPitch <= 128, "a swizzle's width");
    // where the 16 bytes c of a slot lie
    static __device__ __forceinline__ uint32_t at(uint32_t slot, uint32_t c) {
        return slot * kPitch + ((c ^ ((slot * kPitch >> 7) & (kPitch / 16 - 1))) << 4);
    }
};

// With G softmax warpgroups each has NR / G rows of every tile; then comes a warp for each other role.
template <int G>
constexpr int kThreads = (G + 1) * 128;
constexpr int kReaders = 1 + 1 + 1;  // of an item, besides the softmax warps: loader, products, values
constexpr int kHalfSm = 113 * 1024;  // of shared memory

// What a group's warps tell each other when the references move and at an item's end: per warp a row's maximum, or
// sum. One group's notes lie in the weights' place, while no product reads that; two groups are not at the same step.
template <int N>
struct Notes {
    float part[4][N];
};
struct Nothing {};
template <int N, int G>
struct alignas(16) Group : std::conditional<G == 1, Nothing, Notes<N>>::type {
    uint64_t vote;
    int again[3];  // votes in turn: some weight is too large
};

template <int NR, int G>
struct alignas(16) Shared : Common {
    uint64_t s_full[2], p_ready, pv_done;
    Group<NR / G, G> group[G];
};

// A barrier of a group's warps; what lies between the two calls needs no one.
struct Vote {
    uint32_t bar, parity;
    Limit limit;
    __device__ __forceinline__ void arrive() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) bar_arrive(bar);
    }
    __device__ __forceinline__ bool pass() {
        const bool ok = wait(bar, parity, limit);
        parity ^= 1u;
        return ok;
    }
};

__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tc_ld16(uint32_t col, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : SV_R8(r, 0), SV_R8(r, 8)
                 : "r"(col));
}
__device__ __forceinline__ void tc_ld1(uint32_t col, uint32_t& r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(col));
}
__device__ __forceinline__ void tc_st1(uint32_t col, uint32_t r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(col), "r"(r) : "memory");
}
__device__ __forceinline__ void tc_ld4(uint32_t col, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(col));
}
// e4m3 weights in pairs: what rounding gives, and 2^kLow of what it leaves
template <int kLow>
__device__ __forceinline__ void split_weights(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = e4m3x2(a, b);
    const float2 x = from_e4m3x2(hi);
    lo = e4m3x2((a - x.x) * (1 << kLow), (b - x.y) * (1 << kLow));
}

// The rows that see a slot, as bits, the first of them row0.
__device__ __forceinline__ uint32_t rows_seeing(const Params& P, const Item& it, const Tree* tree, int32_t slot, uint32_t bad,
                                                int32_t row0) {
    if (slot < it.lo || slot >= it.end || (bad >> (slot % kTile >> 3) & 1u)) return 0;
    const int32_t i = slot - it.past, w = P.a.window;  // its place in the chunk, if it has one
    if (!rarely(tree)) {
        // (compared without i + w, which a window near 2^31 takes past an int32)
        const int32_t first = max(0, i), last = w > 0 && i < it.nt - w ? i + w - 1 : it.nt - 1;
        return prefix32((last + 1) * P.G - row0) & ~prefix32(first * P.G - row0);
    }
    if (i < 0 && w <= 0) return prefix32(it.nt * P.G - row0);
    uint32_t m = 0;
#pragma unroll 1
    for (int32_t t = 0; t < it.nt; ++t)
        if (i < 0 ? tree->depth[t] - i < w : tree->above[t] >> i & 1u) m |= prefix32((t + 1) * P.G - row0) & ~prefix32(t * P.G - row0);
    return m;
}

template <int K, int NR, int G>
__device__ __forceinline__ void softmax_role(const Params& P, Shared<NR, G>& sh, char* weights) {
    using KT = KindOf<K>;
    using T = typename KT::T;
    using Wt = Weights<K, NR>;
    const AttendArgs& A = P.a;
    constexpr int N = NR / G;  // the group's rows, from row0 on
    const int k = threadIdx.x & 127, lane = threadIdx.x & 31, warp = k >> 5, row0 = threadIdx.x / 128 * N;
    Group<N, G>& mine = sh.group[threadIdx.x / 128];
    const uint32_t lanes = (uint32_t)(k & ~31) << 16, tmem = sh.tmem + lanes + row0, p_smem = smem_u32(weights);
    const uint32_t o_col = tmem + 2 * NR;
    const uint32_t p_ready = smem_u32(&sh.p_ready), pv_done = smem_u32(&sh.pv_done);
    Notes<N>& notes = *(G == 1 ? reinterpret_cast<Notes<N>*>(weights) : reinterpret_cast<Notes<N>*>(&mine));
    static_assert(sizeof(Notes<N>) <= Wt::kBytes, "the notes fit");
    constexpr int kParts = K == kE4m3 ? 2 : 1;
    const int32_t D = A.pool.dim;
    const Limit limit{&sh.gave_up, P.polls};
    Vote vote{smem_u32(&mine.vote), 0, limit};
    uint32_t steps = 0, tiles = 0, votes = 0;  // votes: on weights, modulo 3
    bool owed = false;  // a vote of the last item's end has been given and not passed: others may still read the notes
    Items walk(P, sh);
    Item it;
#pragma unroll 1
    while (walk.next(it)) {
        const Tree* tree = A.chunk.parents ? &walk.tree() : nullptr;
        // taken from one lane: the same in all, so that the branches on it are the warp's. None or less: a group without work
        const int32_t rows = __shfl_sync(kAll, min(N, it.nt * P.G - row0), 0);
        bool flip;
        const float unit = score_unit(A, it.h, flip);
        float l[N], off[N], u[K == kE4m3 ? N : 1];  // weights are 2^(u s + off)
        u[0] = unit;
        // The loops below take four rows at a time. Those past the item's last have another sequence's queries, or what
        // an earlier item left (e4m3: and an unset factor): their weights are zero, or nothing would keep their scores
        // from voting on the references, and so from changing the roundings of the item's own rows.
#pragma unroll
        for (int r = 0; r < N; ++r) {
            l[r] = 0.f;
            off[r] = r < rows ? Wt::kShift : -INFINITY;
        }
        // every warp settles the references by itself, from the same notes: a lane has a row's (off again, and whether
        // there is a reference at all)
        float own_off = Wt::kShift;
        bool own = false, unset = true;
#pragma unroll 1
        for (int32_t j = 0; j < it.n; ++j, ++steps) {
            const uint32_t buf = steps & 1;
            if (!wait(smem_u32(&sh.s_full[buf]), steps >> 1 & 1, limit)) return;
            tc_after();
            if (K == kE4m3 && j == 0)
#pragma unroll
                for (int r = 0; r < (K == kE4m3 ? N : 1); r += 4) {
                    if (r >= rows) break;
#pragma unroll
                    for (int e = 0; e < (K == kE4m3 ? 4 : 1); ++e)
                        u[r + e] = row_unit(unit, sh.q_down[walk.ring.i * sh.q_rows + row0 + r + e]);
                }
            const uint32_t s_col = tmem + buf * NR;
            const int32_t k0 = (it.tile + j) * kTile;
            const uint32_t ring = (tiles + j) % kNotes;
            const uint32_t bad = sh.bad[0][ring];
            const bool cut = k0 < max(it.lo, it.mixed_lo) || k0 + kTile > min(it.mixed_hi, it.end) || bad;
            uint32_t seen = ~0u;
            if (rarely(cut)) seen = rows_seeing(P, it, tree, k0 + k, bad, row0);
            uint32_t s[N];
            // Once, mostly: while the votes come in that no weight is too large, the weights are taken as if none were.
            bool fresh = unset;
#pragma unroll 1
            for (;;) {
#pragma unroll
                for (int c = 0; c < N; c += 16) {
                    if (c > 0 && c >= rows) break;
                    tc_ld16(s_col + c, s + c);
                }
                tc_wait_ld();
                if (rarely(cut))
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        if (r >= rows) break;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(seen >> (r + e) & 1u)) s[r + e] = 0xff800000u;
                    }
                // the weights' logarithms against the references (where there is none yet, against 0)
                float top = -INFINITY;
#pragma unroll
                for (int r = 0; r < N; r += 4) {
                    if (r >= rows) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = fmaf(__uint_as_float(s[r + e]), u[K == kE4m3 ? r + e : 0], off[r + e]);
                        s[r + e] = __float_as_uint(y);
                        top = fmaxf(top, y);
                    }
                }
                if (!fresh) {
                    // no one passes this vote before everyone has read the last but one's word
                    if (k == 0) mine.again[votes == 2 ? 0 : votes + 1] = 0;
                    if (__any_sync(kAll, top > Wt::kMost) && lane == 0) mine.again[votes] = 1;
                    vote.arrive();
                } else {
                    if (owed && !vote.pass()) return;
                    owed = false;
                    if (j > 0) {  // O is whole, and the notes' place free, once the last step's product has been
                        if (!wait(pv_done, (steps - 1) & 1, limit)) return;
                        tc_after();
                    }
                    // the rows' maxima, by warp, then of all
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        if (r >= rows) break;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = warp_max(__uint_as_float(s[r + e]));
                            if (lane == r + e) notes.part[warp][r + e] = x;
                        }
                    }
                    vote.arrive();
                    if (!vote.pass()) return;
                    const int r0 = lane % N;
                    const float mx = fmaxf(fmaxf(notes.part[0][r0], notes.part[1][r0]), fmaxf(notes.part[2][r0], notes.part[3][r0])) -
                                     Wt::kShift;
                    vote.arrive();
                    // from none to the maximum, if there is one; else upwards only
                    const float d = r0 >= rows ? 0.f : own ? fmaxf(mx, 0.f) : mx != -INFINITY ? mx : 0.f;
                    const bool moved = __any_sync(kAll, own && d > 0.f);
                    const float fac = own ? exp2_fast(-d) : 1.f;
                    own_off -= d;
                    own = own || mx != -INFINITY;
                    unset = __any_sync(kAll, r0 < rows && !own);
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        if (r >= rows) break;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = __shfl_sync(kAll, d, r + e);
                            s[r + e] = __float_as_uint(__uint_as_float(s[r + e]) - x);
                            off[r + e] -= x;
                        }
                    }
                    if (rarely(moved)) {
#pragma unroll
                        for (int r = 0; r < N; ++r) l[r] *= __shfl_sync(kAll, fac, r);
#pragma unroll 1
                        for (int c = 0; c < kParts * N; c += 16) {
                            if (c % N >= rows) continue;
                            const uint32_t col = o_col + (c >= N ? NR - N : 0) + c;
                            uint32_t o[16];
                            tc_ld16(col, o);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(kAll, fac, c % N + i));
                            tc_st16(col, o);
                        }
                        tc_wait_st();
                    }
                }
#pragma unroll
                for (int r = 0; r < N; r += 4) {
                    if (r >= rows) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r + e] = __float_as_uint(exp2_fast(__uint_as_float(s[r + e])));
                }
                if (!vote.pass()) return;
                if (fresh) break;
                fresh = mine.again[votes];
                votes = votes == 2 ? 0 : votes + 1;
                if (!fresh) break;
            }
            uint32_t pk[N / 2];  // 16 bits: pairs; e4m3: hi in the first half, lo in the second
#pragma unroll
            for (int r = 0; r < N; r += 4) {
                if (r >= rows) break;
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = __uint_as_float(s[r + e]);
                    l[r + e] += p[e];
                }
                if (K != kE4m3) {
                    pk[r / 2] = from_float2<T>(p[0], p[1]);
                    pk[r / 2 + 1] = from_float2<T>(p[2], p[3]);
                } else {
                    uint32_t a, b, c, d;
                    split_weights<Wt::kLow>(p[0], p[1], a, c);
                    split_weights<Wt::kLow>(p[2], p[3], b, d);
                    pk[r / 4] = a | b << 16;
                    pk[N / 4 + r / 4] = c | d << 16;
                }
            }
            // the weights' place is free once the last step's product has been
            if (j > 0 && !wait(pv_done, (steps - 1) & 1, limit)) return;
            constexpr int kWide = N * KT::kBytes / 16;  // 16 bytes of a part
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
                for (int c = 0; c < kWide; ++c) {
                    if (c * (16 / KT::kBytes) >= rows) break;
                    const uint32_t* v = pk + part * (N / 4) + 4 * c;
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                                     p_smem + Wt::at(k, part * (NR / 16) + row0 / N * kWide + c)),
                                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                 : "memory");
                }
            const bool mixed = mixed_tile(it, k0);
            if (rarely(mixed)) {  // before p_ready: the tile cannot be released, nor its barrier move on, until then
                const uint32_t v = tiles + j;
                if (!wait(smem_u32(&sh.value[v % P.v_slots]), (v / P.v_slots) & 1, limit)) return;
            }
            fence_async();
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_ready);
            if (rarely(mixed)) {
                // rows that see a non-finite value, which the product met as zero, get it added here
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) any |= sh.odd[ring][i];
                if (rarely(any)) {
                    if (!wait(pv_done, steps & 1, limit)) return;
                    tc_after();
#pragma unroll 1
                    for (int i = 0; i < 4; ++i)
#pragma unroll 1
                        for (uint32_t w = sh.odd[ring][i]; w; w &= w - 1) {
                            const int32_t slot = k0 + 32 * i + __ffs(w) - 1;
                            const int64_t at = place_of(A.pool, it.b, slot) + it.h * A.pool.s_head + k;
                            float x = 0.f;
                            if (k < D) {
                                if (K == kE4m3) x = (((const uint8_t*)A.pool.v)[at] & 0x7f) == 0x7f ? NAN : 0.f;
                                else x = (float)((const T*)A.pool.v)[at];
                            }
                            if (isfinite(x)) x = 0.f;
                            const uint32_t m = rows_seeing(P, it, tree, slot, bad, row0);
#pragma unroll 1
                            for (int c = 0; c < rows; ++c) {
                                uint32_t o;
                                tc_ld1(o_col + c, o);
                                tc_wait_ld();
                                if (m >> c & 1u) o = __float_as_uint(__uint_as_float(o) + x);
                                __syncwarp();
                                tc_st1(o_col + c, o);
                                tc_wait_st();
                            }
                        }
                    tc_before();
                }
            }
        }
        tiles += it.n;

        // the item's end: the rows' sums over the lanes
        // of four rows at a time: lanes trade until each has one row's, then add it up
        float sum[N / 4];
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            sum[q] = 0.f;
            if (4 * q >= rows) break;
            float* x = l + 4 * q;
            const bool up = lane & 16, right = lane & 8;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float give = up ? x[e] : x[e + 2], keep = up ? x[e + 2] : x[e];
                x[e] = keep + __shfl_xor_sync(kAll, give, 16);
            }
            const float give = right ? x[0] : x[1], keep = right ? x[1] : x[0];
            sum[q] = keep + __shfl_xor_sync(kAll, give, 8);
#pragma unroll
            for (int o = 4; o; o >>= 1) sum[q] += __shfl_xor_sync(kAll, sum[q], o);
        }
        if (!wait(pv_done, (steps - 1) & 1, limit)) return;
        tc_after();
        if (!(lane & 7))
#pragma unroll
            for (int q = 0; q < N / 4; ++q) notes.part[warp][4 * q + (lane >> 3 & 2) + (lane >> 3 & 1)] = sum[q];
        vote.arrive();
        if (!vote.pass()) return;
        const int r0 = lane % N;
        const float total = (notes.part[0][r0] + notes.part[1][r0]) + (notes.part[2][r0] + notes.part[3][r0]);
        vote.arrive();
        owed = true;
        const bool alone = it.begins && it.finishes;
        const size_t part = (size_t)(2 * blockIdx.x + (it.begins ? 1 : 0)) * P.part_rows + row0;
        // What a row's O is scaled by. Here and in lse the quotient and the logarithm are the short ones, 2 ulp and 2^-22 off:
        // out is rounded to 2^-9 or 2^-12 next, and an exponential before them is 2^-22 off as well.
        float f = 1.f;
        if (alone) f = total == 0.f ? 0.f : __fdividef(A.pool.v_scale ? A.pool.v_scale[it.h] : 1.f, total);
        if (k < rows && k < N) {
            if (alone) {
                const int32_t row = row0 + k, t = row / P.G;
                if (A.lse)
                    A.lse[(int64_t)(it.row0 + it.t0 + t) * A.q_heads + it.h * P.G + row - t * P.G] =
                        total == 0.f ? -INFINITY : (__log2f(total) - own_off) * kLn2;
            } else {
                P.part_ml[part + k] = make_float2(own ? -own_off : -INFINITY, total);
            }
        }
        const int32_t dp = K == kE4m3 || D > 64 ? 128 : 64;
        const int32_t t0 = row0 / P.G;
        int32_t g = row0 - t0 * P.G;
        T* out = (T*)A.out + ((int64_t)(it.row0 + it.t0 + t0) * A.q_heads + it.h * P.G + g) * D + k;
        float* out_part = P.part_o + part * dp + k;
#pragma unroll 1
        for (int c = 0; c < rows; c += 4) {
            uint32_t o[4], o_low[4];
            tc_ld4(o_col + c, o);
            if (K == kE4m3) tc_ld4(o_col + NR + c, o_low);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = __uint_as_float(o[i]);
                if (K == kE4m3) x = fmaf(__uint_as_float(o_low[i]), 1.f / (1 << Wt::kLow), x);
                x *= __shfl_sync(kAll, f, c + i);
                if (k < D && c + i < rows) {
                    if (alone) *out = (T)x;
                    else out_part[(c + i) * dp] = x;
                }
                out += D;
                if (++g == P.G) {  // the next token's heads
                    g = 0;
                    out += (int64_t)(A.q_heads - P.G) * D;
                }
            }
        }
        tc_before();
    }
}

// The products, by one thread, in the order in which they become possible: a tile's scores, into one of two buffers, once
// its keys are in (an item's first: its queries too); its outputs, once its weights and values are. Scores run up to two
// tiles ahead, also into the next item.
template <int K, int NR, int G>
__device__ __forceinline__ void product_role(const Params& P, Shared<NR, G>& sh, uint32_t q_smem, uint32_t p_smem, uint32_t k_smem,
                                             uint32_t v_smem) {
    constexpr bool k8 = K == kE4m3;
    constexpr int parts = k8 ? 2 : 1;
    constexpr uint32_t fmt = K == kBf16 ? 1u : 0u;
    using Wt = Weights<K, NR>;
    const int32_t D = P.a.pool.dim;
    const int32_t depth = (D + KindOf<K>::kStep - 1) / KindOf<K>::kStep;
    const uint32_t slot_bytes = P.halves * kHalf;
    // float accumulators, 128 lanes, NR columns; of O both operands' rows lie along the depth
    const uint32_t id = 1u << 4 | fmt << 7 | fmt << 10 | (uint32_t)(kTile >> 4) << 24;
    const uint32_t id_s = id | (uint32_t)(NR >> 3) << 17, id_o = id | (uint32_t)(Wt::kColumns >> 3) << 17 | 3u << 15;
    const uint32_t tmem = __shfl_sync(kAll, sh.tmem, 0), o_at = tmem + 2 * NR;
    const uint32_t k_full = smem_u32(sh.k_full), k_empty = smem_u32(sh.k_empty), v_empty = smem_u32(sh.v_empty),
                   value = smem_u32(sh.value), s_full = smem_u32(sh.s_full), p_ready = smem_u32(&sh.p_ready),
                   pv_done = smem_u32(&sh.pv_done), q_full = smem_u32(sh.q_full), q_empty = smem_u32(sh.q_empty);
    const uint32_t q_part = (uint32_t)P.q_part >> 4, p = operand(p_smem, 16);
    const bool leader = elect();
    const Limit limit{&sh.gave_up, P.polls};
    uint32_t ahead = 0, scores = 0, outputs = 0, polls = 0;
    uint32_t notes = 0;  // 16 bits a buffer: the first and last step of the outputs' depth, an item's first tile
    int32_t j = 0, n = 0;
    Ring kr, vr, qr;
    Items walk(P, sh);
    Item it;
    bool more = walk.next(it);
    n = __shfl_sync(kAll, it.n, 0);
#pragma unroll 1
    while (more || ahead > 0) {
        if (more && ahead < 2 && (j > 0 || ready(q_full + 8 * qr.i, qr.parity)) && ready(k_full + 8 * kr.i, kr.parity)) {
            tc_after();
            const uint32_t q = operand(q_smem + qr.i * P.q_bytes, 16);
            const uint32_t buf = scores & 1, a = operand(k_smem + kr.i * slot_bytes, 16), d = tmem + buf * NR;
            if (leader) {
#pragma unroll
                for (int part = 0; part < parts; ++part)
#pragma unroll 1
                    for (int i = 0; i < depth; ++i) {
                        const uint32_t in = (i & 3) * 32 >> 4;
                        mma_ss<k8>(d, a + (i >> 2) * (kHalf >> 4) + in, q + (k8 ? part : i >> 2) * q_part + in, id_s, part + i > 0);
                    }
                tc_commit(s_full + 8 * buf);
                tc_commit(k_empty + 8 * kr.i);
                if (j + 1 == n) tc_commit(q_empty + 8 * qr.i);
            }
            __syncwarp();
            int32_t lo, hi;
            steps_of<K>(it, (it.tile + j) * kTile, lo, hi);
            notes = (notes & ~(0xffffu << 16 * buf)) | (uint32_t)(lo | hi << 4 | (j == 0) << 8) << 16 * buf;
            kr.step(P.k_slots);
            ++scores;
            ++ahead;
            polls = 0;
            if (++j == n) {
                j = 0;
                qr.step(P.q_bufs);
                more = walk.next(it);
                n = __shfl_sync(kAll, it.n, 0);
            }
        } else if (ahead > 0 && ready(p_ready, outputs & 1) && ready(value + 8 * vr.i, vr.parity)) {
            tc_after();
            // D <= 64: the upper 64 lanes repeat the lower ones' columns
            const uint32_t a = operand(v_smem + vr.i * slot_bytes, slot_bytes > kHalf ? kHalf : 0);
            const uint32_t note = __shfl_sync(kAll, notes, 0) >> 16 * (outputs & 1);
            const int32_t lo = note & 15u, hi = note >> 4 & 15u;
            const uint32_t add = (note >> 8 & 1u) ^ 1u;
            if (leader) {
#pragma unroll 1
                for (int i = lo; i < hi; ++i)
                    mma_mixed<k8, Wt::kHigh>(o_at, a + (i * KindOf<K>::kStep * 128 >> 4), p + (i * KindOf<K>::kStep * Wt::kPitch >> 4), id_o,
                                             i > lo ? 1u : add);
                tc_commit(pv_done);
                tc_commit(v_empty + 8 * vr.i);
            }
            __syncwarp();
            vr.step(P.v_slots);
            ++outputs;
            --ahead;
            polls = 0;
        } else if ((++polls & 255u) == 0) {
            if (polls >> 4 >= limit.polls) *limit.gave_up = 1;  // these do not sleep: 0.1 us each, half a second in all
            if (__any_sync(kAll, *limit.gave_up)) break;
        }
    }
    // products under way end before the tensor memory is given back
    if (leader) tc_commit(smem_u32(&sh.drain));
    __syncwarp();
    drain(smem_u32(&sh.drain), 0);
}

template <int K, int NR, int G>
__global__ void __launch_bounds__(kThreads<G>, G == 1 ? 2 : 1)
    k_attend_few(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                 const __grid_constant__ CUtensorMap qm) {
    constexpr int columns = 4 * NR;  // twice NR for scores, NR (e4m3: twice) for O
    extern __shared__ __align__(1024) char raw[];
    const uint32_t slot_bytes = P.halves * kHalf;
    const uint32_t q_smem = smem_u32(raw), p_smem = q_smem + P.q_bufs * P.q_bytes, k_smem = p_smem + Weights<K, NR>::kBytes,
                   v_smem = k_smem + P.k_slots * slot_bytes;
    char* behind = raw + (v_smem - q_smem) + P.v_slots * slot_bytes;
    Shared<NR, G>& sh = *reinterpret_cast<Shared<NR, G>*>(behind);
    if (q_smem & 1023u) {  // the tiles' swizzle counts on it
        if (threadIdx.x == 0) report(P.a.status, 1u << SV_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, w = tid >> 5;
    if (tid == 0) {
        init_common(sh, 1, 4 * G + kReaders, 1);
        bar_init(smem_u32(&sh.s_full[0]), 1);
        bar_init(smem_u32(&sh.s_full[1]), 1);
        bar_init(smem_u32(&sh.p_ready), 4 * G);
        bar_init(smem_u32(&sh.pv_done), 1);
        for (int g = 0; g < G; ++g) {
            bar_init(smem_u32(&sh.group[g].vote), 4);
            sh.group[g].again[0] = 0;
        }
        sh.q_rows = NR;
        sh.tree = reinterpret_cast<Tree*>(behind + (sizeof(sh) + 15) / 16 * 16);
        sh.q_down = reinterpret_cast<float*>(sh.tree + (P.a.chunk.parents ? kItems : 0));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // query rows past the copies' last one stay zero
    for (int i = tid; i < P.q_bufs * P.q_bytes / 16; i += kThreads<G>) reinterpret_cast<uint4*>(raw)[i] = make_uint4(0, 0, 0, 0);
    fence_async();
    const int role = w - 4 * G;
    if (role == 0 && (tid & 31) == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&km));
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vm));
        if (K != kE4m3) asm volatile("prefetch.tensormap [%0];" ::"l"(&qm));
    }
    begin<kThreads<G>, columns>(P, sh, role == 1);
    // at launch 128 registers a thread for one group, 168 for two
    if (role < 0) {
        if (G == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        softmax_role<K, NR, G>(P, sh, raw + P.q_bufs * P.q_bytes);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (role == 0) load_role(P, sh, k_smem, v_smem, &km, &vm, 0, 1);
        else if (role == 1) product_role<K, NR, G>(P, sh, q_smem, p_smem, k_smem, v_smem);
        else if (role == 2) value_role<K>(P, sh, v_smem);
        else item_role<K, 1>(P, sh, q_smem, &qm);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (role == 1) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "n"(columns));
    }
    if (tid == 0 && sh.gave_up) report(P.a.status, 1u << SV_ERR_TIMEOUT);
}

template <int K, int NR, int G>
cudaError_t launch(Params& P, int sms, cudaStream_t st) {
    const AttendArgs& A = P.a;
    P.ctas = G == 1 ? 2 * sms : sms;
    const int halves = P.halves = K == kE4m3 || A.pool.dim <= 64 ? 1 : 2;
    P.tokens = P.block = A.chunk.max_gamma + 1;
    P.q_box = P.tokens;
    P.q_part = NR * 128;
    P.lead = halves == 2 ? 1 : 2;  // measured on the cases above: others of 0 to 4 are 1 to 30 % slower
    P.q_tile = (K == kE4m3 ? 2 : halves) * P.q_part;
    const int own = (int)(sizeof(Shared<NR, G>) + 15) / 16 * 16 + (A.chunk.parents ? kItems * (int)sizeof(Tree) : 0) +
                    (K == kE4m3 ? kItems * NR * 4 : 0);
    P.q_bytes = P.q_tile;
    auto slots_of = [&](int bufs) {
        const int rest = (G == 1 ? kHalfSm : kSmem) - bufs * P.q_bytes - Weights<K, NR>::kBytes - own;
        return min(2 * kMaxSlots, rest / (halves * kHalf));
    };
    // The next item's queries are fetched (e4m3: and split into parts) under this one's tiles, where that costs no slot.
    P.q_bufs = K == kE4m3 || slots_of(2) == slots_of(1) ? 2 : 1;
    const int slots = slots_of(P.q_bufs), rest = P.q_bufs * P.q_bytes + Weights<K, NR>::kBytes + own;
    P.k_slots = slots / 2;
    P.v_slots = slots - P.k_slots;
    CUtensorMap km, vm, qm;
    if (K != kE4m3 && !encode_queries(&qm, A, K, P.G, P.q_box)) return cudaErrorInvalidValue;
    if (!encode_pool(&km, A.pool, A.pool.k, KindOf<K>::kBytes, K, P.box) ||
        !encode_pool(&vm, A.pool, A.pool.v, KindOf<K>::kBytes, K, P.box))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> allowed{0};
    void* args[] = {&P, &km, &vm, &qm};
    return launch_early((const void*)k_attend_few<K, NR, G>, &allowed, dim3(P.ctas), kThreads<G>, rest + slots * halves * kHalf, st, args);
}

template <int K>
cudaError_t choose(Params& P, int rows, int sms, cudaStream_t st) {
    P.part_rows = kFewRows;
    if (rows <= 16) return launch<K, 16, 1>(P, sms, st);
    return rows <= 32 ? launch<K, 32, 1>(P, sms, st) : launch<K, 64, 2>(P, sms, st);
}

}  // namespace

cudaError_t launch_few(Params& P, int kind, int rows, int sms, cudaStream_t st) {
    return kind == kE4m3 ? choose<kE4m3>(P, rows, sms, st) : kind == kFp16 ? choose<kFp16>(P, rows, sms, st) : choose<kBf16>(P, rows, sms, st);
}

}  // namespace cache
}  // namespace sv
