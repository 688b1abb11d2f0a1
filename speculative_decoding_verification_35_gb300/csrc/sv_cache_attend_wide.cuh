// spec_cache_attend and spec_cache_attend_scored (include/speccache.h): attention of a chunk of new tokens over the paged
// cache. The kernel for chunks of more than 64 rows; kScored: scores capped, biased or seen by a prefix, in two files of
// their own, so that they compile beside the others.
//
// Mathematics. A row (token, query head) with scores z_s = scale q . k_s keeps a reference m and, tile after
// tile of 128 slots, l = sum 2^(z_s log2 e - m) and O = sum 2^(z_s log2 e - m) v_s; out = O / l. When a tile's
// maximum exceeds m by more than a threshold, m moves there and l and O are scaled by 2^(old - new). Partial
// (m, l, O) of disjoint slots merge the same way, so a row's slots can be shared out.
//
// Shape. The query heads of a group share their key head, so a query tile of 128 rows packs 128 / G tokens of G heads,
// and both products run on the tensor cores as 128 x 128 x D (S = Q K^T, O += P V), operands in shared memory,
// S, P and O in tensor memory. A CTA (one per SM) has two such tiles, one for each of its two softmax warpgroups, so
// that the tensor cores work for one while the other is at its exponentials, and a tile of keys and values is read from
// the cache once for 256 rows. Chunks of up to 64 rows have too few rows to fill such tiles and go to
// sv_cache_attend_few.cuh, which turns the products around.
//
// Split. The items' tiles are numbered in one line (sequence, row block, key head, tile), and CTA c of n takes
// those from c W / n to (c + 1) W / n, whatever items they belong to: every SM gets the same number of
// tiles with one long sequence or hundreds of short ones, and a CTA leaves at most two items unfinished. Their
// partials go to the workspace, and a second small launch merges them in a fixed order. Lengths are read
// on the device, so the host needs to know none of them.
//
// Bound by the chain of a stream's tile: scores (512 cycles of the tensor cores at D = 128), softmax (some 1450), outputs
// (512) and what lies between; two streams in turn keep the tensor cores busy 1024 of every 1560 cycles. Measured:
// bfloat16, D = 128, 3 prompts of 700 to 2048 tokens over 1 to 8192 cached, 32 heads in 8 groups: 233 us (230 to 238),
// 1.27 PFLOP/s of what the mask leaves (0.67 of a library product's 1.89), 3 us of them the merge. The same prompts on an
// e4m3 cache take 356 us.
// Scored: a pass over the scores in tensor memory before the softmax's, 32 columns at a time, is latency and multiply-adds (9 or 7
// packed operations for two scores) on top of the chain above: the same prompts, plain 218 us, with a prefix 248 (more is
// seen), capped 399, both 456, by distance 330. In one pass with the weights it was slower: capped 472 and more unrolled, which
// waits for instructions, and 454 rolled, where a pass of its own took 418 at the time.
#pragma once
#include "sv_cache_attend.cuh"

#include <algorithm>

namespace sv {
namespace cache {
namespace wide {

constexpr int kThreads = 512;  // two softmax warpgroups, then a warp for each other role
constexpr int kReaders = 8 + 2 + 2 + 1;
constexpr int kSplitters = 3;  // warps that split the queries for e4m3 caches: two of their own, and the items'

struct Shared : Common {
    uint64_t s_full[2], p_ready[2], pv_done[2];
    uint64_t turn[2];  // the streams' products take turns
};

// ---------------------------------------------------------------------------------------------------------
// the softmax warpgroups
// ---------------------------------------------------------------------------------------------------------
// A row of a query tile as its thread knows it.
struct Row {
    bool real;
    int32_t token;      // chunk token
    int32_t low, limit; // slots low .. limit - 1 are seen, as far as they are not a tree's
    uint32_t above;     // a tree: the chunk tokens it sees
    float sl;           // score units to log2 of the weight, not negative
    float raw;          // kScored: the same before the scores are capped and biased, when sl becomes 1
    int32_t pos;
    float slope;        // kScored: log2 of the weight that a step of distance costs
};

// tl: the row's token within its tile; g: its head within the group.
template <bool kScored>
__device__ __forceinline__ Row row_of(const Params& P, const Item& it, const Items& items, int stream, int32_t tl, int32_t g) {
    const AttendArgs& A = P.a;
    Row row;
    row.token = it.t0 + tl + (stream ? it.split : 0);
    row.real = tl < (stream ? it.nt - it.split : it.split);
    row.above = 0;
    int32_t depth = row.token;
    if (A.chunk.parents && row.real) {
        row.above = items.tree().above[row.token];
        depth = items.tree().depth[row.token];
    }
    const int32_t pos = it.past + depth;
    row.low = A.window > 0 ? max(0, pos - A.window + 1) : 0;
    row.limit = it.past + (A.chunk.parents ? 0 : row.token + 1);
    bool flip;
    row.sl = score_unit(A, it.h, flip);
    if (kScored) {
        row.limit = max(row.limit, it.reach);
        row.pos = pos;
        row.slope = A.slopes && row.real ? A.slopes[it.h * P.G + g] * kLog2e : 0.f;
        row.raw = row.sl;
        if (A.cap > 0.f || A.slopes) row.sl = 1.f;
    }
    return row;
}

// The 128 slots of a tile that a row sees.
__device__ __forceinline__ void seen_of(const Row& row, const Item& it, int32_t k0, uint32_t bad, bool tree, uint32_t* seen) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t at = k0 + 32 * i;
        uint32_t m = prefix32(row.limit - at) & ~prefix32(row.low - at);
        if (tree) {
            const int32_t off = it.past - at;  // chunk token t lies at bit off + t
            if (off > -32 && off < 32) m |= off >= 0 ? row.above << off : row.above >> -off;
        }
        if (bad) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (bad >> (4 * i + g) & 1u) m &= ~(0xffu << (8 * g));
        }
        seen[i] = m;
    }
}

// Adds the non-finite values of the slots in odd that a row sees (and its product met as zero) to its output.
template <int K, int DP>
__device__ __forceinline__ void add_odd(const AttendArgs& A, const Item& it, uint32_t o_col, int32_t k0, const uint32_t* odd,
                                     const uint32_t* seen) {
    using T = typename KindOf<K>::T;
#pragma unroll 1
    for (int c = 0; c < DP; c += 32) {
        uint32_t o[32];
        tc_ld32(o_col + c, o);
        tc_wait_ld();
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
            for (uint32_t w = odd[i] & seen[i]; w; w &= w - 1) {
                const int32_t slot = k0 + 32 * i + __ffs(w) - 1;
                const int64_t at = place_of(A.pool, it.b, slot) + it.h * A.pool.s_head;
#pragma unroll
                for (int d = 0; d < 32; ++d) {
                    float x = 0.f;
                    if (c + d < A.pool.dim) {
                        if (K == kE4m3) x = (((const uint8_t*)A.pool.v)[at + c + d] & 0x7f) == 0x7f ? NAN : 0.f;
                        else x = (float)((const T*)A.pool.v)[at + c + d];
                    }
                    if (!isfinite(x)) o[d] = __float_as_uint(__uint_as_float(o[d]) + x);
                }
            }
        tc_st32(o_col + c, o);
    }
}

// A step turns a tile's scores into its weights, in their place, and sums them. quick_weights reads the scores once
// and counts on the row's reference; where a weight would be too large for it nothing is written, the tile's
// maximum is taken, the reference moves and the step begins again. A row's first tile and the narrow e4m3 weights
// begin with the maximum. What few tiles need (tile_max, hide_tile) is rolled: unrolled, the roles' code misses the
// instruction cache in every step (measured: 1500 cycles a step, 2200 with all unrolled).
__device__ __forceinline__ float tile_max(uint32_t s_col) {
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int q = 0; q < 4; q += 2) {
        uint32_t s[2][32];
        tc_ld32(s_col + 32 * q, s[0]);
        tc_ld32(s_col + 32 * q + 32, s[1]);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top[e] = fmaxf(top[e], fmaxf(__uint_as_float(s[0][i + e]), __uint_as_float(s[1][i + e])));
    }
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}
// Scores of slots that a row does not see become -inf.
__device__ __forceinline__ void hide_tile(uint32_t s_col, const uint32_t* seen) {
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const uint32_t m = q == 0 ? seen[0] : q == 1 ? seen[1] : q == 2 ? seen[2] : seen[3];
        if (__all_sync(kAll, m == ~0u)) continue;
        uint32_t s[32];
        tc_ld32(s_col + 32 * q, s);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(m >> i & 1u)) s[i] = 0xff800000u;
        tc_st32(s_col + 32 * q, s);
    }
    tc_wait_st();
}
// kScored: what becomes of the scores.
struct Scoring {
    Cap cap;
    bool capped, biased;
    float by;
    __device__ __forceinline__ explicit Scoring(const AttendArgs& A)
        : cap(A.cap > 0.f ? A.cap : 1.f), capped(A.cap > 0.f), biased(A.slopes != nullptr), by(capped ? cap.by : 1.f) {}
    // 32 scores of a row, times f, capped, in place; col: where they lie in tensor memory, which is free to be written.
    __device__ __forceinline__ void cap32(uint32_t* s, float f, uint32_t col) const {
        const F2 f2 = pack2(f, f);
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 2) big = fmaxf(big, fmaxf(fabsf(__uint_as_float(s[i])), fabsf(__uint_as_float(s[i + 1]))));
        if (rarely(__any_sync(kAll, big * f > 1.f))) {  // some lie past the cap: in a few instructions
#pragma unroll 1
            for (int c = 0; c < 32; c += 4) {
                uint32_t x[4];
                tc_ld4(col + c, x);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __float_as_uint(cap.of(__uint_as_float(x[i]) * f));
                tc_st4(col + c, x);
            }
            tc_wait_st();
            tc_ld32(col, s);
            tc_wait_ld();
            return;
        }
        auto each = [&](auto&& g) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float a, b;
                unpack2(g(mul2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), f2)), a, b);
                s[i] = __float_as_uint(a);
                s[i + 1] = __float_as_uint(b);
            }
        };
        if (__any_sync(kAll, big * f > Cap::kSmall)) each([&](F2 x) { return cap.near(x, 0); });
        else each([&](F2 x) { return cap.small(x); });
    }
};
// A tile's scores become logarithms of the weights, in their place: a pass of its own.
__device__ __forceinline__ void score_tile(const Scoring& sc, bool tree, const Row& row, const Item& it, const Items& items, uint32_t s_col,
                                        int32_t k0) {
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        uint32_t s[32];
        tc_ld32(s_col + 32 * q, s);
        tc_wait_ld();
        if (sc.capped) sc.cap32(s, row.raw * sc.by, s_col + 32 * q);
        if (sc.biased) {
            const float unit = sc.capped ? 1.f : row.raw;
            const int32_t at = k0 + 32 * q;
            const float far = (float)(row.pos - at);
            const bool nodes = tree && at + 32 > it.past;  // chunk tokens of a tree lie at other positions than their slots
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float d = far - (float)i;
                const int32_t t = at + i - it.past;  // (of the tree, whose earlier tokens may be another block's)
                if (rarely(nodes) && t >= 0 && t < it.t0 + it.nt) d = (float)(row.pos - it.past - items.tree().depth[t]);
                s[i] = __float_as_uint(fmaf(-row.slope, fabsf(d), __uint_as_float(s[i]) * unit));
            }
        }
        tc_st32(s_col + 32 * q, s);
    }
    tc_wait_st();
}
template <int K>
__device__ __forceinline__ void weights32(const uint32_t* x, F2 sl2, F2 off2, F2* sum, uint32_t* pk) {
    using T = typename KindOf<K>::T;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            unpack2(fma2(pack2(__uint_as_float(x[i + e]), __uint_as_float(x[i + e + 1])), sl2, off2), p[e], p[e + 1]);
            p[e] = exp2_fast(p[e]);
            p[e + 1] = exp2_fast(p[e + 1]);
            sum[e >> 1] = add2(sum[e >> 1], pack2(p[e], p[e + 1]));
        }
        if (K != kE4m3) {
            pk[i >> 1] = from_float2<T>(p[0], p[1]);
            pk[(i >> 1) + 1] = from_float2<T>(p[2], p[3]);
        } else {
            uint32_t a, b, c, d;
            split_pair(p[0], p[1], a, c);
            split_pair(p[2], p[3], b, d);
            pk[i >> 2] = a | b << 16;
            pk[8 + (i >> 2)] = c | d << 16;
        }
    }
}
// False, with nothing written, if the weights of some row sum to more than their type may hold. bounded: the row's
// reference has met the tile's maximum, so each weight is 2^(kShift + kSlack) at most and all are written. (Their sum is
// no test then: 128 of that size sum to the limit itself, and as the arguments are rounded, to a little more.)
template <int K>
__device__ __forceinline__ bool quick_weights(uint32_t s_col, float sl, float off, bool real, bool bounded, float& total) {
    const F2 sl2 = pack2(sl, sl), off2 = pack2(off, off);
    F2 sum[2] = {0, 0};
    uint32_t s[2][32], pk[4][16];
    tc_ld32(s_col, s[0]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        tc_wait_ld();
        if (q < 3) tc_ld32(s_col + 32 * q + 32, s[(q + 1) & 1]);
        weights32<K>(s[q & 1], sl2, off2, sum, pk[q]);
    }
    float a, b;
    unpack2(add2(sum[0], sum[1]), a, b);
    total = a + b;
    if (K != kE4m3 && !bounded && __any_sync(kAll, real && total > (K == kBf16 ? 0x1p64f : 0x1p15f))) return false;
#pragma unroll
    for (int q = 0; q < 4; ++q) tc_st16(s_col + 16 * q, pk[q]);
    return true;
}
// O times f, a factor per row.
template <int DP>
__device__ __forceinline__ void rescale(uint32_t o_col, float f) {
#pragma unroll 1
    for (int c = 0; c < DP; c += 32) {
        uint32_t o[32];
        tc_ld32(o_col + c, o);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tc_st32(o_col + c, o);
    }
}

// Among four lanes: what was block b (8 of 32) of lane i becomes block i of lane b.
__device__ __forceinline__ void trade(uint32_t* u, int lane) {
#pragma unroll
    for (int o = 1; o <= 2; o *= 2)
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (!(b & o))
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t &lo = u[8 * b + i], &hi = u[8 * (b + o) + i];
                    const bool up = lane & o;
                    const uint32_t got = __shfl_xor_sync(kAll, up ? lo : hi, o);
                    lo = up ? got : lo;
                    hi = up ? hi : got;
                }
}

template <int K, int DP, bool kScored>
__device__ __forceinline__ void softmax_role(const Params& P, Shared& sh) {
    using KT = KindOf<K>;
    using T = typename KT::T;
    const AttendArgs& A = P.a;
    const int stream = threadIdx.x >> 7, r = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(r & ~31) << 16;
    const uint32_t s_col = sh.tmem + lanes + stream * kTile;
    const uint32_t o_col = sh.tmem + lanes + 256 + stream * DP;
    const uint32_t s_full = smem_u32(&sh.s_full[stream]), p_ready = smem_u32(&sh.p_ready[stream]),
                   pv_done = smem_u32(&sh.pv_done[stream]);
    const int32_t D = A.pool.dim;
    const bool tree = A.chunk.parents != nullptr;
    const Limit limit{&sh.gave_up, P.polls};
    const int32_t tl = r / P.G, g = r - tl * P.G;
    uint32_t steps = 0;   // of this stream, over all items
    uint32_t tiles = 0;   // of the CTA, before this item
    const Scoring scoring(A);  // kScored

    Items walk(P, sh);
    Item it;
#pragma unroll 1
    while (walk.next(it)) {
        Row row = row_of<kScored>(P, it, walk, stream, tl, g);
        float m = -INFINITY, l = 0.f;
        const bool busy = __any_sync(kAll, row.real);
        bool unset = busy;  // some row has no reference yet
#pragma unroll 1
        for (int32_t j = 0; j < it.n; ++j, ++steps) {
            // what needs no scores, before them
            const int32_t k0 = tile_at<kScored>(P, it, j) * kTile;
            const uint32_t ring = (tiles + j) % kNotes;
            const bool whole = __all_sync(kAll, (k0 + kTile <= row.limit && row.low <= k0) || !row.real);
            const bool mixed = mixed_tile(it, k0);
            if (!wait(s_full, steps & 1, limit)) return;
            tc_after();
            if (K == kE4m3 && j == 0) {
                float& unit = kScored && (scoring.capped || scoring.biased) ? row.raw : row.sl;
                unit = row_unit(unit, sh.q_down[walk.ring.i * sh.q_rows + stream * kTile + r]);
            }
            uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
            if (busy) {
                const uint32_t bad = sh.bad[0][ring];
                float sum;
                if (kScored && (scoring.capped || scoring.biased)) score_tile(scoring, tree, row, it, walk, s_col, k0);
                if (!whole || bad) {
                    seen_of(row, it, k0, bad, tree, seen);
                    hide_tile(s_col, seen);
                }
                bool first = K == kE4m3 || unset;
#pragma unroll 1
                for (;; first = true) {
                    if (first) {
                        const float mx = tile_max(s_col);
                        const bool move = row.real && ((mx - m) * row.sl > KT::kSlack || (m == -INFINITY && mx > m));
                        if (__any_sync(kAll, move)) {
                            const float old = m;
                            if (move) m = mx;
                            unset = __any_sync(kAll, row.real && m == -INFINITY);
                            const float f = !move || old == -INFINITY ? 1.f : exp2_fast((old - m) * row.sl);
                            l *= f;
                            if (__any_sync(kAll, move && old != -INFINITY)) {
                                if (!wait(pv_done, (steps - 1) & 1, limit)) return;
                                tc_after();
                                rescale<DP>(o_col, f);
                            }
                        }
                    }
                    if (quick_weights<K>(s_col, row.sl, KT::kShift - (m == -INFINITY ? 0.f : m * row.sl), row.real, first, sum)) break;
                }
                l += sum;
                tc_wait_st();
            }
            if (rarely(mixed)) {  // before p_ready: the tile cannot be released, nor its barrier move on, until then
                const uint32_t v = tiles + j;
                if (!wait(smem_u32(&sh.value[v % P.v_slots]), (v / P.v_slots) & 1, limit)) return;
            }
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_ready);
            if (rarely(mixed)) {
                // rows that see a non-finite value, which the product met as zero, get it added here
                const uint32_t none[4] = {0, 0, 0, 0};
                uint32_t odd[4], any = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) any |= odd[i] = sh.odd[ring][i];
                if (rarely(any && busy)) {
                    if (!wait(pv_done, steps & 1, limit)) return;
                    tc_after();
                    add_odd<K, DP>(A, it, o_col, k0, row.real ? odd : none, seen);
                    tc_wait_st();
                    tc_before();
                }
            }
        }
        tiles += it.n;

        // the item's end
        if (!wait(pv_done, (steps - 1) & 1, limit)) return;
        tc_after();
        const float ref = m == -INFINITY ? -INFINITY : m * row.sl - KT::kShift;
        const bool alone = it.begins && it.finishes;
        const int32_t row_at = it.row0 + row.token;
        const float vs = A.pool.v_scale ? A.pool.v_scale[it.h] : 1.f;
        const float inv = l == 0.f ? 0.f : vs / l;
        const int32_t head = it.h * P.G + g;
        // a row that carries NaN or infinity in its sum stays so: inv is then NaN or zero
        const size_t prow = (size_t)(2 * blockIdx.x + (it.begins ? 1 : 0)) * P.part_rows + stream * kTile + r;
        if (busy) {
            // A lane has a row; four lanes trade, so that they write 128 bytes of one row and then of the next.
            const int64_t at = alone ? ((int64_t)row_at * A.q_heads + head) * D : (int64_t)prow * DP;
            const uint32_t real = __ballot_sync(kAll, row.real) >> (lane & ~3);
            const int part = (lane & 3) * 8;
            const int step = alone ? 64 : 32;  // columns of 128 bytes
#pragma unroll 1
            for (int c = 0; c < D; c += step) {
                uint32_t u[32];
                tc_ld32(o_col + c, u);
                if (alone) {
                    uint32_t o[32];
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        u[i] = from_float2<T>(__uint_as_float(u[2 * i]) * inv, __uint_as_float(u[2 * i + 1]) * inv);
                    tc_ld32(o_col + c + 32, o);  // past D: columns that are not written
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        u[16 + i] = from_float2<T>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                }
                tc_wait_ld();
                trade(u, lane);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int64_t to = __shfl_sync(kAll, at, (lane & ~3) + b);
                    const uint32_t* v = u + 8 * b;
                    if (!(real >> b & 1u)) continue;
                    if (!alone) {
                        if (c + part < D)
                            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(P.part_o + to + c + part), SV_W8(v, 0)
                                         : "memory");
                        continue;
                    }
                    const int d = c + 2 * part;
                    T* out = (T*)A.out + to + d;
                    if (P.wide && d < D) {
                        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out), SV_W8(v, 0) : "memory");
                    } else {
                        if (d < D) *reinterpret_cast<uint4*>(out) = make_uint4(v[0], v[1], v[2], v[3]);
                        if (d + 8 < D) *reinterpret_cast<uint4*>(out + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
            if (row.real) {
                if (!alone) P.part_ml[prow] = make_float2(ref, l);
                else if (A.lse)
                    A.lse[(int64_t)row_at * A.q_heads + head] = l == 0.f ? -INFINITY : ref * kLn2 + logf(l);
            }
        }
        tc_before();
    }
}

// A stream's products, by one thread: S = Q K^T of its next tile follows O += P V of this one, whose P lies where that
// S will. The streams take turns, each turn both products: left to themselves they fall into step, both at their
// products and then both at their exponentials (measured: 4200 cycles a tile of 256 rows, 3050 in turns).
template <int K, int NH, bool kScored>
__device__ __forceinline__ void product_role(const Params& P, Shared& sh, uint32_t q_smem, uint32_t k_smem, uint32_t v_smem,
                                             const uint32_t st) {
    constexpr bool k8 = K == kE4m3;
    constexpr int parts = k8 ? 2 : 1, slot_bytes = NH * kHalf, steps_max = k8 ? 4 : 4 * NH;
    constexpr uint32_t fmt = K == kBf16 ? 1u : 0u;
    const int32_t D = P.a.pool.dim;
    const int32_t depth = (D + KindOf<K>::kStep - 1) / KindOf<K>::kStep;
    // float accumulators, 128 rows; scores are 128 columns wide, outputs D rounded up to 16 with the value
    // operand's rows along the depth
    const uint32_t base = 1u << 4 | fmt << 7 | fmt << 10 | (uint32_t)(kTile >> 4) << 24;
    const uint32_t id_s = base | (uint32_t)(kTile >> 3) << 17;
    const uint32_t id_o = base | 1u << 16 | (uint32_t)((D + 15) / 16 * 2) << 17;
    constexpr uint32_t q_bytes = (k8 ? 2 : NH) * kHalf;
    constexpr uint32_t dp = NH == 1 && !k8 ? 64 : 128;
    const uint32_t tmem = __shfl_sync(kAll, sh.tmem, 0);
    const uint32_t s_at = tmem + st * kTile, o_at = tmem + 256 + st * dp;
    const uint32_t k_full = smem_u32(sh.k_full), k_empty = smem_u32(sh.k_empty), v_empty = smem_u32(sh.v_empty),
                   value = smem_u32(sh.value), s_full = smem_u32(&sh.s_full[st]), p_ready = smem_u32(&sh.p_ready[st]),
                   pv_done = smem_u32(&sh.pv_done[st]), q_empty = smem_u32(sh.q_empty), q_full = smem_u32(sh.q_full);
    const bool leader = elect();
    const Limit limit{&sh.gave_up, P.polls};
    const uint32_t turn[2] = {smem_u32(&sh.turn[st]), smem_u32(&sh.turn[st ^ 1])};
    uint32_t p_parity = 0, turns = 0;
    Ring kr, vr, qr;
    Items walk(P, sh);
    Item it;
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(it)) {
        if (!(ok = wait(q_full + 8 * qr.i, qr.parity, limit))) break;
        tc_after();
        // the same in every lane; taken from one, so that the operands below live in uniform registers
        const int32_t n = __shfl_sync(kAll, it.n, 0);
        const uint32_t q = operand(q_smem + qr.i * P.q_bytes + st * q_bytes, 16), q_done = q_empty + 8 * qr.i;
#pragma unroll 1
        for (int32_t t = -1; t < n; ++t) {  // outputs of tile t, scores of the next
            const bool more = t + 1 < n;
            if (t >= 0 && !(ok = wait(value + 8 * vr.i, vr.parity, limit))) break;
            if (more && !(ok = wait(k_full + 8 * kr.i, kr.parity, limit))) break;
            if (t >= 0) {
                if (!(ok = wait(p_ready, p_parity, limit))) break;
                p_parity ^= 1u;
            }
            if (!(ok = wait(turn[0], turns, limit))) break;
            turns ^= 1u;
            tc_after();
            if (t >= 0) {
                const uint32_t b = operand(v_smem + vr.i * slot_bytes, kHalf);
                const uint32_t add = t > 0;
                int32_t lo, hi;
                steps_of<K>(it, tile_at<kScored>(P, it, t) * kTile, lo, hi);
                if (leader) {
#pragma unroll
                    for (int i = 0; i < kTile / KindOf<K>::kStep; ++i)
                        if (i >= lo && i < hi)
#pragma unroll
                        for (int part = 0; part < parts; ++part)
                            mma_ts<k8>(o_at, s_at + (k8 ? part * 8 + i * 16 : i * 8), b + (i * KindOf<K>::kStep * 128 >> 4), id_o,
                                       i > lo || part > 0 ? 1u : add);
                    if (!more) bar_arrive(turn[1]);
                    tc_commit(pv_done);
                    tc_commit(v_empty + 8 * vr.i);
                }
                __syncwarp();
                vr.step(P.v_slots);
            }
            if (more) {
                const uint32_t k = operand(k_smem + kr.i * slot_bytes, 16);
                if (leader) {
#pragma unroll
                    for (int part = 0; part < parts; ++part)
#pragma unroll
                        for (int i = 0; i < steps_max; ++i) {
                            const uint32_t off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
                            if (i < depth) mma_ss<k8>(s_at, q + (part * kHalf >> 4) + off, k + off, id_s, part + i > 0);
                        }
                    bar_arrive(turn[1]);
                    tc_commit(s_full);
                    tc_commit(k_empty + 8 * kr.i);
                    if (t + 2 == n) tc_commit(q_done);
                }
                __syncwarp();
                kr.step(P.k_slots);
            }
        }
        qr.step(P.q_bufs);
    }
    // products under way end before the tensor memory is given back
    if (leader) tc_commit(smem_u32(&sh.drain));
    __syncwarp();
    drain(smem_u32(&sh.drain), 0);
}

template <int K, int DP, bool kScored>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
             const __grid_constant__ CUtensorMap qm) {
    constexpr int NH = K == kE4m3 ? 1 : DP / 64;
    extern __shared__ __align__(1024) char raw[];
    const uint32_t q_smem = smem_u32(raw), k_smem = q_smem + P.q_bufs * P.q_bytes, v_smem = k_smem + P.k_slots * NH * kHalf;
    char* behind = raw + (v_smem - q_smem) + P.v_slots * NH * kHalf;
    Shared& sh = *reinterpret_cast<Shared*>(behind);
    if (q_smem & 1023u) {  // the tiles' swizzle counts on it
        if (threadIdx.x == 0) report(P.a.status, 1u << SV_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, w = tid >> 5;
    if (tid == 0) {
        init_common(sh, 2, kReaders + (K == kE4m3 ? kSplitters - 1 : 0), K == kE4m3 ? kSplitters : 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_u32(&sh.s_full[i]), 1);
            bar_init(smem_u32(&sh.p_ready[i]), 4);
            bar_init(smem_u32(&sh.pv_done[i]), 1);
            bar_init(smem_u32(&sh.turn[i]), 1);
        }
        sh.q_rows = 2 * kTile;
        sh.tree = reinterpret_cast<Tree*>(behind + (sizeof(Shared) + 15) / 16 * 16);
        sh.q_down = reinterpret_cast<float*>(sh.tree + (P.a.chunk.parents ? kItems : 0));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        bar_arrive(smem_u32(&sh.turn[0]));
    }
    if (w == 8 && (tid & 31) == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&km));
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vm));
        if (K != kE4m3) asm volatile("prefetch.tensormap [%0];" ::"l"(&qm));
    }
    begin<kThreads, 512, kScored>(P, sh, w == 9);
    // 128 registers a thread at launch: 192 + 192 + 64 + 64 for the four warpgroups
    if (w < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        softmax_role<K, DP, kScored>(P, sh);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (w == 8 || w == 10) load_role<kScored>(P, sh, k_smem, v_smem, &km, &vm, w == 10, w == 10);
        else if (w == 9 || w == 13) product_role<K, NH, kScored>(P, sh, q_smem, k_smem, v_smem, w == 13);
        else if (w == 11) value_role<K, kScored>(P, sh, v_smem);
        else if (w == 12) item_role<K, kSplitters, kScored>(P, sh, q_smem, &qm);
        else if (K == kE4m3 && w >= 14) query_role(P, sh, q_smem, w - 14, kSplitters);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (w == 9) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem));
    }
    if (tid == 0 && sh.gave_up) report(P.a.status, 1u << SV_ERR_TIMEOUT);
}

template <int K, int DP, bool kScored>
cudaError_t launch(Params P, int n, cudaStream_t st) {
    constexpr int NH = K == kE4m3 ? 1 : DP / 64;
    const AttendArgs& A = P.a;
    P.tokens = kTile / P.G;
    P.block = 2 * P.tokens;
    P.q_box = min(P.tokens, A.chunk.max_gamma + 1);
    P.q_part = kHalf;
    // measured on prompts of 700 to 2048 tokens: 235 us, with 1, 2, 4 and 5 272, 238, 238
    // and 240. With an e4m3 cache the queries' parts take longer: 3, 6 and 10 make 476, 356 and 387 us of those prompts,
    // and 54, 58 and 66 of 16 trees of 32 tokens, whose items have few rows each: 6 serves the prompts at the trees' cost.
    P.lead = K == kE4m3 ? 6 : 3;
    P.halves = NH;
    P.q_tile = (K == kE4m3 ? 2 : NH) * kHalf;
    P.q_bytes = 2 * P.q_tile;
    P.q_bufs = K == kE4m3 ? 2 : 1;  // the next item's are split into parts, 256 rows by three warps, under this one's tiles
    const int own = (int)(sizeof(Shared) + 15) / 16 * 16 + (A.chunk.parents ? kItems * (int)sizeof(Tree) : 0) +
                    (K == kE4m3 ? kItems * 2 * kTile * 4 : 0);
    const int slots = min(2 * kMaxSlots, (kSmem - own - P.q_bufs * P.q_bytes) / (NH * kHalf));
    P.k_slots = slots / 2;
    P.v_slots = slots - P.k_slots;
    CUtensorMap km, vm, qm;
    if (K != kE4m3 && !encode_queries(&qm, A, K, P.G, P.q_box)) return cudaErrorInvalidValue;
    if (!encode_pool(&km, A.pool, A.pool.k, KindOf<K>::kBytes, K, P.box) ||
        !encode_pool(&vm, A.pool, A.pool.v, KindOf<K>::kBytes, K, P.box))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> allowed{0};
    void* args[] = {&P, &km, &vm, &qm};
    return launch_early((const void*)k_attend<K, DP, kScored>, &allowed, dim3(n), kThreads, P.q_bufs * P.q_bytes + slots * NH * kHalf + own, st, args);
}

}  // namespace wide

template <bool kScored>
cudaError_t launch_wide(const Params& P, int kind, int dp, int n, cudaStream_t st) {
    if (kind == kE4m3) return wide::launch<kE4m3, 128, kScored>(P, n, st);
    if (kind == kFp16) return dp == 128 ? wide::launch<kFp16, 128, kScored>(P, n, st) : wide::launch<kFp16, 64, kScored>(P, n, st);
    return dp == 128 ? wide::launch<kBf16, 128, kScored>(P, n, st) : wide::launch<kBf16, 64, kScored>(P, n, st);
}

}  // namespace cache
}  // namespace sv
