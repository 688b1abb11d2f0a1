// spec_cache_attend (include/speccache.h): attention of a chunk of new tokens over the paged cache.
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
// sv_cache_attend_few.cu, which turns the products around.
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
#include "sv_cache_attend.cuh"

#include <algorithm>

namespace sv {
namespace cache {
namespace {

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
};

// tl: the row's token within its tile.
__device__ __forceinline__ Row row_of(const Params& P, const Item& it, const Items& items, int stream, int32_t tl) {
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

template <int K, int DP>
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

    Items walk(P, sh);
    Item it;
#pragma unroll 1
    while (walk.next(it)) {
        Row row = row_of(P, it, walk, stream, tl);
        float m = -INFINITY, l = 0.f;
        const bool busy = __any_sync(kAll, row.real);
        bool unset = busy;  // some row has no reference yet
#pragma unroll 1
        for (int32_t j = 0; j < it.n; ++j, ++steps) {
            // what needs no scores, before them
            const int32_t k0 = (it.tile + j) * kTile;
            const uint32_t ring = (tiles + j) % kNotes;
            const bool whole = __all_sync(kAll, (k0 + kTile <= row.limit && row.low <= k0) || !row.real);
            const bool mixed = mixed_tile(it, k0);
            if (!wait(s_full, steps & 1, limit)) return;
            tc_after();
            if (K == kE4m3 && j == 0) row.sl = row_unit(row.sl, sh.q_down[walk.ring.i * sh.q_rows + stream * kTile + r]);
            uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
            if (busy) {
                const uint32_t bad = sh.bad[0][ring];
                if (!whole || bad) {
                    seen_of(row, it, k0, bad, tree, seen);
                    hide_tile(s_col, seen);
                }
                float sum;
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
template <int K, int NH>
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
                steps_of<K>(it, (it.tile + t) * kTile, lo, hi);
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

template <int K, int DP>
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
    begin<kThreads, 512>(P, sh, w == 9);
    // 128 registers a thread at launch: 192 + 192 + 64 + 64 for the four warpgroups
    if (w < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        softmax_role<K, DP>(P, sh);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (w == 8 || w == 10) load_role(P, sh, k_smem, v_smem, &km, &vm, w == 10, w == 10);
        else if (w == 9 || w == 13) product_role<K, NH>(P, sh, q_smem, k_smem, v_smem, w == 13);
        else if (w == 11) value_role<K>(P, sh, v_smem);
        else if (w == 12) item_role<K, kSplitters>(P, sh, q_smem, &qm);
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

// Items that several CTAs worked on: one warp a row, the parts in their order. Bound by the latency of a few dependent
// reads from L2, so the first parts are read along with the references, and there are warps for every row at once.
constexpr int kMergeThreads = 256;
template <typename T, int DP>
__global__ void __launch_bounds__(kMergeThreads) k_attend_merge(const __grid_constant__ Params P) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t c = blockIdx.x + 1;
    const Record rec = P.records[c];
    const int32_t i = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);  // the item's row
    if (!rec.parts || i >= rec.tokens * P.G) return;
    const int lane = threadIdx.x & 31;
    constexpr int kPer = DP / 32, kAtOnce = 4;
    const bool in = lane * kPer < P.a.pool.dim;
    const int32_t t = i / P.G, g = i - t * P.G;
    const int32_t r = t < rec.split ? i : kTile + i - rec.split * P.G;
    // the first part is the last item of CTA c - 1, the others the first items of c, c + 1, ...
    auto slot = [&](int32_t part) { return (size_t)(part ? 2 * (c + part - 1) : 2 * (c - 1) + 1) * P.part_rows + r; };
    float x[kAtOnce][kPer];
    auto read = [&](int32_t p0) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[k][e] = 0.f;
            if (p0 + k >= rec.parts || !in) continue;
            const float* o = P.part_o + slot(p0 + k) * DP + lane * kPer;
            if (kPer == 4) *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(o);
            else *reinterpret_cast<float2*>(x[k]) = *reinterpret_cast<const float2*>(o);
        }
    };
    read(0);
    float2 ml = lane < rec.parts ? P.part_ml[slot(lane)] : make_float2(-INFINITY, 0.f);
    float top = ml.x;
#pragma unroll 1
    for (int32_t p = 32 + lane; p < rec.parts; p += 32) top = fmaxf(top, P.part_ml[slot(p)].x);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f, acc[kPer] = {}, wt = 0.f;
#pragma unroll 1
    for (int32_t p = 0; p < rec.parts; p += kAtOnce) {
        if (p % 32 == 0) {
            if (p > 0) ml = p + lane < rec.parts ? P.part_ml[slot(p + lane)] : make_float2(-INFINITY, 0.f);
            wt = p + lane >= rec.parts ? 0.f : top == -INFINITY ? 1.f : exp2_fast(ml.x - base);
            float pl = ml.y * wt;
            for (int o = 16; o; o >>= 1) pl += __shfl_xor_sync(kAll, pl, o);
            l += pl;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float f = __shfl_sync(kAll, wt, (p + k) & 31);
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] = p + k < rec.parts ? fmaf(f, x[k][e], acc[e]) : acc[e];
        }
        if (p + kAtOnce < rec.parts) read(p + kAtOnce);
    }
    const float vs = P.a.pool.v_scale ? P.a.pool.v_scale[rec.head] : 1.f;
    const float inv = l == 0.f ? 0.f : vs / l;
    const int64_t at = (int64_t)(rec.row0 + t) * P.a.q_heads + rec.head * P.G + g;
    if (in) {
        T* out = (T*)P.a.out + at * P.a.pool.dim + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<uint32_t*>(out + e) = from_float2<T>(acc[e] * inv, acc[e + 1] * inv);
    }
    if (P.a.lse && lane == 0) P.a.lse[at] = l == 0.f ? -INFINITY : top * kLn2 + logf(l);
}

template <int K, int DP>
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
    return launch_early((const void*)k_attend<K, DP>, &allowed, dim3(n), kThreads, P.q_bufs * P.q_bytes + slots * NH * kHalf + own, st, args);
}

template <typename T>
cudaError_t merge(Params& P, cudaStream_t st, bool narrow) {
    static std::atomic<unsigned long long> allowed{~0ull};  // it asks for no shared memory
    void* args[] = {&P};
    const void* k = narrow ? (const void*)k_attend_merge<T, 64> : (const void*)k_attend_merge<T, 128>;
    const int warps = kMergeThreads / 32, rows = (int)std::min((int64_t)(P.a.chunk.max_gamma + 1) * P.G, (int64_t)P.part_rows);
    return launch_early(k, &allowed, dim3(P.ctas - 1, (rows + warps - 1) / warps), kMergeThreads, 0, st, args);
}

}  // namespace

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// One layer's keys or values as (dim, token of the page, head, page), copied in boxes of 128 bytes by `box` tokens.
bool encode_pool(CUtensorMap* m, const Pool& p, char* base, int esize, int kind, int box) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.dim, (cuuint64_t)p.page_size, (cuuint64_t)p.heads, (cuuint64_t)p.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.s_token * esize, (cuuint64_t)p.s_head * esize,
                                   (cuuint64_t)p.s_page * esize};
    const cuuint32_t boxes[4] = {(cuuint32_t)(128 / esize), (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = kind == kE4m3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : kind == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encoder()(m, type, 4, base, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries as (dim, head, row), copied in boxes of 128 bytes by the heads of a group by q_box rows.
bool encode_queries(CUtensorMap* m, const AttendArgs& A, int kind, int G, int q_box) {
    const cuuint64_t dims[3] = {(cuuint64_t)A.pool.dim, (cuuint64_t)A.q_heads, (cuuint64_t)A.chunk.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)A.pool.dim * 2, (cuuint64_t)A.q_stride * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)G, (cuuint32_t)q_box}, ones[3] = {1, 1, 1};
    return encoder()(m, kind == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(A.q), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_early(const void* kernel, std::atomic<unsigned long long>* allowed, dim3 grid, int threads, int smem, cudaStream_t st,
                         void** args) {
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // the devices on which the kernel may use all shared memory: setting that twice does no harm
    if (dev >= 64 || !(allowed->load() >> dev & 1u)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed->fetch_or(1ull << dev);
    }
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

namespace {
// Wide partials' row length in floats.
int part_dim(int dim, int kind) { return kind == kE4m3 || dim > 64 ? 128 : 64; }
constexpr size_t kParts = (size_t)2 * (kMaxCtas / 2) * 256;  // rows of all partials: half as many CTAs as in sv_cache_attend_few.cu
static_assert(kParts >= (size_t)2 * kMaxCtas * kFewRows, "the other launch's partials fit");
}  // namespace

size_t attend_workspace(int dim, int cache_dtype) {
    const int dp = part_dim(dim, cache_dtype == SV_E4M3 ? kE4m3 : kBf16);
    return kParts * (dp * sizeof(float) + sizeof(float2)) + kMaxCtas * sizeof(Record);
}

cudaError_t launch_attend(const AttendArgs& A, int dtype, int cache_dtype, cudaStream_t st) {
    const int kind = cache_dtype == SV_E4M3 ? kE4m3 : dtype == SV_F16 ? kFp16 : kBf16;
    const int dp = part_dim(A.pool.dim, kind);
    Params P{};
    P.a = A;
    P.polls = A.spin_limit ? A.spin_limit : kPolls;
    P.G = A.q_heads / A.pool.heads;
    P.box = kTile;
    while (A.pool.page_size % P.box) P.box /= 2;
    P.boxes = kTile / P.box;
    P.tile_pages = kTile / A.pool.page_size;
    P.tile_rest = kTile % A.pool.page_size;
    P.wide = A.pool.dim % 16 == 0 && (uintptr_t)A.out % 32 == 0;
    char* ws = (char*)A.workspace;
    P.part_o = (float*)ws;
    P.part_ml = (float2*)(ws + kParts * dp * sizeof(float));
    P.records = (Record*)(P.part_ml + kParts);
    int dev, sms;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (!encoder()) return cudaErrorNotSupported;
    P.ctas = min(sms, kMaxCtas / 2);
    P.part_rows = 2 * kTile;
    const int n = P.ctas;
    const int64_t rows = (int64_t)(A.chunk.max_gamma + 1) * P.G;
    if (rows <= kFewRows) e = launch_few(P, kind, (int)rows, n, st);
    else if (kind == kE4m3) e = launch<kE4m3, 128>(P, n, st);
    else if (kind == kFp16) e = dp == 128 ? launch<kFp16, 128>(P, n, st) : launch<kFp16, 64>(P, n, st);
    else e = dp == 128 ? launch<kBf16, 128>(P, n, st) : launch<kBf16, 64>(P, n, st);
    if (e != cudaSuccess) return e;
    return kind == kFp16 ? merge<__half>(P, st, dp == 64) : merge<__nv_bfloat16>(P, st, dp == 64);
}

}  // namespace cache
}  // namespace sv
