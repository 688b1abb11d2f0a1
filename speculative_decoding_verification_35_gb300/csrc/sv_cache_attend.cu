// spec_cache_attend (include/speccache.h): attention of a chunk of new tokens over the paged cache.
//
// Mathematics. A row (token, query head) with scores z_s = scale q . k_s keeps a reference m and, tile after
// tile of 128 slots, l = sum 2^(z_s log2 e - m) and O = sum 2^(z_s log2 e - m) v_s; out = O / l. When a tile's
// maximum exceeds m by more than a threshold, m moves there and l and O are scaled by 2^(old - new). Partial
// (m, l, O) of disjoint slots merge the same way, so a row's slots can be shared out.
//
// Shape. The query heads of a group share their key head, so a tile of 128 rows packs 128 / G tokens of G heads
// and both products run on the tensor cores as 128 x 128 x D (S = Q K^T, O += P V), operands in shared memory,
// S, P and O in tensor memory. With few rows most of a tile is padding, which costs nothing that matters: a
// 128-slot tile of 16-bit keys and values takes an SM about 2800 cycles to bring in at the HBM rate and about
// 1000 to multiply.
//
// Streams. A CTA (one per SM) has two softmax warpgroups, each with its own S, P and O, so that the tensor cores
// work for one while the other is at its exponentials. A work item with up to 128 rows gives the streams its
// even and odd tiles and merges the two at its end; one with up to 256 rows gives each stream 128 rows and runs
// every tile for both, which reads it from shared memory twice and from the cache once.
//
// Split. The items' tiles are numbered in one line (sequence, row block, key head, tile), and CTA c of n takes
// those from c W / n to (c + 1) W / n, whatever items they belong to: every SM gets the same number of
// tiles with one long sequence or hundreds of short ones, and a CTA leaves at most two items unfinished. Their
// partials go to the workspace, and a second small launch merges them in a fixed order. Lengths are read
// on the device, so the host needs to know none of them.
#include <cuda.h>

#include "sv_cache.cuh"

namespace sv {
namespace cache {
namespace {

constexpr int kThreads = 384;   // two softmax warpgroups, then warps for loads, products and value tiles
constexpr int kTile = 128;      // slots of a tile, and rows of a query tile
constexpr int kMaxSlots = 12;   // key or value tiles in flight
constexpr int kBadRing = 16;
constexpr int kMaxCtas = 160;
constexpr int kHalf = kTile * 128;  // bytes of 128 rows of 128 bytes, the unit of an operand in shared memory
constexpr int kSmem = 227 * 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------------------------------------------
// element kinds
// ---------------------------------------------------------------------------------------------------------
// kShift: weights are held as 2^kShift w, so that those far below the largest keep their precision in a narrow
// type; kSlack: how far (log2) a weight may exceed the reference before the reference moves. 2^(kShift + kSlack)
// is within the type's range.
// kE4m3: the cache is 8 bits wide and the products are too. A bfloat16 query has 8 significant bits and an
// e4m3 value 4, so q 2^k = hi + lo exactly, but for elements under 2^-11 of the row's largest (k brings it to
// [128, 256)); a weight is hi + lo to 2^-9 of itself. Each product then runs twice, at twice the 16-bit rate,
// and no key or value is converted.
enum Kind { kBf16 = 0, kFp16 = 1, kE4m3 = 2 };
template <int K>
struct KindOf;
template <>
struct KindOf<kBf16> {
    using T = __nv_bfloat16;
    static constexpr float kShift = 0.f, kSlack = 8.f;
    static constexpr int kBytes = 2, kStep = 16;  // of an element; elements a product step takes along its depth
};
template <>
struct KindOf<kFp16> {
    using T = __half;
    static constexpr float kShift = 7.f, kSlack = 8.f;
    static constexpr int kBytes = 2, kStep = 16;
};
template <>
struct KindOf<kE4m3> {
    using T = __nv_bfloat16;
    static constexpr float kShift = 8.f, kSlack = 0.75f;
    static constexpr int kBytes = 1, kStep = 32;
};

// ---------------------------------------------------------------------------------------------------------
// parameters and workspace
// ---------------------------------------------------------------------------------------------------------
struct Record {  // an item that more than one CTA worked on, written by the second of them
    int32_t parts;  // CTAs, 0: none
    int32_t row0;   // its first row
    int32_t tokens, head, two;
    int32_t pad[3];
};

struct Params {
    AttendArgs a;
    int32_t G, tokens;  // query heads per key head; tokens of a query tile, kTile / G
    int32_t q_tiles;    // query tiles that shared memory has room for: 1 or 2
    int32_t slots;      // key or value tiles that fit
    int32_t box;        // slots of one copy, a divisor of the page size and of kTile
    float* part_o;      // [2 n][256][DP]
    float2* part_ml;    // [2 n][256]
    Record* records;    // [n]
};

__host__ __device__ constexpr size_t part_rows() { return (size_t)2 * kMaxCtas * 2 * kTile; }

// ---------------------------------------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// A whole warp waits; false once the CTA has given up (after two seconds without the phase).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
    bool ok = bar_try(bar, parity);
    if (!__all_sync(kAll, ok)) {
        unsigned long long t0 = 0;
        for (uint32_t i = 1; !ok; ++i) {
            ok = bar_try(bar, parity);
            if (!ok && (i & 63u) == 0) {
                const unsigned long long t = now_ns();
                if (!t0) t0 = t;
                if (t - t0 > 2000000000ull) *gave_up = 1;
                if (*gave_up) break;
            }
        }
        ok = __all_sync(kAll, ok);
    }
    return ok;
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int d, int token, int head, int page,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(d), "r"(token), "r"(head), "r"(page), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#define SV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define SV_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
__device__ __forceinline__ void tc_ld32(uint32_t col, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24)
        : "r"(col));
}
__device__ __forceinline__ void tc_st32(uint32_t col, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(col),
        SV_W8(r, 0), SV_W8(r, 8), SV_W8(r, 16), SV_W8(r, 24)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t col, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(col),
        SV_W8(r, 0), SV_W8(r, 8)
        : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t col, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(col), SV_W8(r, 0)
                 : "memory");
}
// Shared-memory operand of 128-byte rows under the 128-byte swizzle; eight rows are 1024 bytes apart. far: bytes
// between column halves of an operand whose rows run along its depth.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t far) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(far >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
template <bool k8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    if (k8)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
    else
        asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(
                         d),
                     "l"(a), "l"(b), "r"(idesc), "r"(add)
                     : "memory");
}
template <bool k8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    if (k8)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t u) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ---------------------------------------------------------------------------------------------------------
// work items
// ---------------------------------------------------------------------------------------------------------
struct Item {
    int32_t b, h, row0;       // sequence, key head, the sequence's first row
    int32_t t0, nt;           // its chunk tokens
    int32_t past;
    int32_t lo, end;          // the slots [lo, end) that some row of it sees
    int32_t tile, n;          // the CTA's tiles: the first (absolute), how many
    bool two;                 // 129 to 256 rows: a query tile per stream
    bool begins, finishes;    // its first and last tiles are among the CTA's
};

__device__ __forceinline__ void span(const Params& P, int32_t T, int32_t past, int32_t p, Item& it, int32_t& first,
                                     int32_t& count) {
    const int32_t per = 2 * P.tokens;
    it.t0 = p * per;
    it.nt = min(per, T - it.t0);
    it.two = it.nt > P.tokens;
    it.past = past;
    it.end = past + it.t0 + it.nt;
    it.lo = 0;
    if (P.a.window > 0) {  // the least position of its rows: the root's in a tree
        const int32_t t = P.a.chunk.parents ? 0 : it.t0;
        it.lo = max(0, past + t - P.a.window + 1);
    }
    first = it.lo / kTile;
    count = (it.end - 1) / kTile - first + 1;
}

// Whether every parent of the tree lies before its node, by one thread.
__device__ __forceinline__ bool tree_ok(const Chunk& c, int32_t b, int32_t T) {
    const int32_t* par = c.parents + c.offs[b];
    bool ok = true;
    for (int j = 1; j < T; ++j) ok &= (uint32_t)par[j - 1] < (uint32_t)j;
    return ok;
}

__device__ __forceinline__ Seq checked_seq(const Params& P, int32_t b) {
    Seq s = seq_of(P.a.chunk, capacity_of(P.a.pool), b);
    if (!s.err && P.a.chunk.parents && !tree_ok(P.a.chunk, b, s.T)) s.err = 1u << SV_ERR_BAD_OFFSETS;
    return s;
}

// Tiles of a sequence over all its row blocks and key heads.
__device__ __forceinline__ long long units_of(const Params& P, const Seq& s) {
    if (s.err) return 0;
    const int32_t per = 2 * P.tokens;
    long long u = 0;
    for (int32_t p = 0; p * per < s.T; ++p) {
        Item it;
        int32_t first, count;
        span(P, s.T, s.past, p, it, first, count);
        u += count;
    }
    return u * P.a.pool.heads;
}

struct Start {  // where a CTA begins
    int32_t b, p, h, j;
    long long left;
};

// The items of a CTA, one after the other. Every warp walks by itself.
struct Walk {
    const Params& P;
    int32_t b, p, h, j, T, past, row0;
    long long left;
    bool fresh;
    __device__ Walk(const Params& P_, const Start& s) : P(P_), b(s.b), p(s.p), h(s.h), j(s.j), left(s.left), fresh(true) {}
    __device__ bool next(Item& it) {
        if (left <= 0) return false;
        if (fresh) {
            for (; b < P.a.chunk.B; ++b) {
                const Seq s = checked_seq(P, b);
                if (!s.err) {
                    T = s.T;
                    past = s.past;
                    row0 = s.row0;
                    break;
                }
            }
            if (b >= P.a.chunk.B) return false;
            fresh = false;
        }
        int32_t first, count;
        span(P, T, past, p, it, first, count);
        it.b = b;
        it.h = h;
        it.row0 = row0;
        it.tile = first + j;
        it.begins = j == 0;
        it.n = (int32_t)min((long long)(count - j), left);
        it.finishes = j + it.n == count;
        left -= it.n;
        j = 0;
        if (++h == P.a.pool.heads) {
            h = 0;
            ++p;
            if (p * 2 * P.tokens >= T) {
                p = 0;
                ++b;
                fresh = true;
            }
        }
        return true;
    }
};

struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots], value[kMaxSlots];  // value: a value tile is in and clean
    uint64_t s_full[2], p_ready[2], pv_done[2];
    uint64_t q_full, q_empty, meet, part, drain;
    uint32_t tmem;
    int gave_up;
    Start start;
    long long scan[kThreads / 32 + 1];
    uint32_t bad[kBadRing];         // per tile: groups of 8 slots that lie on a bad page
    uint32_t odd[kBadRing][4];      // per value tile: slots with a non-finite value that was cleared
    float2 ml[2][kTile];
};

// Where the CTA begins, and the record of an item that its predecessor began. All threads.
__device__ __forceinline__ void plan(const Params& P, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int32_t B = P.a.chunk.B, c = (int32_t)blockIdx.x;
    long long mine = 0, sum = 0;
    for (int32_t b = tid; b < B; b += kThreads) {
        const long long u = units_of(P, checked_seq(P, b));
        if (b == tid) mine = u;
        sum += u;
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) sh.scan[w] = sum;
    if (tid == 0) {
        sh.start.left = 0;
        if (blockIdx.x > 0) P.records[c].parts = 0;
    }
    __syncthreads();
    long long W = 0;
    for (int i = 0; i < kThreads / 32; ++i) W += sh.scan[i];
    // with fewer tiles than CTAs the first W take one each, so that an item's CTAs follow one another
    const int32_t n = (int32_t)min((long long)gridDim.x, W);
    if (c >= n) return;  // the same for the whole CTA
    const long long u0 = W * c / n, u1 = W * (c + 1) / n;
    long long base = 0;
    for (int32_t b0 = 0; b0 < B && base <= u0; b0 += kThreads) {
        const int32_t b = b0 + tid;
        const long long u = b0 == 0 ? mine : b < B ? units_of(P, checked_seq(P, b)) : 0;
        long long incl = u;
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += x;
        }
        __syncthreads();
        if (lane == 31) sh.scan[w] = incl;
        __syncthreads();
        long long before = base, total = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < w) before += sh.scan[i];
            total += sh.scan[i];
        }
        const long long begin = before + incl - u;
        if (u > 0 && u0 >= begin && u0 < begin + u) {
            const Seq s = checked_seq(P, b);
            long long rest = u0 - begin;
            Item it;
            int32_t first, count, p = 0;
            for (;; ++p) {
                span(P, s.T, s.past, p, it, first, count);
                if (rest < (long long)count * P.a.pool.heads) break;
                rest -= (long long)count * P.a.pool.heads;
            }
            const int32_t h = (int32_t)(rest / count), j = (int32_t)(rest - (long long)h * count);
            sh.start.b = b;
            sh.start.p = p;
            sh.start.h = h;
            sh.start.j = j;
            sh.start.left = u1 - u0;
            if (j > 0) {
                // the item began at u0 - j; if the CTA before this one began it, this one records it
                const long long from = u0 - j, to = from + count;
                if (from >= W * (c - 1) / n) {
                    Record r{};
                    const long long last = (to * n - 1) / W;  // the CTA of its last tile
                    r.parts = (int32_t)(last - c) + 2;
                    r.row0 = s.row0 + it.t0;
                    r.tokens = it.nt;
                    r.head = h;
                    r.two = it.two;
                    P.records[c] = r;
                }
            }
        }
        base += total;
    }
}

// ---------------------------------------------------------------------------------------------------------
// the softmax warpgroups
// ---------------------------------------------------------------------------------------------------------
// A row of a query tile as its thread knows it.
struct Row {
    bool real;
    int32_t token, g;   // chunk token, head of the group
    int32_t low, limit; // slots low .. limit - 1 are seen, as far as they are not a tree's
    uint32_t above;     // a tree: the chunk tokens it sees
    float sl;           // score units to log2 of the weight
};

template <int K>
__device__ __forceinline__ void load_queries(const Params& P, const Item& it, int stream, int r, uint32_t q_smem, Row& row) {
    using T = typename KindOf<K>::T;
    const AttendArgs& A = P.a;
    const int32_t D = A.pool.dim;
    const int32_t tl = r / P.G;
    row.g = r - tl * P.G;
    row.token = it.t0 + tl + (it.two && stream ? P.tokens : 0);
    row.real = tl < P.tokens && row.token < it.t0 + it.nt;
    row.above = 0;
    int32_t depth = row.token;
    if (A.chunk.parents) {
        const int32_t* par = A.chunk.parents + (it.row0 - it.b);
        depth = -1;
        if (row.real)
            for (int32_t t = row.token;; t = par[t - 1]) {
                ++depth;
                if (A.window <= 0 || depth < A.window) row.above |= 1u << t;
                if (t == 0) break;
            }
    }
    const int32_t pos = it.past + depth;
    row.low = A.window > 0 ? max(0, pos - A.window + 1) : 0;
    row.limit = it.past + (A.chunk.parents ? 0 : row.token + 1);
    float sl = A.scale * (A.pool.k_scale ? A.pool.k_scale[it.h] : 1.f) * kLog2e;
    const bool flip = sl < 0.f;
    sl = fmaxf(fabsf(sl), 1e-30f);  // a scale of zero: all weights equal, and -inf stays -inf
    row.sl = sl;
    const T* q = (const T*)A.q + (int64_t)(it.row0 + row.token) * A.q_stride + (int64_t)(it.h * P.G + row.g) * D;
    // a query tile shared by both streams is loaded by both, every other 16 bytes each
    const uint32_t base = q_smem + (it.two && stream ? (K == kE4m3 ? 2 : (D > 64 ? 2 : 1)) * kHalf : 0) + r * 128;
    const int begin = it.two ? 0 : stream, by = it.two ? 1 : 2;
    if (K != kE4m3) {
        const int chunks = (D + 15) / 16 * 2;
        for (int c = begin; c < chunks; c += by) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (row.real && c * 8 < D) {
                u = *reinterpret_cast<const uint4*>(q + c * 8);
                if (flip) {
                    u.x ^= 0x80008000u;
                    u.y ^= 0x80008000u;
                    u.z ^= 0x80008000u;
                    u.w ^= 0x80008000u;
                }
            }
            const uint32_t at = base + (c >> 3) * kHalf + (((c & 7) ^ (r & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w)
                         : "memory");
        }
    } else {
        float top = 0.f;
        if (row.real)
            for (int c = 0; c < D / 8; ++c) {
                const uint4 u = *reinterpret_cast<const uint4*>(q + c * 8);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                for (int i = 0; i < 4; ++i) {
                    const float2 f = to_float2<T>(w[i]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
        int e = 0;
        if (top > 0.f && top < INFINITY) e = max(-120, min(120, 7 - ilogbf(top)));
        const float up = exp2f((float)e) * (flip ? -1.f : 1.f);
        row.sl = sl * exp2f((float)-e);
        const int chunks = (D + 31) / 32 * 2;
        for (int c = begin; c < chunks; c += by) {
            uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
            if (row.real && c * 16 < D) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint4 u = *reinterpret_cast<const uint4*>(q + c * 16 + half * 8);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 f = to_float2<T>(w[i]);
                        // an infinite query has no finite parts: its row is NaN, as its softmax is
                        f.x = isinf(f.x) ? NAN : f.x * up;
                        f.y = isinf(f.y) ? NAN : f.y * up;
                        const uint32_t a = e4m3x2(f.x, f.y);
                        const float2 g = from_e4m3x2(a);
                        const uint32_t b = e4m3x2(f.x - g.x, f.y - g.y);
                        hi[half * 2 + (i >> 1)] |= a << (16 * (i & 1));
                        lo[half * 2 + (i >> 1)] |= b << (16 * (i & 1));
                    }
                }
            }
            const uint32_t at = base + (((c & 7) ^ (r & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + kHalf), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]),
                         "r"(lo[3])
                         : "memory");
        }
    }
}

__device__ __forceinline__ uint32_t prefix32(int32_t n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

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

// Slots of the item that some of its rows see and others do not: only there can a value meet a weight of
// zero, and a NaN or infinity be carried into a row that does not see it.
__device__ __forceinline__ bool mixed_tile(const Params& P, const Item& it, int32_t k0) {
    const bool tree = P.a.chunk.parents != nullptr;
    if (it.nt == 1 && !tree) return false;
    if (k0 + kTile > it.past + (tree ? 0 : it.t0 + 1)) return true;
    return P.a.window > 0 && k0 < it.lo + it.nt + (tree ? it.t0 : 0);
}

template <int K, int DP>
__device__ __forceinline__ void softmax_role(const Params& P, Shared& sh, uint32_t q_smem) {
    using KT = KindOf<K>;
    using T = typename KT::T;
    const AttendArgs& A = P.a;
    const int stream = threadIdx.x >> 7, r = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(r & ~31) << 16;
    const uint32_t s_col = sh.tmem + lanes + stream * kTile;
    const uint32_t o_col[2] = {sh.tmem + lanes + 256, sh.tmem + lanes + 256 + DP};
    const uint32_t s_full = smem_u32(&sh.s_full[stream]), p_ready = smem_u32(&sh.p_ready[stream]),
                   pv_done = smem_u32(&sh.pv_done[stream]);
    const uint32_t q_full = smem_u32(&sh.q_full), q_empty = smem_u32(&sh.q_empty);
    const int32_t D = A.pool.dim;
    const bool tree = A.chunk.parents != nullptr;
    volatile int* gave_up = &sh.gave_up;
    uint32_t steps = 0;   // of this stream, over all items
    uint32_t tiles = 0;   // of the CTA, before this item
    uint32_t items = 0, merges = 0;

    Walk walk(P, sh.start);
    Item it, nx;
    Row row, nrow;
    bool more = walk.next(it);
    if (more) {
        load_queries<K>(P, it, stream, r, q_smem, row);
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(q_full);
    }
    while (more) {
        float m = -INFINITY, l = 0.f;
        const bool busy = __any_sync(kAll, row.real);
        const int32_t first = it.two ? 0 : stream, by = it.two ? 1 : 2;
        uint32_t done = 0;
        for (int32_t j = first; j < it.n; j += by, ++done, ++steps) {
            if (!wait(s_full, steps & 1, gave_up)) return;
            tc_after();
            const int32_t k0 = (it.tile + j) * kTile;
            const uint32_t ring = (tiles + j) % kBadRing;
            const uint32_t bad = sh.bad[ring];
            uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
            if (busy) {
                uint32_t s[128];
#pragma unroll
                for (int i = 0; i < 4; ++i) tc_ld32(s_col + 32 * i, s + 32 * i);
                tc_wait_ld();
                const bool whole = (k0 + kTile <= row.limit && row.low <= k0 && !bad) || !row.real;
                if (!__all_sync(kAll, whole)) {
                    seen_of(row, it, k0, bad, tree, seen);
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (!(seen[c >> 5] >> (c & 31) & 1u)) s[c] = 0xff800000u;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 128; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(s[c]));
                const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                const bool move = (mx - m) * row.sl > KT::kSlack || (m == -INFINITY && mx > m);
                const unsigned movers = __ballot_sync(kAll, move);
                if (movers) {
                    const float old = m;
                    if (move) m = mx;
                    const float f = old == -INFINITY ? 1.f : exp2_fast((old - m) * row.sl);
                    l *= f;
                    if (done > 0 && __any_sync(kAll, move && old != -INFINITY)) {
                        if (!wait(pv_done, (steps - 1) & 1, gave_up)) return;
                        tc_after();
                        for (int c = 0; c < DP; c += 32) {
                            uint32_t o[32];
                            tc_ld32(o_col[stream] + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * (move ? f : 1.f));
                            tc_st32(o_col[stream] + c, o);
                        }
                    }
                }
                const float off = KT::kShift - (m == -INFINITY ? 0.f : m * row.sl);
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16], lo[8];
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[e] = exp2_fast(fmaf(__uint_as_float(s[32 * q + i + e]), row.sl, off));
                            sum[e] += p[e];
                        }
                        if (K != kE4m3) {
                            pk[i >> 1] = from_float2<T>(p[0], p[1]);
                            pk[(i >> 1) + 1] = from_float2<T>(p[2], p[3]);
                        } else {
                            const uint32_t a = e4m3x2(p[0], p[1]), b = e4m3x2(p[2], p[3]);
                            const float2 x = from_e4m3x2(a), y = from_e4m3x2(b);
                            pk[i >> 2] = a | b << 16;
                            lo[i >> 2] = e4m3x2(p[0] - x.x, p[1] - x.y) | e4m3x2(p[2] - y.x, p[3] - y.y) << 16;
                        }
                    }
                    if (K != kE4m3) tc_st16(s_col + 16 * q, pk);
                    else {
                        tc_st8(s_col + 8 * q, pk);
                        tc_st8(s_col + 32 + 8 * q, lo);
                    }
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc_wait_st();
            }
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_ready);
            if (mixed_tile(P, it, k0)) {
                // rows that see a non-finite value, which the product met as zero, get it added here
                const uint32_t v = tiles + j;
                if (!wait(smem_u32(&sh.value[v % P.slots]), (v / P.slots) & 1, gave_up)) return;
                uint32_t odd[4], any = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) any |= odd[i] = sh.odd[ring][i];
                if (any && busy) {
                    if (!wait(pv_done, steps & 1, gave_up)) return;
                    tc_after();
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        tc_ld32(o_col[stream] + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            for (uint32_t w = row.real ? odd[i] & seen[i] : 0u; w; w &= w - 1) {
                                const int32_t slot = k0 + 32 * i + __ffs(w) - 1;
                                const int64_t at = place_of(A.pool, it.b, slot) + it.h * A.pool.s_head;
#pragma unroll
                                for (int d = 0; d < 32; ++d) {
                                    if (c + d >= D) break;
                                    float x;
                                    if (K == kE4m3) {
                                        const uint8_t u = ((const uint8_t*)A.pool.v)[at + c + d];
                                        x = (u & 0x7f) == 0x7f ? NAN : 0.f;
                                    } else {
                                        x = (float)((const T*)A.pool.v)[at + c + d];
                                    }
                                    if (!isfinite(x)) o[d] = __float_as_uint(__uint_as_float(o[d]) + x);
                                }
                            }
                        tc_st32(o_col[stream] + c, o);
                    }
                    tc_wait_st();
                    tc_before();
                }
            }
        }
        tiles += it.n;

        // the next item's queries, as soon as the products of this one have read theirs
        more = walk.next(nx);
        if (more) {
            if (!wait(q_empty, items & 1, gave_up)) return;
            load_queries<K>(P, nx, stream, r, q_smem, nrow);
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(q_full);
        }
        ++items;

        // the item's end
        if (done > 0) {
            if (!wait(pv_done, (steps - 1) & 1, gave_up)) return;
            tc_after();
        }
        float w0 = 1.f, w1 = 0.f, total = l;
        float ref = m == -INFINITY ? -INFINITY : m * row.sl - KT::kShift;
        const bool both = !it.two && it.n > 1;  // the other stream has a part
        if (!it.two) {
            sh.ml[stream][r] = make_float2(ref, l);
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_u32(&sh.meet));
            if (!wait(smem_u32(&sh.meet), merges & 1, gave_up)) return;
            tc_after();
            const float2 a = sh.ml[0][r], b = both ? sh.ml[1][r] : make_float2(-INFINITY, 0.f);
            ref = fmaxf(a.x, b.x);
            const float base = ref == -INFINITY ? 0.f : ref;
            w0 = exp2_fast(a.x - base);
            w1 = exp2_fast(b.x - base);
            if (ref == -INFINITY) w0 = w1 = 1.f;  // sums of zero, or of NaN
            total = a.y * w0 + (both ? b.y * w1 : 0.f);
        }
        const bool alone = it.begins && it.finishes;
        const int32_t row_at = it.row0 + row.token;
        const float vs = A.pool.v_scale ? A.pool.v_scale[it.h] : 1.f;
        const float inv = total == 0.f ? 0.f : vs / total;
        const int32_t head = it.h * P.G + row.g;
        // a row that carries NaN or infinity in its sum stays so: inv is then NaN or zero
        const int c_begin = it.two ? 0 : stream * (DP / 2), c_end = it.two ? DP : c_begin + DP / 2;
        const size_t prow = (size_t)(2 * blockIdx.x + (it.begins ? 1 : 0)) * 256 + (it.two && stream ? kTile : 0) + r;
        if (busy) {
            for (int c = c_begin; c < c_end; c += 32) {
                uint32_t o[32];
                tc_ld32(it.two ? o_col[stream] + c : o_col[0] + c, o);
                if (both) {
                    uint32_t x[32];
                    tc_ld32(o_col[1] + c, x);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * w0 + __uint_as_float(x[i]) * w1);
                } else {
                    tc_wait_ld();
                }
                if (row.real) {
                    if (alone) {
                        T* out = (T*)A.out + ((int64_t)row_at * A.q_heads + head) * D;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            if (c + i < D) {
                                uint4 u;
                                u.x = from_float2<T>(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
                                u.y = from_float2<T>(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                                u.z = from_float2<T>(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
                                u.w = from_float2<T>(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
                                *reinterpret_cast<uint4*>(out + c + i) = u;
                            }
                        }
                    } else {
                        float* out = P.part_o + prow * DP + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (c + i < D)
                                *reinterpret_cast<float4*>(out + i) =
                                    make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                                __uint_as_float(o[i + 3]));
                    }
                }
            }
            if (row.real && (it.two || stream == 0)) {
                if (!alone) P.part_ml[prow] = make_float2(ref, total);
                else if (A.lse)
                    A.lse[(int64_t)row_at * A.q_heads + head] = total == 0.f ? -INFINITY : ref * kLn2 + logf(total);
            }
        }
        if (!it.two) {  // neither stream starts on its O before both have read the two
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_u32(&sh.part));
            if (!wait(smem_u32(&sh.part), merges & 1, gave_up)) return;
            tc_after();
            ++merges;
        }
        it = nx;
        row = nrow;
    }
}

// ---------------------------------------------------------------------------------------------------------
// loads, products, value tiles: one warp each (value tiles: two)
// ---------------------------------------------------------------------------------------------------------
template <int NH>
__device__ __forceinline__ void load_role(const Params& P, Shared& sh, uint32_t kv_smem, const CUtensorMap* km,
                                          const CUtensorMap* vm) {
    const int lane = threadIdx.x & 31;
    const int32_t box = P.box, boxes = kTile / box, ps = P.a.pool.page_size;
    volatile int* gave_up = &sh.gave_up;
    uint32_t load = 0, tile = 0;
    bool ok = true;
    Walk walk(P, sh.start);
    Item it;
    while (ok && walk.next(it)) {
        const int32_t* table = P.a.pool.table + (int64_t)it.b * P.a.pool.table_stride;
        for (int32_t j = 0; j < it.n && ok; ++j, ++tile) {
            const int32_t slot = (it.tile + j) * kTile + lane * box;
            int32_t page = -1, at = 0;
            bool need = lane < boxes && slot < it.end && slot + box > it.lo;
            if (need) {
                const int32_t i = slot / ps;
                at = slot - i * ps;
                page = table[i];
            }
            const bool miss = need && (page < 0 || page >= P.a.pool.pages);
            if (miss) report(P.a.status, 1u << SV_ERR_BAD_OFFSETS);
            need = need && !miss;
            uint32_t bad = miss ? ((1u << (box / 8)) - 1u) << (lane * (box / 8)) : 0u;
            bad = __reduce_or_sync(kAll, bad);
            const uint32_t bytes = __popc(__ballot_sync(kAll, need)) * box * 128 * NH;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++load) {
                const uint32_t slot_i = load % P.slots, full = smem_u32(&sh.full[slot_i]);
                if (load >= (uint32_t)P.slots &&
                    !wait(smem_u32(&sh.empty[slot_i]), (load / P.slots - 1) & 1, gave_up)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (kv == 0) sh.bad[tile % kBadRing] = bad;
                    bar_expect(full, bytes);
                }
                __syncwarp();
                if (need) {
                    const uint32_t dst = kv_smem + slot_i * (NH * kHalf) + lane * box * 128;
#pragma unroll
                    for (int h = 0; h < NH; ++h) copy_box(dst + h * kHalf, kv ? vm : km, h * 64, at, it.h, page, full);
                }
            }
        }
    }
    // copies still under way land before the CTA ends, also where another role gave up
    for (uint32_t i = load > (uint32_t)P.slots ? load - P.slots : 0; i < load; ++i) {
        int none = 0;
        wait(smem_u32(&sh.full[i % P.slots]), (i / P.slots) & 1, &none);
    }
}

template <int K, int NH>
__device__ __forceinline__ void product_role(const Params& P, Shared& sh, uint32_t q_smem, uint32_t kv_smem) {
    constexpr bool k8 = K == kE4m3;
    constexpr int parts = k8 ? 2 : 1, slot_bytes = NH * kHalf;
    constexpr uint32_t fmt = K == kBf16 ? 1u : 0u;
    const int lane = threadIdx.x & 31;
    const int32_t D = P.a.pool.dim;
    const int32_t depth = (D + KindOf<K>::kStep - 1) / KindOf<K>::kStep;
    // float accumulators, 128 rows; scores are 128 columns wide, outputs D rounded up to 16 with the value
    // operand's rows along the depth
    const uint32_t base = 1u << 4 | fmt << 7 | fmt << 10 | (uint32_t)(kTile >> 4) << 24;
    const uint32_t id_s = base | (uint32_t)(kTile >> 3) << 17;
    const uint32_t id_o = base | 1u << 16 | (uint32_t)((D + 15) / 16 * 2) << 17;
    const uint32_t q_bytes = (k8 ? 2 : NH) * kHalf;
    const uint32_t dp = NH == 1 && !k8 ? 64 : 128;
    volatile int* gave_up = &sh.gave_up;
    uint32_t tiles = 0, items = 0, steps[2] = {0, 0};
    Walk walk(P, sh.start);
    Item it;
    bool ok = true;
    while (ok && walk.next(it)) {
        if (!(ok = wait(smem_u32(&sh.q_full), items & 1, gave_up))) break;
        tc_after();
        const int32_t S = it.two ? 2 * it.n : it.n;
        auto scores = [&](int32_t n) {
            const int st = n & 1;
            const int32_t t = it.two ? n >> 1 : n;
            const uint32_t load = 2 * (tiles + t), slot = load % P.slots;
            if (!(it.two && st) && !wait(smem_u32(&sh.full[slot]), (load / P.slots) & 1, gave_up)) return false;
            if (lane == 0) {
                const uint32_t q = q_smem + (it.two && st ? q_bytes : 0), k = kv_smem + slot * slot_bytes;
                const uint32_t d = sh.tmem + st * kTile;
#pragma unroll
                for (int part = 0; part < parts; ++part)
                    for (int i = 0; i < depth; ++i) {
                        const uint32_t off = (i >> 2) * kHalf + (i & 3) * 32;
                        mma_ss<k8>(d, operand(q + part * kHalf + off, 16), operand(k + off, 16), id_s, part + i > 0);
                    }
                tc_commit(smem_u32(&sh.s_full[st]));
                if (!it.two || st) tc_commit(smem_u32(&sh.empty[slot]));
                if (n == S - 1) tc_commit(smem_u32(&sh.q_empty));
            }
            __syncwarp();
            return true;
        };
        auto outputs = [&](int32_t n) {
            const int st = n & 1;
            const int32_t t = it.two ? n >> 1 : n;
            const uint32_t v = tiles + t, slot = (2 * v + 1) % P.slots;
            if (!(it.two && st) && !wait(smem_u32(&sh.value[v % P.slots]), (v / P.slots) & 1, gave_up)) return false;
            if (!wait(smem_u32(&sh.p_ready[st]), steps[st] & 1, gave_up)) return false;
            tc_after();
            if (lane == 0) {
                const uint32_t a = sh.tmem + st * kTile, b = kv_smem + slot * slot_bytes, d = sh.tmem + 256 + st * dp;
#pragma unroll
                for (int part = 0; part < parts; ++part)
#pragma unroll
                    for (int i = 0; i < kTile / KindOf<K>::kStep; ++i)
                        mma_ts<k8>(d, a + part * 32 + i * 8, operand(b + i * KindOf<K>::kStep * 128, kHalf), id_o,
                                   n > 1 || part + i > 0);
                tc_commit(smem_u32(&sh.pv_done[st]));
                if (!it.two || st) tc_commit(smem_u32(&sh.empty[slot]));
            }
            __syncwarp();
            ++steps[st];
            return true;
        };
        ok = scores(0);
        if (ok && S > 1) ok = scores(1);
        for (int32_t n = 0; n < S && ok; ++n) {
            ok = outputs(n);
            if (ok && n + 2 < S) ok = scores(n + 2);
        }
        tiles += it.n;
        ++items;
    }
    // products under way end before the tensor memory is given back
    if (lane == 0) tc_commit(smem_u32(&sh.drain));
    __syncwarp();
    int none = 0;
    wait(smem_u32(&sh.drain), 0, &none);
}

// Value tiles before they are multiplied: rows of slots that no row of the item sees are cleared (they may
// hold anything, and a weight of zero times NaN is NaN), and so are single non-finite values that only some
// rows see; those are noted for the rows that do.
template <int K, int NH>
__device__ __forceinline__ void value_role(const Params& P, Shared& sh, uint32_t kv_smem) {
    const int lane = threadIdx.x & 31, half = (threadIdx.x >> 5) & 1;  // rows 64 half .. 64 half + 63
    volatile int* gave_up = &sh.gave_up;
    uint32_t v = 0;
    Walk walk(P, sh.start);
    Item it;
    while (walk.next(it)) {
        for (int32_t j = 0; j < it.n; ++j, ++v) {
            const uint32_t load = 2 * v + 1, slot = load % P.slots, ring = v % kBadRing;
            if (!wait(smem_u32(&sh.full[slot]), (load / P.slots) & 1, gave_up)) return;
            const int32_t k0 = (it.tile + j) * kTile;
            const uint32_t bad = sh.bad[ring];
            const bool edge = bad || k0 < it.lo || k0 + kTile > it.end, mixed = mixed_tile(P, it, k0);
            uint32_t odd[2] = {0, 0};
            if (edge || mixed) {
                const uint32_t at = kv_smem + slot * (NH * kHalf) + (lane & 7) * 16;
                for (int i = 0; i < 16; ++i) {  // four rows at a time, eight lanes each
                    const int row = half * 64 + i * 4 + (lane >> 3);
                    const int32_t s = k0 + row;
                    const bool clear = s < it.lo || s >= it.end || (bad >> (row >> 3) & 1u);
                    bool found = false;
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const uint32_t a = at + h * kHalf + row * 128;
                        uint32_t u[4];
                        bool write = clear;
                        if (clear) u[0] = u[1] = u[2] = u[3] = 0;
                        else if (mixed) {
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                                         : "r"(a)
                                         : "memory");
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (K == kE4m3) {
#pragma unroll
                                    for (int by = 0; by < 32; by += 8)
                                        if ((u[e] >> by & 0x7fu) == 0x7fu) {
                                            u[e] &= ~(0xffu << by);
                                            write = found = true;
                                        }
                                } else {
                                    constexpr uint32_t top = K == kBf16 ? 0x7f80u : 0x7c00u;
#pragma unroll
                                    for (int by = 0; by < 32; by += 16)
                                        if ((u[e] >> by & top) == top) {
                                            u[e] &= ~(0xffffu << by);
                                            write = found = true;
                                        }
                                }
                            }
                        }
                        if (write)
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                                         "r"(u[3])
                                         : "memory");
                    }
                    const unsigned f = __ballot_sync(kAll, found);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (f >> (8 * k) & 0xffu) odd[i >> 3] |= 1u << ((i & 7) * 4 + k);
                }
                fence_async();
            }
            if (lane == 0) {
                sh.odd[ring][2 * half] = odd[0];
                sh.odd[ring][2 * half + 1] = odd[1];
            }
            __syncwarp();
            if (lane == 0) bar_arrive(smem_u32(&sh.value[v % P.slots]));
        }
    }
}

template <int K, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
    constexpr int NH = K == kE4m3 ? 1 : DP / 64;
    extern __shared__ char raw[];
    __shared__ Shared sh;
    const uint32_t q_smem = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t kv_smem = q_smem + P.q_tiles * (K == kE4m3 ? 2 : NH) * kHalf;
    const int tid = threadIdx.x, w = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            bar_init(smem_u32(&sh.full[i]), 1);
            bar_init(smem_u32(&sh.empty[i]), 1);
            bar_init(smem_u32(&sh.value[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_u32(&sh.s_full[i]), 1);
            bar_init(smem_u32(&sh.p_ready[i]), 4);
            bar_init(smem_u32(&sh.pv_done[i]), 1);
        }
        bar_init(smem_u32(&sh.q_full), 8);
        bar_init(smem_u32(&sh.q_empty), 1);
        bar_init(smem_u32(&sh.meet), 8);
        bar_init(smem_u32(&sh.part), 8);
        bar_init(smem_u32(&sh.drain), 1);
        sh.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (w == 9)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    // sequences that fail: their findings, and zeros in their rows
    for (int32_t b = blockIdx.x; b < P.a.chunk.B; b += gridDim.x) {
        const Seq s = checked_seq(P, b);
        if (!s.err) continue;
        if (tid == 0) report(P.a.status, s.err);
        if (!s.rows_ok) continue;
        const int64_t row = (int64_t)P.a.q_heads * P.a.pool.dim / 8;
        uint4* out = (uint4*)P.a.out + s.row0 * row;
        for (int64_t i = tid; i < s.T * row; i += kThreads) out[i] = make_uint4(0, 0, 0, 0);
        if (P.a.lse)
            for (int64_t i = tid; i < (int64_t)s.T * P.a.q_heads; i += kThreads)
                P.a.lse[(int64_t)s.row0 * P.a.q_heads + i] = -INFINITY;
    }
    if (blockIdx.x == 0 && tid == 0) {
        const int64_t end = (int64_t)P.a.chunk.offs[P.a.chunk.B] + P.a.chunk.B;
        if (end > P.a.chunk.rows || P.a.chunk.offs[0] != 0) report(P.a.status, 1u << SV_ERR_BAD_OFFSETS);
    }
    plan(P, sh);
    tc_before();
    __syncthreads();
    tc_after();
    if (w < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        softmax_role<K, DP>(P, sh, q_smem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (w == 8) load_role<NH>(P, sh, kv_smem, &km, &vm);
        else if (w == 9) product_role<K, NH>(P, sh, q_smem, kv_smem);
        else value_role<K, NH>(P, sh, kv_smem);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (w == 9) {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem));
    }
    if (tid == 0 && sh.gave_up) report(P.a.status, 1u << SV_ERR_TIMEOUT);
}

// Items that several CTAs worked on: one warp a row, the parts in their order.
constexpr int kMergeThreads = 256;
template <typename T, int DP>
__global__ void __launch_bounds__(kMergeThreads) k_attend_merge(const __grid_constant__ Params P) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t c = blockIdx.x + 1;
    const Record rec = P.records[c];
    if (!rec.parts) return;
    const int lane = threadIdx.x & 31;
    const int32_t D = P.a.pool.dim, rows = rec.tokens * P.G;
    constexpr int kPer = DP / 32;
    for (int32_t i = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5); i < rows;
         i += gridDim.y * (kMergeThreads / 32)) {
        const int32_t t = i / P.G, g = i - t * P.G;
        const int32_t r = t < P.tokens ? i : kTile + i - P.tokens * P.G;
        // the first part is the last item of CTA c - 1, the others the first items of c, c + 1, ...
        auto slot = [&](int32_t part) { return (size_t)(part ? 2 * (c + part - 1) : 2 * (c - 1) + 1) * 256 + r; };
        float top = -INFINITY;
        for (int32_t p = lane; p < rec.parts; p += 32) top = fmaxf(top, P.part_ml[slot(p)].x);
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        const float base = top == -INFINITY ? 0.f : top;
        float l = 0.f, acc[kPer] = {};
        for (int32_t p0 = 0; p0 < rec.parts; p0 += 32) {
            float wt = 0.f, pl = 0.f;
            if (p0 + lane < rec.parts) {
                const float2 ml = P.part_ml[slot(p0 + lane)];
                wt = top == -INFINITY ? 1.f : exp2_fast(ml.x - base);
                pl = ml.y * wt;
            }
            for (int o = 16; o; o >>= 1) pl += __shfl_xor_sync(kAll, pl, o);
            l += pl;
            const int32_t n = min(32, rec.parts - p0);
#pragma unroll 4
            for (int32_t k = 0; k < n; ++k) {
                const float f = __shfl_sync(kAll, wt, k);
                const float* o = P.part_o + slot(p0 + k) * DP + lane * kPer;
                if (lane * kPer < D) {
                    float x[kPer];
                    if (kPer == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(o);
                    else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(o);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) acc[e] = fmaf(f, x[e], acc[e]);
                }
            }
        }
        const float vs = P.a.pool.v_scale ? P.a.pool.v_scale[rec.head] : 1.f;
        const float inv = l == 0.f ? 0.f : vs / l;
        const int64_t at = (int64_t)(rec.row0 + t) * P.a.q_heads + rec.head * P.G + g;
        if (lane * kPer < D) {
            T* out = (T*)P.a.out + at * D + lane * kPer;
#pragma unroll
            for (int e = 0; e < kPer; e += 2)
                *reinterpret_cast<uint32_t*>(out + e) = from_float2<T>(acc[e] * inv, acc[e + 1] * inv);
        }
        if (P.a.lse && lane == 0) P.a.lse[at] = l == 0.f ? -INFINITY : top * kLn2 + logf(l);
    }
}

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
bool encode(CUtensorMap* m, const Pool& p, char* base, int esize, int kind, int box) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.dim, (cuuint64_t)p.page_size, (cuuint64_t)p.heads, (cuuint64_t)p.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.s_token * esize, (cuuint64_t)p.s_head * esize,
                                   (cuuint64_t)p.s_page * esize};
    const cuuint32_t boxes[4] = {(cuuint32_t)(128 / esize), (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = kind == kE4m3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : kind == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encoder()(m, type, 4, base, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int K, int DP>
cudaError_t launch(const AttendArgs& A, cudaStream_t st) {
    constexpr int NH = K == kE4m3 ? 1 : DP / 64, q_bytes = (K == kE4m3 ? 2 : NH) * kHalf;
    Params P{};
    P.a = A;
    P.G = A.q_heads / A.pool.heads;
    P.tokens = kTile / P.G;
    P.q_tiles = A.chunk.max_gamma + 1 > P.tokens ? 2 : 1;
    P.slots = min(kMaxSlots, (kSmem - 1024 - (int)sizeof(Shared) - P.q_tiles * q_bytes) / (NH * kHalf));
    P.box = kTile;
    while (A.pool.page_size % P.box) P.box /= 2;
    char* ws = (char*)A.workspace;
    P.part_o = (float*)ws;
    P.part_ml = (float2*)(ws + part_rows() * DP * sizeof(float));
    P.records = (Record*)(P.part_ml + part_rows());
    int dev, sms;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int n = min(sms, kMaxCtas);
    if (!encoder()) return cudaErrorNotSupported;
    CUtensorMap km, vm;
    if (!encode(&km, A.pool, A.pool.k, KindOf<K>::kBytes, K, P.box) || !encode(&vm, A.pool, A.pool.v, KindOf<K>::kBytes, K, P.box))
        return cudaErrorInvalidValue;
    const int smem = 1024 + P.q_tiles * q_bytes + P.slots * NH * kHalf;
    e = cudaFuncSetAttribute(k_attend<K, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem - (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    k_attend<K, DP><<<n, kThreads, smem, st>>>(P, km, vm);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(n - 1, 4);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attend_merge<typename KindOf<K>::T, DP>, P);
}

}  // namespace

size_t attend_workspace(int dim, int cache_dtype) {
    const size_t dp = cache_dtype == SV_E4M3 || dim > 64 ? 128 : 64;
    return part_rows() * (dp * sizeof(float) + sizeof(float2)) + kMaxCtas * sizeof(Record);
}

cudaError_t launch_attend(const AttendArgs& A, int dtype, int cache_dtype, cudaStream_t st) {
    if (cache_dtype == SV_E4M3) return launch<kE4m3, 128>(A, st);
    if (dtype == SV_F16) return A.pool.dim > 64 ? launch<kFp16, 128>(A, st) : launch<kFp16, 64>(A, st);
    return A.pool.dim > 64 ? launch<kBf16, 128>(A, st) : launch<kBf16, 64>(A, st);
}

}  // namespace cache
}  // namespace sv
