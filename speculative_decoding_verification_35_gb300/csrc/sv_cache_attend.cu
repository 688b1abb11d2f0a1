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

#include <atomic>

#include "sv_cache.cuh"

namespace sv {
namespace cache {
namespace {

constexpr int kThreads = 512;   // two softmax warpgroups, then a warp for each other role
constexpr int kTile = 128;      // slots of a tile, and rows of a query tile
constexpr int kMaxSlots = 6;    // key tiles in flight, and value tiles
constexpr int kBadRing = 16;
constexpr int kMaxCtas = 160;
constexpr int kItems = 4;       // items that are known ahead
constexpr int kHalf = kTile * 128;  // bytes of 128 rows of 128 bytes, the unit of an operand in shared memory
constexpr int kSmem = 227 * 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------------------------------------------
// element kinds
// ---------------------------------------------------------------------------------------------------------
// kShift: weights are held as 2^kShift w, so that those far below the largest keep their precision in a narrow
// type; kSlack: how far (log2) a weight may exceed the reference before the reference moves. A tile's 128 weights
// sum to 2^(kShift + kSlack + 7) at most, within the type's range: bfloat16 has float's, and its reference hardly
// ever moves after the first tile. (e4m3: every weight, 2^(kShift + kSlack) <= 448.)
// kE4m3: the cache is 8 bits wide and the products are too. A bfloat16 query has 8 significant bits and an
// e4m3 value 4, so q 2^k = hi + lo exactly, but for elements under 2^-11 of the row's largest (k brings it to
// [128, 256)); a weight is hi + lo to about 2^-9 of itself. Each product then runs twice, at twice the 16-bit rate,
// and no key or value is converted.
enum Kind { kBf16 = 0, kFp16 = 1, kE4m3 = 2 };
template <int K>
struct KindOf;
template <>
struct KindOf<kBf16> {
    using T = __nv_bfloat16;
    static constexpr float kShift = 0.f, kSlack = 56.f;
    static constexpr int kBytes = 2, kStep = 16;  // of an element; elements a product step takes along its depth
};
template <>
struct KindOf<kFp16> {
    using T = __half;
    static constexpr float kShift = 7.f, kSlack = 1.f;
    static constexpr int kBytes = 2, kStep = 16;
};
template <>
struct KindOf<kE4m3> {
    using T = __nv_bfloat16;
    static constexpr float kShift = 7.f, kSlack = 1.75f;
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
    int32_t q_box;      // tokens of one copy into a query tile
    int32_t k_slots, v_slots;  // key and value tiles that shared memory has room for
    int32_t box;        // slots of one copy, a divisor of the page size and of kTile
    int32_t wide;       // output rows lie on 32 bytes
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
// True once the phase is over; may sleep for it, half a microsecond at most.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "n"(500)
        : "memory");
    return ok;
}
// A whole warp waits; false once the CTA has given up (a wait of at least a tenth of a second and a few at most).
constexpr uint32_t kPolls = 1u << 24;
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
    bool ok = bar_try(bar, parity);
#pragma unroll 1
    for (uint32_t i = 1; !__all_sync(kAll, ok); ++i) {
        if (!ok) ok = bar_try(bar, parity);
        if ((i & 255u) == 0) {
            if (i >= kPolls) *gave_up = 1;
            if (__any_sync(kAll, *gave_up)) return false;
        }
    }
    return true;
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int d, int token, int head, int page,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(d), "r"(token), "r"(head), "r"(page), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy_queries(uint32_t dst, const CUtensorMap* map, int d, int head, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(d), "r"(head), "r"(row), "r"(bar)
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
// Shared-memory operand of 128-byte rows under the 128-byte swizzle, eight rows 1024 bytes apart: the low word
// of its descriptor (address, and the bytes between column halves of an operand whose rows run along the depth),
// and the high word, which all share.
constexpr uint32_t kOperandHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t far) {
    return (addr & 0x3ffffu) >> 4 | (far >> 4) << 16;
}
#define SV_MMA(kind, a)                                                                                            \
    "{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.u32 p, %4, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"      \
    "tcgen05.mma.cta_group::1.kind::" kind " [%0], " a ", y, %3, p;\n}"
template <bool k8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    if (k8) asm volatile(SV_MMA("f8f6f4", "x") ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh) : "memory");
    else asm volatile(SV_MMA("f16", "x") ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh) : "memory");
}
template <bool k8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    if (k8) asm volatile(SV_MMA("f8f6f4", "[%1]") ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh) : "memory");
    else asm volatile(SV_MMA("f16", "[%1]") ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh) : "memory");
}
// One thread of a converged warp, always the same.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p;
}
// A position in a ring of n slots and the parity of its current use.
struct Ring {
    uint32_t i = 0, parity = 0;
    __device__ __forceinline__ void step(uint32_t n) {
        if (++i == n) {
            i = 0;
            parity ^= 1;
        }
    }
};
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two floats in one register pair, for the packed multiply-add and add.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 half_pair(uint32_t e4m3) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)e4m3, __NV_E4M3);
    return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t u) { return __half22float2(half_pair(u)); }
// The parts hi and lo of two weights, by way of their half-precision values (2^-11 of them off, where hi + lo is 2^-9).
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 x = __floats2half2_rn(a, b);
    hi = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&x), __NV_SATFINITE, __NV_E4M3);
    const __half2 r = __hsub2(x, half_pair(hi));
    lo = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&r), __NV_SATFINITE, __NV_E4M3);
}

// ---------------------------------------------------------------------------------------------------------
// work items
// ---------------------------------------------------------------------------------------------------------
struct alignas(16) Item {
    int32_t b, h, row0;           // sequence, key head, the sequence's first row
    int32_t t0, nt;               // its chunk tokens
    int32_t past;
    int32_t lo, end;              // the slots [lo, end) that some row of it sees
    int32_t tile, n;              // the CTA's tiles: the first (absolute), how many; 0: no more items
    int32_t mixed_lo, mixed_hi;   // slots below mixed_lo and from mixed_hi on are seen by some of its rows only
    int32_t two;                  // 129 to 256 rows: a query tile per stream
    int32_t begins, finishes;     // its first and last tiles are among the CTA's
    int32_t pad;
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
#pragma unroll 4
    for (int j = 1; j < T; ++j) ok &= (uint32_t)par[j - 1] < (uint32_t)j;
    return ok;
}

__device__ __forceinline__ Seq checked_seq(const Params& P, int32_t b) {
    Seq s = seq_of(P.a.chunk, capacity_of(P.a.pool), b);
    if (!s.err && P.a.chunk.parents && !tree_ok(P.a.chunk, b, s.T)) s.err = 1u << SV_ERR_BAD_OFFSETS;
    return s;
}

// Tiles and row blocks of a sequence, for one key head.
__device__ __forceinline__ void size_of(const Params& P, const Seq& s, long long& tiles, long long& blocks) {
    tiles = blocks = 0;
    if (s.err) return;
#pragma unroll 1
    for (int32_t p = 0; p * 2 * P.tokens < s.T; ++p) {
        Item it;
        int32_t first, count;
        span(P, s.T, s.past, p, it, first, count);
        tiles += count;
        ++blocks;
    }
}

// Where a CTA begins. An item is `lead` units of beginning and ending (its queries' way in, its outputs' way
// out, and the pipeline's filling in between) and a unit a tile; x counts them.
struct Start {
    int32_t b, p, h, T, past, row0;
    int32_t lead, x;
    long long left;
};

struct Shared {  // behind the operand tiles
    uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
    uint64_t value[kMaxSlots];  // a value tile is in and clean
    uint64_t s_full[2], p_ready[2], pv_done[2];
    uint64_t turn[2];           // the streams' products take turns
    uint64_t q_in, q_full, q_empty, meet, part, drain;
    uint64_t item_full[kItems], item_empty[kItems];
    Item item[kItems];
    uint32_t tmem;
    int gave_up;
    Start start;
    long long scan[kThreads / 32], scan2[kThreads / 32];
    int failing;  // some sequence of this CTA's share has a finding
    uint32_t bad[2][kBadRing];      // per key and per value tile: groups of 8 slots that lie on a bad page
    uint32_t odd[kBadRing][4];      // per value tile: slots with a non-finite value that was cleared
    float2 ml[2][kTile];
    float q_down[1];  // e4m3 caches: [2][256], what a row's scores are scaled by, for even and odd items
};
template <int K>
constexpr int shared_bytes() {
    return (int)sizeof(Shared) + (K == kE4m3 ? 2 * 2 * kTile * 4 : 0);
}

// a * b / c of small numbers without the long division.
__device__ __forceinline__ long long share(long long a, int32_t b, int32_t c) {
    const unsigned long long x = (unsigned long long)a * (uint32_t)b;
    return x >> 32 ? (long long)(x / (uint32_t)c) : (long long)((uint32_t)x / (uint32_t)c);
}

// Where the CTA begins, and the record of an item that its predecessor began. All threads.
constexpr int32_t kLead = 5;  // measured: about five tiles' time between an item's last tile and the next one's pace
__device__ __forceinline__ void plan(const Params& P, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int32_t B = P.a.chunk.B, c = (int32_t)blockIdx.x, heads = P.a.pool.heads;
    Seq mine{};
    long long my_tiles = 0, my_blocks = 0, tiles = 0, blocks = 0;
    if (tid == 0) {
        sh.start.left = 0;
        sh.failing = 0;
        if (c > 0) P.records[c].parts = 0;
    }
    bool fails = false;
#pragma unroll 1
    for (int32_t b = tid; b < B; b += kThreads) {
        const Seq s = checked_seq(P, b);
        long long t, n;
        size_of(P, s, t, n);
        fails |= s.err && b % gridDim.x == c;
        tiles += t;
        blocks += n;
        if (b == tid) {
            mine = s;
            my_tiles = t;
            my_blocks = n;
        }
    }
    for (int o = 16; o; o >>= 1) {
        tiles += __shfl_xor_sync(kAll, tiles, o);
        blocks += __shfl_xor_sync(kAll, blocks, o);
    }
    if (lane == 0) {
        sh.scan[w] = tiles;
        sh.scan2[w] = blocks;
    }
    if (__syncthreads_or(fails) && tid == 0) sh.failing = 1;
    tiles = blocks = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        tiles += sh.scan[i];
        blocks += sh.scan2[i];
    }
    tiles *= heads;
    blocks *= heads;
    // With few tiles there is a CTA for each, and an item's beginning is nobody's but its own.
    const int32_t lead = tiles <= 2 * (long long)gridDim.x ? 0 : kLead;
    const long long W = tiles + lead * blocks;
    const int32_t n = (int32_t)min((long long)gridDim.x, tiles);
    if (c >= n) return;  // the same for the whole CTA
    const long long u0 = share(W, c, n), u1 = share(W, c + 1, n);
    long long base = 0;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < B && base <= u0; b0 += kThreads) {
        const int32_t b = b0 + tid;
        if (b0 > 0) {
            my_tiles = my_blocks = 0;
            if (b < B) {
                mine = checked_seq(P, b);
                size_of(P, mine, my_tiles, my_blocks);
            }
        }
        const long long u = (my_tiles + lead * my_blocks) * heads;
        long long incl = u;
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += x;
        }
        if (B > kThreads) {  // else the warps' sums are there already
            __syncthreads();
            if (lane == 31) {
                sh.scan[w] = incl;
                sh.scan2[w] = 0;
            }
            __syncthreads();
        }
        const int32_t sc = B > kThreads ? 1 : heads, lc = B > kThreads ? 0 : lead * heads;
        long long before = base, total = 0;
#pragma unroll 1
        for (int i = 0; i < kThreads / 32; ++i) {
            const long long x = sh.scan[i] * sc + sh.scan2[i] * lc;
            if (i < w) before += x;
            total += x;
        }
        const long long begin = before + incl - u;
        if (u > 0 && u0 >= begin && u0 < begin + u) {
            long long rest = u0 - begin;
            Item it;
            int32_t first, count, p = 0;
#pragma unroll 1
            for (;; ++p) {
                span(P, mine.T, mine.past, p, it, first, count);
                const long long block = (long long)(count + lead) * heads;
                if (rest < block) break;
                rest -= block;
            }
            const int32_t h = (int32_t)(rest / (count + lead)), x = (int32_t)(rest - (long long)h * (count + lead));
            sh.start = {b, p, h, mine.T, mine.past, mine.row0, lead, x, u1 - u0};
            if (x > lead) {
                // the item's first tile is unit `from`; if the CTA before this one had it, this one records the item
                const long long from = u0 - x + lead;
                if (from >= share(W, c - 1, n)) {
                    Record r{};
                    r.parts = (int32_t)(((from + count) * n - 1) / W - c) + 2;  // to the CTA of its last tile
                    r.row0 = mine.row0 + it.t0;
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
// The CTA's items, one after the other, by one warp; a last one of no tiles ends them.
__device__ __forceinline__ void item_role(const Params& P, Shared& sh) {
    const int lane = threadIdx.x & 31;
    const bool tree = P.a.chunk.parents != nullptr;
    const int32_t lead = sh.start.lead;
    int32_t b = sh.start.b, p = sh.start.p, h = sh.start.h, x = sh.start.x;
    int32_t T = sh.start.T, past = sh.start.past, row0 = sh.start.row0;
    long long left = sh.start.left;
    Ring ring;
#pragma unroll 1
    for (uint32_t i = 0;; ++i, ring.step(kItems)) {
        Item it{};
        left -= max(0, lead - x);
        if (left > 0 && T < 0) {  // the next sequence
#pragma unroll 1
            for (; b < P.a.chunk.B; ++b) {
                const Seq s = checked_seq(P, b);
                if (!s.err) {
                    T = s.T;
                    past = s.past;
                    row0 = s.row0;
                    break;
                }
            }
        }
        if (left > 0 && T > 0) {
            int32_t first, count;
            span(P, T, past, p, it, first, count);
            const int32_t j = max(0, x - lead);
            it.b = b;
            it.h = h;
            it.row0 = row0;
            it.tile = first + j;
            it.begins = j == 0;
            it.n = (int32_t)min((long long)(count - j), left);
            it.finishes = j + it.n == count;
            it.mixed_hi = past + (tree ? 0 : it.t0 + 1);
            it.mixed_lo = P.a.window > 0 && (tree || it.nt > 1) ? it.lo + it.nt + (tree ? it.t0 : 0) : 0;
            left -= it.n;
            x = 0;
            if (++h == P.a.pool.heads) {
                h = 0;
                ++p;
                if (p * 2 * P.tokens >= T) {
                    p = 0;
                    ++b;
                    T = -1;
                }
            }
        }
        if (i >= kItems && !wait(smem_u32(&sh.item_empty[ring.i]), ring.parity ^ 1, &sh.gave_up)) return;
        if (lane == 0) {
            sh.item[ring.i] = it;
            bar_arrive(smem_u32(&sh.item_full[ring.i]));
        }
        __syncwarp();
        if (it.n == 0) return;
    }
}

// A role's view of the items.
struct Items {
    Shared& sh;
    Ring ring;
    __device__ __forceinline__ Items(Shared& s) : sh(s) {}
    __device__ __forceinline__ bool next(Item& it) {
        if (!wait(smem_u32(&sh.item_full[ring.i]), ring.parity, &sh.gave_up)) return false;
        it = sh.item[ring.i];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) bar_arrive(smem_u32(&sh.item_empty[ring.i]));
        ring.step(kItems);
        return it.n > 0;
    }
};
constexpr int kItemReaders = 8 + 2 + 2 + 1;

// A row of a query tile as its thread knows it.
struct Row {
    bool real;
    int32_t token;      // chunk token
    int32_t low, limit; // slots low .. limit - 1 are seen, as far as they are not a tree's
    uint32_t above;     // a tree: the chunk tokens it sees
    float sl;           // score units to log2 of the weight, not negative
};

// Scores to log2 of the weights. A negative factor changes the queries' signs; one of zero is kept above it, so
// that -inf stays -inf.
__device__ __forceinline__ float score_unit(const AttendArgs& A, int32_t h, bool& flip) {
    const float sl = A.scale * (A.pool.k_scale ? A.pool.k_scale[h] : 1.f) * kLog2e;
    flip = sl < 0.f;
    return fmaxf(fabsf(sl), 1e-30f);
}

// The nodes that a tree's node t sees (itself and those above it, as far as the window reaches), and its depth.
__device__ __forceinline__ uint32_t lineage(const int32_t* par, int32_t t, int32_t window, int32_t& depth) {
    uint32_t above = 0;
    int32_t d = 0;
#pragma unroll 1
    for (;; t = par[t - 1], ++d) {
        if (window <= 0 || d < window) above |= 1u << t;
        if (t == 0) break;
    }
    depth = d;
    return above;
}

// tl: the row's token within its tile.
__device__ __forceinline__ Row row_of(const Params& P, const Item& it, int stream, int32_t tl) {
    const AttendArgs& A = P.a;
    Row row;
    row.token = it.t0 + tl + (it.two && stream ? P.tokens : 0);
    row.real = tl < P.tokens && row.token < it.t0 + it.nt;
    row.above = 0;
    int32_t depth = row.token;
    if (A.chunk.parents) {
        const int32_t* par = A.chunk.parents + (it.row0 - it.b);
        if (row.real) row.above = lineage(par, row.token, A.window, depth);
    }
    const int32_t pos = it.past + depth;
    row.low = A.window > 0 ? max(0, pos - A.window + 1) : 0;
    row.limit = it.past + (A.chunk.parents ? 0 : row.token + 1);
    bool flip;
    row.sl = score_unit(A, it.h, flip);
    return row;
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

// Only among slots that some rows of the item see and others do not can a value meet a weight of zero, and a NaN
// or infinity be carried into a row that does not see it.
__device__ __forceinline__ bool mixed_tile(const Item& it, int32_t k0) {
    return k0 < it.mixed_lo || max(k0, it.mixed_hi) < min(k0 + kTile, it.end);
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
// False if the weights of some row sum to more than their type holds.
template <int K>
__device__ __forceinline__ bool quick_weights(uint32_t s_col, float sl, float off, bool real, float& total) {
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
    if (K != kE4m3 && __any_sync(kAll, real && total > (K == kBf16 ? 0x1p64f : 0x1p15f))) return false;
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

template <int K, int DP>
__device__ __forceinline__ void softmax_role(const Params& P, Shared& sh) {
    using KT = KindOf<K>;
    using T = typename KT::T;
    const AttendArgs& A = P.a;
    const int stream = threadIdx.x >> 7, r = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(r & ~31) << 16;
    const uint32_t s_col = sh.tmem + lanes + stream * kTile;
    const uint32_t o_col[2] = {sh.tmem + lanes + 256, sh.tmem + lanes + 256 + DP};
    const uint32_t s_full = smem_u32(&sh.s_full[stream]), p_ready = smem_u32(&sh.p_ready[stream]),
                   pv_done = smem_u32(&sh.pv_done[stream]);
    const int32_t D = A.pool.dim;
    const bool tree = A.chunk.parents != nullptr;
    volatile int* gave_up = &sh.gave_up;
    const int32_t tl = r / P.G, g = r - tl * P.G;
    uint32_t steps = 0;   // of this stream, over all items
    uint32_t tiles = 0;   // of the CTA, before this item
    uint32_t items = 0, merges = 0;

    Items walk(sh);
    Item it;
#pragma unroll 1
    for (; walk.next(it); ++items) {
        Row row = row_of(P, it, stream, tl);
        float m = -INFINITY, l = 0.f;
        const bool busy = __any_sync(kAll, row.real);
        const int32_t first = it.two ? 0 : stream, by = it.two ? 1 : 2;
        uint32_t done = 0;
#pragma unroll 1
        for (int32_t j = first; j < it.n; j += by, ++done, ++steps) {
            if (!wait(s_full, steps & 1, gave_up)) return;
            tc_after();
            if (K == kE4m3 && done == 0)
                row.sl *= sh.q_down[(items & 1) * 2 * kTile + (it.two ? stream * kTile : 0) + r];
            const int32_t k0 = (it.tile + j) * kTile;
            const uint32_t ring = (tiles + j) % kBadRing;
            uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
            if (busy) {
                const uint32_t bad = sh.bad[0][ring];
                const bool whole = (k0 + kTile <= row.limit && row.low <= k0 && !bad) || !row.real;
                const bool masked = !__all_sync(kAll, whole);
                if (masked) seen_of(row, it, k0, bad, tree, seen);
                if (masked) hide_tile(s_col, seen);
                float sum;
                bool first = K == kE4m3 || __any_sync(kAll, row.real && m == -INFINITY);
#pragma unroll 1
                for (int attempt = 0; attempt < 2; ++attempt, first = true) {
                    if (first) {
                        const float mx = tile_max(s_col);
                        const bool move = row.real && ((mx - m) * row.sl > KT::kSlack || (m == -INFINITY && mx > m));
                        if (__any_sync(kAll, move)) {
                            const float old = m;
                            if (move) m = mx;
                            const float f = !move || old == -INFINITY ? 1.f : exp2_fast((old - m) * row.sl);
                            l *= f;
                            if (__any_sync(kAll, move && old != -INFINITY)) {
                                if (!wait(pv_done, (steps - 1) & 1, gave_up)) return;
                                tc_after();
                                rescale<DP>(o_col[stream], f);
                            }
                        }
                    }
                    if (quick_weights<K>(s_col, row.sl, KT::kShift - (m == -INFINITY ? 0.f : m * row.sl), row.real, sum)) break;
                }
                l += sum;
                tc_wait_st();
            }
            const bool mixed = mixed_tile(it, k0);
            if (mixed) {  // before p_ready: the tile cannot be released, nor its barrier move on, until then
                const uint32_t v = tiles + j;
                if (!wait(smem_u32(&sh.value[v % P.v_slots]), (v / P.v_slots) & 1, gave_up)) return;
            }
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_ready);
            if (mixed) {
                // rows that see a non-finite value, which the product met as zero, get it added here
                const uint32_t none[4] = {0, 0, 0, 0};
                uint32_t odd[4], any = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) any |= odd[i] = sh.odd[ring][i];
                if (any && busy) {
                    if (!wait(pv_done, steps & 1, gave_up)) return;
                    tc_after();
                    add_odd<K, DP>(A, it, o_col[stream], k0, row.real ? odd : none, seen);
                    tc_wait_st();
                    tc_before();
                }
            }
        }
        tiles += it.n;

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
        const int32_t head = it.h * P.G + g;
        // a row that carries NaN or infinity in its sum stays so: inv is then NaN or zero
        const int c_begin = it.two ? 0 : stream * (DP / 2), c_end = it.two ? DP : c_begin + DP / 2;
        const size_t prow = (size_t)(2 * blockIdx.x + (it.begins ? 1 : 0)) * 256 + (it.two && stream ? kTile : 0) + r;
        if (busy) {
#pragma unroll 1
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
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            u[i] = from_float2<T>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        // lanes write to rows of their own: whole 32-byte sectors halve what that costs
#pragma unroll
                        for (int i = 0; i < 32; i += 16) {
                            const uint32_t* w = u + i / 2;
                            if (P.wide && c + i < D) {
                                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + c + i), SV_W8(w, 0)
                                             : "memory");
                            } else {
                                if (c + i < D) *reinterpret_cast<uint4*>(out + c + i) = make_uint4(w[0], w[1], w[2], w[3]);
                                if (c + i + 8 < D)
                                    *reinterpret_cast<uint4*>(out + c + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    } else {
                        float* out = P.part_o + prow * DP + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (c + i < D)
                                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + i), SV_W8(o, i)
                                             : "memory");
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
    }
}

// ---------------------------------------------------------------------------------------------------------
// loads, products, value tiles: one warp each (value tiles: two)
// ---------------------------------------------------------------------------------------------------------
// Keys (kv 0) or values (kv 1).
template <int NH>
__device__ __forceinline__ void load_role(const Params& P, Shared& sh, uint32_t smem, const CUtensorMap* map, int kv) {
    const int lane = threadIdx.x & 31;
    const int32_t box = P.box, boxes = kTile / box, ps = P.a.pool.page_size;
    const uint32_t full = smem_u32(kv ? sh.v_full : sh.k_full), empty = smem_u32(kv ? sh.v_empty : sh.k_empty);
    const uint32_t slots = kv ? P.v_slots : P.k_slots;
    const bool leader = elect();
    volatile int* gave_up = &sh.gave_up;
    uint32_t tile = 0;
    Ring ring;
    bool ok = true;
    Items walk(sh);
    Item it;
#pragma unroll 1
    while (ok && walk.next(it)) {
        const int32_t* table = P.a.pool.table + (int64_t)it.b * P.a.pool.table_stride;
        // where a lane's box of a tile lies; read a tile ahead
        auto look = [&](int32_t j, bool& need, int32_t& page, int32_t& at) {
            const int32_t slot = (it.tile + j) * kTile + lane * box;
            need = j < it.n && lane < boxes && slot < it.end && slot + box > it.lo;
            page = -1;
            at = 0;
            if (need) {
                const int32_t i = slot / ps;
                at = slot - i * ps;
                page = table[i];
            }
        };
        bool next_need;
        int32_t next_page, next_at;
        look(0, next_need, next_page, next_at);
#pragma unroll 1
        for (int32_t j = 0; j < it.n; ++j, ++tile, ring.step(slots)) {
            bool need = next_need;
            const int32_t page = next_page, at = next_at;
            look(j + 1, next_need, next_page, next_at);
            if (tile >= slots && !wait(empty + 8 * ring.i, ring.parity ^ 1, gave_up)) {
                ok = false;
                break;
            }
            const bool miss = need && (page < 0 || page >= P.a.pool.pages);
            need = need && !miss;
            const uint32_t bytes = __popc(__ballot_sync(kAll, need)) * box * 128 * NH;
            uint32_t bad = 0;
            if (__any_sync(kAll, miss)) {
                if (miss) {
                    report(P.a.status, 1u << SV_ERR_BAD_OFFSETS);
                    bad = ((1u << (box / 8)) - 1u) << (lane * (box / 8));
                }
                bad = __reduce_or_sync(kAll, bad);
            }
            const uint32_t bar = full + 8 * ring.i;
            if (lane == 0) {
                sh.bad[kv][tile % kBadRing] = bad;
                bar_expect(bar, bytes);
            }
            __syncwarp();
            const uint32_t dst = smem + ring.i * (NH * kHalf), todo = __ballot_sync(kAll, need);
            const int32_t head = __shfl_sync(kAll, it.h, 0);
#pragma unroll 1
            for (int i = 0; i < boxes; ++i) {  // one thread issues: from many, each copy would wait for the last
                const int32_t p = __shfl_sync(kAll, page, i), a = __shfl_sync(kAll, at, i);
                if (leader && (todo >> i & 1u)) {
#pragma unroll
                    for (int h = 0; h < NH; ++h) copy_box(dst + i * box * 128 + h * kHalf, map, h * 64, a, head, p, bar);
                }
            }
            __syncwarp();
        }
    }
    // copies still under way land before the CTA ends, also where another role gave up
#pragma unroll 1
    for (uint32_t i = tile > slots ? tile - slots : 0; i < tile; ++i) {
        int none = 0;
        wait(full + 8 * (i % slots), (i / slots) & 1, &none);
    }
}

// A stream's products, by one thread: S = Q K^T of its next tile follows O += P V of this one, whose P lies where that
// S will. Tiles of the other stream's alone are passed on. The streams take turns, each turn both products: left to
// themselves they fall into step, both at their products and then both at their exponentials (measured: 4200 cycles
// a tile of 256 rows).
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
                   pv_done = smem_u32(&sh.pv_done[st]), q_empty = smem_u32(&sh.q_empty);
    const bool leader = elect();
    volatile int* gave_up = &sh.gave_up;
    const uint32_t turn[2] = {smem_u32(&sh.turn[st]), smem_u32(&sh.turn[st ^ 1])};
    uint32_t items = 0, p_parity = 0, turns = 0;
    Ring kr, vr;
    Items walk(sh);
    Item it;
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(it)) {
        if (!(ok = wait(smem_u32(&sh.q_full), items & 1, gave_up))) break;
        tc_after();
        // the same in every lane; taken from one, so that the operands below live in uniform registers
        const bool two = __shfl_sync(kAll, it.two, 0);
        const int32_t n = __shfl_sync(kAll, it.n, 0);
        const uint32_t q = operand(q_smem + (two && st ? q_bytes : 0), 16);
        // this stream's tiles are first, first + by, ...; k_at and v_at: the next tile of either kind
        const int32_t first = two ? 0 : (int32_t)st, by = two ? 1 : 2;
        int32_t k_at = 0, v_at = 0;
        auto pass = [&](int32_t to, int32_t& at, Ring& r, uint32_t full, uint32_t empty, uint32_t slots) {
            for (; at < to; ++at, r.step(slots)) {
                if (!wait(full + 8 * r.i, r.parity, gave_up)) return false;
                if (leader) bar_arrive(empty + 8 * r.i);
            }
            return true;
        };
        auto ready = [&](int32_t t) {  // the tile's keys
            return pass(t, k_at, kr, k_full, k_empty, P.k_slots) && wait(k_full + 8 * kr.i, kr.parity, gave_up);
        };
        auto scores = [&](int32_t t) {
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
                if (t + by >= n) tc_commit(q_empty);
            }
            __syncwarp();
            ++k_at;
            kr.step(P.k_slots);
        };
        auto idle = [&](bool last) {  // a turn without work
            if (!wait(turn[0], turns, gave_up)) return false;
            turns ^= 1u;
            if (leader) {
                bar_arrive(turn[1]);
                if (last) bar_arrive(q_empty);
            }
            return true;
        };
        if (first < n) {
            if (!(ok = ready(first) && wait(turn[0], turns, gave_up))) break;
            turns ^= 1u;
            scores(first);
        } else if (!(ok = idle(true))) {
            break;
        }
        const int32_t rounds = two ? n : (n + 1) / 2;
#pragma unroll 1
        for (int32_t k = 0; k < rounds; ++k) {
            const int32_t t = first + k * by;
            if (t >= n) {
                ok = idle(false);
                break;  // only ever the last round
            }
            const bool more = t + by < n;
            if (!(ok = pass(t, v_at, vr, value, v_empty, P.v_slots) && wait(value + 8 * vr.i, vr.parity, gave_up))) break;
            if (more && !(ok = ready(t + by))) break;
            if (!(ok = wait(p_ready, p_parity, gave_up))) break;
            p_parity ^= 1u;
            if (!(ok = wait(turn[0], turns, gave_up))) break;
            turns ^= 1u;
            tc_after();
            const uint32_t b = operand(v_smem + vr.i * slot_bytes, kHalf);
            const uint32_t add = t > first;
            if (leader) {
#pragma unroll
                for (int i = 0; i < kTile / KindOf<K>::kStep; ++i)
#pragma unroll
                    for (int part = 0; part < parts; ++part)
                        mma_ts<k8>(o_at, s_at + (k8 ? part * 8 + i * 16 : i * 8), b + (i * KindOf<K>::kStep * 128 >> 4), id_o,
                                   part + i > 0 ? 1u : add);
                if (!more) bar_arrive(turn[1]);
                tc_commit(pv_done);
                tc_commit(v_empty + 8 * vr.i);
            }
            __syncwarp();
            ++v_at;
            vr.step(P.v_slots);
            if (more) scores(t + by);
        }
        if (ok) ok = pass(n, k_at, kr, k_full, k_empty, P.k_slots) && pass(n, v_at, vr, value, v_empty, P.v_slots);
        ++items;
    }
    // products under way end before the tensor memory is given back
    if (leader) tc_commit(smem_u32(&sh.drain));
    __syncwarp();
    int none = 0;
    wait(smem_u32(&sh.drain), 0, &none);
}

// The rows of an item's query tiles. 16-bit caches: copied, G heads of q_box tokens at once (rows past the
// sequence's end are another sequence's, or zero: a product's row depends on its own row only). e4m3: split
// into the parts hi and lo, each row brought to [128, 256) by a power of two.
template <int K, int NH>
__device__ __forceinline__ bool load_queries(const Params& P, Shared& sh, const Item& it, uint32_t q_smem,
                                             const CUtensorMap* qm, uint32_t items) {
    using T = typename KindOf<K>::T;
    const AttendArgs& A = P.a;
    const int lane = threadIdx.x & 31;
    const uint32_t q_full = smem_u32(&sh.q_full);
    bool flip;
    score_unit(A, it.h, flip);
    if (K != kE4m3) {
        const uint32_t bar = flip ? smem_u32(&sh.q_in) : q_full;
        if (lane == 0) {
            bar_expect(bar, (it.two ? 2 : 1) * NH * P.q_box * P.G * 128);
            for (int t = 0; t < (it.two ? 2 : 1); ++t)
#pragma unroll
                for (int h = 0; h < NH; ++h)
                    copy_queries(q_smem + (t * NH + h) * kHalf, qm, h * 64, it.h * P.G, it.row0 + it.t0 + t * P.tokens, bar);
        }
        __syncwarp();
        if (!flip) return true;
        if (!wait(bar, items & 1, &sh.gave_up)) return false;
#pragma unroll 1
        for (int i = lane; i < (it.two ? 2 : 1) * NH * kHalf / 16; i += 32) {
            uint32_t u[4];
            const uint32_t at = q_smem + i * 16;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at));
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(u[0] ^ 0x80008000u), "r"(u[1] ^ 0x80008000u),
                         "r"(u[2] ^ 0x80008000u), "r"(u[3] ^ 0x80008000u)
                         : "memory");
        }
    } else {
        const int32_t D = A.pool.dim, rows = it.nt * P.G, tile_rows = P.tokens * P.G;
        const T* q = (const T*)A.q + (int64_t)(it.row0 + it.t0) * A.q_stride + (int64_t)it.h * P.G * D;
        // half a warp a row, eight elements a lane; eight rows under way
        const int c = lane & 15;
#pragma unroll 1
        for (int32_t r0 = lane >> 4; r0 - (lane >> 4) < rows; r0 += 8) {
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int32_t r = r0 + 2 * k;
                u[k] = make_uint4(0, 0, 0, 0);
                if (r < rows && c * 8 < D) {
                    const int32_t t = r / P.G, g = r - t * P.G;
                    u[k] = *reinterpret_cast<const uint4*>(q + t * A.q_stride + (int64_t)g * D + c * 8);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int32_t r = r0 + 2 * k;
                const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                float2 f[4];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = to_float2<T>(w[i]);
                    top = fmaxf(top, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
                }
                for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
                int e = 0;
                if (top > 0.f && top < INFINITY) e = max(-120, min(120, 7 - ilogbf(top)));
                const float up = __int_as_float((127 + e) << 23);
                uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // an infinite query has no finite parts: its row is NaN, as its softmax is
                    const float x = isinf(f[i].x) ? NAN : flip ? -f[i].x * up : f[i].x * up;
                    const float y = isinf(f[i].y) ? NAN : flip ? -f[i].y * up : f[i].y * up;
                    const uint32_t a = e4m3x2(x, y);
                    const float2 b = from_e4m3x2(a);
                    hi[i >> 1] |= a << (16 * (i & 1));
                    lo[i >> 1] |= e4m3x2(x - b.x, y - b.y) << (16 * (i & 1));
                }
                if (r < rows) {
                    const int32_t at = r < tile_rows ? r : r - tile_rows;
                    const uint32_t dst = q_smem + (r < tile_rows ? 0 : 2 * kHalf) + at * 128 +
                                         (((c >> 1) ^ (at & 7)) << 4) + (c & 1) * 8;
                    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(dst), "r"(hi[0]), "r"(hi[1]) : "memory");
                    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(dst + kHalf), "r"(lo[0]), "r"(lo[1]) : "memory");
                    if (c == 0)
                        sh.q_down[(items & 1) * 2 * kTile + (r < tile_rows ? 0 : kTile) + at] = __int_as_float((127 - e) << 23);
                }
            }
        }
    }
    fence_async();
    __syncwarp();
    if (lane == 0) bar_arrive(q_full);
    return true;
}

// Rows [lo, hi) of a value tile set to zero. A whole row is the same 128 bytes under any swizzle.
template <int NH>
__device__ __forceinline__ void clear_rows(uint32_t at, int32_t lo, int32_t hi) {
    lo = max(lo, 0);
    hi = min(hi, kTile);
#pragma unroll 2
    for (int32_t i = lo * 8 + (threadIdx.x & 31); i < hi * 8; i += 32)
#pragma unroll
        for (int h = 0; h < NH; ++h)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at + h * kHalf + i * 16), "r"(0) : "memory");
}

// Non-finite elements of rows [lo, hi): cleared, and their rows noted.
template <int K, int NH>
__device__ __forceinline__ void scan_rows(uint32_t at, int32_t lo, int32_t hi, uint32_t bad, uint32_t* odd) {
    constexpr int bits = K == kE4m3 ? 8 : 16;
    constexpr uint32_t unit = K == kE4m3 ? 0x01010101u : 0x00010001u;
    constexpr uint32_t top = unit * (K == kE4m3 ? 0x7fu : K == kBf16 ? 0x7f80u : 0x7c00u), high = unit << (bits - 1);
#pragma unroll 4
    for (int32_t i = lo * 8 + (threadIdx.x & 31); i < hi * 8; i += 32)
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const uint32_t a = at + h * kHalf + i * 16;
            uint32_t u[4], any = 0;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(a));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t t = ~u[e] & top;  // an element of zeros: its exponent is all ones
                any |= (t - unit) & ~t & high;
            }
            if (any && !(bad >> (i >> 6) & 1u)) {
                bool found = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int by = 0; by < 32; by += bits) {
                        constexpr uint32_t one = (1u << bits) - 1u;
                        if ((u[e] >> by & top & one) == (top & one)) {
                            u[e] &= ~(one << by);
                            found = true;
                        }
                    }
                if (found) {
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
                                 : "memory");
                    atomicOr(&odd[i >> 8], 1u << (i >> 3 & 31));
                }
            }
        }
}

// Queries, and value tiles before they are multiplied: rows of slots that no row of the item sees are cleared
// (they may hold anything, and a weight of zero times NaN is NaN), and so are single non-finite values that only
// some rows see; those are noted for the rows that do.
template <int K, int NH>
__device__ __forceinline__ void value_role(const Params& P, Shared& sh, uint32_t q_smem, uint32_t v_smem,
                                           const CUtensorMap* qm) {
    const int lane = threadIdx.x & 31;
    volatile int* gave_up = &sh.gave_up;
    uint32_t v = 0, items = 0;
    Ring ring;
    Items walk(sh);
    Item it;
#pragma unroll 1
    for (; walk.next(it); ++items) {
        if (items > 0 && !wait(smem_u32(&sh.q_empty), (items - 1) & 1, gave_up)) return;
        if (!load_queries<K, NH>(P, sh, it, q_smem, qm, items)) return;
#pragma unroll 1
        for (int32_t j = 0; j < it.n; ++j, ++v, ring.step(P.v_slots)) {
            if (!wait(smem_u32(&sh.v_full[ring.i]), ring.parity, gave_up)) return;
            const int32_t k0 = (it.tile + j) * kTile;
            const uint32_t bad = sh.bad[1][v % kBadRing];
            const bool mixed = mixed_tile(it, k0);
            if (bad || k0 < it.lo || k0 + kTile > it.end || mixed) {
                const uint32_t at = v_smem + ring.i * (NH * kHalf);
                // rows no one sees lie before the first and after the last one that is seen
                clear_rows<NH>(at, 0, it.lo - k0);
                clear_rows<NH>(at, it.end - k0, kTile);
                if (bad)
#pragma unroll 1
                    for (int g = 0; g < 16; ++g)
                        if (bad >> g & 1u) clear_rows<NH>(at, 8 * g, 8 * g + 8);
                if (mixed) {
                    if (lane < 4) sh.odd[v % kBadRing][lane] = 0;
                    __syncwarp();
                    const int32_t lo = max(0, it.lo - k0), hi = min(kTile, it.end - k0);
                    scan_rows<K, NH>(at, lo, min(hi, it.mixed_lo - k0), bad, sh.odd[v % kBadRing]);
                    scan_rows<K, NH>(at, max(lo, it.mixed_hi - k0), hi, bad, sh.odd[v % kBadRing]);
                }
                fence_async();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(smem_u32(&sh.value[ring.i]));
        }
    }
}

template <int K, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
             const __grid_constant__ CUtensorMap qm) {
    constexpr int NH = K == kE4m3 ? 1 : DP / 64;
    extern __shared__ __align__(1024) char raw[];
    const uint32_t q_smem = smem_u32(raw), k_smem = q_smem + P.q_tiles * (K == kE4m3 ? 2 : NH) * kHalf,
                   v_smem = k_smem + P.k_slots * NH * kHalf;
    Shared& sh = *reinterpret_cast<Shared*>(raw + (v_smem - q_smem) + P.v_slots * NH * kHalf);
    if (q_smem & 1023u) {  // the tiles' swizzle counts on it
        if (threadIdx.x == 0) report(P.a.status, 1u << SV_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, w = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            bar_init(smem_u32(&sh.k_full[i]), 1);
            bar_init(smem_u32(&sh.k_empty[i]), 2);
            bar_init(smem_u32(&sh.v_full[i]), 1);
            bar_init(smem_u32(&sh.v_empty[i]), 2);
            bar_init(smem_u32(&sh.value[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_u32(&sh.s_full[i]), 1);
            bar_init(smem_u32(&sh.p_ready[i]), 4);
            bar_init(smem_u32(&sh.pv_done[i]), 1);
            bar_init(smem_u32(&sh.turn[i]), 1);
        }
        bar_init(smem_u32(&sh.q_in), 1);
        bar_init(smem_u32(&sh.q_full), 1);
        bar_init(smem_u32(&sh.q_empty), 2);
        bar_init(smem_u32(&sh.meet), 8);
        bar_init(smem_u32(&sh.part), 8);
        bar_init(smem_u32(&sh.drain), 2);
        for (int i = 0; i < kItems; ++i) {
            bar_init(smem_u32(&sh.item_full[i]), 1);
            bar_init(smem_u32(&sh.item_empty[i]), kItemReaders);
        }
        sh.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        bar_arrive(smem_u32(&sh.turn[0]));
    }
    if (w == 8 && (tid & 31) == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&km));
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vm));
        if (K != kE4m3) asm volatile("prefetch.tensormap [%0];" ::"l"(&qm));
    }
    if (w == 9)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    // what is above may run while the stream's previous kernel ends
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    plan(P, sh);
    if (blockIdx.x == 0 && tid == 0) {
        const int64_t end = (int64_t)P.a.chunk.offs[P.a.chunk.B] + P.a.chunk.B;
        if (end > P.a.chunk.rows || P.a.chunk.offs[0] != 0) report(P.a.status, 1u << SV_ERR_BAD_OFFSETS);
    }
    tc_before();
    __syncthreads();
    tc_after();
    // sequences that fail: their findings, and zeros in their rows
    if (sh.failing)
#pragma unroll 1
        for (int32_t b = blockIdx.x; b < P.a.chunk.B; b += gridDim.x) {
            const Seq s = checked_seq(P, b);
            if (!s.err) continue;
            if (tid == 0) report(P.a.status, s.err);
            if (!s.rows_ok) continue;
            const int64_t row = (int64_t)P.a.q_heads * P.a.pool.dim / 8;
            uint4* out = (uint4*)P.a.out + s.row0 * row;
#pragma unroll 1
            for (int64_t i = tid; i < s.T * row; i += kThreads) out[i] = make_uint4(0, 0, 0, 0);
            if (P.a.lse)
#pragma unroll 1
                for (int64_t i = tid; i < (int64_t)s.T * P.a.q_heads; i += kThreads)
                    P.a.lse[(int64_t)s.row0 * P.a.q_heads + i] = -INFINITY;
        }
    // 128 registers a thread at launch: 192 + 192 + 64 + 64 for the four warpgroups
    if (w < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        softmax_role<K, DP>(P, sh);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (w == 8 || w == 10) load_role<NH>(P, sh, w == 8 ? k_smem : v_smem, w == 8 ? &km : &vm, w == 10);
        else if (w == 9 || w == 13) product_role<K, NH>(P, sh, q_smem, k_smem, v_smem, w == 13);
        else if (w == 11) value_role<K, NH>(P, sh, q_smem, v_smem, &qm);
        else if (w == 12) item_role(P, sh);
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
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t c = blockIdx.x + 1;
    const Record rec = P.records[c];
    if (!rec.parts) return;
    const int lane = threadIdx.x & 31;
    const int32_t D = P.a.pool.dim, rows = rec.tokens * P.G;
    constexpr int kPer = DP / 32;
#pragma unroll 1
    for (int32_t i = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5); i < rows;
         i += gridDim.y * (kMergeThreads / 32)) {
        const int32_t t = i / P.G, g = i - t * P.G;
        const int32_t r = t < P.tokens ? i : kTile + i - P.tokens * P.G;
        // the first part is the last item of CTA c - 1, the others the first items of c, c + 1, ...
        auto slot = [&](int32_t part) { return (size_t)(part ? 2 * (c + part - 1) : 2 * (c - 1) + 1) * 256 + r; };
        float top = -INFINITY;
#pragma unroll 1
        for (int32_t p = lane; p < rec.parts; p += 32) top = fmaxf(top, P.part_ml[slot(p)].x);
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        const float base = top == -INFINITY ? 0.f : top;
        float l = 0.f, acc[kPer] = {};
#pragma unroll 1
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

// Queries as (dim, head, row), copied in boxes of 128 bytes by the heads of a group by q_box rows.
bool encode_queries(CUtensorMap* m, const AttendArgs& A, int kind, int G, int q_box) {
    const cuuint64_t dims[3] = {(cuuint64_t)A.pool.dim, (cuuint64_t)A.q_heads, (cuuint64_t)A.chunk.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)A.pool.dim * 2, (cuuint64_t)A.q_stride * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)G, (cuuint32_t)q_box}, ones[3] = {1, 1, 1};
    return encoder()(m, kind == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(A.q), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
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
    P.q_box = min(P.tokens, A.chunk.max_gamma + 1);
    const int slots = min(2 * kMaxSlots, (kSmem - shared_bytes<K>() - P.q_tiles * q_bytes) / (NH * kHalf));
    P.k_slots = slots / 2;
    P.v_slots = slots - P.k_slots;
    P.box = kTile;
    while (A.pool.page_size % P.box) P.box /= 2;
    P.wide = A.pool.dim % 16 == 0 && (uintptr_t)A.out % 32 == 0;
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
    CUtensorMap km, vm, qm;
    if (K != kE4m3 && !encode_queries(&qm, A, K, P.G, P.q_box)) return cudaErrorInvalidValue;
    if (!encode(&km, A.pool, A.pool.k, KindOf<K>::kBytes, K, P.box) || !encode(&vm, A.pool, A.pool.v, KindOf<K>::kBytes, K, P.box))
        return cudaErrorInvalidValue;
    const int smem = P.q_tiles * q_bytes + slots * NH * kHalf + shared_bytes<K>();
    static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use all shared memory
    if (dev >= 64 || !(allowed.load() >> dev & 1u)) {
        e = cudaFuncSetAttribute(k_attend<K, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed.fetch_or((uint64_t)1 << dev);
    }
    // both launches may begin before the one ahead of them has ended; they wait for it where they need it
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_attend<K, DP>, P, km, vm, qm);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(n - 1, 4);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
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
