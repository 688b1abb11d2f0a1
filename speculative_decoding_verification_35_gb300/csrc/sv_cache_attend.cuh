// Shared by the attention kernels of spec_cache_attend (sv_cache_attend_wide.cuh: up to 256 rows a work item,
// sv_cache_attend_few.cuh: up to 64): how the work is numbered and shared out, the warps that load and clean, and
// the PTX beneath. The heads of the two files say why they are made as they are.
#pragma once
#include <cuda.h>

#include <atomic>

#include "sv_cache.cuh"

namespace sv {
namespace cache {

constexpr int kTile = 128;      // slots of a tile
constexpr int kMaxSlots = 6;    // key tiles in flight, and value tiles
constexpr int kNotes = 8;       // tiles whose notes (bad pages, non-finite values) are kept: as many as are in flight,
                                // with those whose scores run ahead
constexpr int kItems = 3;       // items that are known ahead
constexpr int kMaxCtas = 320;   // of any launch
constexpr int kHalf = kTile * 128;  // bytes of 128 rows of 128 bytes, the unit of an operand in shared memory
constexpr int kSmem = 227 * 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xffffffffu;

// What is rarely so: its code is put aside, so that what runs lies closer together in the instruction cache.
__device__ __forceinline__ bool rarely(bool x) { return __builtin_expect(x, 0); }

// ---------------------------------------------------------------------------------------------------------
// element kinds
// ---------------------------------------------------------------------------------------------------------
// kShift: weights are held as 2^kShift w, so that those far below the largest keep their precision in a narrow
// type; kSlack: how far (log2) a weight may exceed the reference before the reference moves. A tile's 128 weights
// sum to 2^(kShift + kSlack + 7) at most, within the type's range: bfloat16 has float's, and its reference hardly
// ever moves after the first tile. (e4m3: every weight, 2^(kShift + kSlack) <= 448.)
// Weights of 16-bit caches are rounded to the values' type, because a product's two operands share one. What that leaves
// off could be a second operand, as it is for e4m3, but would cost half of the tensor cores' work again in the wide
// kernel, which they bound together with the softmax, and in the other one of three tile slots (its weights' tile
// would take 8 KB more where 16 bytes are free). Sums and lse have the weights unrounded.
// kE4m3: the cache is 8 bits wide and the products are too. A bfloat16 query has 8 significant bits and an
// e4m3 value 4, so q 2^k = hi + lo exactly, but for elements under 2^-9 of the row's largest (k brings it to
// [128, 256)), which are off by 2^-10 at most, e4m3's least half step; a weight is hi + lo to about 2^-9 of itself. Each
// product then runs twice, at twice the 16-bit rate, and no key or value is converted.
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
    int32_t tokens, head, split;
    int32_t pad[3];
};

struct Params {
    AttendArgs a;
    int32_t G;          // query heads per key head
    int32_t block;      // tokens of an item
    int32_t tokens;     // tokens of a query tile; an item with more has two tiles
    int32_t q_box;      // tokens of one copy into a query tile
    int32_t halves;     // 128-byte columns of a row of keys, values and 16-bit queries: 1 or 2
    int32_t q_part;     // bytes from a query tile's hi part to its lo part (e4m3)
    int32_t q_tile;     // bytes from a query tile to the next
    int32_t q_bytes, q_bufs;  // of an item's query tiles; how many items' there is room for, 1 or 2
    int32_t k_slots, v_slots;  // key and value tiles that shared memory has room for
    int32_t box, boxes; // slots of one copy, a divisor of the page size and of kTile; copies of a tile
    int32_t tile_pages, tile_rest;  // kTile in whole pages, and the slots left over
    int32_t wide;       // output rows lie on 32 bytes
    int32_t ctas;       // of the launch
    int32_t part_rows;  // rows of a partial result
    int32_t lead;       // what an item's beginning and end cost, in tiles
    uint32_t polls;     // of a wait, before it gives up
    float* part_o;      // [2 n][part_rows][64 or 128]
    float2* part_ml;    // [2 n][part_rows]
    Record* records;    // [n]
};

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
// True once the phase is over; sleeps for it, 4 us at most (measured, with and without a hint of another time).
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok;
}
// A whole warp waits, a second at most; false, and the CTA gives up, if that was not enough. (Short, as it stands in some
// thirty places: the limit is read only where the first look was in vain.)
constexpr uint32_t kPolls = 1u << 18;
struct Limit {
    volatile int* gave_up;
    uint32_t polls;  // kPolls, but for tests
};
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Limit limit) {
    uint32_t i = 0;
#pragma unroll 1
    do
        if (__all_sync(kAll, bar_try(bar, parity))) return true;
    while (++i < limit.polls);
    *limit.gave_up = 1;
    return false;
}
// What is under way in any case, copies and products, before the CTA ends: nothing is left to give up.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    int none;
    wait(bar, parity, Limit{&none, kPolls});
}
// Whether the phase is over, for a whole warp.
__device__ __forceinline__ bool ready(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return __all_sync(kAll, ok);
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
__device__ __forceinline__ void tc_ld4(uint32_t col, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(col));
}
__device__ __forceinline__ void tc_st4(uint32_t col, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(col), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
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
// As mma_ss, with a second operand of another swizzle and row pitch.
#define SV_MMA_MIXED(kind)                                                                                          \
    "{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.u32 p, %4, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %6};\n"      \
    "tcgen05.mma.cta_group::1.kind::" kind " [%0], x, y, %3, p;\n}"
template <bool k8, uint32_t kHigh>
__device__ __forceinline__ void mma_mixed(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    if (k8)
        asm volatile(SV_MMA_MIXED("f8f6f4") ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh), "n"(kHigh)
                     : "memory");
    else
        asm volatile(SV_MMA_MIXED("f16") ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh), "n"(kHigh)
                     : "memory");
}
// The lowest n bits.
__device__ __forceinline__ uint32_t prefix32(int32_t n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
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
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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
    int32_t split;                // of these in the first query tile
    int32_t past;
    int32_t lo, end;              // the slots [lo, end) that some row of it sees
    int32_t tile, n;              // the CTA's tiles: the first (absolute), how many; 0: no more items
    int32_t mixed_lo, mixed_hi;   // slots below mixed_lo and from mixed_hi on are seen by some of its rows only
    int32_t begins, finishes;     // its first and last tiles are among the CTA's
    int32_t reach;                // kScored: the slots before it are seen by every token
};

template <bool kScored>
__device__ __forceinline__ void span(const Params& P, int32_t b, int32_t T, int32_t past, int32_t p, Item& it, int32_t& first,
                                     int32_t& count) {
    it.t0 = p * P.block;
    it.nt = min(P.block, T - it.t0);
    it.split = P.tokens == P.block ? it.nt : it.nt > P.tokens ? P.tokens : (it.nt + 1) / 2;
    it.past = past;
    it.end = past + it.t0 + it.nt;
    it.reach = 0;
    if (kScored && P.a.prefix) {
        it.reach = max(0, min(P.a.prefix[b], past + T));
        it.end = max(it.end, it.reach);
    }
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
#pragma unroll 8
    for (int j = 1; j < T; ++j) ok &= (uint32_t)par[j - 1] < (uint32_t)j;
    return ok;
}

__device__ __forceinline__ Seq checked_seq(const Params& P, int32_t b) {
    Seq s = seq_of(P.a.chunk, capacity_of(P.a.pool), b);
    if (!s.err && P.a.chunk.parents && !tree_ok(P.a.chunk, b, s.T)) s.err = 1u << SV_ERR_BAD_OFFSETS;
    return s;
}

// The CTA's j-th tile of an item. Where scores fall with the distance the last tiles come first: from the first to the last a
// row's reference would move at every tile (measured, 32 rows of 4001 slots: 159 us, and 75 backwards).
template <bool kScored>
__device__ __forceinline__ int32_t tile_at(const Params& P, const Item& it, int32_t j) {
    return kScored && P.a.slopes ? it.tile + it.n - 1 - j : it.tile + j;
}

// Tiles and items of a sequence, for one key head.
template <bool kScored>
__device__ __forceinline__ void size_of(const Params& P, int32_t b, const Seq& s, uint32_t& tiles, uint32_t& blocks) {
    tiles = blocks = 0;
    if (s.err) return;
#pragma unroll 1
    for (int32_t p = 0; p * P.block < s.T; ++p) {
        Item it;
        int32_t first, count;
        span<kScored>(P, b, s.T, s.past, p, it, first, count);
        if (tiles >> 31 == 0) tiles += count;  // more are refused, so they need not be counted
        ++blocks;
    }
}

// Where a CTA begins. An item is `lead` units of beginning and ending (its queries' way in, its outputs' way
// out, and the pipeline's filling in between) and a unit a tile; x counts them.
struct Start {
    int32_t b, p, h, T, past, row0;
    int32_t lead, x, left;
    uint32_t W, n, u0;  // units in all, CTAs that have some, and this CTA's first
};

// A tree's nodes: what each sees (bits: itself and those above it, as far as the window reaches), and its depth.
struct Tree {
    uint32_t above[32];
    int32_t depth[32];
};

struct Common {  // of both kernels, behind the operand tiles
    uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
    uint64_t value[kMaxSlots];  // a value tile is in and clean
    uint64_t q_in, q_full[2], q_empty[2], drain;
    uint64_t item_full[kItems], item_empty[kItems];
    Item item[kItems];
    uint32_t tmem;
    int gave_up;
    int failing;  // some sequence of this CTA's share has a finding
    Start start;
    uint32_t bad[2][kNotes];    // per key and per value tile: groups of 8 slots that lie on a bad page
    uint32_t odd[kNotes][4];    // per value tile: slots with a non-finite value that was cleared
    uint32_t scan[2][16];
    float* q_down;  // e4m3 caches: [kItems][q_rows], what a row's scores are scaled by
    Tree* tree;     // trees: [kItems]
    int32_t q_rows;
};

// a b / c, rounded down, without the long division: a = q c + r gives q b + r b / c. b and c below 2^15.
__device__ __forceinline__ uint32_t share(uint32_t a, uint32_t b, uint32_t c) { return a / c * b + a % c * b / c; }

// Where the CTA begins: by all threads, in the end by one,
// whose sequence b it is, `rest` units into it.
template <bool kScored>
__device__ __forceinline__ void begin_at(const Params& P, Common& sh, const Seq& s, int32_t b, uint32_t rest, uint32_t lead,
                                         uint32_t W, uint32_t n, uint32_t u0, uint32_t u1) {
    const uint32_t heads = P.a.pool.heads;
    Item it;
    int32_t first, count, p = 0;
#pragma unroll 1
    for (;; ++p) {
        span<kScored>(P, b, s.T, s.past, p, it, first, count);
        const uint32_t all = (count + lead) * heads;
        if (rest < all) break;
        rest -= all;
    }
    const uint32_t h = rest / (count + lead), x = rest - h * (count + lead);
    sh.start = {b, p, (int32_t)h, s.T, s.past, s.row0, (int32_t)lead, (int32_t)x, (int32_t)(u1 - u0), W, n, u0};
    // its page ids on their way here
    const int32_t slot = (first + (x > lead ? (int32_t)(x - lead) : 0)) * kTile;
    asm volatile("prefetch.global.L1 [%0];" ::"l"(P.a.pool.table + (int64_t)b * P.a.pool.table_stride +
                                                  min(slot / P.a.pool.page_size, P.a.pool.table_stride - 1)));
}

// The record of the item that the CTA begins in, if it is the second one to work on it. Late, by one thread: only the
// merge needs it.
template <bool kScored>
__device__ __forceinline__ void record(const Params& P, const Common& sh) {
    const Start& s = sh.start;
    const uint32_t c = blockIdx.x;
    if (s.left == 0 || s.x <= s.lead) return;
    Item it;
    int32_t first, count;
    span<kScored>(P, s.b, s.T, s.past, s.p, it, first, count);
    // the item's first tile is unit `from`; if the CTA before this one had it, this one records the item
    const uint32_t from = s.u0 - s.x + s.lead;
    if (from < share(s.W, c - 1, s.n)) return;
    uint32_t lo = c, hi = s.n - 1;  // the CTA of its last tile
#pragma unroll 1
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) / 2;
        if (share(s.W, mid, s.n) <= from + count - 1) lo = mid;
        else hi = mid - 1;
    }
    Record r{};
    r.parts = (int32_t)(lo - c) + 2;
    r.row0 = s.row0 + it.t0;
    r.tokens = it.nt;
    r.head = s.h;
    r.split = it.split;
    P.records[c] = r;
}

template <int kThreads, bool kScored>
__device__ __forceinline__ void plan(const Params& P, Common& sh) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int32_t B = P.a.chunk.B, c = (int32_t)blockIdx.x;
    const uint32_t heads = P.a.pool.heads;
    if (tid == 0) {
        sh.start.left = 0;
        sh.failing = 0;
        if (c > 0) P.records[c].parts = 0;
    }
    // Twice over the sequences, kThreads at a time: their sums, then the one that the CTA begins in. (As two rounds of
    // one loop: the code runs once a launch and is fetched from afar.)
    const int used = (min(kThreads, B) + 31) / 32;  // warps that have sequences
    Seq mine{};
    uint32_t my_tiles = 0, my_blocks = 0, lead = 0, W = 0, n = 0, u0 = 0, u1 = 0, base = 0;
    unsigned long long tiles = 0, blocks = 0;
    bool fails = false;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
#pragma unroll 1
        for (int32_t b0 = 0; b0 < B && base <= u0; b0 += kThreads) {
            const int32_t b = b0 + tid;
            if (round == 0 || B > kThreads) {
                my_tiles = my_blocks = 0;
                uint32_t* wrong = &sh.odd[0][0];  // bits: trees of this turn that are none
                if (P.a.chunk.parents) {
                    static_assert(kThreads / 32 <= kNotes * 4, "a word a warp");
                    if (b0 > 0) __syncthreads();  // the last turn's have been read
                    if (tid < kThreads / 32) wrong[tid] = 0;
                    __syncthreads();
#pragma unroll 1
                    for (int i = w; i < min(kThreads, B - b0); i += kThreads / 32) {  // a warp a tree
                        const Seq s = seq_of(P.a.chunk, capacity_of(P.a.pool), b0 + i);
                        int32_t par = 0;
                        if (!s.err && lane > 0 && lane < s.T) par = P.a.chunk.parents[s.row0 - (b0 + i) + lane - 1];
                        const bool ok = __all_sync(kAll, (uint32_t)par < (uint32_t)max(lane, 1));
                        if (!ok && lane == 0) atomicOr(&wrong[i >> 5], 1u << (i & 31));
                    }
                    __syncthreads();
                }
                if (b < B) {
                    mine = seq_of(P.a.chunk, capacity_of(P.a.pool), b);
                    if (!mine.err && P.a.chunk.parents && (wrong[tid >> 5] >> (tid & 31) & 1u)) mine.err = 1u << SV_ERR_BAD_OFFSETS;
                    size_of<kScored>(P, b, mine, my_tiles, my_blocks);
                }
            }
            if (round == 0) {
                fails |= b < B && mine.err && b % gridDim.x == c;
                tiles += my_tiles;
                blocks += my_blocks;
                continue;
            }
            const uint32_t u = (my_tiles + lead * my_blocks) * heads;
            uint32_t incl = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += x;
            }
            if (B > kThreads) {  // else the warps' sums are there already
                __syncthreads();
                if (lane == 31) {
                    sh.scan[0][w] = incl;
                    sh.scan[1][w] = 0;
                }
                __syncthreads();
            }
            const uint32_t sc = B > kThreads ? 1 : heads, lc = B > kThreads ? 0 : lead * heads;
            uint32_t before = base, total = 0;
#pragma unroll 4
            for (int i = 0; i < used; ++i) {
                const uint32_t x = sh.scan[0][i] * sc + sh.scan[1][i] * lc;
                if (i < w) before += x;
                total += x;
            }
            const uint32_t first_unit = before + incl - u;
            if (u > 0 && u0 >= first_unit && u0 < first_unit + u) begin_at<kScored>(P, sh, mine, b, u0 - first_unit, lead, W, n, u0, u1);
            base += total;
        }
        if (round > 0) break;
        // over the warp, 16 bits and the rest: what is clamped there is far too large below
        auto sum = [](unsigned long long v) {
            return __reduce_add_sync(kAll, (uint32_t)v & 0xffffu) +
                   ((unsigned long long)__reduce_add_sync(kAll, (uint32_t)min(v >> 16, 0x3ffffffull)) << 16);
        };
        tiles = sum(tiles);
        blocks = sum(blocks);
        if (lane == 0) {  // a sum too large for 32 bits is kept as too large for what is allowed below
            sh.scan[0][w] = (uint32_t)min(tiles, 0xffffffffull);
            sh.scan[1][w] = (uint32_t)min(blocks, 0xffffffffull);
        }
        if (__syncthreads_or(fails) && tid == 0) sh.failing = 1;
        tiles = blocks = 0;
#pragma unroll 4
        for (int i = 0; i < used; ++i) {
            tiles += sh.scan[0][i];
            blocks += sh.scan[1][i];
        }
        tiles *= heads;
        blocks *= heads;
        // With few tiles there is a CTA for each, and an item's beginning is nobody's but its own.
        lead = tiles <= 2 * gridDim.x ? 0 : P.lead;
        if (tiles + lead * blocks >> 31) {
            if (c == 0 && tid == 0) report(P.a.status, 1u << SV_ERR_CAPACITY);
            return;
        }
        W = (uint32_t)(tiles + lead * blocks);
        n = min(gridDim.x, (uint32_t)tiles);
        if (c >= n) return;  // the same for the whole CTA
        u0 = share(W, c, n);
        u1 = share(W, c + 1, n);
    }
}

// A role's view of the items. An item (and its tree) stays until the role asks for the next one.
struct Items {
    Common& sh;
    const uint32_t polls;
    Ring ring;
    bool held = false;
    __device__ __forceinline__ Items(const Params& P, Common& s) : sh(s), polls(P.polls) {}
    __device__ __forceinline__ bool next(Item& it) {
        if (held) {
            __syncwarp();
            if ((threadIdx.x & 31) == 0) bar_arrive(smem_u32(&sh.item_empty[ring.i]));
            ring.step(kItems);
        }
        if (!wait(smem_u32(&sh.item_full[ring.i]), ring.parity, Limit{&sh.gave_up, polls})) return false;
        it = sh.item[ring.i];
        held = true;
        return it.n > 0;
    }
    __device__ __forceinline__ const Tree& tree() const { return sh.tree[ring.i]; }
};
// x or the least, NaN for NaN (where fmaxf returns the other).
__device__ __forceinline__ float at_least(float x, float least) { return x < least ? least : x; }
// Scores to log2 of the weights. A negative factor changes the queries' signs; one of zero is kept above it, so
// that -inf stays -inf. A NaN stays one: a head whose scale is NaN has no weights.
__device__ __forceinline__ float score_unit(const AttendArgs& A, int32_t h, bool& flip) {
    const float sl = A.scale * (A.pool.k_scale ? A.pool.k_scale[h] : 1.f) * kLog2e;
    flip = sl < 0.f;
    return at_least(fabsf(sl), 1e-30f);
}
// The same for a row whose queries were brought up by a power of two (e4m3): 2^-120 for a row of zeros, so that this
// product, too, is kept above zero.
__device__ __forceinline__ float row_unit(float unit, float down) { return at_least(unit * down, 1e-37f); }

// Capped scores, cap tanh(z / cap), from scores to log2 of the weights (cap log2e tanh(..)). With x = z / cap up to 1, where a
// model keeps most of them, tanh x = x q(x^2), q of degree 6 with q(0) = 1 fitted for the least relative error on [0, 1]
// (6.1e-8; 1.6e-7 with the roundings): nine packed operations for two scores and none of the special-function unit, which
// the weights keep busy. Past 1, 1 - 2 / (1 + 2^(2 x log2 e)): its error, some 2^-22 of one, is as small a part there.
struct Cap {
    F2 c[7], d[4];   // times cap log2e, the highest first; d is for x up to kSmall
    static constexpr float kSmall = 0.55f;
    float by;  // x = s by, for scores of unit 1
    float most;  // cap log2e
    __device__ __forceinline__ explicit Cap(float cap) {
        most = cap * kLog2e;
        by = kLn2 / cap;
        const float q[7] = {0.00105826119f, -0.00625932904f, 0.0203597479f, -0.0534987018f, 0.133264087f, -0.333329868f, 1.f};
#pragma unroll
        for (int i = 0; i < 7; ++i) c[i] = pack2(q[i] * most, q[i] * most);
        const float r[4] = {0.0164375687f, -0.0526718062f, 0.133207249f, -0.333329466f};
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = pack2(r[i] * most, r[i] * most);
    }
    // x up to kSmall, degree 4 (4e-8; 1.2e-7 with the roundings)
    __device__ __forceinline__ F2 small(F2 x) const {
        const F2 y = mul2(x, x);
        F2 p = d[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) p = fma2(p, y, d[i]);
        return mul2(fma2(p, y, c[6]), x);
    }
    // x up to 1; and what is added to the score
    __device__ __forceinline__ F2 near(F2 x, F2 o) const {
        const F2 y = mul2(x, x);
        F2 p = c[0];
#pragma unroll
        for (int i = 1; i < 7; ++i) p = fma2(p, y, c[i]);
        return fma2(p, x, o);
    }
    // any x
    __device__ __forceinline__ float of(float x) const {
        float n, none;
        unpack2(near(pack2(x, x), 0), n, none);
        return fabsf(x) > 1.f ? fmaf(-2.f * most, rcp_fast(1.f + exp2_fast(x * (2.f * kLog2e))), most) : n;
    }
};

// Only among slots that some rows of the item see and others do not can a value meet a weight of zero, and a NaN
// or infinity be carried into a row that does not see it.
__device__ __forceinline__ bool mixed_tile(const Item& it, int32_t k0) {
    return k0 < it.mixed_lo || max(k0, it.mixed_hi) < min(k0 + kTile, it.end);
}

// ---------------------------------------------------------------------------------------------------------
// loads and value tiles
// ---------------------------------------------------------------------------------------------------------
// Tiles of keys (first 0) and values (last 1), or of one of them. P.halves: column halves of 128 bytes a row, one
// after the other in a slot.
template <bool kScored>
__device__ __forceinline__ void load_role(const Params& P, Common& sh, uint32_t k_smem, uint32_t v_smem, const CUtensorMap* km,
                                          const CUtensorMap* vm, int first, int last) {
    const int lane = threadIdx.x & 31;
    const int32_t box = P.box, boxes = P.boxes, ps = P.a.pool.page_size;
    const bool leader = elect();
    const Limit limit{&sh.gave_up, P.polls};
    uint32_t tile = 0, issued[2] = {0, 0};
    Ring rings[2];
    bool ok = true;
    Items walk(P, sh);
    Item it;
#pragma unroll 1
    while (ok && walk.next(it)) {
        const int32_t* table = P.a.pool.table + (int64_t)it.b * P.a.pool.table_stride;
        const int32_t head = __shfl_sync(kAll, it.h, 0), n = __shfl_sync(kAll, it.n, 0);
        // where a lane's box of a tile lies; its page's id is read a tile ahead
        int32_t slot = tile_at<kScored>(P, it, 0) * kTile + lane * box, i = slot / ps, in = slot - i * ps;
        bool next_need = false;
        int32_t next_page = -1, next_at = 0;
#pragma unroll 1
        for (int32_t j = -1; j < n && ok; ++j) {
            bool need = next_need;
            const int32_t page = next_page, at = next_at;
            next_need = j + 1 < n && lane < boxes && slot < it.end && slot + box > it.lo;
            next_at = in;
            next_page = next_need ? table[i] : -1;
            if (kScored && P.a.slopes) {
                slot -= kTile;
                i -= P.tile_pages;
                in -= P.tile_rest;
                if (in < 0) {
                    in += ps;
                    --i;
                }
            } else {
                slot += kTile;
                i += P.tile_pages;
                in += P.tile_rest;
                if (in >= ps) {
                    in -= ps;
                    ++i;
                }
            }
            if (j < 0) continue;
            const bool miss = need && (page < 0 || page >= P.a.pool.pages);
            need = need && !miss;
            const uint32_t todo = __ballot_sync(kAll, need), bytes = __popc(todo) * box * 128 * P.halves;
            uint32_t bad = 0;
            if (rarely(__any_sync(kAll, miss))) {
                if (miss) {
                    report(P.a.status, 1u << SV_ERR_BAD_OFFSETS);
                    bad = ((1u << (box / 8)) - 1u) << (lane * (box / 8));
                }
                bad = __reduce_or_sync(kAll, bad);
            }
#pragma unroll 1
            for (int kv = first; kv <= last; ++kv) {
                Ring r = rings[0];
                if (kv) r = rings[1];
                const uint32_t slots = kv ? P.v_slots : P.k_slots, full = smem_u32(kv ? sh.v_full : sh.k_full) + 8 * r.i,
                               empty = smem_u32(kv ? sh.v_empty : sh.k_empty) + 8 * r.i;
                if (tile >= slots && !(ok = wait(empty, r.parity ^ 1, limit))) break;
                if (lane == 0) {
                    sh.bad[kv][tile % kNotes] = bad;
                    bar_expect(full, bytes);
                }
                __syncwarp();
                const CUtensorMap* map = kv ? vm : km;
                const uint32_t dst = (kv ? v_smem : k_smem) + r.i * (P.halves * kHalf);
#pragma unroll 1
                for (int i = 0; i < boxes; ++i) {  // one thread issues: from many, each copy would wait for the last
                    const int32_t p = __shfl_sync(kAll, page, i), a = __shfl_sync(kAll, at, i);
                    if (leader && (todo >> i & 1u)) {
                        copy_box(dst + i * box * 128, map, 0, a, head, p, full);
                        if (P.halves > 1) copy_box(dst + i * box * 128 + kHalf, map, 64, a, head, p, full);
                    }
                }
                r.step(slots);
                if (kv) {
                    rings[1] = r;
                    ++issued[1];
                } else {
                    rings[0] = r;
                    ++issued[0];
                }
            }
            ++tile;
        }
    }
    // copies still under way land before the CTA ends, also where another role gave up
#pragma unroll 1
    for (int kv = first; kv <= last; ++kv) {
        const uint32_t slots = kv ? P.v_slots : P.k_slots, n = kv ? issued[1] : issued[0];
#pragma unroll 1
        for (uint32_t i = 0; i < slots && i < n; ++i)
            drain(smem_u32(kv ? &sh.v_full[i] : &sh.k_full[i]), (n - 1 - i) / slots & 1);
    }
}

// The rows of an item's query tiles, 16-bit caches: copied, G heads of q_box tokens at once (rows past the sequence's end
// are another sequence's, or zero: a product's row depends on its own row only).
__device__ __forceinline__ bool copy_item_queries(const Params& P, Common& sh, const Item& it, uint32_t q_smem, const CUtensorMap* qm,
                                                  uint32_t items, uint32_t q_full) {
    const AttendArgs& A = P.a;
    const int lane = threadIdx.x & 31;
    const int q_tiles = P.tokens < P.block ? 2 : 1;
    bool flip;
    score_unit(A, it.h, flip);
    const uint32_t bar = flip ? smem_u32(&sh.q_in) : q_full;
    if (lane == 0) {
        bar_expect(bar, q_tiles * P.halves * P.q_box * P.G * 128);
        for (int t = 0; t < q_tiles; ++t)
            for (int h = 0; h < P.halves; ++h)
                copy_queries(q_smem + t * P.q_tile + h * P.q_part, qm, h * 64, it.h * P.G, it.row0 + it.t0 + t * it.split, bar);
    }
    __syncwarp();
    if (!rarely(flip)) return true;
    if (!wait(bar, items & 1, Limit{&sh.gave_up, P.polls})) return false;
#pragma unroll 1
    for (int i = lane; i < q_tiles * P.q_tile / 16; i += 32) {
        uint32_t u[4];
        const uint32_t at = q_smem + i * 16;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at));
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(u[0] ^ 0x80008000u), "r"(u[1] ^ 0x80008000u),
                     "r"(u[2] ^ 0x80008000u), "r"(u[3] ^ 0x80008000u)
                     : "memory");
    }
    fence_async();
    __syncwarp();
    if (lane == 0) bar_arrive(q_full);
    return true;
}

// e4m3 caches: split into the parts hi and lo, each row brought to [128, 256) by a power of two, by `of` warps, of which
// this is number `who`. A lane has a row and goes over it twice, for its largest element and for its parts; wide
// chunks have three warps. (Half a warp a row, with its maximum over the lanes, took four times as long: 60000 cycles
// for 256 rows.)
__device__ __forceinline__ void split_queries(const Params& P, Common& sh, const Item& it, uint32_t q_smem, uint32_t entry, uint32_t q_full,
                                              int who, int of) {
    using T = __nv_bfloat16;
    const AttendArgs& A = P.a;
    const int lane = threadIdx.x & 31;
    bool flip;
    score_unit(A, it.h, flip);
    const int32_t D = A.pool.dim, rows = it.nt * P.G, tile_rows = P.tokens < P.block ? it.split * P.G : rows;
    const T* q = (const T*)A.q + (int64_t)(it.row0 + it.t0) * A.q_stride + (int64_t)it.h * P.G * D;
#pragma unroll 1
    for (int32_t r = 32 * who + lane; r - lane < rows; r += 32 * of) {
        const int32_t t = r / P.G, g = r - t * P.G;
        const T* row = q + t * A.q_stride + (int64_t)g * D;
        const int32_t end = r < rows ? D : 0;
        uint32_t big = 0;  // magnitudes, in pairs
#pragma unroll 1
        for (int32_t d = 0; d < end; d += 64) {
            uint4 u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                u[k] = d + 8 * k < end ? *reinterpret_cast<const uint4*>(row + d + 8 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(big) : "r"(w[i] & 0x7fff7fffu));
            }
        }
        const float top = fmaxf(__uint_as_float(big << 16), __uint_as_float(big & 0xffff0000u));
        const int e = max(-120, min(120, 134 - (int)(__float_as_uint(top) >> 23)));
        const float up = __int_as_float((127 + e) << 23), by = flip ? -up : up;
        const int32_t at = r < tile_rows ? r : r - tile_rows;
        const uint32_t dst = q_smem + (r < tile_rows ? 0 : P.q_tile) + at * 128;
#pragma unroll 1
        for (int32_t c = 0; c < 8; ++c) {  // 16 elements, 16 bytes of each part
            uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (16 * c + 8 * k < end) u = *reinterpret_cast<const uint4*>(row + 16 * c + 8 * k);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = to_float2<T>(w[i]);
                    float x = f.x * by, y = f.y * by;
                    // an infinite query has no finite parts: its row is NaN, as its softmax is
                    if (fabsf(x) == INFINITY) x = NAN;
                    if (fabsf(y) == INFINITY) y = NAN;
                    const uint32_t a = e4m3x2(x, y);
                    const float2 b = from_e4m3x2(a);
                    hi[2 * k + (i >> 1)] |= a << (16 * (i & 1));
                    lo[2 * k + (i >> 1)] |= e4m3x2(x - b.x, y - b.y) << (16 * (i & 1));
                }
            }
            if (r < rows) {
                const uint32_t to = dst + ((c ^ (at & 7)) << 4);
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to + P.q_part), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                             : "memory");
            }
        }
        if (r < rows) sh.q_down[entry * sh.q_rows + (r < tile_rows ? 0 : kTile) + at] = __int_as_float((127 - e) << 23);
    }
    fence_async();
    __syncwarp();
    if (lane == 0) bar_arrive(q_full);
}

// Queries of e4m3 caches by warps of their own.
__device__ __forceinline__ void query_role(const Params& P, Common& sh, uint32_t q_smem, int who, int of) {
    Ring qr;
    Items walk(P, sh);
    Item it;
#pragma unroll 1
    for (uint32_t i = 0; walk.next(it); ++i, qr.step(P.q_bufs)) {
        if (i >= (uint32_t)P.q_bufs && !wait(smem_u32(&sh.q_empty[qr.i]), qr.parity ^ 1, Limit{&sh.gave_up, P.polls})) return;
        split_queries(P, sh, it, q_smem + qr.i * P.q_bytes, walk.ring.i, smem_u32(&sh.q_full[qr.i]), who, of);
    }
}

// The steps of a tile's depth that O += P V takes: those with a slot that some row of the item sees.
template <int K>
__device__ __forceinline__ void steps_of(const Item& it, int32_t k0, int32_t& lo, int32_t& hi) {
    constexpr int step = KindOf<K>::kStep;
    lo = max(0, it.lo - k0) / step;
    hi = (min(kTile, it.end - k0) + step - 1) / step;
}

// Rows [lo, hi) of a value tile set to zero. A whole row is the same 128 bytes under any swizzle.
__device__ __forceinline__ void clear_rows(int halves, uint32_t at, int32_t lo, int32_t hi) {
#pragma unroll 1
    for (int32_t i = lo * 8 + (threadIdx.x & 31); i < hi * 8; i += 32)
        for (int h = 0; h < halves; ++h)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at + h * kHalf + i * 16), "r"(0) : "memory");
}

// 16 bytes' non-finite elements cleared; whether there were any.
template <int K>
__device__ __forceinline__ bool clean16(uint32_t a) {
    constexpr int bits = K == kE4m3 ? 8 : 16;
    constexpr uint32_t one = (1u << bits) - 1u, top = K == kE4m3 ? 0x7fu : K == kBf16 ? 0x7f80u : 0x7c00u;
    bool any = false;
#pragma unroll 1
    for (int e = 0; e < 16; e += 4) {
        uint32_t x, clear = 0;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a + e));
#pragma unroll 1
        for (int by = 0; by < 32; by += bits)
            if ((x >> by & top) == top) clear |= one << by;
        if (!clear) continue;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(a + e), "r"(x & ~clear) : "memory");
        any = true;
    }
    return any;
}

// Non-finite elements of rows [lo, hi): cleared, and their rows noted. A product with zero finds them, for 16 bits:
// x 0 + a is NaN from the first one on. Four reads are under way at a time: one after the other they took 7000 cycles
// of a tile of 128 rows of 256 bytes, so 3000.
template <int K>
__device__ __forceinline__ void scan_rows(int halves, uint32_t at, int32_t lo, int32_t hi, uint32_t bad, uint32_t* odd) {
#pragma unroll 1
    for (int h = 0; h < halves; ++h, at += kHalf)
#pragma unroll 1
        for (int32_t i = lo * 8 + (threadIdx.x & 31); i < hi * 8; i += 128) {
            uint32_t u[4][4], any = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u[k][0] = u[k][1] = u[k][2] = u[k][3] = 0;
                if (i + 32 * k < hi * 8)
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(u[k][0]), "=r"(u[k][1]), "=r"(u[k][2]), "=r"(u[k][3])
                                 : "r"(at + (i + 32 * k) * 16));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (K == kE4m3) any |= ((u[k][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    else if (K == kBf16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(any) : "r"(u[k][e]), "r"(0));
                    else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(any) : "r"(u[k][e]), "r"(0));
                }
            if (!rarely(K == kE4m3 ? any != 0 : (any & 0x7fff7fffu) != 0)) continue;
#pragma unroll 1
            for (int32_t c = i; c < min(hi * 8, i + 128); c += 32)
                if (!(bad >> (c >> 6) & 1u) && clean16<K>(at + c * 16)) atomicOr(&odd[c >> 8], 1u << (c >> 3 & 31));
        }
}

// The CTA's items, one after the other, by one warp, and their queries (e4m3: a part of them, where kSplitters warps do
// that); a last one of no tiles ends them.
template <int K, int kSplitters, bool kScored>
__device__ __forceinline__ void item_role(const Params& P, Common& sh, uint32_t q_smem, const CUtensorMap* qm) {
    const int lane = threadIdx.x & 31;
    const bool tree = P.a.chunk.parents != nullptr;
    const int32_t lead = sh.start.lead;
    const Limit limit{&sh.gave_up, P.polls};
    int32_t b = sh.start.b, p = sh.start.p, h = sh.start.h, x = sh.start.x, left = sh.start.left;
    int32_t T = sh.start.T, past = sh.start.past, row0 = sh.start.row0;
    Ring ring;
    Ring qr;
    uint32_t loads = 0, above = 0;
    int32_t depth = 0;
#pragma unroll 1
    for (uint32_t i = 0;; ++i, ring.step(kItems)) {
        Item it{};
        left -= max(0, lead - x);
        if (rarely(left > 0 && (T < 0 || (tree && i == 0)))) {  // the next sequence (a tree's lanes: nodes)
#pragma unroll 1
            for (; b < P.a.chunk.B; ++b) {
                const Seq s = seq_of(P.a.chunk, capacity_of(P.a.pool), b);
                bool ok = !s.err;
                if (ok && tree) {
                    tree_of(P.a.chunk, b, s.T, depth, above, ok);
                    if (P.a.window > 0 && P.a.window < 32) {  // as far as the window reaches, a step at a time
                        int32_t at = lane, par = 0;
                        if (ok && lane > 0 && lane < s.T) par = P.a.chunk.parents[(int64_t)P.a.chunk.offs[b] + lane - 1];
                        above = 1u << lane;
#pragma unroll 1
                        for (int d = 1; d < P.a.window; ++d) {
                            at = __shfl_sync(kAll, par, at);
                            above |= 1u << at;
                        }
                    }
                }
                if (ok) {
                    T = s.T;
                    past = s.past;
                    row0 = s.row0;
                    break;
                }
            }
        }
        if (left > 0 && T > 0) {
            int32_t first, count;
            span<kScored>(P, b, T, past, p, it, first, count);
            const int32_t j = max(0, x - lead);
            it.b = b;
            it.h = h;
            it.row0 = row0;
            it.tile = first + j;
            it.begins = j == 0;
            it.n = min(count - j, left);
            it.finishes = j + it.n == count;
            it.mixed_hi = past + (tree ? 0 : it.t0 + 1);
            if (kScored) it.mixed_hi = max(it.mixed_hi, it.reach);
            it.mixed_lo = P.a.window > 0 && (tree || it.nt > 1) ? it.lo + it.nt + (tree ? it.t0 : 0) : 0;
            left -= it.n;
            x = 0;
        }
        if (i >= kItems && !wait(smem_u32(&sh.item_empty[ring.i]), ring.parity ^ 1, limit)) break;
        if (tree) {
            sh.tree[ring.i].above[lane] = above;
            sh.tree[ring.i].depth[lane] = depth;
            __syncwarp();
        }
        if (it.n > 0 && ++h == P.a.pool.heads) {
            h = 0;
            ++p;
            if (p * P.block >= T) {
                p = 0;
                ++b;
                T = -1;
            }
        }
        if (lane == 0) {
            sh.item[ring.i] = it;
            bar_arrive(smem_u32(&sh.item_full[ring.i]));
        }
        __syncwarp();
        if (it.n == 0) break;
        if (i >= (uint32_t)P.q_bufs && !wait(smem_u32(&sh.q_empty[qr.i]), qr.parity ^ 1, limit)) break;
        ++loads;
        const uint32_t at = q_smem + qr.i * P.q_bytes, q_full = smem_u32(&sh.q_full[qr.i]);
        if (K == kE4m3) split_queries(P, sh, it, at, ring.i, q_full, kSplitters - 1, kSplitters);
        else if (!copy_item_queries(P, sh, it, at, qm, i, q_full)) break;
        qr.step(P.q_bufs);
    }
    if (lane == 0) record<kScored>(P, sh);
    if (K != kE4m3 && loads > 0) {  // its copies land before the CTA ends, whoever gave up
        bool flip;
        score_unit(P.a, 0, flip);
        if (flip) drain(smem_u32(&sh.q_in), (loads - 1) & 1);
        else
#pragma unroll 1
            for (uint32_t k = loads > (uint32_t)P.q_bufs ? loads - P.q_bufs : 0; k < loads; ++k)
                drain(smem_u32(&sh.q_full[k % P.q_bufs]), k / P.q_bufs & 1);
    }
}

// Value tiles before they are multiplied: rows of slots that no row of the item sees are cleared
// (they may hold anything, and a weight of zero times NaN is NaN), and so are single non-finite values that only
// some rows see; those are noted for the rows that do.
template <int K, bool kScored>
__device__ __forceinline__ void value_role(const Params& P, Common& sh, uint32_t v_smem) {
    const int lane = threadIdx.x & 31;
    const Limit limit{&sh.gave_up, P.polls};
    uint32_t v = 0;
    Ring ring;
    Items walk(P, sh);
    Item it;
#pragma unroll 1
    while (walk.next(it)) {
#pragma unroll 1
        for (int32_t j = 0; j < it.n; ++j, ++v, ring.step(P.v_slots)) {
            if (!wait(smem_u32(&sh.v_full[ring.i]), ring.parity, limit)) return;
            const int32_t k0 = tile_at<kScored>(P, it, j) * kTile;
            const uint32_t bad = sh.bad[1][v % kNotes];
            const bool mixed = mixed_tile(it, k0);
            if (rarely(bad || k0 < it.lo || k0 + kTile > it.end || mixed)) {
                const uint32_t at = v_smem + ring.i * (P.halves * kHalf);
                uint32_t* odd = sh.odd[v % kNotes];
                if (lane < 4) odd[lane] = 0;
                __syncwarp();
                const int32_t lo = max(0, it.lo - k0), hi = min(kTile, it.end - k0);
                int32_t from, to;
                steps_of<K>(it, k0, from, to);
                // rows no one sees lie before the first and after the last one that is seen, or on bad pages
                constexpr int step = KindOf<K>::kStep;
#pragma unroll 1
                for (int g = -2; g < (bad ? 16 : 0); ++g)
                    if (g < 0 || (bad >> g & 1u))
                        clear_rows(P.halves, at, g == -2 ? from * step : g == -1 ? hi : 8 * g, g == -2 ? lo : g == -1 ? to * step : 8 * g + 8);
                if (rarely(mixed))
#pragma unroll 1
                    for (int g = 0; g < 2; ++g)
                        scan_rows<K>(P.halves, at, g ? max(lo, it.mixed_hi - k0) : lo, g ? hi : min(hi, it.mixed_lo - k0), bad, odd);
                fence_async();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(smem_u32(&sh.value[ring.i]));
        }
    }
}

// ---------------------------------------------------------------------------------------------------------
// the kernels' beginning and end
// ---------------------------------------------------------------------------------------------------------
// Barriers of the common part, by one thread. streams: warps at products; readers: warps that read the items; writers: of
// the queries.
__device__ __forceinline__ void init_common(Common& sh, int streams, int readers, int writers) {
#pragma unroll 1
    for (int i = 0; i < kMaxSlots; ++i) {
        bar_init(smem_u32(&sh.k_full[i]), 1);
        bar_init(smem_u32(&sh.k_empty[i]), streams);
        bar_init(smem_u32(&sh.v_full[i]), 1);
        bar_init(smem_u32(&sh.v_empty[i]), streams);
        bar_init(smem_u32(&sh.value[i]), 1);
    }
    bar_init(smem_u32(&sh.q_in), 1);
    for (int i = 0; i < 2; ++i) {
        bar_init(smem_u32(&sh.q_full[i]), writers);
        bar_init(smem_u32(&sh.q_empty[i]), streams);
    }
    bar_init(smem_u32(&sh.drain), streams);
    for (int i = 0; i < kItems; ++i) {
        bar_init(smem_u32(&sh.item_full[i]), 1);
        bar_init(smem_u32(&sh.item_empty[i]), readers);
    }
    sh.gave_up = 0;
}

// After the previous kernel's end: tensor memory, where the CTA begins, and the sequences that fail (their findings, and
// zeros in their rows). All threads; the caller's barrier follows.
// Tensor memory is taken after the wait, and the next kernel let in after that, by the warp that took it: a CTA that held
// some while it waits for a kernel whose CTAs, on the same SM, are yet to take theirs would wait for ever, and so would
// this one for the next kernel's.
template <int kThreads, int kColumns, bool kScored>
__device__ __forceinline__ void begin(const Params& P, Common& sh, bool allocates) {
    const int tid = threadIdx.x;
    // what is above may run while the stream's previous kernel ends
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (allocates) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "n"(kColumns)
                     : "memory");
        // else the SM's other CTA could not allocate before this one ends
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("griddepcontrol.launch_dependents;");
    }
    plan<kThreads, kScored>(P, sh);
    if (blockIdx.x == 0 && tid == 0) {
        const int64_t end = (int64_t)P.a.chunk.offs[P.a.chunk.B] + P.a.chunk.B;
        if (end > P.a.chunk.rows || P.a.chunk.offs[0] != 0) report(P.a.status, 1u << SV_ERR_BAD_OFFSETS);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (!sh.failing) return;
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
}

// Host: a kernel with all of an SM's shared memory, which may begin while the stream's previous one ends.
cudaError_t launch_early(const void* kernel, std::atomic<unsigned long long>* allowed, dim3 grid, int threads, int smem, cudaStream_t st,
                         void** args);
bool encode_pool(CUtensorMap* m, const Pool& p, char* base, int esize, int kind, int box);
bool encode_queries(CUtensorMap* m, const AttendArgs& A, int kind, int G, int q_box);
constexpr int kFewRows = 64;  // rows of a chunk up to which sv_cache_attend_few.cuh serves it
template <bool kScored>
cudaError_t launch_few(Params& P, int kind, int rows, int sms, cudaStream_t st);  // sets P.part_rows and P.ctas
template <bool kScored>
cudaError_t launch_wide(const Params& P, int kind, int dp, int n, cudaStream_t st);

}  // namespace cache
}  // namespace sv
