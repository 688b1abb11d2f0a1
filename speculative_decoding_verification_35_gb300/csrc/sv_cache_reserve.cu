// spec_cache_reserve (include/speccache.h): pages of the cache's pool for what the sequences are to hold, and the chunk's
// slots.
//
// A sequence's pages to give back or to take follow from its length alone; where they come to lie in the queue follows
// from prefix sums over the sequences. One cluster does it all: every CTA makes the same sums, a sequence a thread, and
// the pages and slots that they number are shared out one by one over all threads (a binary search in the sums, in shared
// memory, gives a page its sequence), so that one long prompt is as quick as many short ones. Two barriers order it: what
// is given back lies in the queue before anything is taken, and the new counts are written once no one reads the old
// ones, which they may replace. Where sequences go without, a warp each clears the entries that they wanted.
//
// Bound by the launch and a chain of dependent reads (the offsets and lengths, the queue, the writes): 64 sequences of 6 tokens
// 5.5 us by one CTA (6.2 to 6.5 a call, the host's). 32 prompts of 700 to 8192 tokens, 93000 slots: 11.3 us by 16 CTAs; by one,
// with 64-bit sums and a search for each slot, 130.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "sv_cache.cuh"

namespace cg = cooperative_groups;

namespace sv {
namespace cache {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCtas = 16;
constexpr int kAtOnce = 4, kSmall = 1024;
constexpr unsigned kAll = 0xffffffffu;
typedef unsigned long long u64;

// A block of sequences, one a thread. The sums are those before each sequence, and of all. They are kept to 2^32 - 1, which
// only sums that are refused exceed, and rows that several sequences claim.
struct Block {
    int32_t held[kThreads], need[kThreads], past[kThreads], row0[kThreads];
    int32_t lacks[kThreads];  // its entries from held up to this one it wants and does not get
    bool fine[kThreads];  // has no finding and got what it needs
    uint32_t give[kThreads + 1], take[kThreads + 1], rows[kThreads + 1];
    u64 scan[3][kWarps];
    u64 served;  // pages that the block's sequences take
};

struct Team {
    int rank, size;
    __device__ __forceinline__ void sync() const {
        if (size == 1) {
            __syncthreads();
        } else {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
    }
};

__device__ __forceinline__ u64 inscan(u64 v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(kAll, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += x;
    }
    return v;
}
// The entry of `sums` (kThreads + 1 of them) in which i lies.
__device__ __forceinline__ int find(const uint32_t* sums, uint32_t i) {
    int lo = 0;
#pragma unroll
    for (int o = kThreads / 2; o; o >>= 1)
        if (sums[lo + o] <= i) lo += o;
    return lo;
}
// The queue's entry i behind its head; both below `pages`.
__device__ __forceinline__ int32_t* queue_at(const ReserveArgs& A, uint32_t head, uint32_t i) {
    const uint32_t at = head + i;
    return A.queue + (at < (uint32_t)A.pages ? at : at - (uint32_t)A.pages);
}
// n / page_size for 0 <= n < 2^31: page_recip is 2^(31 + L) / page_size, rounded up, L = page_bits the least with 2^L >= page_size
// (the rounding adds less than 2^L to page_recip page_size, and so less than 1 / page_size to the quotient).
__device__ __forceinline__ int32_t page_of(const ReserveArgs& A, int32_t n) {
    return (int32_t)(((u64)(uint32_t)n * A.page_recip) >> (31 + A.page_bits));
}

// A thread's sequence, and what it gives back, takes and has of rows, by itself and with those before it.
struct Mine {
    int32_t b, held, need, want;  // want: entries of its row, whether it gets them or not
    uint32_t err;
    u64 gives, takes, takes_upto;
};

// The block of the sequences from b0 on, with its sums. All threads; ends with a barrier. Returns what the block gives back.
__device__ __forceinline__ u64 read_block(const ReserveArgs& A, Block& s, int32_t b0, Mine& me, u64& takes) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    me = Mine{};
    me.b = b0 + tid;
    u64 v[3] = {0, 0, 0};  // gives, takes, rows
    if (me.b < A.B) {
        me.held = A.held[me.b];
        int64_t n;
        if (A.lengths) {
            n = A.lengths[me.b];
        } else {
            const Seq q = seq_of(A.chunk, 0x7fffffff, me.b);
            me.err = q.err;
            n = q.past < 0 ? -1 : (int64_t)q.past + q.T;
            if (q.rows_ok) v[2] = (u64)q.T;
            s.past[tid] = q.past;
            s.row0[tid] = q.row0;
        }
        if (me.held < 0 || me.held > A.table_stride) me.err |= 1u << SV_ERR_BAD_OFFSETS;
        const int64_t pages = (n + A.page_size - 1) / A.page_size;
        if (!me.err && n >= 0) me.want = (int32_t)min(pages, (int64_t)A.table_stride);
        if (n < 0 || pages > A.table_stride) me.err |= 1u << SV_ERR_CAPACITY;
        me.need = me.err ? me.held : (int32_t)pages;
        if (!me.err) {
            if (me.need < me.held) v[0] = (u64)(me.held - me.need);
            else v[1] = (u64)(me.need - me.held);
        }
    }
    u64 upto[3], all[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        upto[i] = inscan(v[i]);
        if (lane == 31) s.scan[i][warp] = upto[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const u64 x = s.scan[i][w];
            if (w < warp) upto[i] += x;
            all[i] += x;
        }
        uint32_t* sums = i == 0 ? s.give : i == 1 ? s.take : s.rows;
        sums[tid] = (uint32_t)min(upto[i] - v[i], 0xffffffffull);
        if (tid == 0) sums[kThreads] = (uint32_t)min(all[i], 0xffffffffull);
    }
    s.held[tid] = me.held;
    s.need[tid] = me.need;
    if (tid == 0) s.served = 0;
    me.gives = v[0];
    me.takes = v[1];
    me.takes_upto = upto[1];
    takes = all[1];
    __syncthreads();
    return all[0];
}
// Who gets what it lacks, of `free` pages, after the blocks before took (or would have) `before`. All threads; ends with a barrier.
// Whether some go without.
__device__ __forceinline__ bool serve(Block& s, Mine& me, u64 before, u64 free, bool bad, int32_t B) {
    const int tid = threadIdx.x;
    const bool served = !bad && before + me.takes_upto <= free;
    if (bad || (!served && me.takes)) me.need = me.held;
    if (!bad && !served && me.takes) me.err |= 1u << SV_ERR_CAPACITY;
    const unsigned who = __ballot_sync(kAll, served && me.takes);
    if (who && (tid & 31) == 31 - __clz(who)) atomicMax(&s.served, me.takes_upto);
    s.need[tid] = me.need;
    s.fine[tid] = me.b < B && !me.err && !bad;
    s.lacks[tid] = me.want > me.need ? me.want : 0;
    return __syncthreads_or(me.want > me.need);
}

__global__ void __launch_bounds__(kThreads) k_cache_reserve(const __grid_constant__ ReserveArgs A) {
    __shared__ Block s;
    __shared__ u64 block_base[kMaxReserve / kThreads];  // pages that the blocks before would take
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Team team{(int)blockIdx.x, (int)gridDim.x};
    const int tid = threadIdx.x;
    const uint32_t first = (uint32_t)(team.rank * kThreads + tid), step = (uint32_t)(team.size * kThreads);
    const bool once = A.B <= kThreads;
    const int32_t head = A.state[0], count = A.state[1];
    bool bad = head < 0 || head >= A.pages || count < 0;
    uint32_t err = 0;
    Mine me{};
    u64 takes = 0;

    // what is given back in all
    u64 gives = 0;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B; b0 += kThreads) {
        if (b0 > 0) __syncthreads();
        gives += read_block(A, s, b0, me, takes);
    }
    bad = bad || (u64)count + gives > (u64)A.pages;
    // into the queue, behind its last
    uint32_t given = 0;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B && gives > 0 && !bad; b0 += kThreads) {
        if (!once) {
            __syncthreads();
            read_block(A, s, b0, me, takes);
        }
        for (uint32_t i = first; i < s.give[kThreads]; i += step) {
            const int t = find(s.give, i);
            const int32_t id = A.table[(int64_t)(b0 + t) * A.table_stride + (s.need[t] + (int32_t)(i - s.give[t]))];
            if (id < 0 || id >= A.pages) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
            *queue_at(A, head, (uint32_t)count + given + i) = id;
        }
        given += s.give[kThreads];
    }
    team.sync();
    const u64 free = bad ? 0 : (u64)count + gives;
    // out of it, from the front; and the slots
    u64 base = 0, taken = 0;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B; b0 += kThreads) {
        if (!once) {
            __syncthreads();
            read_block(A, s, b0, me, takes);
        }
        const bool lacking = serve(s, me, base, free, bad, A.B);
        err |= me.err;
        if (tid == 0) block_base[b0 / kThreads] = base;
        const uint32_t served = (uint32_t)s.served, from = (uint32_t)base;  // both below `pages` where pages are taken
        for (uint32_t i = first; i < served; i += step) {
            const int t = find(s.take, i);
            const int32_t id = __ldcg(queue_at(A, head, from + i));
            if (id < 0 || id >= A.pages) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
            A.table[(int64_t)(b0 + t) * A.table_stride + (s.held[t] + (int32_t)(i - s.take[t]))] = id;
        }
        // What lies past a sequence's pages is what it gave back once, and may be another's by now: entries that it wanted and
        // did not get must not pass for its own.
        if (lacking)
#pragma unroll 1
            for (int t = (int)first / 32; t < kThreads; t += (int)step / 32)
                for (int32_t i = s.held[t] + (tid & 31); i < s.lacks[t]; i += 32) A.table[(int64_t)(b0 + t) * A.table_stride + i] = -1;
        if (A.slots) {
            // a warp takes a run of slots, several a lane at once where there are many: the sequence of the run's first is
            // searched for once, and is that of most others in a prompt
            const uint32_t all = s.rows[kThreads], lane = tid & 31, per = all > 2 * step ? kAtOnce : 1;
            for (uint64_t r0 = (uint64_t)(first - lane) * per; r0 < all; r0 += (uint64_t)step * per) {
                int32_t row[kAtOnce], id[kAtOnce], in[kAtOnce];
                const int t0 = find(s.rows, (uint32_t)r0);
                const uint32_t t0_end = s.rows[t0 + 1];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const uint64_t i64 = r0 + 32 * k + lane;
                    row[k] = id[k] = -1;
                    if (k >= (int)per || i64 >= all) continue;
                    const uint32_t i = (uint32_t)i64;
                    const int t = i < t0_end ? t0 : find(s.rows, i);
                    const int32_t j = (int32_t)(i - s.rows[t]), slot = s.past[t] + j, page = page_of(A, slot);
                    row[k] = s.row0[t] + j;
                    if (!s.fine[t]) continue;
                    in[k] = slot - page * A.page_size;
                    id[k] = page < s.held[t] ? A.table[(int64_t)(b0 + t) * A.table_stride + page]
                                             : __ldcg(queue_at(A, head, from + s.take[t] + (uint32_t)(page - s.held[t])));
                    if (id[k] < 0 || id[k] >= A.pages) {
                        report(A.status, 1u << SV_ERR_BAD_OFFSETS);
                        id[k] = -1;
                    }
                }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (row[k] >= 0) A.slots[row[k]] = id[k] < 0 ? -1 : (int64_t)id[k] * A.page_size + in[k];
            }
        }
        if (served) taken = base + served;
        base += takes;
    }
    team.sync();  // no other CTA reads held any more
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B; b0 += kThreads) {
        if (b0 / kThreads % team.size != team.rank) continue;
        if (!once) {
            __syncthreads();
            read_block(A, s, b0, me, takes);
            serve(s, me, block_base[b0 / kThreads], free, bad, A.B);
        }
        if (me.b < A.B) A.out_held[me.b] = me.need;
    }
    if (team.rank == 0) {
        if (bad) err |= 1u << SV_ERR_BAD_OFFSETS;
        err = __reduce_or_sync(kAll, err);
        if ((tid & 31) == 0) report(A.status, err);
        if (tid == 0) {
            A.out_state[0] = bad ? head : (int32_t)(((u64)head + taken) % (u64)A.pages);
            A.out_state[1] = bad ? count : (int32_t)(free - taken);
            if (!A.lengths && A.B > 0) {
                const int64_t end = (int64_t)A.chunk.offs[A.B] + A.B;
                if (end > A.chunk.rows || A.chunk.offs[0] != 0) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
            }
        }
    }
}

}  // namespace

cudaError_t launch_reserve(const ReserveArgs& A, cudaStream_t st) {
    // slots and pages that there may be; a cluster costs a small call what its barriers do
    const int64_t most = A.lengths ? std::min((int64_t)A.B * A.table_stride, (int64_t)A.pages) : (int64_t)A.chunk.rows + A.B;
    const int ctas = most > kSmall ? kMaxCtas : 1;
    ReserveArgs a = A;
    a.page_bits = 0;
    while ((1u << a.page_bits) < (uint32_t)A.page_size) ++a.page_bits;
    a.page_recip = (uint32_t)((((u64)1 << (31 + a.page_bits)) + (uint32_t)A.page_size - 1) / (uint32_t)A.page_size);
    if (ctas > 8) {  // a cluster of that size asks for it, once a device; setting it twice does no harm
        int dev;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        static std::atomic<unsigned long long> allowed{0};
        if (dev >= 64 || !(allowed.load() >> dev & 1u)) {
            e = cudaFuncSetAttribute(k_cache_reserve, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            if (dev < 64) allowed.fetch_or(1ull << dev);
        }
    }
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_cache_reserve, a);
}

}  // namespace cache
}  // namespace sv
