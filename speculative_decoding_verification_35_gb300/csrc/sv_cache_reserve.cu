// spec_cache_reserve (include/speccache.h): pages of the cache's pool for what the sequences are to hold, and the chunk's
// slots.
//
// A sequence's pages to give back or to take follow from its length alone; where they come to lie in the queue follows
// from prefix sums over the sequences. One cluster does it all: every CTA makes the same sums, a sequence a thread, and
// the pages and slots that they number are shared out one by one over all threads (a binary search in the sums, in shared
// memory, gives a page its sequence), so that one long prompt is as quick as many short ones. Two barriers order it: what
// is given back lies in the queue before anything is taken, and the new counts are written once no one reads the old
// ones, which they may replace.
//
// Bound by the launch and a chain of dependent reads (the offsets and lengths, the queue, the writes).
#include <cooperative_groups.h>

#include <algorithm>

#include "sv_cache.cuh"

namespace cg = cooperative_groups;

namespace sv {
namespace cache {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCtas = 8;
constexpr unsigned kAll = 0xffffffffu;
typedef unsigned long long u64;

// A block of sequences, one a thread.
struct Block {
    int32_t held[kThreads], need[kThreads], past[kThreads], row0[kThreads];
    bool fine[kThreads];                                              // has no finding and got what it needs
    u64 give[kThreads + 1], take[kThreads + 1], rows[kThreads + 1];  // sums before each
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
__device__ __forceinline__ int find(const u64* sums, u64 i) {
    int lo = 0;
#pragma unroll
    for (int o = kThreads / 2; o; o >>= 1)
        if (sums[lo + o] <= i) lo += o;
    return lo;
}

// The queue's entry i behind its head; i < pages.
__device__ __forceinline__ int32_t* queue_at(const ReserveArgs& A, int64_t head, u64 i) {
    const u64 at = (u64)head + i;
    return A.queue + (at < (u64)A.pages ? at : at - (u64)A.pages);
}

// The block of the sequences from b0 on: what they need, and the sums. before: pages that earlier blocks would take;
// count: free pages, with those given back. All threads; ends with a barrier. Returns the thread's finding.
__device__ __forceinline__ uint32_t read_block(const ReserveArgs& A, Block& s, int32_t b0, u64 before, u64 count, bool bad) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t b = b0 + tid;
    uint32_t err = 0;
    int32_t held = 0, need = 0;
    u64 v[3] = {0, 0, 0};  // gives, takes, rows
    if (b < A.B) {
        held = A.held[b];
        int64_t n;
        if (A.lengths) {
            n = A.lengths[b];
        } else {
            const Seq q = seq_of(A.chunk, 0x7fffffff, b);
            err = q.err;
            n = (int64_t)q.past + q.T;
            if (q.past < 0) n = -1;
            if (q.rows_ok) v[2] = (u64)q.T;
            s.past[tid] = q.past;
            s.row0[tid] = q.row0;
        }
        if (held < 0 || held > A.table_stride) err |= 1u << SV_ERR_BAD_OFFSETS;
        const int64_t pages = (n + A.page_size - 1) / A.page_size;
        if (n < 0 || pages > A.table_stride) err |= 1u << SV_ERR_CAPACITY;
        need = err || bad ? held : (int32_t)pages;
        if (!err && !bad) {
            if (need < held) v[0] = (u64)(held - need);
            else v[1] = (u64)(need - held);
        }
    }
    u64 upto[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        upto[i] = inscan(v[i]);
        if (lane == 31) s.scan[i][warp] = upto[i];
    }
    if (tid == 0) s.served = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        u64 x = upto[i];
        for (int w = 0; w < warp; ++w) x += s.scan[i][w];
        u64* sums = i == 0 ? s.give : i == 1 ? s.take : s.rows;
        sums[tid] = x - v[i];
        if (tid == kThreads - 1) sums[kThreads] = x;
        upto[i] = x;
    }
    const bool served = before + upto[1] <= count;
    if (!served && v[1]) err |= 1u << SV_ERR_CAPACITY;
    if (served && v[1]) atomicMax(&s.served, upto[1]);
    s.held[tid] = held;
    s.need[tid] = served || !v[1] ? need : held;
    s.fine[tid] = b < A.B && !err && !bad;
    __syncthreads();
    return err;
}

__global__ void __launch_bounds__(kThreads) k_cache_reserve(const __grid_constant__ ReserveArgs A) {
    __shared__ Block s;
    __shared__ u64 block_base[kMaxReserve / kThreads];  // pages that the blocks before would take
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Team team{(int)blockIdx.x, (int)gridDim.x};
    const int tid = threadIdx.x;
    const u64 me = (u64)team.rank * kThreads + tid, step = (u64)team.size * kThreads;
    const bool once = A.B <= kThreads;
    const int64_t head = A.state[0];
    int64_t count = A.state[1];
    const u64 pages = (u64)A.pages;
    bool bad = head < 0 || head >= A.pages || count < 0;
    uint32_t err = 0;

    // what is given back in all
    u64 gives = 0;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B; b0 += kThreads) {
        if (b0 > 0) __syncthreads();
        read_block(A, s, b0, 0, 0, false);
        gives += s.give[kThreads];
    }
    if (bad || (u64)count + gives > pages) bad = true;
    if (bad) gives = 0;
    // into the queue, behind its last
    u64 base = 0;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B && gives > 0; b0 += kThreads) {
        if (!once) {
            __syncthreads();
            read_block(A, s, b0, 0, 0, false);
        }
        for (u64 i = me; i < s.give[kThreads]; i += step) {
            const int t = find(s.give, i);
            const int32_t id = A.table[(int64_t)(b0 + t) * A.table_stride + s.need[t] + (int64_t)(i - s.give[t])];
            if (id < 0 || id >= A.pages) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
            *queue_at(A, head, (u64)count + base + i) = id;
        }
        base += s.give[kThreads];
    }
    team.sync();
    const u64 free = bad ? 0 : (u64)count + gives;
    // out of it, from the front; and the slots
    base = 0;
    u64 taken = 0;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B; b0 += kThreads) {
        if (b0 > 0) __syncthreads();
        err |= read_block(A, s, b0, base, free, bad);
        if (tid == 0) block_base[b0 / kThreads] = base;
        const u64 served = s.served;
        for (u64 i = me; i < served; i += step) {
            const int t = find(s.take, i);
            const int32_t id = __ldcg(queue_at(A, head, base + i));
            if (id < 0 || id >= A.pages) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
            A.table[(int64_t)(b0 + t) * A.table_stride + s.held[t] + (int64_t)(i - s.take[t])] = id;
        }
        if (A.slots)
            for (u64 i = me; i < s.rows[kThreads]; i += step) {
                const int t = find(s.rows, i);
                const int32_t j = (int32_t)(i - s.rows[t]);
                int64_t at = -1;
                if (s.fine[t]) {
                    const int32_t slot = s.past[t] + j, k = slot / A.page_size;
                    const int32_t id = k < s.held[t] ? A.table[(int64_t)(b0 + t) * A.table_stride + k]
                                                     : __ldcg(queue_at(A, head, base + s.take[t] + (u64)(k - s.held[t])));
                    if (id >= 0 && id < A.pages) at = (int64_t)id * A.page_size + (slot - k * A.page_size);
                    else report(A.status, 1u << SV_ERR_BAD_OFFSETS);
                }
                A.slots[s.row0[t] + j] = at;
            }
        if (served) taken = base + served;
        base += s.take[kThreads];
        if (once) break;
    }
    team.sync();  // no other CTA reads held any more
#pragma unroll 1
    for (int32_t b0 = 0; b0 < A.B; b0 += kThreads) {
        if (b0 / kThreads % team.size != team.rank) continue;
        if (!once) {
            __syncthreads();
            read_block(A, s, b0, block_base[b0 / kThreads], free, bad);
        }
        if (b0 + tid < A.B) A.out_held[b0 + tid] = s.need[tid];
    }
    if (team.rank == 0) {
        if (bad) err |= 1u << SV_ERR_BAD_OFFSETS;
        err = __reduce_or_sync(kAll, err);
        if ((tid & 31) == 0) report(A.status, err);
        if (tid == 0) {
            A.out_state[0] = bad ? (int32_t)head : (int32_t)(((u64)head + taken) % pages);
            A.out_state[1] = bad ? (int32_t)count : (int32_t)(free - taken);
            if (!A.lengths && A.B > 0) {
                const int64_t end = (int64_t)A.chunk.offs[A.B] + A.B;
                if (end > A.chunk.rows || A.chunk.offs[0] != 0) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
            }
        }
    }
}

}  // namespace

cudaError_t launch_reserve(const ReserveArgs& A, cudaStream_t st) {
    const int ctas = 1;
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
    return cudaLaunchKernelEx(&cfg, k_cache_reserve, A);
}

}  // namespace cache
}  // namespace sv
