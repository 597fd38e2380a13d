// memq_page_plan.cu -- memq_page_plan: the bookkeeping of one serving step over a paged cache.  From
// every request's lengths it gives back the pages that are no longer needed, takes the pages that the
// new tokens need off the stack of free pages, and writes block tables, lengths, offsets and slots.
//
//   have = ceil(cached / page), need = ceil((keep + new) / page)
//   push = max(0, have - need) pages leave the request's table, in (request, column) order
//   pop  = max(0, need - have) pages enter it, in the same order, from the stack's top
//
// Everything follows from prefix sums over the requests (tokens, pushes, pops): a request is served
// when the pops up to and including its own fit on the stack, so the sums of those that are served are
// the sums over all, and no request waits for another's verdict.  Every CTA forms the sums of all
// requests itself (at most 4096, out of L2); then a thread serves a page or a token, which it finds by
// bisection in the sums.  Pops may take what was pushed by the same call: a cluster of CTAs, with one
// barrier between the two, rather than a grid, which would need two launches.
//
// A step is bound by latency.  1 request: one CTA, 4.5 us; 1024 requests with 27,000 new tokens: a cluster of 8, 9.6 us,
// of three prefix sums behind one another, the barrier and a bisection a thread.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "memq.h"
#include "memq_dev.cuh"

namespace memq {
namespace {

__device__ unsigned int g_plan_fault = 0;
constexpr unsigned int kFaultInput = 32;  // a length, a count or a page index was out of range

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxSeqs = 4096;
constexpr int kPer = kMaxSeqs / kPlanThreads;  // requests a thread
constexpr int kClusterCtas = 8;
constexpr int kMaxCached = 1 << 30;

struct PlanArgs {
    const int32_t *cached, *keep, *fresh;
    int32_t *table, *free_pages;
    const int32_t *n_free;
    int32_t *kv_len, *n_free_out, *cu_q, *slots, *positions, *granted;
    int n_seq, n_tok, max_pages, page_shift, n_pages;
    int wide;  // slots and positions are 16-byte aligned
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Every thread of the cluster; what was written before is visible after it, in global memory too.
__device__ __forceinline__ void cluster_sync() {
    __threadfence();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix over the CTA's threads; `total` is the sum over all.
__device__ __forceinline__ long long block_prefix(long long v, long long *warp_sums, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += up;
    }
    __syncthreads();  // the sums of an earlier call have been read
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    long long s = warp_sums[lane];
    long long run = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(kFullMask, run, o);
        if (lane >= o) run += up;
    }
    total = __shfl_sync(kFullMask, run, 31);
    const long long before = __shfl_sync(kFullMask, run - s, warp);
    return before + incl - v;
}

// The request that item `k` belongs to: the last whose first item is at or before k.  Requests without
// items share their first with the next one, so the last is the one that owns it.
__device__ __forceinline__ int owner_of(const int32_t *first, int n, int k) {
    int lo = 0, hi = n;  // first[lo] <= k < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= k) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads, 1) page_plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t smem[];
    __shared__ long long warp_sums[kPlanWarps];
    static_assert(kPlanWarps == 32, "a warp sums the warps' sums");
    // per request: first token, first push, first pop, pages before, pages needed (-1: not served), kept rows
    int32_t *tok0 = smem, *push0 = tok0 + a.n_seq + 1, *pop0 = push0 + a.n_seq, *have_of = pop0 + a.n_seq,
            *need_of = have_of + a.n_seq, *keep_of = need_of + a.n_seq;
    const int tid = threadIdx.x;
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    griddep_launch_dependents();
    griddep_wait();

    const int page = 1 << a.page_shift;
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    const int per = (a.n_seq + kPlanThreads - 1) / kPlanThreads, b0 = tid * per;
    int cached[kPer], keep[kPer], fresh[kPer];
    bool bad = false;
    long long tokens = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        cached[i] = keep[i] = fresh[i] = 0;
        const int b = b0 + i;
        if (i >= per || b >= a.n_seq) continue;
        const int c = __ldcg(a.cached + b), f = __ldcg(a.fresh + b);
        const int k = a.keep ? __ldcg(a.keep + b) : c;
        cached[i] = static_cast<int>(min(static_cast<long long>(max(c, 0)), cap));
        keep[i] = min(max(k, 0), cached[i]);
        fresh[i] = min(max(f, 0), kMaxCached);
        bad = bad || cached[i] != c || keep[i] != k || fresh[i] != f;
        tokens += fresh[i];
    }
    int free_now = __ldcg(a.n_free);
    if (free_now < 0 || free_now > a.n_pages) {
        bad = true;
        free_now = min(max(free_now, 0), a.n_pages);
    }
    long long total_tok, total_push, total_pop;
    long long tok = block_prefix(tokens, warp_sums, total_tok);
    int have[kPer], need[kPer];
    long long pushes = 0, pops = 0;
    bool room[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = b0 + i;
        have[i] = need[i] = 0;
        room[i] = false;
        if (i >= per || b >= a.n_seq) continue;
        tok0[b] = static_cast<int>(min(tok, static_cast<long long>(a.n_tok)));
        tok += fresh[i];
        const long long want = static_cast<long long>(keep[i]) + fresh[i];
        room[i] = want <= cap && (fresh[i] == 0 || tok <= a.n_tok);  // (behind too many tokens, those without any)
        bad = bad || tok > a.n_tok;
        have[i] = static_cast<int>((static_cast<long long>(cached[i]) + page - 1) >> a.page_shift);
        need[i] = room[i] ? static_cast<int>((want + page - 1) >> a.page_shift) : have[i];
        pushes += max(0, have[i] - need[i]);
        pops += max(0, need[i] - have[i]);
    }
    long long push = block_prefix(pushes, warp_sums, total_push);
    long long pop = block_prefix(pops, warp_sums, total_pop);
    // a stack that holds more pages than there are was given pages twice
    if (free_now + total_push > a.n_pages) bad = true;
    const long long stack = min(free_now + total_push, static_cast<long long>(a.n_pages));
    // requests are served up to the first whose pages do not fit: the pops of those are the longest
    // prefix of all that is no more than the stack
    long long taken = 0;
    bool ok[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = b0 + i;
        ok[i] = false;
        if (i >= per || b >= a.n_seq) continue;
        const int n = max(0, need[i] - have[i]);
        push0[b] = static_cast<int>(min(push, static_cast<long long>(a.n_pages)));
        push += max(0, have[i] - need[i]);
        pop0[b] = static_cast<int>(min(pop, static_cast<long long>(0x7fffffff)));
        pop += n;
        ok[i] = room[i] && (n == 0 || pop <= stack);
        if (n > 0 && ok[i]) taken = pop;
        have_of[b] = have[i];
        need_of[b] = ok[i] ? need[i] : -1;
        keep_of[b] = keep[i];
    }
    if (tid == 0) tok0[a.n_seq] = static_cast<int>(min(total_tok, static_cast<long long>(a.n_tok)));
    // the largest prefix that was served, over the CTA
    {
        long long m = taken;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
        __syncthreads();
        if ((tid & 31) == 0) warp_sums[tid >> 5] = m;
        __syncthreads();
        m = warp_sums[tid & 31];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
        taken = m;
    }
    if (bad && rank == 0) atomicOr(&g_plan_fault, kFaultInput);

    const int stride = ranks * kPlanThreads, first = rank * kPlanThreads + tid;
    const int n_push = static_cast<int>(min(total_push, static_cast<long long>(a.n_pages - free_now)));
    for (int k = first; k < n_push; k += stride) {
        const int b = owner_of(push0, a.n_seq, k);
        const int col = max(need_of[b], 0) + (k - push0[b]);
        a.free_pages[free_now + k] = __ldcg(a.table + static_cast<int64_t>(b) * a.max_pages + min(col, a.max_pages - 1));
    }
    // Every CTA has read the lengths, which the outputs may replace, and the pushed pages are on the stack.
    if (ranks > 1)
        cluster_sync();
    else
        __syncthreads();
    if (rank == 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = b0 + i;
            if (i >= per || b >= a.n_seq) continue;
            a.cu_q[b] = tok0[b];
            a.kv_len[b] = ok[i] ? keep[i] + fresh[i] : cached[i];
            a.granted[b] = ok[i];
        }
        if (tid == 0) {
            a.cu_q[a.n_seq] = tok0[a.n_seq];
            *a.n_free_out = static_cast<int>(stack - taken);
        }
    }
    const int top = static_cast<int>(stack) - 1, n_pop = static_cast<int>(taken);
    for (int k = first; k < n_pop; k += stride) {
        const int b = owner_of(pop0, a.n_seq, k);
        a.table[static_cast<int64_t>(b) * a.max_pages + have_of[b] + (k - pop0[b])] = __ldcg(a.free_pages + top - k);
    }
    // Four tokens next to one another a thread: one bisection, and a store of 16 bytes where the outputs lie so.
    const int live = tok0[a.n_seq];
    for (int t0 = 4 * first; t0 < a.n_tok; t0 += 4 * stride) {
        int slot[4], pos[4], col_then = -1, page_then = -1, b = t0 < live ? owner_of(tok0, a.n_seq, t0) : 0, b_then = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i;
            slot[i] = pos[i] = -1;
            if (t >= live) continue;
            while (tok0[b + 1] <= t) ++b;  // (t < live = tok0[n_seq])
            pos[i] = keep_of[b] + (t - tok0[b]);
            if (need_of[b] < 0) continue;
            const int col = pos[i] >> a.page_shift;
            if (col != col_then || b != b_then) {
                page_then = col < have_of[b] ? __ldcg(a.table + static_cast<int64_t>(b) * a.max_pages + col)
                                             : __ldcg(a.free_pages + top - (pop0[b] + col - have_of[b]));
                col_then = col;
                b_then = b;
            }
            if (page_then >= 0 && page_then < a.n_pages)
                slot[i] = (page_then << a.page_shift) + (pos[i] & (page - 1));
            else
                atomicOr(&g_plan_fault, kFaultInput);
        }
        if (a.wide && t0 + 4 <= a.n_tok) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < a.n_tok) {
                    a.slots[t0 + i] = slot[i];
                    a.positions[t0 + i] = pos[i];
                }
        }
    }
}

constexpr int kMaxDevices = 64;

constexpr int smem_bytes(int n_seq) { return (n_seq * 6 + 1) * static_cast<int>(sizeof(int32_t)); }

// Allows the kernel the shared memory of the most requests on the current device, once: the allowance is the
// function's, for all host threads, and the default one holds for the warps' sums beside it too.
bool allow() {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kMaxSeqs)) !=
        cudaSuccess)
        return false;
    if (dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
    return true;
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; }

}  // namespace
}  // namespace memq

// Internal: this translation unit's device fault word (not part of the public header).
int memq_internal_fault_plan(unsigned int *out, bool clear) {
    if (cudaMemcpyFromSymbol(out, memq::g_plan_fault, sizeof(unsigned int)) != cudaSuccess) return 1;
    if (!clear) return 0;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(memq::g_plan_fault, &zero, sizeof(zero)) == cudaSuccess ? 0 : 1;
}

extern "C" int memq_page_plan(const int32_t *cached, const int32_t *keep, const int32_t *new_tok, int32_t *block_table,
                              int32_t *free_pages, const int32_t *n_free, int32_t *kv_len, int32_t *n_free_out,
                              int32_t *cu_q, int32_t *slots, int32_t *positions, int32_t *granted, int n_seq,
                              int64_t n_tok, int max_pages, int page_size, int64_t n_pages, void *stream) {
    using namespace memq;
    if (n_seq < 0 || n_seq > kMaxSeqs || n_tok < 0 || n_tok > (1 << 24) || page_size < 16 || page_size > 1024 ||
        (page_size & (page_size - 1)) != 0 || n_pages < 0 || n_pages > 0x7fffffffLL / page_size || max_pages < 0 ||
        max_pages > kMaxCached / page_size)
        return MEMQ_ERR_SHAPE;
    if (n_seq == 0) return n_tok == 0 ? MEMQ_OK : MEMQ_ERR_SHAPE;
    if (n_pages < 1 || max_pages < 1) return MEMQ_ERR_SHAPE;
    if (!cached || !new_tok || !block_table || !free_pages || !n_free || !kv_len || !n_free_out || !cu_q || !granted ||
        (n_tok > 0 && (!slots || !positions)))
        return MEMQ_ERR_NULL;
    for (const void *p : {static_cast<const void *>(cached), static_cast<const void *>(keep),
                          static_cast<const void *>(new_tok), static_cast<const void *>(block_table),
                          static_cast<const void *>(free_pages), static_cast<const void *>(n_free),
                          static_cast<const void *>(kv_len), static_cast<const void *>(n_free_out),
                          static_cast<const void *>(cu_q), static_cast<const void *>(slots),
                          static_cast<const void *>(positions), static_cast<const void *>(granted)})
        if (misaligned4(p)) return MEMQ_ERR_ALIGN;
    PlanArgs a{cached, keep, new_tok, block_table, free_pages, n_free, kv_len, n_free_out, cu_q, slots, positions,
               granted, n_seq, static_cast<int>(n_tok), max_pages, __builtin_ctz(static_cast<unsigned>(page_size)),
               static_cast<int>(n_pages),
               ((reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(positions)) & 15) == 0};
    if (!allow()) return MEMQ_ERR_LAUNCH;
    // One CTA serves what its threads hold in one round; more of it is shared by a cluster.
    const bool small = n_seq <= kPlanThreads && n_tok <= 4 * kPlanThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(small ? 1 : kClusterCtas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes(n_seq));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, page_plan_kernel, a) == cudaSuccess ? MEMQ_OK : MEMQ_ERR_LAUNCH;
}
