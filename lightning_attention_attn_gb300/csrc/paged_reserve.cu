// Page bookkeeping of one serving step, from the requests' lengths, on the
// GPU: returns the pages of finished requests to the free stack, takes pages
// for the step's new tokens from it, and writes block table, slot, position
// and offset of every new token.
//
// For request b with old tokens in the cache (0 if it just finished) and
// new_b more, have = ceil(old / page), want = ceil((old + new_b) / page):
//     need_b = want - have, upto_b = sum_{b' <= b} need_b'
//     served iff want fits the table row and (need_b = 0 or upto_b <= free)
// and page i of its need comes from the free stack's entry
// free - 1 - (upto_b - need_b) - i.  Prefix sums only, so the result does not
// depend on the order in which threads run.
//
// Latency-bound: a few kilobytes of lengths, then one slot and one position a
// token.  One launch of one cluster: every CTA computes the prefix sums for
// itself (a few hundred lengths) and takes a share of the tokens; the
// cluster's barrier separates the pushes and all reads of the lengths from
// the pops and the updates, so lengths and count may be updated in place.
// One CTA up to kSmallTokens tokens, else eight (the portable cluster size).
#include <cuda_runtime.h>

#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSmallTokens = 4096;
constexpr int kCluster = 8;

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Inclusive prefix sum over the block's threads; *all is the block's sum.
__device__ __forceinline__ long long block_scan(long long x, long long *warp_sums, long long *all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    __syncthreads();  // the previous scan's readers are done
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += v;
    }
    *all = __shfl_sync(0xffffffffu, w, 31);
    const long long below = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
    return x + (warp == 0 ? 0 : below);
}

__device__ __forceinline__ int blocks_of(long long tokens, int page) {
    return (int)((tokens + page - 1) / page);
}

__global__ void __launch_bounds__(kThreads)
paged_reserve_kernel(const PagedReserveArgs a, int ctas) {
    extern __shared__ int smem[];
    __shared__ long long warp_sums[32];
    int *cu = smem;                  // [B + 1] first new token of a request
    int *old = cu + a.batch + 1;     // [B] tokens before the step; ~tokens if not served
    int *top = old + a.batch;        // [B] stack entry of a request's first new page

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int rank = ctas > 1 ? cluster_rank() : 0;
    const int lane = threadIdx.x & 31, warp = rank * kWarps + (threadIdx.x >> 5);
    const int warps = ctas * kWarps;
    const long long capacity = min((long long)a.table_width * a.page_size, 0x7fffffffLL);
    long long count = min(max(__ldcg(a.free_count), 0), a.num_pages);

    // pages that finished requests return, in the order of requests and blocks
    if (a.finished) {
        long long base = 0;
        for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
            const int b = b0 + threadIdx.x;
            int n = 0;
            if (b < a.batch && a.finished[b])
                n = blocks_of(min((long long)max(__ldcg(a.seq_lens + b), 0), capacity), a.page_size);
            long long all;
            const long long upto = block_scan(n, warp_sums, &all) + base;
            if (b < a.batch) {
                top[b] = (int)min(count + upto - n, (long long)a.num_pages);
                old[b] = n;
            }
            base += all;
        }
        __syncthreads();
        for (int b = warp; b < a.batch; b += warps)
            for (int i = lane; i < old[b]; i += 32)
                if (top[b] + i < a.num_pages)
                    a.free_pages[top[b] + i] = __ldcg(a.block_table + (size_t)b * a.table_stride + i);
        count = min(count + base, (long long)a.num_pages);
        __syncthreads();
    }

    // pages and offsets of the new tokens
    long long tokens = 0, taken = 0, left = count;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long was = 0, add = 0;
        int need = 0;
        bool fits = true;
        if (b < a.batch) {
            was = max(__ldcg(a.seq_lens + b), 0);
            if (a.finished && a.finished[b]) was = 0;
            add = max(__ldcg(a.new_lens + b), 0);
            fits = was + add <= capacity;
            if (fits) need = blocks_of(was + add, a.page_size) - blocks_of(was, a.page_size);
        }
        long long all, all_need;
        const long long upto = block_scan(add, warp_sums, &all) + tokens;
        const long long upto_need = block_scan(need, warp_sums, &all_need) + taken;
        if (b < a.batch) {
            const bool ok = fits && (need == 0 || upto_need <= count);
            cu[b] = (int)min(upto - add, 0x7fffffffLL);
            old[b] = ok ? (int)was : ~(int)was;
            top[b] = (int)(count - 1 - (upto_need - need));  // used by served requests only
            if (ok && need > 0) left = min(left, count - upto_need);
        }
        tokens += all;
        taken += all_need;
    }
    if (threadIdx.x == 0) cu[a.batch] = (int)min(tokens, 0x7fffffffLL);
    // the stack after the step: the smallest remainder that a served request left
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) left = min(left, __shfl_xor_sync(0xffffffffu, left, o));
        __syncthreads();
        if (lane == 0) warp_sums[threadIdx.x >> 5] = left;
        __syncthreads();
        left = warp_sums[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) left = min(left, __shfl_xor_sync(0xffffffffu, left, o));
    }

    // every read of the lengths, the count and finished rows is done, every
    // push is visible
    if (ctas > 1) cluster_barrier(); else __syncthreads();

    const int end = cu[a.batch];
    for (int t = rank * kThreads + threadIdx.x; t < a.num_tokens; t += ctas * kThreads) {
        int slot = -1, position = 0;
        if (t < end) {
            int lo = 0, hi = a.batch;  // the last request with cu[b] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid; else hi = mid;
            }
            const int was = old[lo];
            if (was >= 0) {
                position = was + (t - cu[lo]);
                const int blk = position / a.page_size;
                const int have = blocks_of(was, a.page_size);
                const int page = blk < have
                                     ? __ldcg(a.block_table + (size_t)lo * a.table_stride + blk)
                                     : __ldcg(a.free_pages + (top[lo] - (blk - have)));
                slot = page < 0 || page >= a.num_pages ? -1 : page * a.page_size + (position - blk * a.page_size);
            }
        }
        a.slots[t] = slot;
        a.positions[t] = position;
    }
    for (int b = warp; b < a.batch; b += warps) {
        const int was = old[b];
        if (was < 0) continue;
        const int have = blocks_of(was, a.page_size);
        const int want = blocks_of((long long)was + (cu[b + 1] - cu[b]), a.page_size);
        for (int i = have + lane; i < want; i += 32)
            a.block_table[(size_t)b * a.table_stride + i] = __ldcg(a.free_pages + (top[b] - (i - have)));
    }
    for (int b = rank * kThreads + threadIdx.x; b < a.batch; b += ctas * kThreads) {
        const int was = old[b];
        a.cu_seqlens[b + 1] = cu[b + 1];
        a.served[b] = was >= 0;
        a.seq_lens_out[b] = was >= 0 ? was + (cu[b + 1] - cu[b]) : ~was;
    }
    if (rank == 0 && threadIdx.x == 0) {
        a.cu_seqlens[0] = 0;
        a.free_count_out[0] = (int)left;
    }
}

}  // namespace

cudaError_t paged_reserve(const PagedReserveArgs &a) {
    const size_t smem = sizeof(int) * (3 * (size_t)a.batch + 1);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            paged_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)(sizeof(int) * (3 * (size_t)kReserveMaxBatch + 1)));
        if (e != cudaSuccess) return e;
    }
    const int ctas = a.num_tokens > kSmallTokens ? kCluster : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_reserve_kernel, a, ctas);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace la
