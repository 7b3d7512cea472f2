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
// depend on the order in which threads run; the requests served with a need
// are the first ones that have one.
//
// Latency-bound: a few kilobytes of lengths, then a slot and a position a
// token.  One CTA computes the prefix sums; up to kSmallTokens tokens it writes
// the slots too (one launch).  For more (prompts) a second kernel, over all
// SMs, reads the lengths after the step and the offsets that the first has
// written and fills slots, positions and table, so lengths and count may be
// updated in place.  Measured: a step of 128 requests, 12 of them ending with 3000 pages,
// 6.8 us; 16 prompts of 270K tokens 8.0 us (7.4 in a graph; 38 when one cluster of eight
// CTAs did it all).
#include <cuda_runtime.h>

#include "la_internal.h"

namespace la {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillBlocks = 152 * 2;
constexpr int kSmallTokens = 4096;
constexpr int kFlight = 4;  // dependent loads a thread keeps in flight

struct Pair {
    long long x, y;
};

// Inclusive prefix sums of two values over the block's threads, and the
// block's totals.  sums: two rows of 32.
__device__ __forceinline__ Pair block_scan(long long x, long long y, long long (*sums)[32], Pair *all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += u, y += v;
    }
    __syncthreads();  // the previous scan's readers are done
    if (lane == 31) sums[0][warp] = x, sums[1][warp] = y;
    __syncthreads();
    // the warps' sums, scanned by every warp
    long long u = lane < warps ? sums[0][lane] : 0, v = lane < warps ? sums[1][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long p = __shfl_up_sync(0xffffffffu, u, o), q = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) u += p, v += q;
    }
    all->x = __shfl_sync(0xffffffffu, u, 31);
    all->y = __shfl_sync(0xffffffffu, v, 31);
    const long long below_x = __shfl_sync(0xffffffffu, u, warp > 0 ? warp - 1 : 0);
    const long long below_y = __shfl_sync(0xffffffffu, v, warp > 0 ? warp - 1 : 0);
    return {x + (warp > 0 ? below_x : 0), y + (warp > 0 ? below_y : 0)};
}

__device__ __forceinline__ int blocks_of(long long tokens, int page) {
    // 32-bit where it fits (a 64-bit division is many times the work)
    return tokens < 0x7fffffffLL - page ? ((int)tokens + page - 1) / page
                                        : (int)((tokens + page - 1) / page);
}

// The last entry of the ascending at[0 .. n) that is <= v (at[0] is).
__device__ __forceinline__ int last_at(const int *at, int n, int v) {
    int lo = 0;
    while (n - lo > 1) {
        const int mid = (lo + n) >> 1;
        if (at[mid] <= v) lo = mid; else n = mid;
    }
    return lo;
}

// Arrays of the step in shared memory.
struct Step {
    int *cu;     // [B + 1] first new token of a request
    int *old;    // [B] tokens before the step; ~tokens if it is not served
    int *taken;  // [B + 1] pages taken by the requests before
};
__device__ __forceinline__ Step step_arrays(int *smem, int batch) {
    return {smem, smem + batch + 1, smem + 2 * batch + 1};
}

// Slots and positions of the new tokens, and the table's new blocks; thread
// `i` of `n`.  top: the stack entry of the first page taken; pages: how many are.
__device__ __forceinline__ void fill(const PagedReserveArgs &a, const Step &s, int top, int pages, int i,
                                     int n) {
    const int end = s.cu[a.batch];
    for (int t0 = i; t0 < a.num_tokens; t0 += kFlight * n) {
        int page[kFlight], position[kFlight], row[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int t = t0 + f * n;
            page[f] = -1;
            position[f] = row[f] = 0;
            if (t >= min(end, a.num_tokens)) continue;
            const int b = last_at(s.cu, a.batch, t);
            const int was = s.old[b];
            if (was < 0) continue;
            position[f] = was + (t - s.cu[b]);
            const int blk = position[f] / a.page_size;
            row[f] = position[f] - blk * a.page_size;
            const int have = blocks_of(was, a.page_size);
            // new blocks from the stack: the table may not hold them yet
            page[f] = blk < have ? __ldcg(a.block_table + (size_t)b * a.table_stride + blk)
                                 : __ldcg(a.free_pages + (top - s.taken[b] - (blk - have)));
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int t = t0 + f * n;
            if (t >= a.num_tokens) break;
            a.slots[t] = page[f] < 0 || page[f] >= a.num_pages ? -1 : page[f] * a.page_size + row[f];
            a.positions[t] = position[f];
        }
    }
    // from the last thread down: the first ones have tokens
    for (int j = n - 1 - i; j < pages; j += n) {
        const int b = last_at(s.taken, a.batch, j);
        const int blk = blocks_of(s.old[b], a.page_size) + (j - s.taken[b]);
        a.block_table[(size_t)b * a.table_stride + blk] = __ldcg(a.free_pages + (top - j));
    }
}

template <bool FILL>
__global__ void __launch_bounds__(kMaxThreads)
paged_reserve_kernel(const __grid_constant__ PagedReserveArgs a) {
    extern __shared__ int smem[];
    __shared__ long long sums[2][32];
    const Step s = step_arrays(smem, a.batch);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int threads = blockDim.x;
    const long long capacity = min((long long)a.table_width * a.page_size, 0x7fffffffLL);
    long long count = min(max(__ldcg(a.free_count), 0), a.num_pages);

    // a request's length, finish mark and new tokens; those of the first
    // `threads` requests are loaded once
    int len = 0, add = 0;
    bool ended = false;
    auto load = [&](int b) {
        len = add = 0;
        ended = false;
        if (b < a.batch) {
            len = max(__ldcg(a.seq_lens + b), 0);
            add = max(__ldcg(a.new_lens + b), 0);
            ended = a.finished && a.finished[b] != 0;
        }
    };
    load(threadIdx.x);

    // pages that finished requests return, in the order of requests and blocks
    if (a.finished) {
        long long base = 0;
        for (int b0 = 0; b0 < a.batch; b0 += threads) {
            const int b = b0 + threadIdx.x;
            if (b0 > 0) load(b);
            const int n = ended ? blocks_of(min((long long)len, capacity), a.page_size) : 0;
            Pair all;
            const Pair upto = block_scan(n, 0, sums, &all);
            if (b < a.batch) s.taken[b] = (int)min(count + base + upto.x - n, (long long)a.num_pages);
            base += all.x;
        }
        __syncthreads();
        // entry j of the push: block j - (entries before) of the request that holds it
        const int top = (int)count, most = (int)min(count + base, (long long)a.num_pages);
        for (int j0 = top + threadIdx.x; j0 < most; j0 += kFlight * threads) {
            int page[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int j = j0 + i * threads;
                if (j >= most) break;
                const int b = last_at(s.taken, a.batch, j);
                page[i] = __ldcg(a.block_table + (size_t)b * a.table_stride + (j - s.taken[b]));
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (j0 + i * threads < most) a.free_pages[j0 + i * threads] = page[i];
        }
        count = min(count + base, (long long)a.num_pages);
        if (a.batch > threads) load(threadIdx.x);
        __syncthreads();
    }

    // offsets of the new tokens, pages for them
    Pair base = {0, 0};
    long long left = count;
    for (int b0 = 0; b0 < a.batch; b0 += threads) {
        const int b = b0 + threadIdx.x;
        if (b0 > 0) load(b);
        const long long was = ended ? 0 : len;
        const bool fits = was + add <= capacity;
        const int need =
            fits ? blocks_of(was + add, a.page_size) - blocks_of(was, a.page_size) : 0;
        Pair all;
        Pair upto = block_scan(add, need, sums, &all);
        upto.x += base.x, upto.y += base.y;
        if (b < a.batch) {
            const bool ok = fits && (need == 0 || upto.y <= count);
            s.cu[b] = (int)min(upto.x - add, 0x7fffffffLL);
            s.old[b] = ok ? (int)was : ~(int)was;
            s.taken[b] = (int)min(upto.y - need, 0x7fffffffLL);
            if (ok && need > 0) left = min(left, count - upto.y);
            a.cu_seqlens[b + 1] = (int)min(upto.x, 0x7fffffffLL);
            a.served[b] = ok;
            a.seq_lens_out[b] = (int)(ok ? was + add : was);
        }
        base.x += all.x, base.y += all.y;
    }
    if (threadIdx.x == 0) {
        s.cu[a.batch] = (int)min(base.x, 0x7fffffffLL);
        a.cu_seqlens[0] = 0;
    }
    // the stack after the step: below the last page that a served request took
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) left = min(left, __shfl_xor_sync(0xffffffffu, left, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[0][threadIdx.x >> 5] = left;
    __syncthreads();
    left = (threadIdx.x & 31) < threads >> 5 ? sums[0][threadIdx.x & 31] : count;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) left = min(left, __shfl_xor_sync(0xffffffffu, left, o));
    if (threadIdx.x == 0) a.free_count_out[0] = (int)left;
    if (FILL) fill(a, s, (int)count - 1, (int)(count - left), threadIdx.x, threads);
}

// The second kernel of a long step: every CTA takes the step's arrays from the
// first one's results.
__global__ void __launch_bounds__(kFillThreads)
paged_fill_kernel(const __grid_constant__ PagedReserveArgs a) {
    extern __shared__ int smem[];
    __shared__ long long sums[2][32];
    const Step s = step_arrays(smem, a.batch);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    long long base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kFillThreads) {
        const int b = b0 + threadIdx.x;
        int need = 0, was = 0, from = 0;
        bool ok = false;
        if (b < a.batch) {
            from = __ldcg(a.cu_seqlens + b);
            const int len = __ldcg(a.seq_lens_out + b);
            ok = __ldcg(a.served + b) != 0;
            // (not from the offsets, which stop at 2^31 - 1)
            was = ok ? len - max(__ldcg(a.new_lens + b), 0) : len;
            if (ok) need = blocks_of(len, a.page_size) - blocks_of(was, a.page_size);
        }
        Pair all;
        const Pair upto = block_scan(need, 0, sums, &all);
        if (b < a.batch) {
            s.cu[b] = from;
            s.old[b] = ok ? was : ~was;
            s.taken[b] = (int)(base + upto.x - need);
        }
        base += all.x;
    }
    if (threadIdx.x == 0) s.cu[a.batch] = __ldcg(a.cu_seqlens + a.batch);
    __syncthreads();
    const int pages = (int)base;
    fill(a, s, __ldcg(a.free_count_out) + pages - 1, pages, blockIdx.x * kFillThreads + threadIdx.x,
         gridDim.x * kFillThreads);
}

}  // namespace

cudaError_t paged_reserve(const PagedReserveArgs &a) {
    const size_t smem = sizeof(int) * (3 * (size_t)a.batch + 2);
    const size_t most = sizeof(int) * (3 * (size_t)kReserveMaxBatch + 2);
    const bool small = a.num_tokens <= kSmallTokens;
    auto kern = small ? paged_reserve_kernel<true> : paged_reserve_kernel<false>;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e == cudaSuccess && !small)
            e = cudaFuncSetAttribute(paged_fill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)most);
        if (e != cudaSuccess) return e;
    }
    // a thread per request (and, where it writes them, per token); at least 512 for the
    // pages of finished requests, hundreds each
    int threads = small && a.num_tokens > a.batch ? a.num_tokens : a.batch;
    const int least = a.finished ? 512 : 128;
    threads = threads > kMaxThreads ? kMaxThreads : threads < least ? least : (threads + 31) / 32 * 32;
    e = launch_dependent(kern, 1, threads, smem, a.stream, a);
    if (e == cudaSuccess && !small) {
        const int blocks = (a.num_tokens + kFillThreads - 1) / kFillThreads;
        e = launch_dependent(paged_fill_kernel, blocks < kFillBlocks ? blocks : kFillBlocks,
                             kFillThreads, smem, a.stream, a);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace la
