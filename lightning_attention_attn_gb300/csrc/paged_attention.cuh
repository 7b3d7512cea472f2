// Softmax attention of one new token per request over a paged key-value
// cache, the work split over the cache's length and joined: the kernels of the whole
// cache (paged_decode.cu), of chosen pages (paged_sparse.cu) and of the tokens behind a shared
// prefix (paged_prefix.cu).
//
// For request b with len tokens in the cache, query head h and its key-value
// head (h / G, G = num_heads / num_kv_heads):
//     s_t = scale q_h . k_t,   out_h = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m)
// in one pass with the running maximum m and sum l of a softmax, in fp32.
//
// Bound: every key and value is read once, G flops a byte of bf16 cache, so
// the kernel is a stream over HBM and its layout serves the loads.
//
// Split.  The work is cut into tiles of kTile tokens of one unit (a request's
// key-value head, or 16 query heads of one).  The tiles of all units, one after the
// other, are divided evenly (but for the cost of starting a unit) among a fixed
// number of CTAs, whatever the lengths are: no host copy of the lengths, no plan, the
// same launch for one long request and for many ragged ones.  A unit that lies inside one
// CTA's range is finished there; a piece of a unit leaves its unnormalised sums, maxima and
// exponential sums in the workspace (a CTA has at most two such pieces: the
// end of one unit and the start of another), and a second kernel joins the
// pieces of each unit in the order of their tokens.  Where the table bounds the
// lengths to short ones, a cluster of CTAs a unit takes the place of both.
//
// Inside a CTA each warp streams its own token groups through its own ring
// of shared-memory stages (cp.async, 16 bytes a lane) with its own running
// maximum, so the main loop has no block-wide barrier; the warps' results are
// joined once per piece.
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_internal.h"
#include "sm100_ptx.cuh"

namespace la {
namespace {

// Whose tokens a kernel streams.
enum class Kv {
    kOwn,     // all tokens of each request
    kChosen,  // the tokens of chosen pages of each request and key-value head
    kBehind,  // all tokens of each request, joined with the pieces of a shared prefix before it
    kPrefix   // the tokens of that prefix, for query heads of several requests (rows)
};

constexpr int kTile = 64;     // tokens of one tile of the work split
// Starting a unit (its page table, queries and first loads one after the other, then
// the warps' join) takes a CTA about as long as streaming kOverheadBytes.  100 requests
// of 1 to 3000 tokens, 8 key-value heads of 128, bf16: 64, 96, 128, 160, 192 KB give
// 108, 104, 101, 98, 98 us; 128 of 1 to 1500, 64 wide: 45, 42, 41, 42, 43.
constexpr int kOverheadBytes = 160 << 10;
template <typename T, int D>
constexpr int kOverhead = kOverheadBytes / (2 * kTile * D * (int)sizeof(T));  // in tiles
constexpr int kStages = 3;    // of a warp's ring: two in flight, one read
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_huge_valf();
// The running maximum is -kInf until a token is present and at least kLowest from there on,
// so that scores that are all -infinity (0 / 0: NaN) are told from no tokens (zeros).
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    // an invalid row is filled with zeros, nothing is read
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
// The same, of what is read once: it leaves L2 before what is not (the attention of 128 requests of up to 2048 own
// tokens beside a prefix of 8K, which each of four units reads: 144 -> 142 us, with other splits 160 -> 150).
__device__ __forceinline__ uint64_t once_policy() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid, uint64_t policy) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(n), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // 2 ulp; 0 below 2^-126
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
// x as two bf16 numbers, hi + lo, off by at most 2^-16 |x|: x cut off after hi's bits, and
// what that leaves (and 2^-23 x more, for where it leaves nothing).  So both have x's
// sign and neither is 0 unless x is (or, for lo, below 2^-110), and an infinity times x is
// what it is times either.  Rounding x to the nearest hi instead halves the error (2e-6 of an
// output before its own rounding, instead of 4e-6, and the same time) but lets lo be 0
// or of the other sign, which makes NaN of an infinite key or value.
struct Parts {
    uint32_t hi, lo;  // of a pair
};
__device__ __forceinline__ Parts parts_of(float x, float y) {
    constexpr float kUp = 1.f + 0x1p-23f;
    const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
    return {__byte_perm(u, v, 0x7632), pack2(fmaf(x, kUp, -__uint_as_float(u & 0xffff0000u)),
                                             fmaf(y, kUp, -__uint_as_float(v & 0xffff0000u)))};
}

// ------------------------------------------------------------ work split
// What the kernel before may have written (it can still be running when this one is
// scheduled) is never read as constant data: the lengths, which the join reads before
// its wait, through L2 (an SM's L1 may hold what an earlier call read at the same place), the rest with
// plain loads behind the wait, or what stands for it (wait_before_reads).  (A table entry serves
// several groups: reading it through L2 each time cost 4 to 15 %.)
// Length of request b as the kernels use it: inside [0, table capacity].
__device__ __forceinline__ int own_len(const PagedDecodeArgs &a, int b) {
    return min(max(__ldcg(a.seq_lens + b), 0), a.max_tokens);
}
// Blocks of n tokens (n + page_size could pass 32 bits).
__device__ __forceinline__ int blocks_of(int n, int page_size) { return n > 0 ? (n - 1) / page_size + 1 : 0; }
// Tokens that the kernels pass for it: with chosen pages, those of its entries that count,
// as if every page were full.
template <Kv KV> __device__ __forceinline__ int request_len(const PagedDecodeArgs &a, int b) {
    const int n = own_len(a, b);
    if constexpr (KV == Kv::kChosen)
        return min(blocks_of(n, a.page_size), a.chosen_count) * a.page_size;
    return n;
}
// Cost of a unit of `len` tokens, in tiles: the overhead of starting it, then its
// tiles.  A cut inside the overhead is a cut before the first tile.
template <int OVERHEAD> __device__ __forceinline__ int unit_cost(int len) {
    return len > 0 ? OVERHEAD + (len + kTile - 1) / kTile : 0;
}

// Where CTA `cta`'s range begins.  The costs of all units, request by request,
// are cut into ranges of `chunk`, CTA c taking [c chunk, (c + 1) chunk): ranges(all) of them.
struct Place {
    long long all, chunk, w;  // cost of all units, of a range, start of this one
    long long unit0;          // start of request b's units
    int b;
};

// Whole block (kThr threads): false where the CTA has no range.  The lengths are
// read once for up to kThr requests.
template <Kv KV, int kThr, int OVERHEAD, typename F>
__device__ __forceinline__ bool find_place(const PagedDecodeArgs &a, int units, int cta, Place &p, F ranges) {
    constexpr int kW = kThr / 32;
    __shared__ long long sums[kW];
    __shared__ long long found[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long total;
    // inclusive prefix sum of the costs of requests b0 .. b0 + kThr - 1
    auto scan = [&](int b0, int &t) {
        const int i = b0 + threadIdx.x;
        t = i < a.batch ? unit_cost<OVERHEAD>(request_len<KV>(a, i)) : 0;
        long long s = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += v;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = s;
        if (threadIdx.x == 0) found[0] = -1;
        __syncthreads();
        long long below = 0;
        total = 0;
#pragma unroll
        for (int v = 0; v < kW; ++v) {
            if (v < warp) below += sums[v];
            total += sums[v];
        }
        return s + below;
    };
    int t;
    long long upto = scan(0, t), sum = total;
    for (int b0 = kThr; b0 < a.batch; b0 += kThr) {
        int unused;
        scan(b0, unused);
        sum += total;
    }
    p.all = sum * units;
    const int r = ranges(p.all);
    p.chunk = max((p.all + r - 1) / r, 1LL);
    p.w = cta * p.chunk;
    if (p.w >= p.all) return false;
    long long base = 0;
    for (int b0 = 0;; b0 += kThr) {
        if (b0 > 0 || a.batch > kThr) upto = scan(b0, t);
        // one request holds w: the first whose inclusive count passes it
        if (t > 0 && p.w >= (base + upto - t) * units && p.w < (base + upto) * units) {
            found[0] = b0 + threadIdx.x;
            found[1] = base + upto - t;
        }
        __syncthreads();
        if (found[0] >= 0 || b0 + kThr >= a.batch) break;
        base += total;
    }
    p.b = (int)found[0];
    p.unit0 = found[1] * units;
    return p.b >= 0;
}

// n / d of two costs: 32-bit where it fits.
__device__ __forceinline__ int tiles_div(long long n, int d) {
    return (n >> 32) == 0 ? (int)((uint32_t)n / (uint32_t)d) : (int)(n / d);
}

// The first request from b on that has tokens, and how many (whole warps); a.batch: none.
// Idle rows of a large batch are passed 128 at a time: 5000 of them between two requests of
// 30000 tokens take 95 us (none of them 35), one by one, each load behind the last, 1105.
template <Kv KV>
__device__ __forceinline__ int next_request(const PagedDecodeArgs &a, int b, int &len) {
    constexpr int kLook = 4;
    const int lane = threadIdx.x & 31;
    for (; b < a.batch; b += 32 * kLook) {
        int lens[kLook];
#pragma unroll
        for (int i = 0; i < kLook; ++i) {
            const int at = b + i * 32 + lane;
            lens[i] = at < a.batch ? request_len<KV>(a, at) : 0;
        }
#pragma unroll
        for (int i = 0; i < kLook; ++i) {
            const uint32_t has = __ballot_sync(0xffffffffu, lens[i] > 0);
            if (has) {
                const int first = __ffs(has) - 1;
                len = __shfl_sync(0xffffffffu, lens[i], first);
                return b + i * 32 + first;
            }
        }
    }
    return a.batch;
}

// Where piece `first` (of a unit that CTA c does not hold whole) of CTA c lives in
// the workspace: sums of `rows` heads x D, then their maxima and exponential
// sums.
template <int D>
__device__ __forceinline__ float *piece_at(const PagedDecodeArgs &a, int c, bool first, int rows) {
    return a.workspace + ((size_t)c * 2 + (first ? 0 : 1)) * rows * (D + 2);
}

// Tiles of a shared prefix, and how many of all units' a CTA streams.
__device__ __forceinline__ int prefix_tiles(const PrefixPieces &f) {
    return (min(max(__ldcg(f.len), 0), f.max_tokens) + f.tile - 1) / f.tile;
}
__device__ __forceinline__ long long prefix_chunk(const PrefixPieces &f, int tiles, int ranges) {
    return ((long long)f.units * tiles + ranges - 1) / ranges;
}

// SMs for the prefix on the tensor cores where the own tokens' split kernel can run on the others meanwhile
// (and has as many ranges as those hold at once): the number for which both are done first, or all SMs, one
// kernel behind the other, which costs kBehindUs more.  A tile takes an SM about kTileUs (two where the groups
// share it), kBesideUs beside the other kernel; own tokens, `cost` tiles of them, stream at kHbm, from
// fewer than kFullSms SMs at that share of it.  A tile's times, from the prefix alone and from what bounds the calls
// below: 128 wide 1.2 (shared) to 1.5 us and 2.0 beside, 64 wide 0.9 to 1.1 and 1.2 to 1.5.  Measured,
// 64 and 8 heads of 128 (of 64), for the rule's choice / the best of ten numbers / all SMs: 128
// requests of up to 2048 own tokens behind 8K 145 / 144 / 175 us (104 / 103 / 116), of up to 8192 behind 2K 335 / 335 /
// 362 (192 / 192 / 203), 64 of up to 2048 behind 32K 153 / 153 / 168 (117 / 114 / 121), 256 of up to 1024 behind 4K
// 160 / 154 / 176, 32 of up to 8192 behind 16K 135 / 131 / 158 (87 / 85 / 101), 16 of up to 16K behind 128K 207 / 195 /
// 210 (123 / 123 / 136).  With 304 ranges, in waves of what is free, the first took 162 (149 then).
template <int D> constexpr float kTileUs = D == 128 ? 1.5f : 1.1f;
template <int D> constexpr float kBesideUs = D == 128 ? 2.f : 1.4f;
constexpr float kHbm = 6.7e6f /* bytes a us */, kFullSms = 110.f, kBehindUs = 20.f;

// (Whole warps; a lane a number.)
template <int D> __device__ __forceinline__ int ranges_beside(const PrefixPieces &f, int tiles, long long cost) {
    const int lane = threadIdx.x & 31, n = f.ctas - 4 * lane;
    const float work = (float)prefix_chunk(f, tiles, n) * (f.parts == 1 ? 2.f : 1.f);  // tiles of an SM
    const float stream = (float)cost * (kTile * D * 4) / kHbm;
    const float beside = stream / fminf(1.f, (f.ctas - n) / kFullSms);
    const uint32_t us = __float_as_uint(lane ? fmaxf(work * kBesideUs<D>, beside)
                                                  : work * kTileUs<D> + stream + kBehindUs);
    const uint32_t least = __reduce_min_sync(0xffffffffu, us);
    return f.ctas - 4 * (__ffs(__ballot_sync(0xffffffffu, us == least)) - 1);
}

// The range of `chunk` that place w is in: 32-bit where it fits.
__device__ __forceinline__ int range_of(long long w, long long chunk) {
    return ((w | chunk) >> 32) == 0 ? (int)((uint32_t)w / (uint32_t)chunk) : (int)(w / chunk);
}

// Where columns d .. d + 3 of a row's sums in a piece are, and its maximum and exponential sum.
struct PieceRow {
    const float *x, *m;
};
// Those of a shared prefix's pieces of a row of the output, in the order of their tokens: the row's unit's
// part of every CTA that streamed some of the unit's tiles (PrefixPieces).
struct PrefixRow {
    const float *x = nullptr, *m = nullptr;
    size_t size = 0;
    int n = 0;

    __device__ __forceinline__ PrefixRow(const PagedDecodeArgs &a, size_t row, int d) {
        const PrefixPieces &f = a.prefix;
        const int tiles = prefix_tiles(f);
        if (tiles == 0) return;
        const int b = (int)(row / a.num_heads), head = (int)(row - (size_t)b * a.num_heads);
        const int kvh = head / a.group, r = b * a.group + head - kvh * a.group;
        const int unit = kvh * f.units_per_head + r / f.unit_rows, in = r % f.unit_rows;
        const long long chunk = prefix_chunk(f, tiles, __ldcg(f.ranges)), w = (long long)unit * tiles;
        const int c0 = range_of(w, chunk), c1 = range_of(w + tiles - 1, chunk);
        // (the further parts of a CTA with a single tile are empty, and not written)
        const int parts = chunk == 1 ? 1 : f.parts;
        const size_t slot = (size_t)f.stride * (a.head_dim + 2);
        n = (c1 - c0 + 1) * parts;
        size = slot * (chunk == 1 ? f.parts : 1);
        const float *at = f.pieces + (size_t)(c0 + unit) * f.parts * slot;
        x = at + (size_t)in * a.head_dim + d;
        m = at + (size_t)f.stride * a.head_dim + 2 * in;
    }
    __device__ __forceinline__ PieceRow piece(int i) const { return {x + i * size, m + i * size}; }
};

// Four columns of one head's softmax in the making: maximum, exponential sum,
// unnormalised values.
struct Partial {
    float m, sum;
    float4 acc;

    __device__ Partial() : m(-kInf), sum(0.f), acc(make_float4(0.f, 0.f, 0.f, 0.f)) {}

    // Adds pieces from, from + step, ... of a list, kFlight of them in flight together.
    template <typename F> __device__ __forceinline__ void add_list(int from, int n, int step, F at) {
        constexpr int kFlight = 8;
        for (int i0 = from; i0 < n; i0 += kFlight * step) {
            float4 x[kFlight];
            float2 ms[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const int i = i0 + f * step;
                x[f] = make_float4(0.f, 0.f, 0.f, 0.f);
                ms[f] = make_float2(-kInf, 0.f);
                if (i < n) {
                    const PieceRow p = at(i);
                    x[f] = __ldcg(reinterpret_cast<const float4 *>(p.x));
                    ms[f] = __ldcg(reinterpret_cast<const float2 *>(p.m));
                }
            }
            add<kFlight>(ms, x);
        }
    }

    // Adds N others: their maxima and sums in ms, values in x.
    template <int N>
    __device__ __forceinline__ void add(const float2 (&ms)[N], const float4 (&x)[N]) {
        float top = m;
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, ms[i].x);
        const float base = top == -kInf ? 0.f : top;
        const float k = ex2(m - base);
        m = top;
        sum *= k;
        acc.x *= k, acc.y *= k, acc.z *= k, acc.w *= k;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float e = ex2(ms[i].x - base);
            sum = fmaf(ms[i].y, e, sum);
            acc.x = fmaf(x[i].x, e, acc.x);
            acc.y = fmaf(x[i].y, e, acc.y);
            acc.z = fmaf(x[i].z, e, acc.z);
            acc.w = fmaf(x[i].w, e, acc.w);
        }
    }
    // Writes columns d .. d + 3 of the output's row (and its lse).
    template <typename T, Kv KV>
    __device__ __forceinline__ void write(const PagedDecodeArgs &a, size_t row, int d) {
        if constexpr (KV == Kv::kBehind) {
            const PrefixRow f(a, row, d);
            add_list(0, f.n, 1, [&](int i) { return f.piece(i); });
        }
        const float r = m == -kInf ? 0.f : 1.f / sum;  // no token; a sum of 0 gives NaN
        T *o = static_cast<T *>(a.out) + row * a.head_dim + d;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack2(acc.x * r, acc.y * r), pack2(acc.z * r, acc.w * r));
        else
            *reinterpret_cast<float4 *>(o) = make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
        if (a.lse && d == 0)
            a.lse[row] = sum != 0.f ? (m + log2f(sum)) * (1.f / kLog2e) : -kInf;
    }
};

// Dependent launches: the lengths, the table and the cache may have been written by the kernel
// before.  Behind a shared prefix that kernel is the prefix's, all of whose CTAs have waited for whatever wrote
// them before this one is scheduled.  That orders the two but makes nothing visible here: for that the prefix's
// kernel then releases f.ranges[2], and every thread here acquires it (which also lets go of L1's lines) in place of
// a wait.  Only the prefix's pieces are still to come, and what reads
// those waits for them (in the cluster kernel every CTA before its rows; the split kernel does not read
// them, but its last CTA waits, so that whoever waits for this kernel has waited for the prefix's too).  The
// join behind the split kernel reads the lengths before its wait, through L2: the split kernel has not waited,
// but does not run before the prefix's has.  (128 requests of up to 2048 own tokens behind 8K: 142 us; with the
// table through L2 in place of the acquire 154.)
template <Kv KV> __device__ __forceinline__ void wait_before_reads(const PagedDecodeArgs &a) {
    if constexpr (KV != Kv::kBehind) ptx::grid_dependency_wait();
    else ptx::load_acquire(a.prefix.ranges + 2);
    ptx::grid_launch_dependents();
}
template <Kv KV> __device__ __forceinline__ void wait_before_rows() {
    if constexpr (KV == Kv::kBehind) ptx::grid_dependency_wait();
}

// Zeros for the requests without tokens, which are nobody's tiles.
template <typename T>
__device__ __forceinline__ void write_empty(const PagedDecodeArgs &a) {
    const int row = a.num_heads * a.head_dim;
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (own_len(a, b) != 0) continue;
        for (int i = threadIdx.x; i < row; i += blockDim.x)
            static_cast<T *>(a.out)[(size_t)b * row + i] = T(0.f);
        if (a.lse)
            for (int i = threadIdx.x; i < a.num_heads; i += blockDim.x)
                a.lse[(size_t)b * a.num_heads + i] = -kInf;
    }
}

// What a core leaves in shared memory, and its sum over the warps.
template <typename Core>
__device__ __forceinline__ Partial warps_sum(const unsigned char *smem, int h, int d) {
    const float *ow = reinterpret_cast<const float *>(smem);
    const float2 *ml = reinterpret_cast<const float2 *>(ow + Core::W * Core::ROWS * Core::D);
    float2 ms[Core::W];
    float4 x[Core::W];
#pragma unroll
    for (int w = 0; w < Core::W; ++w) {
        ms[w] = ml[w * Core::ROWS + h];
        x[w] = *reinterpret_cast<const float4 *>(ow + (w * Core::ROWS + h) * Core::D + d);
    }
    Partial p;
    p.add<Core::W>(ms, x);
    return p;
}

// Where the tokens of a unit lie.  Token t of the unit is row t % page_size of the page of its
// block t / page_size; with chosen pages that block is an entry of the choice, whose block
// may be none of the request's (then, as behind the request's last token, nothing is there).
template <Kv KV> struct Tokens {
    const int32_t *pages, *chosen;
    int len, blocks;

    __device__ __forceinline__ Tokens(const PagedDecodeArgs &a, int b, int kvh)
        : pages(a.block_table + (KV == Kv::kPrefix ? 0 : (size_t)b * a.table_stride)),
          chosen(nullptr), len(0), blocks(0) {
        if constexpr (KV == Kv::kChosen) {
            chosen = a.chosen + ((size_t)b * a.num_kv_heads + kvh) * a.chosen_count;
            len = own_len(a, b);
            blocks = blocks_of(len, a.page_size);
        }
    }
    // The block and row of token t (-1: behind t1).
    __device__ __forceinline__ void block(const PagedDecodeArgs &a, int t, int t1, int &blk, int &row) const {
        blk = -1;
        row = 0;
        if (t < t1) {
            blk = t / a.page_size;
            row = t - blk * a.page_size;
            if constexpr (KV == Kv::kChosen) blk = chosen[blk];
        }
    }
    // Its page, or -1; pages that are none are left to the page's first use.
    __device__ __forceinline__ int page(const PagedDecodeArgs &a, int blk, int row) const {
        if constexpr (KV == Kv::kChosen)
            return blk >= 0 && blk < blocks && row < len - blk * a.page_size ? pages[blk] : -1;
        return blk >= 0 ? pages[blk] : -1;
    }
    // Page and row of token t at once.
    __device__ __forceinline__ void locate(const PagedDecodeArgs &a, int t, int t1, int &page, int &row) const {
        page = -1;
        row = 0;
        if (t < t1) {
            const int blk = t / a.page_size;
            row = t - blk * a.page_size;
            page = pages[blk];
        }
    }
};

// Query row h of a unit.
template <Kv KV, typename T, int D>
__device__ __forceinline__ const T *query_row(const PagedDecodeArgs &a, int b, int kvh, int head0, int h) {
    if constexpr (KV == Kv::kPrefix) {
        const int r = head0 + h, request = r / a.group;
        return static_cast<const T *>(a.q) + (size_t)request * a.q_stride +
               (size_t)(kvh * a.group + r - request * a.group) * D;
    }
    return static_cast<const T *>(a.q) + (size_t)b * a.q_stride + (size_t)(head0 + h) * D;
}

// The table's entries are read a group ahead of their use (the choice's two groups ahead).  The tokens of group g of a
// piece from token t0 are t0 + g GROUP .. + GROUP - 1, of which `in` is the lane's; its warp takes every W-th
// group.  BRANCH: an entry is loaded where its block is found, in one branch, rather than behind it by whether there
// is a block.  bf16, in a branch / behind it: 1 x 128K tokens 88.6 / 88.9 us, a step of 20 requests 58.5 / 58.8, 1 x 300
// tokens 5.20 / 5.28; fp32, 33 requests: 29.9 / 29.2.
template <Kv KV, int AHEAD, int GROUP, int W, bool BRANCH> struct Finder {
    Tokens<KV> at;
    int page, row;   // of the group that is issued next
    int blk2, row2;  // of the one behind it (chosen pages only)

    __device__ __forceinline__ Finder(const PagedDecodeArgs &a, int b, int kvh) : at(a, b, kvh) {}
    __device__ __forceinline__ void start(const PagedDecodeArgs &a, int t0, int in, int g, int t1,
                                          int (&page0)[AHEAD], int (&row0)[AHEAD]) {
        if constexpr (KV != Kv::kChosen && BRANCH) {
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) at.locate(a, t0 + (g + s * W) * GROUP + in, t1, page0[s], row0[s]);
            at.locate(a, t0 + (g + AHEAD * W) * GROUP + in, t1, page, row);
            return;
        }
        int blk0[AHEAD], blk;
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) at.block(a, t0 + (g + s * W) * GROUP + in, t1, blk0[s], row0[s]);
        at.block(a, t0 + (g + AHEAD * W) * GROUP + in, t1, blk, row);
        if constexpr (KV == Kv::kChosen) at.block(a, t0 + (g + (AHEAD + 1) * W) * GROUP + in, t1, blk2, row2);
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) page0[s] = at.page(a, blk0[s], row0[s]);
        page = at.page(a, blk, row);
    }
    // To group g, which is issued next.
    __device__ __forceinline__ void next(const PagedDecodeArgs &a, int t0, int in, int g, int t1) {
        if constexpr (KV == Kv::kChosen) {
            page = at.page(a, blk2, row2);
            row = row2;
            at.block(a, t0 + (g + W) * GROUP + in, t1, blk2, row2);
        } else if constexpr (BRANCH) {
            at.locate(a, t0 + g * GROUP + in, t1, page, row);
        } else {
            int blk;
            at.block(a, t0 + g * GROUP + in, t1, blk, row);
            page = at.page(a, blk, row);
        }
    }
};

// --------------------------------------------------------------- bf16 core
// A core streams tokens [t0, t1) of one unit through the block and leaves, per
// warp and head, the sums [W][ROWS][D] and (maximum, exponential sum) [W][ROWS] in shared
// memory (every warp has written when the block next synchronises).
//
// Heads of the query in the columns of the products (N = 8, NT such tiles):
//     S^T [16 tokens x 8] = K [16 x D] Q^T,   O^T [D x 8] += V^T [D x 16] P^T
// K and V are the A operands straight from shared memory (V transposed by
// ldmatrix), so up to 8 (16) query heads share one read of the cache and no
// row of an MMA is padding when G is 8 (16).  P^T is S^T's accumulator as two
// bf16 operands (P = hi + lo, 2^-16 relative; parts_of): the tensor pipe is idle most of
// the time and the second product keeps the error far below the output's rounding.
// fp32 queries are split alike.  O^T of a group is added to the running sums on the CUDA
// cores: the tensor core drops the bits that do not fit where the CUDA cores round to
// nearest, which over the 500 groups a warp adds up at 64 requests of 9K to 32K tokens made
// the sums 7e-6 too small (now 1e-7).  It costs 2 % at 64 wide with 16 heads a kv head
// (37.2 -> 38.1 us), less than 0.5 % elsewhere.
// mma.sync rather than tcgen05: with 8 columns the products keep the tensor pipe 12 to
// 15 % busy while HBM is at its limit, and accumulators in registers feed the softmax
// without a trip through tensor memory.
// Four warps of a 16-token, 8 KB stage (D = 128) or eight of 4 KB (D = 64): two CTAs
// an SM either way, 128 KB in flight.  Measured, 8 key-value heads of 128: 128 requests of
// 1K to 32K tokens 1260 us (7.0 TB/s), one of 128K 88 us, 20 of 4096 58 us; of 64, 20 x
// 8192 59 us (with four warps 70).  One CTA of eight warps an SM instead: 62 us for the
// 20 x 4096, 40 instead of 31 for 100 requests up to 600 tokens.  (Of the variants one, 64 wide
// with fp32 queries of 9 to 16 heads, spills: 48 bytes at its 128 registers.)
template <Kv KV_, int D_, int NT, bool QF32>
struct Bf16Core {
    using T = __nv_bfloat16;
    static constexpr Kv KV = KV_;
    static constexpr int D = D_, ROWS = 8 * NT, W = D == 128 ? 4 : 8, kThreads = 32 * W;
    static constexpr int kGroup = 16;               // tokens of one warp step
    static constexpr int kRow = D * 2;              // bytes of a token row
    static constexpr int kMat = kGroup * kRow;      // bytes of K (V) of a stage
    static constexpr int kStageBytes = 2 * kMat;
    static constexpr int kSmem = W * kStages * kStageBytes;

    static __device__ __forceinline__ void stream(const PagedDecodeArgs &a, unsigned char *smem, int b,
                                                  int kvh, int head0, int heads, int t0, int t1) {
        constexpr int KS = D / 16;   // k steps of S, row tiles of O^T
        constexpr int CH = D / 8;    // 16-byte chunks of a row
        constexpr int RPI = 32 / CH; // rows one warp-wide copy covers
        constexpr int kAhead = NT == 1 ? 4 : 2;  // fragments loaded ahead (registers)
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int g = lane >> 2, c2 = (lane & 3) * 2;
        const uint32_t ring = ptx::smem_u32(smem) + warp * kStages * kStageBytes;
        const int crow = lane / CH, cch = lane % CH;
        // ldmatrix row addresses: K as rows, V transposed
        const int krow = lane & 15, kchunk = lane >> 4;
        const int vrow = (lane & 7) + ((lane >> 4) << 3), vchunk = (lane >> 3) & 1;

        const int groups = (t1 - t0 + kGroup - 1) / kGroup;  // of the whole piece
        // This warp's groups: warp, warp + W, ...; lane r < 16 finds row
        // r of a group: its offset inside a key (value) head's page, or -1.
        Finder<KV, kStages - 1, kGroup, W, true> find(a, b, kvh);
        // the prefix's kernel runs beside this one and reads its keys and values again for every unit
        uint64_t policy = 0;
        if constexpr (KV == Kv::kBehind) policy = once_policy();
        // Issues the copies of one group; returns the mask of its present rows.
        auto issue = [&](int stage, int page, int row) -> uint32_t {
            if (page >= a.num_pages) page = -1;  // first use of the table's entry, a group after its load
            const uint32_t have = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
            const uint32_t dk = ring + stage * kStageBytes, dv = dk + kMat;
#pragma unroll
            for (int i = 0; i < kGroup / RPI; ++i) {
                const int r = i * RPI + crow;
                const int pg = __shfl_sync(0xffffffffu, page, r);
                const int rw = __shfl_sync(0xffffffffu, row, r);
                const bool ok = pg >= 0;
                const size_t in = ((size_t)kvh * a.page_size + rw) * D + cch * 8;
                const size_t p = ok ? pg : 0;
                const uint32_t off = r * kRow + ((cch ^ (r & 7)) << 4);
                const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + p * a.k_page_stride + in;
                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + p * a.v_page_stride + in;
                if constexpr (KV == Kv::kBehind) {
                    cp_async16(dk + off, k, ok, policy);
                    cp_async16(dv + off, v, ok, policy);
                } else {
                    cp_async16(dk + off, k, ok);
                    cp_async16(dv + off, v, ok);
                }
            }
            return have;
        };

        // The first groups' table entries together, then bf16 queries, then the copies
        // (fp32 queries, which are converted, behind them): one latency of each.
        int page0[kStages - 1], row0[kStages - 1];
        find.start(a, t0, lane & 15, warp, t1, page0, row0);

        // queries as B operands, scaled after the product
        uint32_t qb[NT][KS][2], ql[QF32 ? NT : 1][QF32 ? KS : 1][2];
        if (!QF32) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const __nv_bfloat16 *qp = query_row<KV, __nv_bfloat16, D>(a, b, kvh, head0, nt * 8 + g) + c2;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qb[nt][ks][i] = nt * 8 + g < heads ? __ldcg(reinterpret_cast<const uint32_t *>(
                                                                 qp + ks * 16 + i * 8))
                                                           : 0u;
            }
        }
        uint32_t have[kStages];
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            have[s] = issue(s, page0[s], row0[s]);  // copies nothing past the end
            cp_commit();
        }
        if (QF32) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float *qp = query_row<KV, float, D>(a, b, kvh, head0, nt * 8 + g) + c2;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float2 x = make_float2(0.f, 0.f);
                        if (nt * 8 + g < heads)
                            x = __ldcg(reinterpret_cast<const float2 *>(qp + ks * 16 + i * 8));
                        const Parts p = parts_of(x.x, x.y);
                        qb[nt][ks][i] = p.hi;
                        ql[nt][ks][i] = p.lo;
                    }
            }
        }
        float o[NT][KS][4];
        float mx[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = mx[nt][1] = -kInf;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                o[nt][ks][0] = o[nt][ks][1] = o[nt][ks][2] = o[nt][ks][3] = 0.f;
        }

        int stage = 0;
        for (int grp = warp; grp < groups; grp += W) {
            // refill the stage that was read last (its readers are this warp)
            {
                const int nx = grp + (kStages - 1) * W;
                const int ns = stage == 0 ? kStages - 1 : stage - 1;
                __syncwarp();
                have[kStages - 1] = 0;
                if (nx < groups) have[kStages - 1] = issue(ns, find.page, find.row);
                cp_commit();
                find.next(a, t0, lane & 15, nx + W, t1);
            }
            cp_wait<kStages - 1>();
            __syncwarp();
            const uint32_t kb = ring + stage * kStageBytes, vb = kb + kMat;

            // Few warps share an SM, so a warp's own latencies count: the
            // fragments are loaded ahead of their products, and the scores are summed in
            // two (with split queries four) independent chains.
            float s[NT][4], s2[NT][4], s3[QF32 ? NT : 1][4], s4[QF32 ? NT : 1][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[nt][i] = s2[nt][i] = 0.f;
                    if (QF32) s3[nt][i] = s4[nt][i] = 0.f;
                }
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += kAhead) {
                uint32_t ka[kAhead][4];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    ldsm4(ka[i], kb + krow * kRow +
                                     (((2 * (k0 + i) + kchunk) ^ (krow & 7)) << 4));
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int ks = k0 + i;
                        mma16816(i & 1 ? s2[nt] : s[nt], ka[i], qb[nt][ks][0], qb[nt][ks][1]);
                        if (QF32)
                            mma16816(i & 1 ? s4[nt] : s3[nt], ka[i], ql[nt][ks][0], ql[nt][ks][1]);
                    }
            }
            uint32_t va[kAhead][4];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                ldsm4_t(va[i], vb + vrow * kRow + (((2 * i + vchunk) ^ (vrow & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[nt][i] += s2[nt][i];
                    if (QF32) s[nt][i] += s3[nt][i] + s4[nt][i];
                }
            const bool v0 = (have[0] >> g) & 1, v1 = (have[0] >> (g + 8)) & 1;
            const float least = have[0] ? kLowest : -kInf;
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // this lane's two heads
                    s[nt][j] = v0 ? s[nt][j] * a.scale_log2 : -kInf;
                    s[nt][2 + j] = v1 ? s[nt][2 + j] * a.scale_log2 : -kInf;
                }
                float t0m = fmaxf(fmaxf(s[nt][0], s[nt][2]), least);
                float t1m = fmaxf(fmaxf(s[nt][1], s[nt][3]), least);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    t0m = fmaxf(t0m, __shfl_xor_sync(0xffffffffu, t0m, d));
                    t1m = fmaxf(t1m, __shfl_xor_sync(0xffffffffu, t1m, d));
                }
                // a maximum that rose rescales what was summed
                if (__any_sync(0xffffffffu, t0m > mx[nt][0] || t1m > mx[nt][1])) {
                    const float n0 = fmaxf(mx[nt][0], t0m), n1 = fmaxf(mx[nt][1], t1m);
                    const float f0 = n0 == -kInf ? 1.f : ex2(mx[nt][0] - n0);
                    const float f1 = n1 == -kInf ? 1.f : ex2(mx[nt][1] - n1);
                    mx[nt][0] = n0;
                    mx[nt][1] = n1;
                    l[nt][0] *= f0;
                    l[nt][1] *= f1;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        o[nt][ks][0] *= f0;
                        o[nt][ks][1] *= f1;
                        o[nt][ks][2] *= f0;
                        o[nt][ks][3] *= f1;
                    }
                }
                const float b0 = mx[nt][0] == -kInf ? 0.f : mx[nt][0];
                const float b1 = mx[nt][1] == -kInf ? 0.f : mx[nt][1];
                const float p0 = ex2(s[nt][0] - b0), p1 = ex2(s[nt][1] - b1);
                const float p2 = ex2(s[nt][2] - b0), p3 = ex2(s[nt][3] - b1);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                const Parts a0 = parts_of(p0, p1), a1 = parts_of(p2, p3);
                ph[nt][0] = transpose8x8(a0.hi);
                ph[nt][1] = transpose8x8(a1.hi);
                pl[nt][0] = transpose8x8(a0.lo);
                pl[nt][1] = transpose8x8(a1.lo);
            }
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += kAhead) {
                if (k0 > 0) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i)
                        ldsm4_t(va[i], vb + vrow * kRow +
                                           (((2 * (k0 + i) + vchunk) ^ (vrow & 7)) << 4));
                }
                float x[kAhead][NT][4];  // the group's products
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        x[i][nt][0] = x[i][nt][1] = x[i][nt][2] = x[i][nt][3] = 0.f;
                        mma16816(x[i][nt], va[i], pl[nt][0], pl[nt][1]);
                    }
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(x[i][nt], va[i], ph[nt][0], ph[nt][1]);
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[nt][k0 + i][j] += x[i][nt][j];
            }
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) have[i] = have[i + 1];
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        cp_wait<0>();

        // the warps' results
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], d);
        float *ow = reinterpret_cast<float *>(smem);
        float2 *ml = reinterpret_cast<float2 *>(ow + W * ROWS * D);
        __syncthreads();  // every warp has read its stages
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (g == 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ml[warp * ROWS + nt * 8 + c2 + j] = make_float2(mx[nt][j], l[nt][j]);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ow[(warp * ROWS + nt * 8 + c2 + (i & 1)) * D + ks * 16 + g + (i >> 1) * 8] =
                        o[nt][ks][i];
        }
    }
};

// --------------------------------------------------------------- fp32 core
// The CUDA cores (fp32 products, as the library's other fp32 paths).  ROWS (4, 8 or
// 16) query heads of a unit.
//   scores   LPT lanes share a token; each keeps DPL dimensions of all queries in
//            registers, and a transposing reduction over the LPT lanes leaves one
//            head's score in each
//   softmax  over the group's scores in shared memory, lane = (head, token), so
//            every exponential is taken once
//   values   a lane owns four columns of all heads (of every other token where 16
//            lanes cover a row)
// A group is 16 tokens of 64 dimensions or 8 of 128: 8 KB a stage, as in bf16.
// 16 requests of 64K / (kv heads) tokens, 128 wide: 165 us with one query head a kv head (6.5
// TB/s), 170 with four, 178 with eight (6.0), 335 with 16 (3.2).  There it is bound by the
// latencies of its own instructions, not by a pipe: twice the instructions of eight heads
// (a lane keeps four dimensions, so every score goes through more of the reduction, and
// the weights of 16 heads are read back), issued in 47 % of the slots by two warps a
// scheduler, the fp32 pipe 44 % and the shared memory 36 % busy, HBM at 39 %.
template <Kv KV_, int D_, int ROWS_>
struct F32Core {
    using T = float;
    static constexpr Kv KV = KV_;
    static constexpr int D = D_, ROWS = ROWS_, W = 4, kThreads = 32 * W;
    static constexpr int kGrp = 1024 / D;           // tokens of a group
    static constexpr int DPL = ROWS == 16 ? 4 : 8;  // dimensions of a lane's scores
    static constexpr int LPT = D / DPL;             // lanes of a token
    static constexpr int kMat = kGrp * D;           // floats of K (V) of a stage
    static constexpr int kScores = W * kGrp * ROWS;
    static constexpr int kSmem = sizeof(float) * (kScores + W * kStages * 2 * kMat);

    static __device__ __forceinline__ void stream(const PagedDecodeArgs &a, unsigned char *smem, int b,
                                                  int kvh, int head0, int heads, int t0, int t1) {
        constexpr int TPP = 32 / LPT;    // tokens whose scores a pass computes
        constexpr int TS = 32 / ROWS;    // tokens of a softmax step
        constexpr int CH = D / 4;        // 16-byte chunks of a row
        constexpr int RPI = 32 / CH;     // rows of a warp-wide copy, tokens of a value step
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float *base = reinterpret_cast<float *>(smem);
        float *pw = base + warp * kGrp * ROWS;  // [kGrp][ROWS] of this warp
        float *ring = base + kScores + warp * kStages * 2 * kMat;
        const uint32_t ring_u = ptx::smem_u32(ring);
        const int sub = lane % LPT, sh = lane % ROWS;
        // the head whose score the reduction leaves in this lane
        int my_head = 0;
        {
            int n = ROWS;
#pragma unroll
            for (int o = LPT / 2; o > 0; o >>= 1)
                if (n > 1) {
                    n >>= 1;
                    if (lane & o) my_head += n;
                }
        }

        const int groups = (t1 - t0 + kGrp - 1) / kGrp;
        Finder<KV, kStages - 1, kGrp, W, false> find(a, b, kvh);
        auto issue = [&](int stage, int page, int row) -> uint32_t {
            if (page >= a.num_pages) page = -1;  // first use of the table's entry, a group after its load
            const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
            const uint32_t dk = ring_u + stage * 2 * kMat * 4, dv = dk + kMat * 4;
            const int ch = lane % CH;
#pragma unroll
            for (int i = 0; i < kGrp / RPI; ++i) {
                const int r = i * RPI + lane / CH;
                const int pg = __shfl_sync(0xffffffffu, page, r);
                const int rw = __shfl_sync(0xffffffffu, row, r);
                const bool ok = pg >= 0;
                const size_t p = ok ? pg : 0;
                const size_t in = ((size_t)kvh * a.page_size + rw) * D + ch * 4;
                const uint32_t off = r * D * 4 + ((ch ^ (r & 7)) << 4);
                cp_async16(dk + off, static_cast<const float *>(a.k) + p * a.k_page_stride + in, ok);
                cp_async16(dv + off, static_cast<const float *>(a.v) + p * a.v_page_stride + in, ok);
            }
            return have;
        };
        int page0[kStages - 1], row0[kStages - 1];
        find.start(a, t0, lane % kGrp, warp, t1, page0, row0);
        uint32_t have[kStages];
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            have[s] = issue(s, page0[s], row0[s]);
            cp_commit();
        }

        // chunk sub + i LPT of every query row
        float2 q[ROWS][DPL / 2];
#pragma unroll
        for (int h = 0; h < ROWS; ++h)
#pragma unroll
            for (int i = 0; i < DPL / 4; ++i) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (h < heads)
                    x = __ldcg(reinterpret_cast<const float4 *>(query_row<KV, float, D>(a, b, kvh, head0, h) +
                                                                (sub + i * LPT) * 4));
                q[h][2 * i] = make_float2(x.x, x.y);
                q[h][2 * i + 1] = make_float2(x.z, x.w);
            }
        float2 o[ROWS][2];
        float mx = -kInf, l = 0.f;  // of head sh (l: this lane's tokens)
#pragma unroll
        for (int h = 0; h < ROWS; ++h) o[h][0] = o[h][1] = make_float2(0.f, 0.f);

        int stage = 0;
        for (int grp = warp; grp < groups; grp += W) {
            {
                const int ns = stage == 0 ? kStages - 1 : stage - 1;
                __syncwarp();
                have[kStages - 1] = issue(ns, find.page, find.row);  // copies nothing past the end
                cp_commit();
                find.next(a, t0, lane % kGrp, grp + kStages * W, t1);
            }
            cp_wait<kStages - 1>();
            __syncwarp();
            const float *kb = ring + stage * 2 * kMat, *vb = kb + kMat;

#pragma unroll
            for (int t = 0; t < kGrp; t += TPP) {
                const int r = t + lane / LPT;
                float2 acc[ROWS];
#pragma unroll
                for (int i = 0; i < DPL / 4; ++i) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(
                        kb + r * D + (((sub + i * LPT) ^ (r & 7)) << 2));
#pragma unroll
                    for (int h = 0; h < ROWS; ++h) {
                        const float2 lo = make_float2(k4.x, k4.y), hi = make_float2(k4.z, k4.w);
                        acc[h] = i == 0 ? ptx::f2_mul(lo, q[h][0]) : ptx::f2_fma(lo, q[h][2 * i], acc[h]);
                        acc[h] = ptx::f2_fma(hi, q[h][2 * i + 1], acc[h]);
                    }
                }
                float v[ROWS];
#pragma unroll
                for (int h = 0; h < ROWS; ++h) v[h] = acc[h].x + acc[h].y;
                int n = ROWS;
#pragma unroll
                for (int d = LPT / 2; d > 0; d >>= 1) {
                    if (n > 1) {
                        n >>= 1;
                        const bool up = lane & d;
#pragma unroll
                        for (int i = 0; i < ROWS / 2; ++i)
                            if (i < n) {
                                const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
                                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
                            }
                    } else {
                        v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
                    }
                }
                pw[r * ROWS + my_head] = v[0];  // lanes of one head write the same sum
            }
            __syncwarp();
            float p[kGrp / TS];
            float top = have[0] ? kLowest : -kInf;
#pragma unroll
            for (int i = 0; i < kGrp / TS; ++i) {
                const int t = i * TS + lane / ROWS;
                p[i] = (have[0] >> t) & 1 ? pw[t * ROWS + sh] * a.scale_log2 : -kInf;
                top = fmaxf(top, p[i]);
            }
#pragma unroll
            for (int d = ROWS; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (__any_sync(0xffffffffu, top > mx)) {
                const float nm = fmaxf(mx, top);
                const float f = nm == -kInf ? 1.f : ex2(mx - nm);
                mx = nm;
                l *= f;
#pragma unroll
                for (int h = 0; h < ROWS; ++h) {
                    const float fh = __shfl_sync(0xffffffffu, f, h);
                    o[h][0] = ptx::f2_mul(o[h][0], make_float2(fh, fh));
                    o[h][1] = ptx::f2_mul(o[h][1], make_float2(fh, fh));
                }
            }
            const float mb = mx == -kInf ? 0.f : mx;
#pragma unroll
            for (int i = 0; i < kGrp / TS; ++i) {
                p[i] = ex2(p[i] - mb);
                l += p[i];
                pw[(i * TS + lane / ROWS) * ROWS + sh] = p[i];
            }
            __syncwarp();
#pragma unroll
            for (int t = 0; t < kGrp; t += RPI) {
                const int r = t + lane / CH;
                const float4 v4 = *reinterpret_cast<const float4 *>(vb + r * D + (((lane % CH) ^ (r & 7)) << 2));
                const float2 lo = make_float2(v4.x, v4.y), hi = make_float2(v4.z, v4.w);
#pragma unroll
                for (int h = 0; h < ROWS; h += 4) {
                    const float4 p4 = *reinterpret_cast<const float4 *>(pw + r * ROWS + h);
                    const float pp[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[h + j][0] = ptx::f2_fma(lo, make_float2(pp[j], pp[j]), o[h + j][0]);
                        o[h + j][1] = ptx::f2_fma(hi, make_float2(pp[j], pp[j]), o[h + j][1]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) have[i] = have[i + 1];
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        cp_wait<0>();
#pragma unroll
        for (int d = ROWS; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);


        // the warps' results
        float *ow = base;
        float2 *ml = reinterpret_cast<float2 *>(ow + W * ROWS * D);
        __syncthreads();  // every warp has read its stages and scores
        if (lane < ROWS) ml[warp * ROWS + lane] = make_float2(mx, l);
#pragma unroll
        for (int h = 0; h < ROWS; ++h) {
            float4 x = make_float4(o[h][0].x, o[h][0].y, o[h][1].x, o[h][1].y);
            if (RPI == 2) {  // the other half's tokens
                x.x += __shfl_xor_sync(0xffffffffu, x.x, 16);
                x.y += __shfl_xor_sync(0xffffffffu, x.y, 16);
                x.z += __shfl_xor_sync(0xffffffffu, x.z, 16);
                x.w += __shfl_xor_sync(0xffffffffu, x.w, 16);
            }
            if (lane < CH) *reinterpret_cast<float4 *>(ow + (warp * ROWS + h) * D + lane * 4) = x;
        }
    }
};

// ------------------------------------------------------------ split kernel
template <typename Core>
__global__ void __launch_bounds__(Core::kThreads, 2)
paged_split_kernel(const __grid_constant__ PagedDecodeArgs a) {
    constexpr int D = Core::D, ROWS = Core::ROWS;
    constexpr int kOver = kOverhead<typename Core::T, D>;
    extern __shared__ __align__(128) unsigned char smem[];

    wait_before_reads<Core::KV>(a);
    const int units = a.num_kv_heads * a.head_groups;
    Place at;
    const bool any = find_place<Core::KV, Core::kThreads, kOver>(a, units, blockIdx.x, at, [&](long long all) {
        int ranges = kPagedCtas;
        if constexpr (Core::KV == Kv::kBehind) {
            const PrefixPieces &f = a.prefix;
            const int tiles = f.share ? prefix_tiles(f) : 0;
            const int sms = tiles > 0 ? f.ctas - ranges_beside<D>(f, tiles, all) : 0;
            if (sms > 0) ranges = 2 * sms;
            if (blockIdx.x == 0 && threadIdx.x == 0) f.ranges[1] = ranges;
        }
        return ranges;
    });
    long long w0 = any ? at.w : 0, unit0 = any ? at.unit0 : 0;
    const long long w1 = any ? min(at.all, w0 + at.chunk) : 0;
    int b = any ? at.b : 0;
    int len = any ? request_len<Core::KV>(a, b) : 0;
    bool first = true;
    while (w0 < w1 && b < a.batch) {
        const int tiles = (len + kTile - 1) / kTile, cost = unit_cost<kOver>(len);
        if (w0 >= unit0 + (long long)cost * units) {
            unit0 += (long long)cost * units;
            b = next_request<Core::KV>(a, b + 1, len);
            continue;
        }
        const int unit = tiles_div(w0 - unit0, cost);
        const int at0 = (int)(w0 - unit0 - (long long)unit * cost);
        const int at1 = (int)min((long long)cost, at0 + (w1 - w0));
        const int tile0 = max(at0 - kOver, 0), tile1 = at1 - kOver;
        w0 += at1 - at0;
        if (tile1 <= 0) continue;  // only overhead: the next CTA starts the unit
        const int kvh = unit / a.head_groups, hg = unit % a.head_groups;
        const int head0 = kvh * a.group + hg * ROWS;
        const int heads = min(ROWS, a.group - hg * ROWS);

        Core::stream(a, smem, b, kvh, head0, heads, tile0 * kTile, min(len, tile1 * kTile));
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == tiles;
        float *ws = piece_at<D>(a, blockIdx.x, first, ROWS);
        for (int i = threadIdx.x; i < heads * (D / 4); i += Core::kThreads) {
            const int h = i / (D / 4), d = (i % (D / 4)) * 4;
            Partial p = warps_sum<Core>(smem, h, d);
            if (whole) {
                const size_t row = (size_t)b * a.num_heads + head0 + h;
                if constexpr (Core::KV == Kv::kBehind) {  // the join adds the prefix
                    *reinterpret_cast<float4 *>(a.prefix.own + row * D + d) = p.acc;
                    if (d == 0) *reinterpret_cast<float2 *>(a.prefix.own_stat + 2 * row) = make_float2(p.m, p.sum);
                } else {
                    p.write<typename Core::T, Core::KV>(a, row, d);
                }
            } else {
                *reinterpret_cast<float4 *>(ws + h * D + d) = p.acc;
                if (d == 0) *reinterpret_cast<float2 *>(ws + ROWS * D + 2 * h) = make_float2(p.m, p.sum);
            }
        }
        __syncthreads();  // shared memory is the ring again
        first = false;
    }
    if constexpr (Core::KV != Kv::kBehind)
        write_empty<typename Core::T>(a);
    else if (blockIdx.x == gridDim.x - 1)
        ptx::grid_dependency_wait();  // this kernel ends behind the prefix's
}

// ---------------------------------------------------------- cluster kernel
// Short tables: one cluster a unit, each CTA a run of its tiles, joined through
// the cluster's shared memory: one launch, no workspace.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 peer_load2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

template <typename Core, int S>
__global__ void __launch_bounds__(Core::kThreads, 2)
paged_cluster_kernel(const __grid_constant__ PagedDecodeArgs a) {
    constexpr int D = Core::D, ROWS = Core::ROWS;
    extern __shared__ __align__(128) unsigned char smem[];
    wait_before_reads<Core::KV>(a);

    // a one-dimensional grid of one-dimensional clusters: the rank in the
    // cluster is the block's index modulo its size
    const int rank = blockIdx.x % S, units = a.num_kv_heads * a.head_groups;
    const int b = blockIdx.x / S / units, unit = blockIdx.x / S % units;
    const int kvh = unit / a.head_groups, hg = unit % a.head_groups;
    const int head0 = kvh * a.group + hg * ROWS;
    const int heads = min(ROWS, a.group - hg * ROWS);
    const int len = request_len<Core::KV>(a, b);
    const int share = ((len + kTile - 1) / kTile + S - 1) / S * kTile;  // tokens of a CTA
    const int t0 = rank * share, t1 = min(len, t0 + share);
    const bool any = t0 < t1;
    if (any) Core::stream(a, smem, b, kvh, head0, heads, t0, t1);
    wait_before_rows<Core::KV>();
    __syncthreads();
    const size_t row0 = (size_t)b * a.num_heads + head0;
    if (S == 1) {
        for (int i = threadIdx.x; i < heads * (D / 4); i += Core::kThreads) {
            const int h = i / (D / 4), d = (i % (D / 4)) * 4;
            Partial p = any ? warps_sum<Core>(smem, h, d) : Partial();
            p.write<typename Core::T, Core::KV>(a, row0 + h, d);
        }
        return;
    }
    // this CTA's sums, behind the warps'
    float *acc = reinterpret_cast<float *>(smem) + Core::W * ROWS * (D + 2);
    static_assert(sizeof(float) * (Core::W + 1) * ROWS * (D + 2) <= Core::kSmem, "shared memory");
    float2 *ms = reinterpret_cast<float2 *>(acc + ROWS * D);
    for (int i = threadIdx.x; i < heads * (D / 4); i += Core::kThreads) {
        const int h = i / (D / 4), d = (i % (D / 4)) * 4;
        const Partial p = any ? warps_sum<Core>(smem, h, d) : Partial();
        *reinterpret_cast<float4 *>(acc + h * D + d) = p.acc;
        if (d == 0) ms[h] = make_float2(p.m, p.sum);
    }
    cluster_barrier();
    const uint32_t acc_u = ptx::smem_u32(acc), ms_u = ptx::smem_u32(ms);
    for (int i = rank * Core::kThreads + threadIdx.x; i < heads * (D / 4); i += S * Core::kThreads) {
        const int h = i / (D / 4), d = (i % (D / 4)) * 4;
        float2 m[S];
        float4 x[S];
#pragma unroll
        for (int r = 0; r < S; ++r) {
            m[r] = peer_load2(peer_smem(ms_u + h * 8, r));
            x[r] = peer_load4(peer_smem(acc_u + (h * D + d) * 4, r));
        }
        Partial p;
        p.add<S>(m, x);
        p.write<typename Core::T, Core::KV>(a, row0 + h, d);
    }
    cluster_barrier();  // no CTA leaves while its shared memory is read
}

// -------------------------------------------------------------------- join
// Adds the pieces of the units that several CTAs hold, in the order of their
// tokens.  Block c - 1 looks at the start of CTA c's range: where it lies inside a
// unit, the block joins a share of that unit's heads (each of the unit's k cuts
// has a block; block j of them takes the heads j, j + k, ...).  At most
// kPagedCtas - 1 units are cut, whatever the batch.  A thread takes four columns of
// every slices-th piece with a running maximum, its loads in flight together; the
// slices are added in order.
template <int D, int ROWS> constexpr int kJoinThreads = ROWS * D / 4 > 256 ? ROWS * D / 4 : 256;

template <Kv KV, typename T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads<D, ROWS>)
paged_join_kernel(const __grid_constant__ PagedDecodeArgs a) {
    constexpr int kJoin = kJoinThreads<D, ROWS>;
    __shared__ float4 part[kJoin];
    __shared__ float2 stat[kJoin];
    const int units = a.num_kv_heads * a.head_groups;
    // The lengths were complete before the main kernel let this one be
    // scheduled; the pieces are read after the wait.
    Place at;
    const int c = blockIdx.x + 1;
    constexpr int kOver = kOverhead<T, D>;
    const bool any = find_place<KV, kJoin, kOver>(a, units, c, at, [](long long) { return kPagedCtas; });
    int unit = 0, c0 = 0, c1 = 0;
    long long u0 = 0;
    if (any) {
        const int cost = unit_cost<kOver>(request_len<KV>(a, at.b));
        unit = tiles_div(at.w - at.unit0, cost);
        u0 = at.unit0 + (long long)unit * cost;
        // the CTAs of the unit's first tile (behind its overhead) and of its last
        c0 = (int)((u0 + kOver) / at.chunk);
        c1 = (int)((u0 + cost - 1) / at.chunk);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!any || c <= c0) return;  // no cut here
    const int pieces = c1 - c0 + 1, cuts = c1 - c0;

    const int kvh = unit / a.head_groups, hg = unit % a.head_groups;
    const int head0 = kvh * a.group + hg * ROWS;
    const int heads = min(ROWS, a.group - hg * ROWS);
    const int mine = c - c0 - 1;  // this block among the unit's
    if (mine >= heads) return;
    const int n = (heads - mine + cuts - 1) / cuts;  // its heads: mine, mine + cuts, ...

    const int cols = n * (D / 4);  // at most kJoin
    const int slices = kJoin / cols;
    const int slice = threadIdx.x / cols, col = threadIdx.x - slice * cols;
    const int h = mine + (col / (D / 4)) * cuts, d = (col % (D / 4)) * 4;
    Partial p;
    if (slice < slices) {
        // the first piece ends CTA c0's range (and is all of it if it began
        // there), the others begin theirs
        const bool whole = c0 * at.chunk >= u0;
        constexpr int kFlight = 4;
        for (int i0 = slice; i0 < pieces; i0 += kFlight * slices) {
            float4 x[kFlight];
            float2 ms[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const int i = i0 + f * slices;
                x[f] = make_float4(0.f, 0.f, 0.f, 0.f);
                ms[f] = make_float2(-kInf, 0.f);
                if (i < pieces) {
                    const float *at_i = piece_at<D>(a, c0 + i, i > 0 || whole, ROWS);
                    x[f] = __ldcg(reinterpret_cast<const float4 *>(at_i + h * D + d));
                    ms[f] = __ldcg(reinterpret_cast<const float2 *>(at_i + ROWS * D + 2 * h));
                }
            }
            p.add<kFlight>(ms, x);
        }
    }
    part[threadIdx.x] = p.acc;
    stat[threadIdx.x] = make_float2(p.m, p.sum);
    __syncthreads();
    if (slice > 0) return;
    for (int i = 1; i < slices; ++i) {
        const float2 ms[1] = {stat[threadIdx.x + i * cols]};
        const float4 x[1] = {part[threadIdx.x + i * cols]};
        p.add<1>(ms, x);
    }
    p.write<T, KV>(a, (size_t)at.b * a.num_heads + head0 + h, d);
}

// Behind a shared prefix: a block takes `heads_per_block` heads of a unit, with or without own tokens, and adds
// the own pieces of the unit (or the sums of one that a CTA held whole) and the prefix's, a slice of
// threads every slices-th of them.
constexpr int kBehindJoin = 256;

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kBehindJoin)
paged_behind_join_kernel(const __grid_constant__ PagedDecodeArgs a, int heads_per_block) {
    constexpr int kOver = kOverhead<T, D>;
    __shared__ float4 part[kBehindJoin];
    __shared__ float2 stat[kBehindJoin];
    __shared__ long long costs[2][kBehindJoin / 32];
    const int units = a.num_kv_heads * a.head_groups;
    const int blocks = (min(ROWS, a.group) + heads_per_block - 1) / heads_per_block;  // of a unit
    const int hb = blockIdx.x % blocks, u = blockIdx.x / blocks, unit = u % units, b = u / units;
    const int kvh = unit / a.head_groups, hg = unit % a.head_groups;
    const int head0 = kvh * a.group + hg * ROWS + hb * heads_per_block;
    const int n = min(heads_per_block, min(ROWS, a.group - hg * ROWS) - hb * heads_per_block);
    // costs of the requests before b, and of all (the lengths before the wait: wait_before_reads)
    const int len = request_len<Kv::kBehind>(a, b);
    long long below = 0, all = 0;
    for (int i = threadIdx.x; i < a.batch; i += kBehindJoin) {
        const int c = unit_cost<kOver>(request_len<Kv::kBehind>(a, i));
        all += c;
        if (i < b) below += c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        below += __shfl_xor_sync(0xffffffffu, below, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if ((threadIdx.x & 31) == 0) {
        costs[0][threadIdx.x >> 5] = below;
        costs[1][threadIdx.x >> 5] = all;
    }
    __syncthreads();
    below = all = 0;
#pragma unroll
    for (int w = 0; w < kBehindJoin / 32; ++w) {
        below += costs[0][w];
        all += costs[1][w];
    }
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (n <= 0) return;  // (the last unit of a head may have fewer rows)
    const int ranges = __ldcg(a.prefix.ranges + 1);
    const long long chunk = max((all * units + ranges - 1) / ranges, 1LL);
    const int cost = unit_cost<kOver>(len);
    const long long u0 = below * units + (long long)unit * cost;
    const int c0 = range_of(u0 + kOver, chunk), c1 = range_of(u0 + max(cost, 1) - 1, chunk);
    const bool starts = c0 * chunk >= u0;  // CTA c0's range begins with the unit
    const int own = len > 0 ? c1 - c0 + 1 : 0;

    const int cols = n * (D / 4);  // at most kBehindJoin
    const int slices = kBehindJoin / cols;
    const int slice = threadIdx.x / cols, col = threadIdx.x - slice * cols;
    const int h = col / (D / 4), d = (col % (D / 4)) * 4;
    const size_t row = (size_t)b * a.num_heads + head0 + h;
    Partial p;
    if (slice < slices) {
        const PrefixRow f(a, row, d);
        p.add_list(slice, own + f.n, slices, [&](int i) -> PieceRow {
            if (i >= own) return f.piece(i - own);
            if (own == 1) return {a.prefix.own + row * D + d, a.prefix.own_stat + 2 * row};
            const int r = hb * heads_per_block + h;
            const float *at = piece_at<D>(a, c0 + i, i > 0 || starts, ROWS);
            return {at + r * D + d, at + ROWS * D + 2 * r};
        });
    }
    part[threadIdx.x] = p.acc;
    stat[threadIdx.x] = make_float2(p.m, p.sum);
    __syncthreads();
    if (slice > 0) return;
    for (int i = 1; i < slices; ++i) {
        const float2 ms[1] = {stat[threadIdx.x + i * cols]};
        const float4 x[1] = {part[threadIdx.x + i * cols]};
        p.add<1>(ms, x);
    }
    p.write<T, Kv::kOwn>(a, row, d);
}

// Opts a kernel into its dynamic shared memory, once per device (concurrent first
// calls may both do it, which is harmless).
template <auto Kern> cudaError_t allow_smem(int smem) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

template <typename Core, int S> cudaError_t launch_cluster(const PagedDecodeArgs &a) {
    constexpr auto kern = paged_cluster_kernel<Core, S>;
    cudaError_t e = allow_smem<kern>(Core::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * a.num_kv_heads * a.head_groups * S);
    cfg.blockDim = dim3(Core::kThreads);
    cfg.dynamicSmemBytes = Core::kSmem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// When the cluster kernel serves a call: up to kClusterTiles tiles a CTA, with as many CTAs
// a unit, at most eight, as fit the SMs at once; units of one CTA may be up to
// kClusterWaves times what fits.  64 query and 8 key-value heads of 128, cluster / split kernel:
// 1 x 300 tokens 4.9 / 6.6 us, 16 x 512 8.1 / 11.9, 16 x 1000 11.5 / 15.0, 8 x 2000 11.9 /
// 14.4, 128 x 128 15.7 / 19.8, 64 x 256 13.0 / 16.2; beyond it, with 16 tiles, 1 x 8000
// 14.8 / 12.0.
constexpr int kClusterTiles = 8;
constexpr int kClusterWaves = 4;

// CTAs of a unit's cluster, 0: the split kernel.
template <typename Core> int cluster_size(const PagedDecodeArgs &a) {
    // What the table can hold bounds the lengths, which only the GPU knows.
    const long units = (long)a.batch * a.num_kv_heads * ((a.group + Core::ROWS - 1) / Core::ROWS);
    const int most = Core::KV == Kv::kChosen ? min(a.max_tokens, a.chosen_count * a.page_size) : a.max_tokens;
    const int tiles = (most + kTile - 1) / kTile;
    int size = 8;
    while (size > 1 && (size > tiles || units * size > kPagedCtas)) size >>= 1;
    return tiles <= kClusterTiles * size && units * size <= kClusterWaves * kPagedCtas ? size : 0;
}

template <typename Core> cudaError_t launch(PagedDecodeArgs a) {
    a.head_groups = (a.group + Core::ROWS - 1) / Core::ROWS;
    switch (cluster_size<Core>(a)) {
        case 0: break;
        case 1: return launch_cluster<Core, 1>(a);
        case 2: return launch_cluster<Core, 2>(a);
        case 4: return launch_cluster<Core, 4>(a);
        default: return launch_cluster<Core, 8>(a);
    }

    using T = typename Core::T;
    constexpr int D = Core::D, ROWS = Core::ROWS;
    constexpr auto kern = paged_split_kernel<Core>;
    cudaError_t e = allow_smem<kern>(Core::kSmem);
    if (e == cudaSuccess)
        e = launch_dependent(kern, kPagedCtas, Core::kThreads, Core::kSmem, a.stream, a);
    if (e != cudaSuccess) return e;
    if constexpr (Core::KV == Kv::kBehind) {
        // one head a block (most slices a row) while that fills the GPU no more than a few times
        const long units = (long)a.batch * a.num_kv_heads * a.head_groups;
        const int rows = min(ROWS, a.group);
        int heads = 1;
        while (heads < 1024 / D && heads < rows && units * ((rows + heads - 1) / heads) > 8 * kPagedCtas) heads *= 2;
        const long blocks = units * ((rows + heads - 1) / heads);
        if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
        e = launch_dependent(paged_behind_join_kernel<T, D, ROWS>, (unsigned)blocks, kBehindJoin, 0,
                             a.stream, a, heads);
    } else {
        e = launch_dependent(paged_join_kernel<Core::KV, T, D, ROWS>, kPagedCtas - 1, kJoinThreads<D, ROWS>, 0,
                             a.stream, a);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Query heads of a unit: as many as share a key-value head, up to 16.  Further heads are a
// further unit, which streams the cache once more: a unit's sums fill the registers at 16
// heads.  64 query heads over bf16 keys and values of 0.54 GB each: 4 to 16 heads a kv head
// 165 to 175 us, 32 heads 325.
template <Kv KV, int D>
cudaError_t dispatch(const PagedDecodeArgs &a, bool bf16, bool q_f32 = false) {
    if (!bf16)
        return a.group <= 4   ? launch<F32Core<KV, D, 4>>(a)
               : a.group <= 8 ? launch<F32Core<KV, D, 8>>(a)
                              : launch<F32Core<KV, D, 16>>(a);
    if constexpr (KV == Kv::kOwn)  // the queries of a whole step
        if (q_f32) return a.group <= 8 ? launch<Bf16Core<KV, D, 1, true>>(a) : launch<Bf16Core<KV, D, 2, true>>(a);
    return a.group <= 8 ? launch<Bf16Core<KV, D, 1, false>>(a) : launch<Bf16Core<KV, D, 2, false>>(a);
}

}  // namespace
}  // namespace la
