// Bounds of the keys of every cache page, and the choice of the pages that a query attends to by
// the largest q . k that those bounds allow.
//
// For a page with keys k_t, channel by channel
//     lo_d = min_t k_td,   hi_d = max_t k_td,
// and for a query q
//     q . k_t <= s = sum_d max(q_d lo_d, q_d hi_d) = sum_d (q+_d max(lo_d, hi_d) + q-_d min(lo_d, hi_d))
// with q+ = max(q, 0), q- = min(q, 0) (the second form holds for any two numbers, in whatever order).  A
// block's score is the largest s of the query heads that share the key-value head; the `count` blocks
// with the largest scores are chosen, ties to the lower block.
//
// The choice is that of scores in 64 bits: two blocks whose scores differ by less than fp32 (or the
// tensor core) resolves would otherwise be chosen by the order of the additions.  So the scores are
// first taken in fp32 with a bound on their error, e = kSlack sum|q| max|bound| (the largest of the
// heads and of the unit's pages) + 2^-118 (2 D results of less than 2^-126, which are not off in proportion to
// themselves), and with T the count-th largest of them
//     s > T + 2 e  is chosen,   s < T - 2 e  is not,
// whatever the true scores are; those in between (a few) are taken again in 64 bits and ranked, and of their
// heads only those that fp32 cannot tell from the largest (the fp64 pipe does two lanes a cycle: all
// heads of them took 120 of 180 us for 128 requests of 1K to 32K tokens, 64 query heads).
// Where e is not finite (an infinity or NaN among bounds or queries) all blocks and heads are.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_internal.h"
#include "sm100_ptx.cuh"

namespace la {
namespace {

constexpr float kInf = __builtin_huge_valf();
constexpr int kSms = 152;

// ------------------------------------------------------------------ bounds
// Minimum and maximum that keep NaN, of a 16-byte chunk's elements.
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kUp = 0x7f807f80u, kDown = 0xff80ff80u;  // +-infinity
    static __device__ __forceinline__ uint32_t low(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t high(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};
template <> struct Chunk<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kUp = 0x7f800000u, kDown = 0xff800000u;
    static __device__ __forceinline__ uint32_t low(uint32_t a, uint32_t b) {
        float r;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        return __float_as_uint(r);
    }
    static __device__ __forceinline__ uint32_t high(uint32_t a, uint32_t b) {
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        return __float_as_uint(r);
    }
};

__device__ __forceinline__ int clamped(const int32_t *p, int most) {
    return min(max(__ldcg(p), 0), most);
}

// Bound: every new key is read once.  One warp takes a block of a request and a key-value head: its new
// rows are contiguous, 16 bytes a lane, kFlight rows of each lane in flight.  `splits` CTAs a request
// share its blocks.  9 prompts of 500 to 32K tokens, pages of 16, 8 key-value heads of 128: 53 us (6.2
// TB/s); one token of 128 requests 5.5 us (latency: lengths, table, old bounds).
constexpr int kBoundsWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32)
paged_bounds_kernel(const __grid_constant__ PagedBoundsArgs a, int splits) {
    using C = Chunk<T>;
    constexpr int LPR = D / C::N;   // lanes of a row
    constexpr int RPI = 32 / LPR;   // rows of a warp-wide load
    constexpr int kFlight = 8;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int b = blockIdx.x / splits, split = blockIdx.x - b * splits;
    const int first = clamped(a.first + b, a.max_tokens), len = clamped(a.seq_lens + b, a.max_tokens);
    if (first >= len) return;
    const int block0 = first / a.page_size, blocks = (len - 1) / a.page_size + 1 - block0;
    const long long tasks = (long long)blocks * a.num_kv_heads;
    const int lane = threadIdx.x & 31, chunk = lane % LPR;
    for (long long task = split * kBoundsWarps + (threadIdx.x >> 5); task < tasks;
         task += (long long)splits * kBoundsWarps) {
        const int i = (int)(task / a.num_kv_heads), kvh = (int)(task - (long long)i * a.num_kv_heads);
        const int blk = block0 + i, page = a.block_table[(size_t)b * a.table_stride + blk];
        if (page < 0 || page >= a.num_pages) continue;
        const int t0 = blk * a.page_size;  // at most len - 1
        const int r0 = max(first - t0, 0), r1 = min(len - t0, a.page_size);
        const uint4 *rows = reinterpret_cast<const uint4 *>(
            static_cast<const T *>(a.k) + (size_t)page * a.k_page_stride + (size_t)kvh * a.page_size * D);
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            lo[w] = C::kUp;
            hi[w] = C::kDown;
        }
        for (int r = r0 + lane / LPR; r < r1; r += RPI * kFlight) {
            uint4 x[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f)  // behind the last row: the last one once more
                x[f] = rows[(size_t)min(r + f * RPI, r1 - 1) * LPR + chunk];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const uint32_t *u = reinterpret_cast<const uint32_t *>(&x[f]);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    lo[w] = C::low(lo[w], u[w]);
                    hi[w] = C::high(hi[w], u[w]);
                }
            }
        }
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                lo[w] = C::low(lo[w], __shfl_xor_sync(0xffffffffu, lo[w], o));
                hi[w] = C::high(hi[w], __shfl_xor_sync(0xffffffffu, hi[w], o));
            }
        if (lane >= LPR) continue;
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.bounds) +
                                               (size_t)page * a.bounds_page_stride + (size_t)kvh * 2 * D);
        if (r0 > 0) {  // the page had tokens
            const uint4 p = out[chunk], q = out[LPR + chunk];
            const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                lo[w] = C::low(lo[w], u[w]);
                hi[w] = C::high(hi[w], v[w]);
            }
        }
        out[chunk] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        out[LPR + chunk] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

// ------------------------------------------------------------------ scores
// A unit is a request's key-value head.  `splits` warps share its blocks, 16 at a time; each leaves
// the fp32 scores and its largest |bound|.  Units whose blocks are all chosen have no scores.
// Bound: every bound is read once (G query heads do G flops a byte).  128 requests of 1K to 32K tokens, pages of
// 64, 64 and 8 heads of 128: 45 us with the choice, this kernel two thirds of it (138 MB at 4.2 TB/s under a
// profiler: three dependent latencies before a warp's first bounds, the next tile's loads behind this one's products,
// and requests of 16 to 512 blocks).  Spills at its 128 registers: 16 bytes (bf16, up to 8 heads of 128 a key-value
// head), 124 (bf16, more heads), 8 and 16 (fp32).
constexpr int kScoreWarps = 4;   // of a CTA, all of one unit
constexpr int kScoreTile = 16;   // blocks of a warp's step

struct SelectSpace {
    int splits;        // warps of a unit
    bool scored;       // some requests may have more blocks than are chosen
    size_t exact, approx, most, ready, bytes;  // offsets
};

SelectSpace select_space(int64_t units, int64_t width) {
    SelectSpace s;
    int64_t n = (int64_t)kSms * 48 / (units > 0 ? units : 1) + 1;
    const int64_t tiles = (width + kScoreTile - 1) / kScoreTile;
    n = n < tiles ? n : tiles;
    // no more than keep a warp's step below 2^16 blocks, which indices have room for behind the last block (at most
    // 2^31 - 2^16 are scored); 2432 warps run at once
    constexpr int64_t kMost = (0x7fffffff - kMaxTokens) / kScoreTile / kScoreWarps * kScoreWarps - kScoreWarps;
    n = n < kMost ? n : kMost;
    n = (n + kScoreWarps - 1) / kScoreWarps;
    s.splits = (int)(n < 1 ? 1 : n) * kScoreWarps;
    s.scored = true;
    s.exact = 0;
    s.approx = (size_t)(units * width) * sizeof(double);
    s.most = s.approx + (size_t)(units * width) * sizeof(float);
    s.ready = s.most + (size_t)units * s.splits * sizeof(float);
    s.bytes = s.ready + sizeof(int);
    return s;
}

__device__ __forceinline__ int unit_blocks(const PagedSelectArgs &a, int b) {
    const int n = clamped(a.seq_lens + b, a.max_tokens);
    return n > 0 ? (n - 1) / a.page_size + 1 : 0;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// bf16: 16 blocks x 8 heads a product, blocks in its rows.  A sum does not depend on the order of
// its terms, so a lane's 16-byte chunks of a row are operands as they are loaded, with the same
// elements of the query beside them.  The products are exact; the tensor core's sum of 16 of them and the running
// one keeps at least 23 bits of the largest, so 2 D / 16 such sums are off by at most
// 2 D / 16 * 17 * 2^-23 of the sum of |terms|, which sum|q| max|bound| exceeds.
// All chunks of a tile are loaded at once (8 KB a warp where D is 128), the table's entries a tile ahead.
template <int D, int NT> struct Bf16Scores {
    using T = __nv_bfloat16;
    static constexpr int HEADS = 8 * NT;  // of one pass
    static constexpr float kSlack = 2 * D / 16 * 17 * 0x1p-23f;

    static __device__ __forceinline__ void run(const PagedSelectArgs &a, int b, int kvh, int split, int splits,
                                               float *scores, float &most) {
        constexpr int CPL = 2 * D / 32;  // chunks of a lane: t, t + 4, ... of a row's minima and maxima
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int32_t *pages = a.block_table + (size_t)b * a.table_stride;
        const T *bounds = static_cast<const T *>(a.bounds) + (size_t)kvh * 2 * D;
        uint32_t top = 0;  // largest |bound| of either half
        for (int h0 = 0; h0 < a.group; h0 += HEADS) {
            const int heads = min(HEADS, a.group - h0);
            int page[2];  // of rows g and g + 8 of the tile
            auto find = [&](int i0) {
#pragma unroll
                for (int r = 0; r < 2; ++r) page[r] = i0 + r * 8 + g < a.table_width ? pages[i0 + r * 8 + g] : -1;
            };
            find(split * kScoreTile);
            uint32_t q[NT][CPL / 2][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 *qp = reinterpret_cast<const uint4 *>(
                    static_cast<const T *>(a.q) + (size_t)b * a.q_stride +
                    (size_t)(kvh * a.group + h0 + n * 8 + g) * D);
#pragma unroll
                for (int c = 0; c < CPL / 2; ++c) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (n * 8 + g < heads) x = __ldcg(qp + t + 4 * c);
                    q[n][c][0] = x.x, q[n][c][1] = x.y, q[n][c][2] = x.z, q[n][c][3] = x.w;
                }
            }
            // (the first entries and the queries are on their way beside the length)
            const int blocks = unit_blocks(a, b);
            if (blocks <= a.count) return;  // all of them are chosen
            for (int i0 = split * kScoreTile; i0 < blocks; i0 += splits * kScoreTile) {
                uint4 x[2][CPL];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const bool there = i0 + r * 8 + g < blocks && page[r] >= 0 && page[r] < a.num_pages;
                    const uint4 *p = reinterpret_cast<const uint4 *>(
                        bounds + (there ? (size_t)page[r] : 0) * a.bounds_page_stride) + t;
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        x[r][c] = make_uint4(0, 0, 0, 0);
                        if (there) x[r][c] = p[4 * c];
                    }
                }
                find(i0 + splits * kScoreTile);
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int c = 0; c < CPL / 2; ++c) {
                        uint32_t *u = reinterpret_cast<uint32_t *>(&x[r][c]);
                        uint32_t *v = reinterpret_cast<uint32_t *>(&x[r][CPL / 2 + c]);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t low = Chunk<T>::low(u[w], v[w]);
                            v[w] = Chunk<T>::high(u[w], v[w]);
                            u[w] = low;
                        }
                    }
                float s[NT][4] = {};
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    const uint32_t *u = reinterpret_cast<const uint32_t *>(&x[0][c]);
                    const uint32_t *v = reinterpret_cast<const uint32_t *>(&x[1][c]);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        top = __vmaxu2(top, u[w] & 0x7fff7fffu);
                        top = __vmaxu2(top, v[w] & 0x7fff7fffu);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t e[4];  // the query's negative elements beside minima, the others beside maxima
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t y = q[n][c % (CPL / 2)][w];
                            const uint32_t neg = ((y >> 15) & 0x00010001u) * 0xffffu;
                            e[w] = c < CPL / 2 ? y & neg : y & ~neg;
                        }
                        mma16816(s[n], u[0], v[0], u[1], v[1], e[0], e[1]);
                        mma16816(s[n], u[2], v[2], u[3], v[3], e[2], e[3]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float m = -kInf;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (n * 8 + 2 * t + j < heads) m = fmaxf(m, s[n][2 * r + j]);
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    const int i = i0 + r * 8 + g;
                    if (t == 0 && i < blocks) {
                        if (h0 > 0) m = fmaxf(m, scores[i]);
                        scores[i] = m;
                    }
                }
            }
        }
        const uint32_t u = max(top & 0xffffu, top >> 16);
        most = __uint_as_float(u << 16);
    }
};

// fp32: D / 4 lanes a block, four channels of a lane; sums of 8 products and log2(D / 4) levels, each
// rounded: off by at most 13 * 2^-24 < 2^-20 of the sum of |terms|.
template <int D> struct F32Scores {
    using T = float;
    static constexpr int HEADS = 8;
    static constexpr float kSlack = 0x1p-20f;

    static __device__ __forceinline__ void run(const PagedSelectArgs &a, int b, int kvh, int split, int splits,
                                               float *scores, float &most) {
        constexpr int LPB = D / 4, BPI = 32 / LPB;  // lanes of a block, blocks of a load
        constexpr int kFlight = 4;
        const int lane = threadIdx.x & 31, sub = lane % LPB;
        const int32_t *pages = a.block_table + (size_t)b * a.table_stride;
        const T *bounds = static_cast<const T *>(a.bounds) + (size_t)kvh * 2 * D;
        most = 0.f;
        // lane l < 16: the entry of block l of a tile, read a tile ahead
        auto entry = [&](int i0) {
            return lane < kScoreTile && i0 + lane < a.table_width ? pages[i0 + lane] : -1;
        };
        for (int h0 = 0; h0 < a.group; h0 += HEADS) {
            const int heads = min(HEADS, a.group - h0);
            int page = entry(split * kScoreTile);
            float2 up[HEADS][2], down[HEADS][2];
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (h < heads)
                    x = __ldcg(reinterpret_cast<const float4 *>(static_cast<const T *>(a.q) + (size_t)b * a.q_stride +
                                                          (size_t)(kvh * a.group + h0 + h) * D) + sub);
                up[h][0] = make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f));
                up[h][1] = make_float2(fmaxf(x.z, 0.f), fmaxf(x.w, 0.f));
                down[h][0] = make_float2(fminf(x.x, 0.f), fminf(x.y, 0.f));
                down[h][1] = make_float2(fminf(x.z, 0.f), fminf(x.w, 0.f));
            }
            // (the first entries and the queries are on their way beside the length)
            const int blocks = unit_blocks(a, b);
            if (blocks <= a.count) return;  // all of them are chosen
            for (int i0 = split * kScoreTile; i0 < blocks; i0 += splits * kScoreTile) {
                const int here = i0 + lane < blocks && page < a.num_pages ? page : -1;
                page = entry(i0 + splits * kScoreTile);
#pragma unroll 1
                for (int j0 = 0; j0 < kScoreTile; j0 += BPI * kFlight) {
                    float4 lo[kFlight], hi[kFlight];
#pragma unroll
                    for (int f = 0; f < kFlight; ++f) {
                        const int from = __shfl_sync(0xffffffffu, here, j0 + f * BPI + lane / LPB);
                        const float4 *p = reinterpret_cast<const float4 *>(
                            bounds + (size_t)max(from, 0) * a.bounds_page_stride);
                        lo[f] = hi[f] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (from >= 0) {
                            const float4 u = p[sub], v = p[LPB + sub];
                            lo[f] = make_float4(min_nan(u.x, v.x), min_nan(u.y, v.y), min_nan(u.z, v.z),
                                                min_nan(u.w, v.w));
                            hi[f] = make_float4(max_nan(u.x, v.x), max_nan(u.y, v.y), max_nan(u.z, v.z),
                                                max_nan(u.w, v.w));
                        }
                    }
#pragma unroll
                    for (int f = 0; f < kFlight; ++f) {
                        most = max_nan(most, max_nan(max_nan(fabsf(lo[f].x), fabsf(lo[f].y)),
                                                     max_nan(fabsf(lo[f].z), fabsf(lo[f].w))));
                        most = max_nan(most, max_nan(max_nan(fabsf(hi[f].x), fabsf(hi[f].y)),
                                                     max_nan(fabsf(hi[f].z), fabsf(hi[f].w))));
                        float v[HEADS];
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) {
                            float2 s = ptx::f2_mul(make_float2(hi[f].x, hi[f].y), up[h][0]);
                            s = ptx::f2_fma(make_float2(hi[f].z, hi[f].w), up[h][1], s);
                            s = ptx::f2_fma(make_float2(lo[f].x, lo[f].y), down[h][0], s);
                            s = ptx::f2_fma(make_float2(lo[f].z, lo[f].w), down[h][1], s);
                            v[h] = s.x + s.y;
                        }
                        // the heads' sums over the block's lanes, one head's in each in the end
                        int n = HEADS, mine = 0;
#pragma unroll
                        for (int o = LPB / 2; o > 0; o >>= 1) {
                            if (n > 1) {
                                n >>= 1;
                                const bool high = lane & o;
                                if (high) mine += n;
#pragma unroll
                                for (int k = 0; k < HEADS / 2; ++k)
                                    if (k < n) {
                                        const float keep = high ? v[k + n] : v[k], give = high ? v[k] : v[k + n];
                                        v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                                    }
                            } else {
                                v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                            }
                        }
                        float m = mine < heads ? v[0] : -kInf;
#pragma unroll
                        for (int o = LPB / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const int i = i0 + j0 + f * BPI + lane / LPB;
                        if (sub == 0 && i < blocks) {
                            if (h0 > 0) m = fmaxf(m, scores[i]);
                            scores[i] = m;
                        }
                    }
                }
            }
        }
    }
};

template <typename S>
__global__ void __launch_bounds__(kScoreWarps * 32, 4)
paged_score_kernel(const __grid_constant__ PagedSelectArgs a, const __grid_constant__ SelectSpace w) {
    ptx::grid_dependency_wait();
    // for the choice, which has no wait for what wrote the arguments
    ptx::release_to_next(reinterpret_cast<int *>(static_cast<char *>(a.workspace) + w.ready));
    ptx::grid_launch_dependents();
    const int ctas = w.splits / kScoreWarps;
    const int unit = blockIdx.x / ctas;
    const int b = unit / a.num_kv_heads, kvh = unit - b * a.num_kv_heads;
    const int split = (blockIdx.x - unit * ctas) * kScoreWarps + (threadIdx.x >> 5);
    char *base = static_cast<char *>(a.workspace);
    float *scores = reinterpret_cast<float *>(base + w.approx) + (size_t)unit * a.table_width;
    float most = 0.f;
    S::run(a, b, kvh, split, w.splits, scores, most);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((threadIdx.x & 31) == 0)
        reinterpret_cast<float *>(base + w.most)[(size_t)unit * w.splits + split] = most;
}

// ------------------------------------------------------------------ choice
// One CTA a unit.  The blocks' keys (the scores' order as unsigned integers) stay in shared memory, up to
// kKeys of them; further ones are made again from the scores where they are wanted.
constexpr int kPick = 256, kPickWarps = kPick / 32;
constexpr int kRanked = 64;   // candidates that are ranked by comparing all with all
constexpr int kKeys = 8192;
constexpr uint32_t kAbsent = 0u, kKept = ~0u;  // of no finite score

// Order of the values as unsigned integers; -0 and 0 are one value.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}

struct PickSpace {
    int hist[256];
    int2 warps[2][kPickWarps];
    int pair[2];
    float norm, most;
    int found;
    int last;          // last block of the ranking's least value that is chosen
    uint64_t least;    // that value
    int list[kRanked];
};

// Sums over the CTA of x and y, to every thread.  (Two places in turn: one barrier.)
__device__ __forceinline__ int2 block_sum(PickSpace &s, int turn, int x, int y) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    if ((threadIdx.x & 31) == 0) s.warps[turn][threadIdx.x >> 5] = make_int2(x, y);
    __syncthreads();
    int2 t = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kPickWarps; ++w) {
        t.x += s.warps[turn][w].x;
        t.y += s.warps[turn][w].y;
    }
    return t;
}

// The rank-th largest (from 1) of the keys that key(i, k) gives for i < n, and how many of those
// that equal it are among the rank largest, of the bits from kLow up.  Eight bits a pass.
template <int kLow, typename K, typename F>
__device__ __forceinline__ K radix_pick(PickSpace &s, int n, int rank, int &equal, F key) {
    constexpr int kTop = sizeof(K) * 8 - 8;
    K prefix = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += kPick) s.hist[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int shift = kTop; shift >= kLow; shift -= 8) {
        for (int i = threadIdx.x; i < n; i += kPick) {
            K k;
            if (key(i, k) && (shift == kTop || (k >> (shift + 8)) == (prefix >> (shift + 8))))
                atomicAdd(&s.hist[(int)(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (threadIdx.x < 32) {  // lane l: bins 255 - 8 l .. 248 - 8 l, from the top
            const int top = 255 - 8 * threadIdx.x;
            int bins[8], mine = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) mine += bins[i] = s.hist[top - i];
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if ((int)threadIdx.x >= o) upto += v;
            }
            const int above = upto - mine;
            if (above < rank && upto >= rank) {
                int left = rank - above, bin = top;
                bool found = false;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!found) {
                        if (bins[i] >= left) {
                            found = true;
                            bin = top - i;
                        } else {
                            left -= bins[i];
                        }
                    }
                s.pair[0] = bin;
                s.pair[1] = left;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) s.hist[top - i] = 0;
        }
        __syncthreads();
        prefix |= (K)s.pair[0] << shift;
        rank = s.pair[1];
    }
    equal = rank;
    return prefix;
}

// The score of a block in 64 bits (whole warp).  err: the fp32 scores' error, which these sums of D
// products have too (4 of a lane, 5 levels); where it is not finite the formula is taken
// word by word, and NaN counts as infinity, so that it is not overlooked.
template <typename T, int D>
__device__ __forceinline__ double exact_score(const PagedSelectArgs &a, int b, int kvh, int page, float err) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const T *lo = static_cast<const T *>(a.bounds) + (size_t)page * a.bounds_page_stride +
                  (size_t)kvh * 2 * D + lane * E;
    const T *q = static_cast<const T *>(a.q) + (size_t)b * a.q_stride + (size_t)kvh * a.group * D + lane * E;
    float l[E], h[E];
#pragma unroll
    for (int d = 0; d < E; ++d) {
        l[d] = fminf((float)lo[d], (float)lo[D + d]);
        h[d] = fmaxf((float)lo[d], (float)lo[D + d]);
    }
    double most = -(double)kInf;
    auto add = [&](int g, bool plain) {
        double sum = 0.0;
#pragma unroll
        for (int d = 0; d < E; ++d) {
            const float x = (float)q[g * D + d];
            if (plain) {  // finite numbers
                sum = fma((double)x, (double)(x < 0.f ? l[d] : h[d]), sum);
            } else {
                const double m = (double)x * (double)(float)lo[d], n = (double)x * (double)(float)lo[D + d];
                sum += m != m || n != n ? m + n : fmax(m, n);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (sum != sum) sum = (double)kInf;
        most = fmax(most, sum);
    };
    if (!(err < 1e30f)) {
        for (int g = 0; g < a.group; ++g) add(g, false);
        return most;
    }
    // fp32 sums of 8 heads at a time: lane i gets that of head i % 8
    auto eight = [&](int g0) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.f;
            const int g = min(g0 + i, a.group - 1);  // (the last one again)
#pragma unroll
            for (int d = 0; d < E; ++d) {
                const float x = (float)q[g * D + d];
                v[i] = fmaf(x, x < 0.f ? l[d] : h[d], v[i]);
            }
        }
        int n = 8;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            n >>= 1;
            const bool high = lane & o;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < n) {
                    const float keep = high ? v[k + n] : v[k], give = high ? v[k] : v[k + n];
                    v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8);
        return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
    };
    float sums = eight(0), first = sums;
    for (int g0 = 8; g0 < a.group; g0 += 8) first = fmaxf(first, eight(g0));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) first = fmaxf(first, __shfl_xor_sync(0xffffffffu, first, o));
    for (int g0 = 0; g0 < a.group; g0 += 8) {
        if (g0 > 0) sums = eight(g0);
        uint32_t near = __ballot_sync(0xffffffffu, lane < 8 && g0 + lane < a.group && sums >= first - 2.02f * err);
        for (; near; near &= near - 1) add(g0 + __ffs(near) - 1, true);
    }
    return most;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPick, 4)
paged_pick_kernel(const __grid_constant__ PagedSelectArgs a, const __grid_constant__ SelectSpace w,
                  float slack, int cap) {
    __shared__ PickSpace s;
    extern __shared__ uint32_t keys[];  // [cap]
    const int unit = blockIdx.x, b = unit / a.num_kv_heads, kvh = unit - b * a.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s.norm = s.most = 0.f;
    // Behind the scores' kernel, all of whose CTAs have waited for whatever wrote the lengths, the table, the
    // queries and the bounds before this one is scheduled.  That orders the two but makes nothing visible here: for
    // that the scores' kernel then releases w.ready (its value means nothing), and every thread here acquires
    // it (which also lets go of L1's lines).  Only the scores are still to come: what else is wanted is read before
    // the wait for them.
    if (w.scored) {
        ptx::load_acquire(reinterpret_cast<const int *>(static_cast<char *>(a.workspace) + w.ready));
        ptx::grid_launch_dependents();
    } else {
        ptx::grid_dependency_wait();
    }
    const int blocks = unit_blocks(a, b);
    const int32_t *pages = a.block_table + (size_t)b * a.table_stride;
    int32_t *out = a.selected + (size_t)unit * a.count;
    const char *base = static_cast<const char *>(a.workspace);
    const float *approx = reinterpret_cast<const float *>(base + w.approx) + (size_t)unit * a.table_width;
    double *exact = reinterpret_cast<double *>(static_cast<char *>(a.workspace) + w.exact) +
                    (size_t)unit * a.table_width;
    const bool scored = blocks > a.count;
    auto there = [&](int i) {
        const int p = pages[i];
        return p >= 0 && p < a.num_pages;
    };
    auto make_key = [&](int i, bool is, float x) -> uint32_t {
        if (!is) return kAbsent;
        // (as differences: the sums could pass 32 bits)
        if (!scored || i < a.keep_first || blocks - 1 - i < a.keep_last) return kKept;
        return x == x ? key_of(x) : 1u << 31;  // (no key of NaN may be one of the two above)
    };
    auto key_at = [&](int i) {
        return i < cap ? keys[i] : make_key(i, there(i), scored ? __ldcg(approx + i) : 0.f);
    };
    // which pages are there, and the queries' part of the scores' error, before the wait
    for (int i = tid; i < min(blocks, cap); i += kPick) keys[i] = there(i);
    if (scored) {
        float norm = 0.f;
        for (int h = warp; h < a.group; h += kPickWarps) {
            const T *q = static_cast<const T *>(a.q) + (size_t)b * a.q_stride + (size_t)(kvh * a.group + h) * D;
            float x = 0.f;
#pragma unroll
            for (int d = 0; d < D; d += 32) x += fabsf((float)q[d + lane]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            norm = max_nan(norm, x);
        }
        __syncthreads();
        // nonnegative floats (and NaN, the largest) have the order of their bits
        if (lane == 0) atomicMax(reinterpret_cast<int *>(&s.norm), __float_as_int(norm) & 0x7fffffff);
    }
    if (w.scored) ptx::grid_dependency_wait();
    else ptx::grid_launch_dependents();
    int present = 0, forced = 0;
    constexpr int kFlight = 4;
    for (int i0 = tid; i0 < blocks; i0 += kFlight * kPick) {
        float x[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int i = i0 + f * kPick;
            x[f] = scored && i < blocks ? __ldcg(approx + i) : 0.f;
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int i = i0 + f * kPick;
            if (i >= blocks) break;
            const uint32_t k = make_key(i, i < cap ? keys[i] != 0 : there(i), x[f]);
            if (i < cap) keys[i] = k;
            present += k != kAbsent;
            forced += k == kKept;
        }
    }
    if (scored) {
        float most = 0.f;
        const float *mp = reinterpret_cast<const float *>(base + w.most) + (size_t)unit * w.splits;
        for (int i = tid; i < w.splits; i += kPick) most = max_nan(most, __ldcg(mp + i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (lane == 0) atomicMax(reinterpret_cast<int *>(&s.most), __float_as_int(most) & 0x7fffffff);
    }
    const int2 all = block_sum(s, 0, present, forced);  // (its barrier is the keys' and the error's too)
    present = all.x;
    forced = all.y;

    // keys above `above` are chosen, keys below `below` are not; those between by rank, if there are too many
    uint32_t above = 0u, below = 0u;  // all that are there
    bool ranked = false;
    int turn = 1;  // the place for sums over the CTA that is free
    if (present > a.count) {
        int need = a.count - forced;  // of the others; at least 0
        const float err = fmaf(slack, s.most * s.norm, 0x1p-118f);
        const bool finite = err < 1e30f;  // false for NaN
        if (need == 0) {
            above = below = kKept - 1;
        } else {
            if (finite) {
                int equal;
                const uint32_t k = radix_pick<8, uint32_t>(s, blocks, need, equal, [&](int i, uint32_t &key) {
                    key = key_at(i);
                    return key != kAbsent && key != kKept;
                });
                // T to 2^-15 of itself, which is near enough to e that a fourth pass would not pay.  (2 e, and
                // room for the rounding of these two sums: e is at least 2^-20 of |T|)
                above = key_of(value_of(k | 255u) + 2.25f * err);
                below = key_of(value_of(k) - 2.25f * err);
            } else {
                above = kKept - 1;
                below = kAbsent + 1;
            }
            auto in_band = [&](int i) {
                const uint32_t k = key_at(i);
                return k >= below && k <= above && k != kAbsent;
            };
            int sure = 0, maybe = 0;
            for (int i = tid; i < blocks; i += kPick) {
                const uint32_t k = key_at(i);
                sure += k > above && k != kKept;
                maybe += k >= below && k <= above && k != kAbsent;
            }
            if (tid == 0) s.found = 0;
            const int2 sums = block_sum(s, turn, sure, maybe);
            turn = 0;
            need -= sums.x;
            maybe = sums.y;
            if (maybe > need) {
                ranked = true;
                if (maybe <= kRanked) {
                    for (int i = tid; i < blocks; i += kPick)
                        if (in_band(i)) s.list[atomicAdd(&s.found, 1)] = i;
                    __syncthreads();
                    for (int c = warp; c < maybe; c += kPickWarps) {
                        const double x = exact_score<T, D>(a, b, kvh, pages[s.list[c]], err);
                        if (lane == 0) exact[s.list[c]] = x;
                    }
                    __syncthreads();
                    if (tid < maybe) {
                        const int mine = s.list[tid];
                        const uint64_t key = key_of(exact[mine]);
                        int before = 0;
                        for (int c = 0; c < maybe; ++c) {
                            const uint64_t other = key_of(exact[s.list[c]]);
                            before += other > key || (other == key && s.list[c] < mine);
                        }
                        if (before == need - 1) {
                            s.least = key;
                            s.last = mine;
                        }
                    }
                    __syncthreads();
                } else {
                    for (int i = warp; i < blocks; i += kPickWarps)
                        if (in_band(i)) {
                            const double x = exact_score<T, D>(a, b, kvh, pages[i], err);
                            if (lane == 0) exact[i] = x;
                        }
                    __syncthreads();
                    int equal;
                    const uint64_t k = radix_pick<0, uint64_t>(s, blocks, need, equal, [&](int i, uint64_t &key) {
                        if (!in_band(i)) return false;
                        key = key_of(exact[i]);
                        return true;
                    });
                    // the `equal`-th block that has the least value
                    if (warp == 0) {
                        int seen = 0;
                        for (int i0 = 0; i0 < blocks && seen < equal; i0 += 32) {
                            const int i = i0 + lane;
                            const bool is = i < blocks && in_band(i) && key_of(exact[i]) == k;
                            const uint32_t m = __ballot_sync(0xffffffffu, is);
                            if (is && seen + __popc(m & ((1u << lane) - 1)) == equal - 1) {
                                s.least = k;
                                s.last = i;
                            }
                            seen += __popc(m);
                        }
                    }
                    __syncthreads();
                }
            }
        }
    }

    // the chosen blocks in ascending order
    int at = 0;
    for (int i0 = 0; i0 < blocks && at < a.count; i0 += kPick, turn ^= 1) {
        const int i = i0 + tid;
        const uint32_t k = i < blocks ? key_at(i) : kAbsent;
        bool take = k != kAbsent && k >= below;
        if (take && ranked && k <= above) {
            const uint64_t key = key_of(exact[i]);
            take = key > s.least || (key == s.least && i <= s.last);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, take);
        if (lane == 0) s.warps[turn][warp].x = __popc(m);
        __syncthreads();
        int before = at;
#pragma unroll
        for (int v = 0; v < kPickWarps; ++v) {
            const int n = s.warps[turn][v].x;
            if (v < warp) before += n;
            at += n;
        }
        const int place = before + __popc(m & ((1u << lane) - 1));
        if (take && place < a.count) out[place] = i;
    }
    for (int i = at + tid; i < a.count; i += kPick) out[i] = -1;
}

template <typename T, int D> cudaError_t launch_bounds_kernel(const PagedBoundsArgs &a) {
    // CTAs of a request: enough for all SMs from few requests, no more than its table has work for
    long splits = ((long)kSms * 8 + a.batch - 1) / a.batch;
    const long most = ((long)a.table_width * a.num_kv_heads + kBoundsWarps - 1) / kBoundsWarps;
    splits = splits < most ? splits : most;
    splits = splits > 1 ? splits : 1;
    if (splits * a.batch > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_dependent(paged_bounds_kernel<T, D>, (unsigned)(splits * a.batch),
                                           kBoundsWarps * 32, 0, a.stream, a, (int)splits);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename S, int D> cudaError_t launch_select(const PagedSelectArgs &a) {
    const int64_t units = (int64_t)a.batch * a.num_kv_heads;
    SelectSpace w = select_space(units, a.table_width);
    w.scored = a.table_width > a.count;
    const int cap = a.table_width < kKeys ? a.table_width : kKeys;
    cudaError_t e = cudaSuccess;
    if (w.scored)
        e = launch_dependent(paged_score_kernel<S>, (unsigned)(units * (w.splits / kScoreWarps)),
                             kScoreWarps * 32, 0, a.stream, a, w);
    if (e == cudaSuccess)
        e = launch_dependent(paged_pick_kernel<typename S::T, D>, (unsigned)units, kPick, cap * sizeof(uint32_t),
                             a.stream, a, w, S::kSlack, cap);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t paged_bounds(const PagedBoundsArgs &a, bool bf16) {
    if (a.head_dim == 128)
        return bf16 ? launch_bounds_kernel<__nv_bfloat16, 128>(a) : launch_bounds_kernel<float, 128>(a);
    if (a.head_dim == 64)
        return bf16 ? launch_bounds_kernel<__nv_bfloat16, 64>(a) : launch_bounds_kernel<float, 64>(a);
    return cudaErrorNotSupported;
}

int64_t paged_select_workspace(int64_t batch, int64_t num_kv_heads, int64_t table_width) {
    if ((double)batch * num_kv_heads * ((double)table_width + 1) > 0x1p56) return -1;
    return (int64_t)select_space(batch * num_kv_heads, table_width).bytes;
}

cudaError_t paged_select(const PagedSelectArgs &a, bool bf16) {
    if (a.head_dim == 128)
        return !bf16          ? launch_select<F32Scores<128>, 128>(a)
               : a.group <= 8 ? launch_select<Bf16Scores<128, 1>, 128>(a)
                              : launch_select<Bf16Scores<128, 2>, 128>(a);
    if (a.head_dim == 64)
        return !bf16          ? launch_select<F32Scores<64>, 64>(a)
               : a.group <= 8 ? launch_select<Bf16Scores<64, 1>, 64>(a)
                              : launch_select<Bf16Scores<64, 2>, 64>(a);
    return cudaErrorNotSupported;
}

}  // namespace la
