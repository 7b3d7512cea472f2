// The attention over a shared prefix on the tensor cores (tcgen05 + TMEM), bf16: for the query
// heads of all requests that share a key-value head (its rows), tile by tile of 128 tokens,
//     S = Q K^T,   P = e^(scale S - m),   X = P V,   o <- o f + X,   l <- l f + sum P
// with the running maximum m of each row and f = e^(m before - m).  A CTA leaves m, l and the
// unnormalised o of its part of a unit (PrefixPieces); see paged_prefix.cu for the split.
//
// Bound: a row does 4 D flops a token, so with many rows the tensor core bounds the kernel, with few
// (and K and V read once for all of them) HBM.
//
// P is passed as two bf16 parts (parts_of: off by at most 2^-16 of each weight, as in the attention
// of one request), which makes P V two products instead of one: 1536 tensor cycles a 128 x 128
// tile instead of 1024.  One part would double the error that the output's own rounding leaves.
// X is taken anew for every tile and added to o in registers: rounded to nearest, where the tensor
// core's own accumulation over a long prefix drops the bits that do not fit, and a maximum
// that moves costs a product in registers instead of a pass through tensor memory.
//
// A CTA has two groups of 128 rows, A and B, which share every tile of K and V in shared memory:
// the tensor core works on one group's products while the other group's 256 threads take its
// exponentials.  Where a key-value head has no more than 128 rows, both groups have the same
// rows and every other tile each, and leave a part each.
//
// TMEM (512 columns): S of A and B 128 columns each, X of A and B 128 each.  P takes the place of S:
// 16 tokens' scores are 16 columns, their weights 8 columns of high and 8 of low parts.
//
// Warp roles (640 threads):
//   warps 0-7    rows of A: two threads a row, each with 64 of a tile's tokens and half of
//                the columns of o; warps 8-15 those of B
//   warps 16, 17 MMA issuers of A and B: S of the next tile follows P V of this one at once (one
//                thread's MMAs run in the order of their issue, so S does not overtake the P V that
//                reads P in its place)
//   warps 18, 19 copies of K and V (cp.async: a page's rows are contiguous, but pages are of any
//                size and lie anywhere), each half of a tile's tokens, into a ring of four tiles
// Every wait is bounded; one that gives up sets the CTA's abort flag, all roles leave, copies and MMAs
// are drained, TMEM is freed and the device error word is raised.
#include "paged_attention.cuh"

namespace la {

__device__ unsigned int g_prefix_error = 0;  // bit 0: a bounded wait gave up

namespace {

using namespace ptx;

constexpr int kTokens = kPrefixTile;  // of a tile
constexpr int kRows = 128;            // of a group
constexpr int kGroupWarps = 8;
constexpr int kIssue0 = 16, kCopy0 = 18, kCopyWarps = 2;
constexpr int kTcThreads = 640;
constexpr int kRing = 4;              // tiles of shared memory: K and V of two tiles of tokens
constexpr uint32_t kAtoms = kTokens * 128;  // 128 rows of 64 bf16
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kColX = 256;
static_assert(kTokens == 128 && kRows == 128, "operand shapes");

struct TcShared {
    uint64_t full[kRing], empty[kRing];
    uint64_t q_ready[2], s_full[2], p_ready[2], done[2];
    uint32_t have[2][4];        // present tokens of a tile of K, by ring slot
    uint32_t mask[2][2][4];     // the same for the rows: group, tile & 1
    uint32_t tmem_base;
    int abort;
    float part[2][2][2][kRows];  // group, tile & 1, half: a row's maximum over the half's tokens
};

template <int D> struct TcSizes {
    static constexpr uint32_t kTile = kTokens * D * 2;
    static constexpr uint32_t kRingAt = 2 * kRows * D * 2;  // behind Q of A and B
    static constexpr uint32_t kCtrl = kRingAt + kRing * kTile;
    static constexpr uint32_t kSmem = kCtrl + sizeof(TcShared) + 1024;  // + alignment slack
};

// Byte offset of 16-byte chunk c of row r in an operand of 128 rows: 64-column halves of
// 128-byte swizzled rows.
__device__ __forceinline__ uint32_t place(int r, int c) {
    return (uint32_t)(c >> 3) * kAtoms + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, kTimeoutNs));
}
// Barrier of the 64 threads of a row quarter; true where all of them say so.
__device__ __forceinline__ bool pair_and(int id, bool ok) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
                 "barrier.cta.red.and.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(id), "r"((uint32_t)ok) : "memory");
    return r != 0;
}
// A CTA's parts of units, in order.
struct Walk {
    long long w, end;
    int tiles;         // of the prefix
    int unit, tile, n;  // this part: tiles tile .. tile + n - 1 of the unit
    int at, done = 0;   // the CTA's tiles before it, with it

    __device__ __forceinline__ bool next() {
        if (w >= end) return false;
        at = done;
        unit = range_of(w, tiles);
        tile = (int)(w - (long long)unit * tiles);
        n = (int)min((long long)(tiles - tile), end - w);
        w += n;
        done += n;
        return true;
    }
};

// kShared: the two groups have rows of their own and share the tiles; otherwise they have the same
// rows, A the CTA's tiles 0, 2, ... and B 1, 3, ...: each sees every use of its slots of the ring, whose
// barriers tell a use only from the one before it.
template <int D, bool kShared>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_prefix_tc_kernel(const __grid_constant__ PagedDecodeArgs a) {
    using Z = TcSizes<D>;
    constexpr int KS = D / 16;          // K steps of S
    constexpr int CH = D / 8;           // 16-byte chunks of a row
    constexpr int kUnitRows = kShared ? 2 * kRows : kRows;
    constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t kIdescX = idesc_bf16_f32(128, D, 0, 1);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    TcShared &cs = *reinterpret_cast<TcShared *>(base + Z::kCtrl);
    const uint32_t sb = smem_u32(base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();

    const PrefixPieces &f = a.prefix;
    const int len = min(max(__ldcg(f.len), 0), f.max_tokens);
    Walk walk;
    walk.tiles = prefix_tiles(f);
    if (walk.tiles == 0) return;
    const long long chunk = prefix_chunk(f, walk.tiles);
    walk.w = blockIdx.x * chunk;
    walk.end = min(walk.w + chunk, (long long)f.units * walk.tiles);
    if (walk.w >= walk.end) return;
    const int all_rows = a.batch * a.group;

    auto bar = [&](const uint64_t &b) { return smem_u32(&b); };
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar(cs.full[i]), kCopyWarps);
            mbar_init(bar(cs.empty[i]), kShared ? 2 : 1);  // the issuers that read the tile
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(cs.q_ready[x]), kGroupWarps);
            mbar_init(bar(cs.s_full[x]), 2);  // the MMAs, and the issuer's mask
            mbar_init(bar(cs.p_ready[x]), kGroupWarps);
            mbar_init(bar(cs.done[x]), 1);
        }
        cs.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&cs.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns start at column 0: a constant for the issuers, whose operands have to be uniform
    const uint32_t tmem = __shfl_sync(0xffffffffu, cs.tmem_base, 0);
    volatile int *abort_flag = &cs.abort;
    const bool tmem_ok = tmem == 0;  // never expected to fail
    auto ring = [&](int slot) { return sb + Z::kRingAt + slot * Z::kTile; };

    if (!tmem_ok) {
        // leave TMEM alone; the error word is raised below
    } else if (warp < 2 * kGroupWarps) {
        // ================= rows =================
        const int x = warp / kGroupWarps, quarter = warp & 3, half = (warp >> 2) & 1;
        const int r = quarter * 32 + lane;  // row of the group, TMEM lane
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + x * 128 + half * 64;
        const uint32_t tx = tmem + lanes + kColX + x * 128 + half * (D / 2);
        const int pair = 1 + x * 4 + quarter;
        const uint32_t s_bar = bar(cs.s_full[x]);
        uint32_t steps = 0;  // completions of s_full
        bool ok = true;
        while (ok && walk.next()) {
            const int kvh = walk.unit / f.units_per_head;
            const int in_unit = (kShared ? x * kRows : 0) + r;
            const int row = (walk.unit - kvh * f.units_per_head) * kUnitRows + in_unit;
            const int n = kShared ? walk.n : (walk.n - ((x - walk.at) & 1) + 1) / 2;
            if (n > 0) {  // this thread's half of its row of Q
                const int request = row / a.group;
                const uint4 *qp = reinterpret_cast<const uint4 *>(
                    static_cast<const __nv_bfloat16 *>(a.q) + (size_t)request * a.q_stride +
                    (size_t)(kvh * a.group + row - request * a.group) * D);
                const uint32_t q_at = sb + x * (kRows * D * 2);
#pragma unroll
                for (int c = 0; c < CH / 2; ++c) {
                    const int ch = half * (CH / 2) + c;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (row < all_rows) v = __ldcg(qp + ch);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q_at + place(r, ch)),
                                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(cs.q_ready[x]));
            }
            float2 o[D / 4];
#pragma unroll
            for (int i = 0; i < D / 4; ++i) o[i] = make_float2(0.f, 0.f);
            float m = -kInf;
            float2 l2 = make_float2(0.f, 0.f);
            // o <- (o + X) f
            auto add_x = [&](float k) {
                const bool scale = __any_sync(0xffffffffu, k != 1.f);
                const float2 k2 = make_float2(k, k);
#pragma unroll
                for (int c = 0; c < D / 2; c += 16) {
                    float v[16];
                    tmem_ld16(tx + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[c / 2 + i] = f2_add(o[c / 2 + i], make_float2(v[2 * i], v[2 * i + 1]));
                    if (scale) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[c / 2 + i] = f2_mul(o[c / 2 + i], k2);
                    }
                }
            };
            const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
            for (int j = 0; j < n; ++j) {
                ok = warp_wait(s_bar, steps & 1, abort_flag);
                ++steps;
                tc_fence_after();
                const uint32_t *mask = cs.mask[x][j & 1];
                const uint32_t h0 = mask[2 * half], h1 = mask[2 * half + 1];
                const bool whole = (mask[0] & mask[1] & mask[2] & mask[3]) == 0xffffffffu;
                const bool some = (mask[0] | mask[1] | mask[2] | mask[3]) != 0;
                float top = some ? kLowest : -kInf;
                if (ok) {
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        float v[32];
                        tmem_ld32(ts + c, v);
                        tmem_wait_ld();
                        if (!whole) {
                            const uint32_t h = c ? h1 : h0;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if ((h >> i) & 1) top = fmaxf(top, v[i] * a.scale_log2);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 t = f2_mul(make_float2(v[2 * i], v[2 * i + 1]), sc2);
                                top = fmaxf(top, fmaxf(t.x, t.y));
                            }
                        }
                    }
                }
                cs.part[x][j & 1][half][r] = top;
                ok = pair_and(pair, ok);
                if (!ok) break;
                top = fmaxf(top, *const_cast<volatile float *>(&cs.part[x][j & 1][half ^ 1][r]));
                const float now = fmaxf(m, top);
                const float k = now == m ? 1.f : ex2(m - now);
                m = now;
                if (j > 0) add_x(k);  // X of the tile before: S came after it
                l2 = f2_mul(l2, make_float2(k, k));
                const float b = m == -kInf ? 0.f : -m;
                const float2 b2 = make_float2(b, b);
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    float v[16];
                    tmem_ld16(ts + c, v);
                    tmem_wait_ld();
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 t = f2_fma(make_float2(v[2 * i], v[2 * i + 1]), sc2, b2);
                        float2 p = make_float2(ex2(t.x), ex2(t.y));
                        if (!whole) {
                            const uint32_t h = (c & 32 ? h1 : h0) >> ((c & 16) + 2 * i);
                            p.x = h & 1 ? p.x : 0.f;
                            p.y = h & 2 ? p.y : 0.f;
                        }
                        l2 = f2_add(l2, p);
                        const Parts q = parts_of(p.x, p.y);
                        w[i] = q.hi;
                        w[8 + i] = q.lo;
                    }
                    tmem_st16(ts + c, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(cs.p_ready[x]));
            }
            if (!ok) break;
            float l = l2.x + l2.y;
            if (n > 0) {
                ok = warp_wait(s_bar, steps & 1, abort_flag);
                ++steps;
                tc_fence_after();
                if (ok) add_x(1.f);
                tc_fence_before();
                // (the buffer of tile n - 2: its last readers have passed tile n - 1's barrier)
                cs.part[x][n & 1][half][r] = l;
                ok = pair_and(pair, ok);
                if (!ok) break;
                l += *const_cast<volatile float *>(&cs.part[x][n & 1][half ^ 1][r]);
            }
            if (row < all_rows) {
                float *slot = f.pieces + ((size_t)(blockIdx.x + walk.unit) * f.parts + (kShared ? 0 : x)) *
                                             f.stride * (D + 2);
                float *at = slot + (size_t)in_unit * D + half * (D / 2);
#pragma unroll
                for (int c = 0; c < D / 4; c += 2)
                    *reinterpret_cast<float4 *>(at + 2 * c) = make_float4(o[c].x, o[c].y, o[c + 1].x, o[c + 1].y);
                if (half == 0)
                    *reinterpret_cast<float2 *>(slot + (size_t)f.stride * D + 2 * in_unit) = make_float2(m, l);
            }
        }
    } else if (warp < kCopy0) {
        // ================= MMA issuers =================
        const int x = warp - kIssue0;
        const uint64_t dq = sdesc_sw128(sb + x * (kRows * D * 2), 16, 1024);
        const uint32_t t_s = x * 128, t_x = kColX + x * 128;
        uint32_t parts = 0, tiles = 0;
        bool ok = true;
        while (ok && walk.next()) {
            const int first = kShared ? 0 : (x - walk.at) & 1, step = kShared ? 1 : 2;
            if (first < walk.n) {
                ok = warp_wait(bar(cs.q_ready[x]), parts & 1, abort_flag);
                ++parts;
            }
            int j = 0;
            for (int i = first; ok && i < walk.n; i += step, ++j, ++tiles) {
                const int t = walk.at + i, ks = (2 * t) & (kRing - 1), vs = ks + 1;
                const uint32_t ph = (t >> 1) & 1;
                ok = warp_wait(bar(cs.full[ks]), ph, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (lane < 4) cs.mask[x][j & 1][lane] = cs.have[t & 1][lane];
                const uint64_t dk = sdesc_sw128(ring(ks), 16, 1024);
                __syncwarp();
                if (elect_one()) {
#pragma unroll
                    for (uint32_t k = 0; k < KS; ++k)
                        mma_bf16(t_s, dq + (uint64_t)((k & 3u) * 2 + (k >> 2) * (kAtoms >> 4)),
                                 dk + (uint64_t)((k & 3u) * 2 + (k >> 2) * (kAtoms >> 4)), kIdescS, k ? 1u : 0u);
                    mma_commit(bar(cs.s_full[x]));
                    mma_commit(bar(cs.empty[ks]));
                    mbar_arrive(bar(cs.s_full[x]));
                }
                __syncwarp();
                ok = warp_wait(bar(cs.p_ready[x]), tiles & 1, abort_flag) &&
                     warp_wait(bar(cs.full[vs]), ph, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dv = sdesc_sw128(ring(vs), kAtoms, 1024);
                if (elect_one()) {
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) {
                        mma_bf16_tmem_a(t_x, t_s + 16 * k + 8, dv + (uint64_t)(128u * k), kIdescX, k ? 1u : 0u);
                        mma_bf16_tmem_a(t_x, t_s + 16 * k, dv + (uint64_t)(128u * k), kIdescX, 1u);
                    }
                    mma_commit(bar(cs.empty[vs]));
                }
                __syncwarp();
            }
            if (ok && j > 0 && elect_one()) {
                mma_commit(bar(cs.s_full[x]));
                mbar_arrive(bar(cs.s_full[x]));
            }
            __syncwarp();
        }
        // all MMAs have to be finished before TMEM is released
        if (elect_one()) mma_commit(bar(cs.done[x]));
        __syncwarp();
        int no_abort = 0;
        warp_wait(bar(cs.done[x]), 0, &no_abort);
    } else {
        // ================= copies =================
        // Rows c * 64 .. + 63 of every tile; lane l finds rows l and l + 32 of them.
        const int w = warp - kCopy0;
        const int first = w * 64;
        int pending = 0;  // copies (groups) that have not been reported
        int reported = 0, issued = 0;
        bool ok = true;
        auto report = [&]() {  // the oldest of them has landed
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(cs.full[reported & (kRing - 1)]));
            ++reported;
            --pending;
        };
        auto drain = [&]() {
            if (pending == 2) {
                cp_wait<1>();
                report();
            }
            if (pending == 1) {
                cp_wait<0>();
                report();
            }
        };
        auto locate = [&](int tile, int(&page)[2], int(&rw)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = tile * kTokens + first + i * 32 + lane;
                page[i] = -1;
                rw[i] = 0;
                if (t < len) {
                    const int blk = t / a.page_size;
                    rw[i] = t - blk * a.page_size;
                    page[i] = a.block_table[blk];
                    if (page[i] >= a.num_pages) page[i] = -1;
                }
            }
        };
        auto copy = [&](const __nv_bfloat16 *cache, int64_t page_stride, int kvh, const int(&page)[2],
                        const int(&rw)[2]) -> bool {
            const int slot = issued & (kRing - 1);
            const uint32_t parity = ((issued / kRing) & 1) ^ 1;
            if (!__all_sync(0xffffffffu, mbar_try_wait(bar(cs.empty[slot]), parity))) {
                drain();  // nothing to do but report what has come
                if (!warp_wait(bar(cs.empty[slot]), parity, abort_flag)) return false;
            }
            if ((issued & 1) == 0) {  // K: which of its tokens there are
                const uint32_t lo = __ballot_sync(0xffffffffu, page[0] >= 0);
                const uint32_t hi = __ballot_sync(0xffffffffu, page[1] >= 0);
                if (lane == 0) {
                    cs.have[(issued >> 1) & 1][2 * w] = lo;
                    cs.have[(issued >> 1) & 1][2 * w + 1] = hi;
                }
            }
            constexpr int RPI = 32 / CH;  // rows of a warp-wide copy
            const int ch = lane % CH;
            const uint32_t dst = ring(slot);
#pragma unroll
            for (int i = 0; i < 64 / RPI; ++i) {
                const int rr = i * RPI + lane / CH;  // of the warp's 64
                const int pg = __shfl_sync(0xffffffffu, page[i * RPI / 32], rr & 31);
                const int rowp = __shfl_sync(0xffffffffu, rw[i * RPI / 32], rr & 31);
                const __nv_bfloat16 *src = cache + (size_t)max(pg, 0) * page_stride +
                                           ((size_t)kvh * a.page_size + rowp) * D + ch * 8;
                cp_async16(dst + place(first + rr, ch), src, pg >= 0);
            }
            cp_commit();
            ++issued;
            if (++pending > 2) {
                cp_wait<2>();
                report();
            }
            return true;
        };
        int page[2], rw[2];
        while (ok && walk.next()) {
            const int kvh = walk.unit / f.units_per_head;
            locate(walk.tile, page, rw);
            for (int i = 0; ok && i < walk.n; ++i) {
                int page2[2], rw2[2];
                locate(walk.tile + i + 1, page2, rw2);  // the table is read a tile ahead
                ok = copy(static_cast<const __nv_bfloat16 *>(a.k), a.k_page_stride, kvh, page, rw) &&
                     copy(static_cast<const __nv_bfloat16 *>(a.v), a.v_page_stride, kvh, page, rw);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    page[e] = page2[e];
                    rw[e] = rw2[e];
                }
            }
        }
        if (ok) drain();
        cp_wait<0>();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && (cs.abort || !tmem_ok)) atomicOr(&g_prefix_error, 1u);
}

template <int D, bool kShared> cudaError_t launch_tc(const PagedDecodeArgs &a) {
    constexpr auto kern = paged_prefix_tc_kernel<D, kShared>;
    constexpr int smem = (int)TcSizes<D>::kSmem;
    static_assert(TcSizes<D>::kSmem <= 232448, "shared memory budget");
    cudaError_t e = allow_smem<kern>(smem);
    if (e == cudaSuccess) e = launch_dependent(kern, a.prefix.ctas, kTcThreads, smem, a.stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t paged_prefix_tc(const PagedDecodeArgs &a) {
    const bool shared = a.prefix.parts == 1;
    if (a.head_dim == 128) return shared ? launch_tc<128, true>(a) : launch_tc<128, false>(a);
    if (a.head_dim == 64) return shared ? launch_tc<64, true>(a) : launch_tc<64, false>(a);
    return cudaErrorNotSupported;
}

cudaError_t take_prefix_device_error(unsigned int *err) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_prefix_error, sizeof(v));
    if (e == cudaSuccess && v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_prefix_error, &zero, sizeof(zero));
    }
    if (e == cudaSuccess) *err = v;
    return e;
}

}  // namespace la
