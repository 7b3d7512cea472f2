// The attention over a shared prefix on the tensor cores (tcgen05 + TMEM), bf16: for the query
// heads of all requests that share a key-value head (its rows), tile by tile of 128 tokens,
//     S = Q K^T,   P = e^(scale S - m),   X = P V,   o <- o f + X,   l <- l f + sum P
// with a base m of each row near its running maximum and f = e^(m before - m).  A CTA leaves m, l and the
// unnormalised o of its part of a unit (PrefixPieces); see paged_prefix.cu for the split.
//
// Bound: a row does 4 D flops a token, so with many rows the tensor core bounds the kernel, with few (and
// K and V read once for all of them) HBM.  Measured, 8 key-value heads of 128, 64 query heads: 32
// requests behind 64K tokens 107 us with all that follows (0.64 PFLOP/s of the formula's products, 0.96
// of those that are done; the tensor pipe is busy 52 % of this kernel's cycles), 16 requests behind 128K
// 127 us (4.2 TB/s), one 109 us (4.9 TB/s).  What bounds it then is the chain of a group's tile, about
// 5000 cycles by cycle stamps: P V and the next S (1536 on the tensor core), the weights, and 500 to 800
// from each of them to the threads that wait for it; two chains in turn keep the tensor core busy for
// three fifths of it.  Half the exponentials moved to FMAs, or none of the low parts, change the time by 0
// to 4 %.  A third group finds no room in tensor memory.  At its 96 registers the kernel spills: 128 and 168
// bytes at 128 wide (tiles shared by the groups, and not), 84 and 68 at 64; which role does has not been told apart.
//
// P is passed as two bf16 parts (parts_of: off by at most 2^-16 of each weight, as in the attention
// of one request), which makes P V two products instead of one: 1536 tensor cycles a 128 x 128
// tile instead of 1024.  One part would add as much error again as the output's own rounding.
// X is taken anew for every tile and added to o in registers: rounded to nearest, where the tensor
// core's own accumulation over a long prefix drops the bits that do not fit, and a maximum
// that moves costs a product in registers instead of a pass through tensor memory.
//
// A CTA has two groups of 128 rows, A and B, which share every tile of K and V in shared memory:
// the tensor core works on one group's products while the other group's 256 threads take its
// exponentials.  Where a key-value head has no more than 128 rows, both groups have the same
// rows and every other tile each, and leave a part each.
//
// TMEM (512 columns): S of A and B 128 columns each, X 128, Q of A and B 64 each.  P takes the place of
// S: 8 tokens' scores are 8 columns, their weights 4 columns of high and 4 of low parts, which together
// are one K step of 16; its operand V is the 8 tokens' rows twice (a stride of 0 between groups of 8
// rows).  Q is there because a 128 x 128 product of two operands in shared memory was issued at half the
// rate (about 1100 cycles for S instead of 512); the room for it comes from X, which the two groups
// share: a group takes its X to registers while its own next S runs, before the other group's P V needs
// the place.
//
// Warp roles (640 threads):
//   warps 0-7    rows of A: two threads a row, each with 64 of a tile's tokens and half of
//                the columns of o; warps 8-15 those of B
//   warps 16, 17 MMA issuers of A and B: P V of a tile, then the group's next S (one thread's MMAs run in the
//                order of their issue, so S does not overtake the P V that reads P in its place).  The one
//                place of X keeps the groups half a period apart; in step, the tensor core would idle while
//                both take exponentials
//   warp 18      copies of K and V into a ring of three tiles: TMA boxes of as many rows as divide
//                both a page and a tile, where those are at least eight; other page sizes and the rows behind
//                the prefix's end (which may hold anything, and are read as zeros) row by row with cp.async
//   warp 19      only gives up registers
// Every wait is bounded; one that gives up sets the CTA's abort flag, all roles leave, copies and MMAs
// are drained, TMEM is freed and the device error word is raised.
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "paged_attention.cuh"

namespace la {

__device__ unsigned int g_prefix_error = 0;  // bit 0: a bounded wait gave up

namespace {

using namespace ptx;

constexpr int kTokens = kPrefixTile;  // of a tile
constexpr int kRows = 128;            // of a group
constexpr int kGroupWarps = 8;
constexpr int kIssue0 = 16, kCopy = 18;
constexpr int kTcThreads = 640;
constexpr int kTiles = 3;             // tiles of tokens in shared memory
constexpr int kRing = 2 * kTiles;     // their K and V
constexpr uint32_t kAtoms = kTokens * 128;  // 128 rows of 64 bf16
// Weights are taken against a base that may lie below the row's maximum: the maximum of the tiles
// before, so that a tile's weights need not wait for its own.  A tile whose maximum is more than kRedo above is
// taken again (S once more, then its maximum first), and the weights are e^(s - base) 2^-kRedo, so at most 1, and
// sums of the largest values pass the type's range no earlier than against the maximum itself.  (The
// factor is part of the base where the sums are written.  What it takes from the other end, weights of less than
// 2^-102 of the largest whose low part may be 0, is below the 2^-100 that infinite values are promised.)
// A base that is kMove below is moved after the tile.  (log2)
constexpr float kRedo = 8.f, kMove = 4.f;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kColX = 256, kColQ = 384;
static_assert(kTokens == 128 && kRows == 128, "operand shapes");

struct TcShared {
    uint64_t full[kTiles], empty[kTiles];
    uint64_t q_ready[2], s_full[2], p_ready[2], x_full[2], done[2];
    alignas(16) uint32_t have[kTiles][4];  // present tokens of a tile, by its place in the ring
    uint32_t tmem_base;
    int redo[2];                // the group wants S of its tile once more
    int abort;
    alignas(1024) float part[2][3][2][kRows];  // group, tile & 1, half: a row's maximum over the half's tokens
};

template <int D> struct TcSizes {
    static constexpr uint32_t kTile = kTokens * D * 2;
    static constexpr uint32_t kCtrl = kRing * kTile;
    static constexpr uint32_t kSmem = kCtrl + sizeof(TcShared) + 1024;  // + alignment slack
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, kTimeoutNs));
}
// Whether the phase is complete, without a wait.
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// The same for the warps that hold rows, without a call: their registers would have to be stored for it.
__device__ __forceinline__ bool row_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
        while (!(ok = mbar_try_wait_sleep(bar, parity, 200000u)) && !*abort)
            if (globaltimer_ns() - t0 > kTimeoutNs) *abort = 1;
    }
    return __all_sync(0xffffffffu, ok);
}
// Barrier of a group's 256 threads; true where any of them says so.
__device__ __forceinline__ bool group_any(int id, bool some) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
                 "barrier.cta.red.or.pred q, %1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(id), "r"((uint32_t)some) : "memory");
    return r != 0;
}
__device__ __forceinline__ void st_part(uint32_t at, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ float ld_part(uint32_t at) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}
// Gives registers of the other warps to those that hold rows: 512 threads of 104 and 128 of 64 are the 640
// of 96 that the kernel is launched with.
template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
static_assert(512 * 104 + 128 * 64 <= kTcThreads * 96, "registers");

// The weights of 8 scores of a row in their place: the sum to l, the high parts (as parts_of has
// them) of tokens 2 i and 2 i + 1 to element i, the low ones to element i + 4.
__device__ __forceinline__ void weights_of(float (&v)[8], float scale, float base, float2 &l) {
    const float2 up = make_float2(1.f + 0x1p-23f, 1.f + 0x1p-23f);
    uint32_t lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = f2_fma(make_float2(v[2 * i], v[2 * i + 1]), make_float2(scale, scale),
                                make_float2(base, base));
        const float2 p = make_float2(ex2(t.x), ex2(t.y));
        l = f2_add(l, p);
        const uint32_t x = __float_as_uint(p.x), y = __float_as_uint(p.y);
        const float2 rest = f2_fma(p, up, make_float2(__uint_as_float((x & 0xffff0000u) ^ 0x80000000u),
                                                      __uint_as_float((y & 0xffff0000u) ^ 0x80000000u)));
        v[i] = __uint_as_float(__byte_perm(x, y, 0x7632));
        lo[i] = pack2(rest.x, rest.y);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 + i] = __uint_as_float(lo[i]);
}
// Bits 0, 2, 4, ... of x.
__device__ __forceinline__ uint16_t every_other(uint32_t x) {
    x &= 0x55555555u;
    x = (x | x >> 1) & 0x33333333u;
    x = (x | x >> 2) & 0x0f0f0f0fu;
    x = (x | x >> 4) & 0x00ff00ffu;
    return (uint16_t)(x | x >> 8);
}
// A CTA's parts of units, in order: `left` tiles from tile `tile` of unit `unit` on.
struct Walk {
    int tiles;    // of the prefix
    int left, at; // the CTA's tiles behind this part, before it
    int unit, tile, n;  // this part: tiles tile .. tile + n - 1 of the unit

    __device__ __forceinline__ bool next() {
        if (left == 0) return false;
        at += n;
        tile = n ? 0 : tile;  // (the first part may begin anywhere, the others begin their unit)
        unit += n ? 1 : 0;
        n = min(tiles - tile, left);
        left -= n;
        return true;
    }
};

// kShared: the two groups have rows of their own and share the tiles; otherwise they have the same
// rows, A the CTA's tiles 0, 2, ... and B 1, 3, ...
template <int D, bool kShared>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_prefix_tc_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, int box) {
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
    if (warp == kCopy && lane == 0 && box) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    grid_dependency_wait();
    release_to_next(a.prefix.ranges + 2);
    grid_launch_dependents();

    const PrefixPieces &f = a.prefix;
    const int len = min(max(__ldcg(f.len), 0), f.max_tokens);
    Walk walk;
    bool alone;  // a CTA has a single tile
    walk.tiles = prefix_tiles(f);
    if (walk.tiles == 0) return;
    int ranges = f.ctas;
    if (f.share) {
        __shared__ long long sums[kTcThreads / 32];
        long long own = 0;
        for (int i = threadIdx.x; i < a.batch; i += kTcThreads)
            own += unit_cost<kOverhead<__nv_bfloat16, D>>(own_len(a, i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
        if (lane == 0) sums[warp] = own;
        __syncthreads();
        own = 0;
#pragma unroll
        for (int i = 0; i < kTcThreads / 32; ++i) own += sums[i];
        // (a request's units: its key-value heads, and up to 16 query heads of each)
        ranges = ranges_beside<D>(f, walk.tiles, own * a.num_kv_heads * ((a.group + 15) / 16));
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *f.ranges = ranges;
    if ((int)blockIdx.x >= ranges) return;
    {
        const long long chunk = prefix_chunk(f, walk.tiles, ranges), w = blockIdx.x * chunk;
        const long long end = min(w + chunk, (long long)f.units * walk.tiles);
        if (w >= end) return;
        walk.unit = range_of(w, walk.tiles);
        walk.tile = (int)(w - (long long)walk.unit * walk.tiles);
        walk.left = (int)(end - w);
        walk.at = walk.n = 0;
        alone = chunk == 1;
    }
    const int all_rows = a.batch * a.group;

    auto bar = [&](const uint64_t &b) { return smem_u32(&b); };
    if (threadIdx.x == 0) {
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(bar(cs.full[i]), 1);
            mbar_init(bar(cs.empty[i]), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(cs.q_ready[x]), kGroupWarps);
            mbar_init(bar(cs.s_full[x]), 2);  // the MMAs, and the issuer for the copies' `have`
            mbar_init(bar(cs.p_ready[x]), 1 + kGroupWarps);  // P, and the place of X from the other group
            mbar_init(bar(cs.x_full[x]), 1);
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
    auto ring = [&](int slot) { return sb + slot * Z::kTile; };

    if (warp < 2 * kGroupWarps)
        more_registers<104>();
    else
        fewer_registers<64>();
    if (!tmem_ok) {
        // leave TMEM alone; the error word is raised below
    } else if (warp < 2 * kGroupWarps) {
        // ================= rows =================
        const int x = warp / kGroupWarps, quarter = warp & 3, half = (warp >> 2) & 1;
        const int r = quarter * 32 + lane;  // row of the group, TMEM lane
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + x * 128 + half * 64;
        const uint32_t tx = tmem + lanes + kColX + half * (D / 2);
        const int group = 1 + x;
        // A negative scale goes into the signs of Q, so that the largest score is the largest S, and a
        // scale of 0 into Q as a whole, so that an S of -infinity has weight 0 whatever the scale (0 times
        // an infinite or NaN query is NaN).
        const float scale = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
        auto scaled = [&](uint32_t x) {
            if (a.scale_log2 != 0.f) return x ^ flip;
            return ((x & 0x7f80u) == 0x7f80u ? 0x7fffu : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 0x7fff0000u : 0u);
        };
        // where the two threads of a row exchange a number: halves and tiles apart by powers of two
        constexpr uint32_t kOther = kRows * 4, kNext = 2 * kOther;
        const uint32_t mine = smem_u32(&cs.part[x][0][half][r]);
        const bool leads = (threadIdx.x & (32 * kGroupWarps - 1)) == 0;
        uint32_t tiles = 0, steps = 0;  // of this group so far: tiles, and its S
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
                    (size_t)(kvh * a.group + row - request * a.group) * D) + half * (CH / 2);
                const uint32_t q_at = tmem + lanes + kColQ + x * 64 + half * (D / 4);
#pragma unroll
                for (int c = 0; c < CH / 2; c += 4) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (row < all_rows) v = __ldcg(qp + c + i);
                        w[4 * i] = scaled(v.x);
                        w[4 * i + 1] = scaled(v.y);
                        w[4 * i + 2] = scaled(v.z);
                        w[4 * i + 3] = scaled(v.w);
                    }
                    tmem_st16(q_at + 4 * c, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(cs.q_ready[x]));
            }
            float2 o[D / 4];
#pragma unroll
            for (int i = 0; i < D / 4; ++i) o[i] = make_float2(0.f, 0.f);
            float m = -kInf;
            float2 l2 = make_float2(0.f, 0.f);
            // Another base.
            auto rescale = [&](float to) {
                const float k = to == m ? 1.f : ex2(m - to);
                m = to;
                l2 = f2_mul(l2, make_float2(k, k));
#pragma unroll
                for (int i = 0; i < D / 4; ++i) o[i] = f2_mul(o[i], make_float2(k, k));
            };
            // o <- o + X of the tile before, while the tensor core takes the next S
            auto add_x = [&]() -> bool {
                if (!row_wait(bar(cs.x_full[x]), (tiles - 1) & 1, abort_flag)) return false;
                tc_fence_after();
                constexpr int kBlocks = D / 32;  // of 16 columns
                float v[2][16];
                tmem_ld16(tx, v[0]);
                tmem_ld16(tx + 16, v[1]);
#pragma unroll
                for (int c = 0; c < kBlocks; c += 2) {
                    tmem_wait_ld();
                    if (c + 2 == kBlocks) {  // X is in registers: its place is the other group's
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(cs.p_ready[x ^ 1]));
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            o[c * 8 + e * 8 + i] =
                                f2_add(o[c * 8 + e * 8 + i], make_float2(v[e][2 * i], v[e][2 * i + 1]));
                        if (c + 2 < kBlocks) tmem_ld16(tx + 16 * (c + 2 + e), v[e]);
                    }
                }
                return true;
            };
            bool based = false;   // there is a base (the same for all rows)
            float next = -kInf;   // the base of the next tile
            for (int j = 0; j < n; ++j, ++tiles) {
                if (j > 0) {
                    ok = add_x();
                    if (__any_sync(0xffffffffu, next != m)) rescale(next);
                }
                while (true) {
                    if (ok) ok = row_wait(bar(cs.s_full[x]), steps & 1, abort_flag);
                    ++steps;
                    tc_fence_after();
                    const int at = (kShared ? walk.at + j : 2 * (int)tiles + x) % kTiles;
                    const uint4 mask = *reinterpret_cast<const uint4 *>(cs.have[at]);
                    if (ok && (mask.x & mask.y & mask.z & mask.w) != 0xffffffffu) {
                        // tokens that are not there: S is -infinity
#pragma unroll 1
                        for (int c = 0; c < 64; c += 16) {
                            const uint32_t word = half ? c & 32 ? mask.w : mask.z : c & 32 ? mask.y : mask.x;
                            const uint32_t here = word >> (c & 16);
                            float v[16];
                            tmem_ld16(ts + c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = (here >> i) & 1 ? v[i] : -kInf;
                            tmem_st16(ts + c, reinterpret_cast<const uint32_t (&)[16]>(v));
                        }
                        tmem_wait_st();
                    }
                    float top = -kInf;
                    if (!based) {  // the row's maximum first
                        if (ok) {
#pragma unroll 1
                            for (int c = 0; c < 64; c += 16) {
                                float v[16];
                                tmem_ld16(ts + c, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; i += 2) top = fmaxf(fmaxf(top, v[i]), v[i + 1]);
                            }
                        }
                        st_part(mine + 2 * kNext, top);
                        ok = !group_any(group, !ok);
                        if (!ok) break;
                        top = fmaxf(top, ld_part((mine ^ kOther) + 2 * kNext)) * scale;
                        based = (mask.x | mask.y | mask.z | mask.w) != 0;
                        rescale(fmaxf(m, fmaxf(top, based ? kLowest : -kInf)));
                        top = -kInf;
                    }
                    const float b = m == -kInf ? 0.f : -(m + kRedo);
                    float2 sum = make_float2(0.f, 0.f);
                    if (ok) {
                        float v[2][8];
                        tmem_ld8(ts, v[0]);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            float (&u)[8] = v[c & 1];
                            tmem_wait_ld();
                            if (c < 7) tmem_ld8(ts + 8 * c + 8, v[(c + 1) & 1]);
#pragma unroll
                            for (int i = 0; i < 8; i += 2) top = fmaxf(fmaxf(top, u[i]), u[i + 1]);
                            weights_of(u, scale, b, sum);
                            tmem_st8(ts + 8 * c, reinterpret_cast<const uint32_t (&)[8]>(u));
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    // (two places in turn: a partner may be reading the one of the tile before)
                    st_part(mine + (tiles & 1) * kNext, top);
                    const bool again = group_any(group, !ok || top * scale > m + kRedo);
                    if (again) ok = !group_any(group, !ok);  // one outcome for all warps
                    if (!ok) break;
                    if (leads) {
                        cs.redo[x] = again;
                        mbar_arrive(bar(cs.p_ready[x]));
                    }
                    if (!again) {
                        l2 = f2_add(l2, sum);
                        top = fmaxf(top, ld_part((mine ^ kOther) + (tiles & 1) * kNext)) * scale;
                        next = top > m + kMove ? top : m;
                        break;
                    }
                    based = false;
                }
                if (!ok) break;
            }
            if (!ok) break;
            float l = l2.x + l2.y;
            if (n > 0) {
                ok = add_x();
                st_part(mine + 2 * kNext, l);
                ok = !group_any(group, !ok);
                if (!ok) break;
                l += ld_part((mine ^ kOther) + 2 * kNext);
            }
            if (row < all_rows && (n > 0 || !alone)) {
                float *slot = f.pieces + ((size_t)(blockIdx.x + walk.unit) * f.parts + (kShared ? 0 : x)) *
                                             f.stride * (D + 2);
                float *at = slot + (size_t)in_unit * D + half * (D / 2);
#pragma unroll
                for (int c = 0; c < D / 4; c += 2)
                    *reinterpret_cast<float4 *>(at + 2 * c) = make_float4(o[c].x, o[c].y, o[c + 1].x, o[c + 1].y);
                if (half == 0)
                    *reinterpret_cast<float2 *>(slot + (size_t)f.stride * D + 2 * in_unit) = make_float2(m + kRedo, l);
            }
        }
    } else if (warp < kCopy) {
        // ================= MMA issuers =================
        // What an issuer does between two of its items (about 60 instructions, each behind the last) is as
        // long as the items themselves; with one for each group it passes while the other's run.  A waits
        // for as few things as there can be: a tile (K and V together), and its group's weights
        // together with the other group's word that X has been taken.
        const int x = warp - kIssue0;
        const uint32_t s_at = x * 128, q_at = kColQ + x * 64;
        const uint32_t s_full = bar(cs.s_full[x]), x_full = bar(cs.x_full[x]), p_ready = bar(cs.p_ready[x]);
        // the group's tiles of the CTA: t = first, first + step, ...
        const int total = walk.left, step = kShared ? 1 : 2, first = kShared ? 0 : x;
        int part_end = 0;                  // tiles of the parts entered so far
        bool fresh = false;                // the group's Q has not been waited for
        uint32_t parts = 0, weights = 0;   // phases of q_ready and p_ready
        // Whether tile t is the group's first of a part, whose Q is then to be waited for.
        auto is_fresh = [&](int t) {
            while (t >= part_end) {
                walk.next();
                part_end = walk.at + walk.n;
                fresh = true;
            }
            return fresh;
        };
        auto wait_tile = [&](int t) -> bool {
            return warp_wait(bar(cs.full[t % kTiles]), (t / kTiles) & 1, abort_flag);
        };
        // (by one lane, with operands that the whole warp has computed: else each MMA becomes a loop)
        auto issue_s = [&](uint64_t dk) {
#pragma unroll
            for (uint32_t i = 0; i < KS; ++i)
                mma_bf16_tmem_a(s_at, q_at + 8 * i, dk + (uint64_t)((i & 3u) * 2 + (i >> 2) * (kAtoms >> 4)), kIdescS,
                                i ? 1u : 0u);
            mma_commit(s_full);
            mbar_arrive(s_full);
        };
        auto issue_x = [&](uint64_t dv, uint32_t empty) {
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i)
                mma_bf16_tmem_a(kColX, s_at + 8 * i, dv + (uint64_t)(64u * i), kIdescX, i ? 1u : 0u);
            mma_commit(x_full);
            // K could be wanted once more until the weights were there; B's P V comes behind A's, whose X
            // has been taken
            if (!kShared || x) mma_commit(empty);
        };
        auto start = [&](int t) -> bool {  // S of a tile, waiting for Q where that is new
            if (is_fresh(t)) {
                if (!warp_wait(bar(cs.q_ready[x]), parts & 1, abort_flag)) return false;
                ++parts;
                fresh = false;
            }
            if (!wait_tile(t)) return false;
            tc_fence_after();
            const uint64_t dk = sdesc_sw128(ring(t % kTiles * 2), 16, 1024);
            if (elect_one()) issue_s(dk);
            __syncwarp();
            return true;
        };
        if (x == 0 && lane < kGroupWarps) mbar_arrive(p_ready);  // nobody's X is in the first item's way
        __syncwarp();
        bool ok = first >= total || start(first);
        for (int t = first; ok && t < total; t += step) {
            const int at = t % kTiles, next = (t + step) % kTiles;
            const bool more = t + step < total, same = more && !is_fresh(t + step);
            const uint64_t dv = sdesc_sw128(ring(2 * at + 1), kAtoms, 0), dk = sdesc_sw128(ring(2 * next), 16, 1024);
            const uint32_t empty = bar(cs.empty[at]);
            while (ok) {
                ok = warp_wait(p_ready, weights++ & 1, abort_flag);
                if (!ok || !*const_cast<volatile int *>(&cs.redo[x])) break;
                const uint64_t dk_now = sdesc_sw128(ring(2 * at), 16, 1024);
                if (lane < kGroupWarps) mbar_arrive(p_ready);  // X has been taken already
                tc_fence_after();
                __syncwarp();
                if (elect_one()) issue_s(dk_now);
                __syncwarp();
            }
            if (!ok) break;
            // P V of the tile and the group's next S go out together where nothing is to be waited for.  (Where the
            // groups do not share the tiles, the next one comes into the place of the one before this, which has
            // been used up only now that its X is taken: not before, the barrier could not tell the two.)
            const bool follows =
                same && __all_sync(0xffffffffu, test_wait(bar(cs.full[next]), ((t + step) / kTiles) & 1));
            tc_fence_after();
            if (elect_one()) {
                issue_x(dv, empty);
                if (follows) issue_s(dk);
            }
            __syncwarp();
            if (!follows && more) ok = start(t + step);
        }
        // all MMAs have to be finished before TMEM is released
        if (elect_one()) mma_commit(bar(cs.done[x]));
        __syncwarp();
        int no_abort = 0;
        warp_wait(bar(cs.done[x]), 0, &no_abort);
    } else if (warp == kCopy) {
        // ================= copies =================
        // Row by row: two lanes a row (32 bytes, a sector, at a time), lane l the rows l / 2 + 16 i, from one
        // pointer each, without an exchange of addresses.
        constexpr int kMine = 8;  // rows of a lane
        int issued = 0;           // tiles
        bool ok = true, unsaid = false;  // the last tile's copies (cp.async) have not been reported
        auto report = [&](int tile) {  // whose copies have landed
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(cs.full[tile % kTiles]));
        };
        // Pages and offsets inside a page of this lane's rows of a tile (page -1: not there).
        auto locate = [&](int tile, int(&page)[kMine], uint32_t(&in)[kMine]) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int t = tile * kTokens + i * 16 + (lane >> 1);
                page[i] = -1;
                in[i] = 0;
                if (t < len) {
                    const int blk = t / a.page_size;
                    in[i] = t - blk * a.page_size;
                    page[i] = a.block_table[blk];
                    if (page[i] >= a.num_pages) page[i] = -1;
                }
            }
        };
        auto copy = [&](uint32_t at, const void *cache, int64_t page_stride, int kvh, const int(&page)[kMine],
                        const uint32_t(&in)[kMine]) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const bool there = page[i] >= 0;
                const char *src = static_cast<const char *>(cache) + (lane & 1) * 16 +
                                  ((there ? (size_t)page[i] * page_stride : 0) +
                                   ((size_t)kvh * a.page_size + in[i]) * D) * 2;
                const int r = i * 16 + (lane >> 1);
                const uint32_t dst = at + r * 128, turn = (r & 7) << 4, odd = (lane & 1) << 4;
#pragma unroll
                for (int c = 0; c < CH; c += 2)  // chunk c + lane & 1
                    cp_async16(dst + (c >> 3) * kAtoms + ((((c & 7) << 4) | odd) ^ turn), src + c * 16, there);
            }
        };
        // Whole tiles of pages that `box` rows divide: lane l has the TMA copy of rows
        // l / halves * box .. of 64-column half l % halves.  A page that is none is out of the map's
        // range and read as zeros.
        constexpr int kHalves = D / 64;
        auto find_box = [&](int tile, int &page, int &in) {
            const int t = tile * kTokens + lane / kHalves * box;
            page = -1;
            in = 0;
            if (lane < kTokens / box * kHalves && t < len) {
                const int blk = t / a.page_size;
                in = t - blk * a.page_size;
                page = a.block_table[blk];
            }
        };
        auto tma = [&](uint32_t at, uint32_t full, const CUtensorMap &map, int kvh, int page, int in) {
            if (lane < kTokens / box * kHalves)
                tma_load_3d(at + lane % kHalves * kAtoms + lane / kHalves * box * 128, &map, full,
                            lane % kHalves * 64, kvh * a.page_size + in, page);
            __syncwarp();
        };
        int page[kMine], page_at = -1, in_at = 0;
        uint32_t in[kMine];
        while (ok && walk.next()) {
            const int kvh = walk.unit / f.units_per_head;
            if (box) find_box(walk.tile, page_at, in_at);
            for (int i = 0; ok && i < walk.n; ++i) {
                const int tile = walk.tile + i;
                const bool whole = box && (tile + 1) * kTokens <= len;
                const int page_now = page_at >= 0 && page_at < a.num_pages ? page_at : -1, in_now = in_at;
                if (whole) find_box(tile + 1, page_at, in_at);  // the table is read a tile ahead
                else locate(tile, page, in);
                const int slot = issued % kTiles;
                const uint32_t empty = bar(cs.empty[slot]), parity = ((issued / kTiles) & 1) ^ 1;
                if (unsaid && (whole || !__all_sync(0xffffffffu, mbar_try_wait(empty, parity)))) {
                    cp_wait<0>();
                    report(issued - 1);
                    unsaid = false;
                }
                ok = warp_wait(empty, parity, abort_flag);
                if (!ok) break;
                const uint32_t k_at = ring(2 * slot), v_at = ring(2 * slot + 1), full = bar(cs.full[slot]);
                if (whole) {
                    // lane l < 16: tokens 8 l .. + 7
                    const int eight = __shfl_sync(0xffffffffu, page_now, (lane & 15) * 8 / box * kHalves);
                    if (lane < 16) reinterpret_cast<uint8_t *>(cs.have[slot])[lane] = eight >= 0 ? 0xff : 0;
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(full, 2 * Z::kTile);
                    __syncwarp();
                    tma(k_at, full, map_k, kvh, page_now, in_now);
                    tma(v_at, full, map_v, kvh, page_now, in_now);
                    ++issued;
                } else {
#pragma unroll
                    for (int e = 0; e < kMine; ++e) {  // rows 16 e .. + 15, from every other lane
                        const uint32_t both = __ballot_sync(0xffffffffu, page[e] >= 0);
                        if (lane == 0) reinterpret_cast<uint16_t *>(cs.have[slot])[e] = every_other(both);
                    }
                    copy(k_at, a.k, a.k_page_stride, kvh, page, in);
                    copy(v_at, a.v, a.v_page_stride, kvh, page, in);
                    cp_commit();
                    if (unsaid) {
                        cp_wait<1>();
                        report(issued - 1);
                    }
                    unsaid = true;
                    ++issued;
                }
            }
        }
        cp_wait<0>();
        if (unsaid) report(issued - 1);
        // No TMA copy may be landing when the CTA exits.  (Of a CTA that ran to its end all have been used.)
        int no_abort = 0;
        if (!ok)
            for (int i = max(0, issued - kTiles); i < issued; ++i)
                warp_wait(bar(cs.full[i % kTiles]), (i / kTiles) & 1, &no_abort);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && (cs.abort || !tmem_ok)) atomicOr(&g_prefix_error, 1u);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// A cache as [pages][Hkv * page_size][D] bf16, box = `box` rows of 64 columns, 128-byte swizzle.
bool make_map(CUtensorMap *m, const void *cache, int64_t page_stride, const PagedDecodeArgs &a, int box) {
    const EncodeTiledFn enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.num_kv_heads * a.page_size,
                                (cuuint64_t)a.num_pages};
    const cuuint64_t strides[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)page_stride * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1}, ones[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(cache), dims, strides, boxes, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kShared> cudaError_t launch_tc(const PagedDecodeArgs &a) {
    constexpr auto kern = paged_prefix_tc_kernel<D, kShared>;
    constexpr int smem = (int)TcSizes<D>::kSmem;
    static_assert(TcSizes<D>::kSmem <= 232448, "shared memory budget");
    // rows of a box: the largest power of two that divides a page, up to a tile; caches that no map
    // can describe (a stride or a size past its range) go without
    int box = a.page_size & -a.page_size;
    box = box > kTokens ? kTokens : box;
    CUtensorMap map_k = {}, map_v = {};
    if (box < 8 || a.num_pages == 0 || (int64_t)a.num_kv_heads * a.page_size > 0x7fffffffLL ||
        !make_map(&map_k, a.k, a.k_page_stride, a, box) || !make_map(&map_v, a.v, a.v_page_stride, a, box))
        box = 0;
    cudaError_t e = allow_smem<kern>(smem);
    if (e == cudaSuccess)
        e = launch_dependent(kern, a.prefix.ctas, kTcThreads, smem, a.stream, a, map_k, map_v, box);
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
