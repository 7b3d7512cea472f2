// Attention of one new token per request where all requests share a prefix: the prefix's
// keys and values are streamed for the batch, not for each request.
//
// With the prefix's tokens u and the request's own tokens t, a softmax over both is
//     out = (e^(m' - m) A' + e^(m'' - m) A'') / (e^(m' - m) l' + e^(m'' - m) l''),   m = max(m', m''),
// from the maximum, exponential sum and weighted sum of either part.  A first kernel leaves those
// of the prefix for all query heads; the kernels over the requests' own tokens (paged_attention.cuh)
// add them where they write a row, or leave theirs for a join of both.
//
// Split.  The query heads of all requests that share a key-value head are its rows; a unit is
// some of them.  The tiles of all units, one unit after the other, are cut into equal ranges for
// a fixed number of CTAs, so a long prefix is spread over the GPU however few the requests are; a
// CTA leaves its part of each unit in a slot of its own (PrefixPieces).
#include "paged_attention.cuh"

namespace la {
namespace {

// fp32: the streaming core of paged_attention.cuh on up to 16 rows.  (bf16: paged_prefix_tc.cu.)
// Bound: the FMAs' latency at 7 warps an SM (244 registers).  33 requests behind 4001 tokens, 16 and 4 heads
// of 64: 40 us with their own tokens, this kernel about 28 of them (19 TFLOP/s; under a profiler 35).
template <typename Core>
__global__ void __launch_bounds__(Core::kThreads, 2)
paged_prefix_kernel(const __grid_constant__ PagedDecodeArgs a) {
    constexpr int D = Core::D, ROWS = Core::ROWS;
    extern __shared__ __align__(128) unsigned char smem[];
    ptx::grid_dependency_wait();
    ptx::release_to_next(a.prefix.ranges + 2);
    ptx::grid_launch_dependents();
    const PrefixPieces &f = a.prefix;
    const int len = min(max(__ldcg(f.len), 0), f.max_tokens);
    const int tiles = prefix_tiles(f);
    if (tiles == 0) return;
    if (blockIdx.x == 0 && threadIdx.x == 0) *f.ranges = f.ctas;
    const long long chunk = prefix_chunk(f, tiles, f.ctas);
    long long w0 = blockIdx.x * chunk;
    const long long w1 = min(w0 + chunk, (long long)f.units * tiles);
    while (w0 < w1) {
        const int unit = range_of(w0, tiles);
        const int tile0 = (int)(w0 - (long long)unit * tiles), tile1 = (int)min((long long)tiles, tile0 + (w1 - w0));
        w0 += tile1 - tile0;
        const int kvh = unit / f.units_per_head, row0 = (unit - kvh * f.units_per_head) * ROWS;
        const int rows = min(ROWS, a.batch * a.group - row0);
        Core::stream(a, smem, 0, kvh, row0, rows, tile0 * kTile, min(len, tile1 * kTile));
        __syncthreads();
        float *slot = f.pieces + (size_t)(blockIdx.x + unit) * ROWS * (D + 2);
        for (int i = threadIdx.x; i < rows * (D / 4); i += Core::kThreads) {
            const int h = i / (D / 4), d = (i % (D / 4)) * 4;
            const Partial p = warps_sum<Core>(smem, h, d);
            *reinterpret_cast<float4 *>(slot + h * D + d) = p.acc;
            if (d == 0) *reinterpret_cast<float2 *>(slot + ROWS * D + 2 * h) = make_float2(p.m, p.sum);
        }
        __syncthreads();  // shared memory is the ring again
    }
}

template <typename Core> cudaError_t launch_prefix(const PagedDecodeArgs &a) {
    constexpr auto kern = paged_prefix_kernel<Core>;
    cudaError_t e = allow_smem<kern>(Core::kSmem);
    if (e == cudaSuccess)
        e = launch_dependent(kern, kPagedCtas, Core::kThreads, Core::kSmem, a.stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D> cudaError_t run(PagedDecodeArgs a, const int32_t *prefix_table, bool bf16) {
    // the split kernel runs beside the prefix's, the cluster kernel's CTAs would wait on their SMs
    if (bf16)
        a.prefix.share = (a.group <= 8 ? cluster_size<Bf16Core<Kv::kBehind, D, 1, false>>(a)
                                       : cluster_size<Bf16Core<Kv::kBehind, D, 2, false>>(a)) == 0;
    PagedDecodeArgs p = a;
    p.block_table = prefix_table;
    cudaError_t e;
    if (bf16) {
        e = paged_prefix_tc(p);
    } else {
        e = a.prefix.unit_rows == 4   ? launch_prefix<F32Core<Kv::kPrefix, D, 4>>(p)
            : a.prefix.unit_rows == 8 ? launch_prefix<F32Core<Kv::kPrefix, D, 8>>(p)
                                      : launch_prefix<F32Core<Kv::kPrefix, D, 16>>(p);
    }
    return e != cudaSuccess ? e : dispatch<Kv::kBehind, D>(a, bf16);
}

}  // namespace

PrefixPieces paged_prefix_pieces(int64_t batch, int64_t num_heads, int64_t num_kv_heads, bool bf16) {
    PrefixPieces f;
    const int64_t rows = batch * (num_heads / num_kv_heads);
    if (bf16) {
        // up to 128 rows: two parts of every other tile each
        const bool shared = rows > 128;
        f.unit_rows = shared ? 256 : 128;
        f.parts = shared ? 1 : 2;
        f.tile = kPrefixTile;
        f.ctas = kPrefixCtas;
        f.stride = shared ? 256 : (int)(rows + 7) / 8 * 8;
    } else {
        f.unit_rows = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
        f.tile = kTile;
        f.ctas = kPagedCtas;
        f.stride = f.unit_rows;
    }
    f.units_per_head = (int)((rows + f.unit_rows - 1) / f.unit_rows);
    f.units = (int)(f.units_per_head * num_kv_heads);
    return f;
}

cudaError_t paged_prefix_decode(const PagedDecodeArgs &a, const int32_t *prefix_table, bool bf16) {
    // No prefix, no kernel in front of those that are behind one, which rely on it.
    if (a.prefix.max_tokens == 0) return paged_decode(a, bf16, !bf16);
    if (a.head_dim == 128) return run<128>(a, prefix_table, bf16);
    if (a.head_dim == 64) return run<64>(a, prefix_table, bf16);
    return cudaErrorNotSupported;
}

}  // namespace la
