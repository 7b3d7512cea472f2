// Per-head RMS norm of queries and keys with the position rotation in the
// same pass, its backward pass, and the variant that writes keys and values
// into the slots of a paged cache.
//
// For a row x of head_dim elements (one token, one head), with w the norm's
// weight and R(p) the rotation of position p on the first rotary_dim elements:
//     n = x r w,  r = (mean(x^2) + eps)^-1/2,   y = R(p) n
// and backward, with g = R(p)^T dy:
//     dw = sum over rows of g x r
//     dx = r (w g - x r mean(w g x r))
// Everything between the load of x and the store of y is fp32; y is rounded
// once.
//
// Memory-bound: a row is read once and written once (backward: two reads, one
// write), so the layout serves the loads and keeps the instructions few.  A lane
// holds two chunks of four elements of a row, placed so that both elements of
// every rotated pair are its own: chunk u and chunk u + rotary_dim / 8 inside the
// rotated part (either layout of the pairs), likewise two chunks behind it.  So
// no element crosses lanes; D / 8 lanes share a row, 32 / (D / 8) rows (a pass) a
// warp instruction.  A warp takes up to U * G passes of one token and one kind
// (query, key or value heads) and issues all their loads first, asynchronously
// into shared memory: 4 KB a warp (backward 8) in flight without registers or block-wide
// barriers, while the token's cosines and sines and the weights arrive.  Those are
// folded into two coefficients an element, y = r (x A + partner(x) B) with
// A = w cos, B = +-w' sin, applied with packed fp32 pairs.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_internal.h"
#include "sm100_ptx.cuh"

namespace la {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 swapped(float2 x) { return make_float2(x.y, x.x); }

// A chunk of four elements as two fp32 pairs, from memory and back.
__device__ __forceinline__ void load_chunk(const __nv_bfloat16 *p, float2 *x) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    x[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    x[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ void load_chunk(const float *p, float2 *x) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = make_float2(v.x, v.y);
    x[1] = make_float2(v.z, v.w);
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16 *p, const float2 *x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0].x, x[0].y);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[1].x, x[1].y);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void store_chunk(float *p, const float2 *x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 16 : 0;  // otherwise zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Waits until group g of N has arrived.
template <int N> __device__ __forceinline__ void cp_wait_group(int g) {
    if (g == 0) cp_wait<N - 1>();
    else if (N > 1 && g == 1) cp_wait<(N > 1 ? N - 2 : 0)>();
    else if (N > 2 && g == 2) cp_wait<(N > 2 ? N - 3 : 0)>();
    else cp_wait<0>();
}

// A lane's coefficients of its token's rotation, y = x ca + partner(x) cb for its
// four pairs (two of each chunk; ea, eb: the chunks' first elements); the
// transposed rotation (sign -1) has the sines negated.
template <bool INTER>
__device__ __forceinline__ void load_rotation(const NormRopeArgs &a, int token, int ea, int eb,
                                              float sign, float2 (&ca)[4], float2 (&cb)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) ca[i] = twice(1.f), cb[i] = twice(0.f);
    if (ea >= a.rotary_dim) return;
    // positions are checked nowhere on the host: clamped, so every read stays
    // inside the table
    const int pos = min(max(__ldcg(a.positions + token), 0), a.rotary_rows - 1);
    const float *row = a.rotary + (size_t)pos * a.rotary_dim;
    const int half = a.rotary_dim >> 1;
    if (INTER) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int i = (c ? eb : ea) >> 1;
            const float2 cs = __ldg(reinterpret_cast<const float2 *>(row + i));
            const float2 sn = __ldg(reinterpret_cast<const float2 *>(row + half + i));
            ca[2 * c] = twice(cs.x);
            ca[2 * c + 1] = twice(cs.y);
            cb[2 * c] = make_float2(-sign * sn.x, sign * sn.x);
            cb[2 * c + 1] = make_float2(-sign * sn.y, sign * sn.y);
        }
    } else {  // chunk b holds the partners of chunk a
        const float4 cs = __ldg(reinterpret_cast<const float4 *>(row + ea));
        const float4 sn = __ldg(reinterpret_cast<const float4 *>(row + half + ea));
        ca[0] = ca[2] = make_float2(cs.x, cs.y);
        ca[1] = ca[3] = make_float2(cs.z, cs.w);
        cb[2] = make_float2(sign * sn.x, sign * sn.y);
        cb[3] = make_float2(sign * sn.z, sign * sn.w);
        cb[0] = make_float2(-cb[2].x, -cb[2].y);
        cb[1] = make_float2(-cb[3].x, -cb[3].y);
    }
}

// The rotated partner of pair i.
template <bool INTER> __device__ __forceinline__ float2 partner(const float2 (&x)[4], int i) {
    return INTER ? swapped(x[i]) : x[i ^ 2];
}

template <int L> __device__ __forceinline__ float row_sum(float s) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <typename T, int D, int U, int G, bool BACK, bool INTER>
__global__ void __launch_bounds__(32 * kWarps, BACK ? 5 : 8)
qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    constexpr int L = D / 8;            // lanes per row
    constexpr int R = 32 / L;           // rows per pass
    constexpr int N = U * G;            // passes of an item
    constexpr int kRows = R * N;
    constexpr int kArrays = BACK ? 2 : 1;
    constexpr int kCopies = 8 * (int)sizeof(T) / 16;  // 16-byte copies a lane makes of a pass
    __shared__ __align__(16) T stage[kWarps][kArrays][N][R * D];

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L, u0 = lane % L;
    // the lane's chunks: a rotated pair of chunks, or two behind the rotated part
    const int pairs = a.rotary_dim / 8;  // lanes of the rotated part
    const bool rotated = u0 < pairs;     // elsewhere no partner's infinity or NaN reaches an element
    const int ea = 4 * (rotated ? u0 : pairs + u0);
    const int eb = ea + (rotated ? a.rotary_dim / 2 : (D - a.rotary_dim) / 2);

    const int nq = (a.set[0].heads + kRows - 1) / kRows;
    const int nk = (a.set[1].heads + kRows - 1) / kRows;
    const int nv = (a.set[2].heads + kRows - 1) / kRows;
    const int per = nq + nk + nv;
    const unsigned items = (unsigned)a.num_tokens * per;  // the caller bounds the rows by 2^31

    // This lane's columns of the weights' gradients: fp32 sums, a warp's rows one after the
    // other, then the rows of a pass, the warps and the blocks (1.4e-7 off in 1021 fp32 tokens,
    // where a 64-bit sum rounded at the end is 0.8e-7 off).
    float2 dw[2][4];
    if (BACK) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[0][i] = dw[1][i] = twice(0.f);
    }

    for (unsigned item = blockIdx.x * kWarps + warp; item < items; item += gridDim.x * kWarps) {
        const int token = (int)(item / per), c = (int)item - token * per;
        const int kind = c < nq ? 0 : c < nq + nk ? 1 : 2;
        const NormRopeRows &s = a.set[kind];
        const int first = (kind == 0 ? c : kind == 1 ? c - nq : c - nq - nk) * kRows;
        const int left = s.heads - first;  // rows of this item (and of later ones)

        // A pass is R * D contiguous elements, 16 bytes of it each copy of a lane.
        // Items that have all their rows (most do) need no checks.
        const bool full = left >= kRows;
        const char *xp = static_cast<const char *>(s.x) + (size_t)token * s.x_stride +
                         (size_t)first * D * sizeof(T) + lane * 16;
        const char *gp = BACK ? static_cast<const char *>(s.dy) + (size_t)token * s.dy_stride +
                                    (size_t)first * D * sizeof(T) + lane * 16
                              : nullptr;
        const uint32_t to = ptx::smem_u32(&stage[warp][0][0][0]) + lane * 16;
        constexpr uint32_t kPass = R * D * sizeof(T);
        __syncwarp();  // the previous item's rows have been read by all lanes
        if (full) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int j = 0; j < kCopies; ++j) {
                    const uint32_t off = i * kPass + j * 512;
                    cp_async16(to + off, xp + off, true);
                    if (BACK) cp_async16(to + N * kPass + off, gp + off, true);
                }
                if (i % U == U - 1) cp_commit();
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (i * R < left) {  // the same in the whole warp
#pragma unroll
                    for (int j = 0; j < kCopies; ++j) {
                        const bool in = i * R + (lane * 16 + j * 512) / (D * (int)sizeof(T)) < left;
                        const uint32_t off = i * kPass + j * 512;
                        cp_async16(to + off, in ? xp + off : xp - lane * 16, in);
                        if (BACK) cp_async16(to + N * kPass + off, in ? gp + off : gp - lane * 16, in);
                    }
                }
                if (i % U == U - 1) cp_commit();
            }
        }

        // destination of the token's rows: its row of the output, or its slot
        // of the cache (a slot outside the pool is skipped)
        T *out = static_cast<T *>(s.out);
        size_t head = D;
        if (s.cache) {
            const int slot = __ldcg(a.slots + token);
            if (slot < 0 || slot >= a.num_slots) {
                cp_wait<0>();  // the stage is filled anew
                continue;
            }
            const int page = slot / a.page_size;
            out += (size_t)page * (s.out_stride / sizeof(T)) +
                   (size_t)(slot - page * a.page_size) * D;
            head = (size_t)a.page_size * D;
        } else {
            out += (size_t)token * (s.out_stride / sizeof(T));
        }
        out += (first + sub) * head;

        float2 ca[4], cb[4], w[4], item_dw[4];
        const bool norm = s.weight != nullptr;
        if (kind != 2) {
            load_rotation<INTER>(a, token, ea, eb, BACK ? -1.f : 1.f, ca, cb);
            if (norm) {
                load_chunk(s.weight + ea, w);
                load_chunk(s.weight + eb, w + 2);
                if (!BACK) {  // forward: the weights go into the coefficients
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ca[i] = ptx::f2_mul(ca[i], w[i]);
                        cb[i] = ptx::f2_mul(cb[i], partner<INTER>(w, i));
                    }
                }
            }
        }
        if (BACK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) item_dw[i] = twice(0.f);
        }
        T *oa = out + ea, *ob = out + eb;
        const size_t step = R * head;
        float *f32 = s.out_f32 ? static_cast<float *>(s.out) +
                                     ((size_t)token * s.heads + first + sub) * D
                               : nullptr;  // unrounded rows (the queries of a fused step)
        auto rows = [&](auto all) {  // all: the item has all its rows
            constexpr bool FULL = decltype(all)::value;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (!FULL && g * U * R >= left) break;
                cp_wait_group<G>(g);
                __syncwarp();
#pragma unroll
                for (int u = 0; u < U; ++u, oa += step, ob += step) {
                    const int pass = g * U + u;
                    if (!FULL && U > 1 && pass * R >= left) break;
                    const bool in = FULL || pass * R + sub < left;
                    const T *row = &stage[warp][0][pass][sub * D];
                    if (!BACK && kind == 2) {  // values: copied, bit for bit
                        using Chunk = std::conditional_t<sizeof(T) == 2, uint2, uint4>;
                        if (in) {
                            *reinterpret_cast<Chunk *>(oa) = *reinterpret_cast<const Chunk *>(row + ea);
                            *reinterpret_cast<Chunk *>(ob) = *reinterpret_cast<const Chunk *>(row + eb);
                        }
                        continue;
                    }
                    float2 x[4];
                    load_chunk(row + ea, x);
                    load_chunk(row + eb, x + 2);
                    float r = 1.f;
                    if (norm) {
                        float2 ss = ptx::f2_mul(x[0], x[0]);
#pragma unroll
                        for (int i = 1; i < 4; ++i) ss = ptx::f2_fma(x[i], x[i], ss);
                        r = rsqrtf(row_sum<L>(ss.x + ss.y) * (1.f / D) + a.eps);
                        if (!in) r = 0.f;  // a row past the last head stays zero also where eps is 0
                    }
                    const float2 rr = twice(r);
                    if (BACK) {
                        const T *grow = &stage[warp][kArrays - 1][pass][sub * D];
                        float2 dy[4], g4[4];
                        load_chunk(grow + ea, dy);
                        load_chunk(grow + eb, dy + 2);
                        float2 dot = twice(0.f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            g4[i] = ptx::f2_mul(dy[i], ca[i]);
                            if (rotated) g4[i] = ptx::f2_fma(partner<INTER>(dy, i), cb[i], g4[i]);
                            if (norm) {
                                x[i] = ptx::f2_mul(x[i], rr);
                                const float2 p = ptx::f2_mul(g4[i], x[i]);
                                item_dw[i] = ptx::f2_add(item_dw[i], p);
                                dot = ptx::f2_fma(w[i], p, dot);
                                g4[i] = ptx::f2_mul(g4[i], w[i]);
                            }
                        }
                        if (norm) {
                            const float2 m = twice(row_sum<L>(dot.x + dot.y) * (-1.f / D));
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                g4[i] = ptx::f2_mul(rr, ptx::f2_fma(x[i], m, g4[i]));
                        }
                        if (in) store_chunk(oa, g4), store_chunk(ob, g4 + 2);
                    } else {
                        float2 y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            y[i] = ptx::f2_mul(x[i], ca[i]);
                            if (rotated) y[i] = ptx::f2_fma(partner<INTER>(x, i), cb[i], y[i]);
                            if (norm) y[i] = ptx::f2_mul(y[i], rr);
                        }
                        if (in && f32) {
                            store_chunk(f32 + pass * R * D + ea, y);
                            store_chunk(f32 + pass * R * D + eb, y + 2);
                        } else if (in) {
                            store_chunk(oa, y);
                            store_chunk(ob, y + 2);
                        }
                    }
                }
            }
        };
        if (full) rows(std::true_type()); else rows(std::false_type());
        cp_wait<0>();  // also the groups of rows past the last head: none in flight
        if (BACK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kind == 0) dw[0][i] = ptx::f2_add(dw[0][i], item_dw[i]);
                else dw[1][i] = ptx::f2_add(dw[1][i], item_dw[i]);
            }
        }
    }

    if (BACK && a.set[0].weight) {
        // block's sums in a fixed order: rows of a warp, then the warps
        __shared__ float red[kWarps][2][D];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float t = i & 1 ? dw[k][i / 2].y : dw[k][i / 2].x;
#pragma unroll
                for (int o = 16; o >= L; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                if (sub == 0) red[warp][k][(i < 4 ? ea : eb) + (i & 3)] = t;
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps) {
            float t = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) t += (&red[v][0][0])[i];
            a.partial[(size_t)blockIdx.x * 2 * D + i] = t;
        }
    }
}

// dw[c] = sum over blocks of partial[block][c], in a fixed order: 8 columns (one
// 32-byte sector of a partial result) a block, 128 slices of the blocks' axis.
constexpr int kSumCols = 8, kSumSlices = 128;
__global__ void __launch_bounds__(kSumCols *kSumSlices)
norm_weight_sum_kernel(const float *partial, int blocks, int D, float *dwq, float *dwk) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float red[kSumSlices][kSumCols + 1];
    const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
    const int c = blockIdx.x * kSumCols + x;
    float t = 0.f;
#pragma unroll 8
    for (int b = y; b < blocks; b += kSumSlices) t += __ldcg(partial + (size_t)b * 2 * D + c);
    red[y][x] = t;
    __syncthreads();
    const int lane = threadIdx.x & 31, col = threadIdx.x >> 5;
    if (col >= kSumCols) return;
    t = 0.f;
#pragma unroll
    for (int i = 0; i < kSumSlices; i += 32) t += red[i + lane][col];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) {
        const int at = blockIdx.x * kSumCols + col;
        if (at < D) dwq[at] = t; else dwk[at - D] = t;
    }
}

template <typename T, int D, int U, int G, bool BACK>
cudaError_t launch_u(const NormRopeArgs &a) {
    constexpr int kRows = 32 / (D / 8) * U * G;
    long per = 0;
    for (const NormRopeRows &s : a.set) per += (s.heads + kRows - 1) / kRows;
    long grid = (a.num_tokens * per + kWarps - 1) / kWarps;
    // the backward pass keeps its weight sums in registers over a fixed
    // number of blocks, one partial result each
    const long most = BACK ? kNormBackwardBlocks : 0x7fffffffL;
    if (grid > most) grid = most;
    cudaError_t e = launch_dependent(a.interleaved ? qk_norm_rope_kernel<T, D, U, G, BACK, true>
                                                   : qk_norm_rope_kernel<T, D, U, G, BACK, false>,
                                     (unsigned)grid, 32 * kWarps, 0, a.stream, a);
    if (e == cudaSuccess && BACK && a.set[0].weight)
        e = launch_dependent(norm_weight_sum_kernel, (a.dk_weight ? 2 : 1) * D / kSumCols,
                             kSumCols * kSumSlices, 0, a.stream,
                             static_cast<const float *>(a.partial), (int)grid, D, a.dq_weight,
                             a.dk_weight);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D, bool BACK>
cudaError_t launch(const NormRopeArgs &a) {
    // Few rows: one pass a warp spreads them over many SMs.  Many: the token's cosines,
    // sines and weights are loaded once for up to U * G passes.  Measured with 64 + 8 heads of 128,
    // single passes / long items, us, at half the limit, at it, twice and four times it:
    // forward bf16 2.1 / 3.0, 2.5 / 3.0, 2.8 / 3.3, 4.5 / 3.6; fp32 2.2 / 2.4, 2.5 / 2.5, 3.0 / 2.8,
    // 4.6 / 3.6; gradients bf16 4.8 / 5.2, 6.0 / 5.3, 7.3 / 6.3, 9.0 / 7.4; fp32 4.8 / 4.3, 6.1 / 5.2,
    // 7.4 / 6.2, 9.3 / 8.2.  64 wide and with 12 + 4 heads they cross between the same points: the
    // limit is within half a microsecond of each type's own, the gradients' within one.  8192
    // tokens of 64 + 64 bf16 heads, forward: G = 1, 2, 3, 4 take 96, 81, 83, 83 us
    // (a plain copy of the bytes 85; of 64 + 8 heads into the cache 60, 54, 60, 64);
    // gradients, where the sums over a block's rows come on top: 185, 144, 134, 131.
    constexpr int R = 32 / (D / 8);
    constexpr int U = 8 / (int)sizeof(T) / (BACK ? 2 : 1);
    const long rows = (long)a.num_tokens * (a.set[0].heads + a.set[1].heads + a.set[2].heads);
    if (rows <= 152L * 16 * R) return launch_u<T, D, 1, 1, BACK>(a);
    return launch_u<T, D, U, BACK ? 4 : 2, BACK>(a);
}

template <typename T>
cudaError_t dispatch(const NormRopeArgs &a, bool back) {
    if (a.head_dim == 128) return back ? launch<T, 128, true>(a) : launch<T, 128, false>(a);
    if (a.head_dim == 64) return back ? launch<T, 64, true>(a) : launch<T, 64, false>(a);
    return cudaErrorNotSupported;
}

}  // namespace

cudaError_t qk_norm_rope(const NormRopeArgs &a, bool bf16) {
    return bf16 ? dispatch<__nv_bfloat16>(a, false) : dispatch<float>(a, false);
}
cudaError_t qk_norm_rope_backward(const NormRopeArgs &a, bool bf16) {
    return bf16 ? dispatch<__nv_bfloat16>(a, true) : dispatch<float>(a, true);
}

}  // namespace la
