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
// write), so the layout serves the loads.  A row is held by L = 8 to 32 lanes
// of 16 bytes, 32 / L rows (a pass) a warp instruction.  A warp takes up to
// U * G passes of one token and one kind (query, key or value heads) and
// issues all their loads first, asynchronously into shared memory where each lane
// reads back its own 16 bytes: 8 KB a warp in flight without registers or
// barriers, while the token's cosines and sines and the weights arrive.  Those are
// folded into two coefficients an element, y = r (x A + partner(x) B) with
// A = w cos, B = +-w' sin, applied with packed fp32 pairs; the partner's element
// crosses lanes in its stored type (half the shuffles of an fp32 one in bf16).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_internal.h"
#include "sm100_ptx.cuh"

namespace la {
namespace {

constexpr int kWarps = 4;

// 16 stored bytes as fp32 pairs.
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int P = 4;  // pairs
    static __device__ __forceinline__ void unpack(const uint4 &v, float2 (&x)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&x)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[i].x, x[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Vec<float> {
    static constexpr int P = 2;
    static __device__ __forceinline__ void unpack(const uint4 &v, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&x)[2]) {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                          __float_as_uint(x[1].y));
    }
};

template <int P> __device__ __forceinline__ void load_pairs(const float *p, float2 (&x)[P]) {
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p + 2 * i));
        x[i] = make_float2(v.x, v.y);
        x[i + 1] = make_float2(v.z, v.w);
    }
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
// Waits until group g of n has arrived.
template <int N> __device__ __forceinline__ void cp_wait_group(int g) {
    if (g == 0) cp_wait<N - 1>();
    else if (N > 1 && g == 1) cp_wait<(N > 1 ? N - 2 : 0)>();
    else if (N > 2 && g == 2) cp_wait<(N > 2 ? N - 3 : 0)>();
    else cp_wait<0>();
}
__device__ __forceinline__ float2 swapped(float2 x) { return make_float2(x.y, x.x); }
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// The rotated partner of every element of a lane's 16 bytes: in the lane that
// holds the row's other half, or the other element of a pair; zero past
// rotary_dim (where its coefficient is zero too).
template <typename T>
__device__ __forceinline__ void partner(const uint4 &v, const float2 (&x)[Vec<T>::P],
                                        bool interleaved, bool rotated, int src,
                                        float2 (&y)[Vec<T>::P]) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < Vec<T>::P; ++i) y[i] = rotated ? swapped(x[i]) : twice(0.f);
    } else {
        uint4 w;
        w.x = __shfl_sync(0xffffffffu, v.x, src);
        w.y = __shfl_sync(0xffffffffu, v.y, src);
        w.z = __shfl_sync(0xffffffffu, v.z, src);
        w.w = __shfl_sync(0xffffffffu, v.w, src);
        Vec<T>::unpack(rotated ? w : make_uint4(0, 0, 0, 0), y);
    }
}

// A lane's coefficients of its token's rotation, y = x cs + partner(x) sn; the
// transposed rotation (sign -1) has sn negated.
template <int P>
__device__ __forceinline__ void load_rotation(const NormRopeArgs &a, int token, int j0, float sign,
                                              float2 (&cs)[P], float2 (&sn)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) cs[i] = twice(1.f), sn[i] = twice(0.f);
    if (j0 >= a.rotary_dim) return;
    // positions are checked nowhere on the host: clamped, so every read stays
    // inside the table
    const int pos = min(max(__ldg(a.positions + token), 0), a.rotary_rows - 1);
    const float *row = a.rotary + (size_t)pos * a.rotary_dim;
    const int half = a.rotary_dim >> 1;
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float c = __ldg(row + (j0 >> 1) + i), s = sign * __ldg(row + half + (j0 >> 1) + i);
            cs[i] = twice(c);
            sn[i] = make_float2(-s, s);
        }
    } else {
        const bool low = j0 < half;
        const float *c = row + (low ? j0 : j0 - half);
        load_pairs<P>(c, cs);
        load_pairs<P>(c + half, sn);
        const float2 sg = twice(low ? -sign : sign);
#pragma unroll
        for (int i = 0; i < P; ++i) sn[i] = ptx::f2_mul(sn[i], sg);
    }
}

template <int L> __device__ __forceinline__ float row_sum(float s) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <typename T, int D, int U, int G, bool BACK>
__global__ void __launch_bounds__(32 * kWarps)
qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    using V = Vec<T>;
    constexpr int P = V::P;                 // fp32 pairs per lane
    constexpr int L = D / (2 * P);          // lanes per row
    constexpr int R = 32 / L;               // rows per pass
    constexpr int kRows = R * U * G;        // rows of an item
    constexpr size_t kRowBytes = D * sizeof(T);
    constexpr int kArrays = BACK ? 2 : 1;
    __shared__ uint4 stage[kWarps][kArrays][U * G][32];

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L, j0 = (lane % L) * 2 * P;
    const int half = a.rotary_dim >> 1;
    const bool rotated = j0 < a.rotary_dim;
    // first element of the rotated partners, and the lane that holds it
    const int jp = a.interleaved || !rotated ? j0 : j0 < half ? j0 + half : j0 - half;
    const int src = lane + (jp - j0) / (2 * P);

    const int nq = (a.set[0].heads + kRows - 1) / kRows;
    const int nk = (a.set[1].heads + kRows - 1) / kRows;
    const int nv = (a.set[2].heads + kRows - 1) / kRows;
    const int per = nq + nk + nv;
    const int items = a.num_tokens * per;  // fits: the caller bounds the number of rows

    float2 dw[2][P];  // this lane's columns of the weights' gradients
    if (BACK) {
#pragma unroll
        for (int i = 0; i < P; ++i) dw[0][i] = dw[1][i] = twice(0.f);
    }

    for (int item = blockIdx.x * kWarps + warp; item < items; item += gridDim.x * kWarps) {
        const int token = item / per, c = item - token * per;
        const int kind = c < nq ? 0 : c < nq + nk ? 1 : 2;
        const NormRopeRows &s = a.set[kind];
        const int first = (kind == 0 ? c : kind == 1 ? c - nq : c - nq - nk) * kRows;
        const int end = s.heads;
        const int row0 = first + sub;

        const char *xp = static_cast<const char *>(s.x) + (size_t)token * s.x_stride + j0 * sizeof(T);
        const char *gp = BACK ? static_cast<const char *>(s.dy) + (size_t)token * s.dy_stride +
                                    j0 * sizeof(T)
                              : nullptr;
#pragma unroll
        for (int i = 0; i < U * G; ++i) {
            if (first + i * R < end) {  // the same in the whole warp
                const int r = row0 + i * R;
                const bool in = r < end;
                cp_async16(ptx::smem_u32(&stage[warp][0][i][lane]), xp + (in ? r : 0) * kRowBytes, in);
                if (BACK)
                    cp_async16(ptx::smem_u32(&stage[warp][kArrays - 1][i][lane]),
                               gp + (in ? r : 0) * kRowBytes, in);
            }
            if (i % U == U - 1) cp_commit();
        }

        // destination of the token's rows: its row of the output, or its slot
        // of the cache (a slot outside the pool is skipped)
        char *out = static_cast<char *>(s.out);
        size_t head_bytes = kRowBytes;
        if (s.cache) {
            const int slot = __ldg(a.slots + token);
            if (slot < 0 || slot >= a.num_slots) {
                cp_wait<0>();  // the stage is filled anew
                continue;
            }
            const int page = slot / a.page_size;
            out += (size_t)page * s.out_stride + (size_t)(slot - page * a.page_size) * kRowBytes;
            head_bytes *= a.page_size;
        } else {
            out += (size_t)token * s.out_stride;
        }
        out += j0 * sizeof(T);

        float2 ca[P], cb[P], w[P];
        const bool norm = s.weight != nullptr;
        if (kind != 2) {
            load_rotation<P>(a, token, j0, BACK ? -1.f : 1.f, ca, cb);
            if (norm) {
                load_pairs<P>(s.weight + j0, w);
                if (!BACK) {  // forward: the weights go into the coefficients
                    float2 wp[P];
                    load_pairs<P>(s.weight + jp, wp);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        ca[i] = ptx::f2_mul(ca[i], w[i]);
                        cb[i] = ptx::f2_mul(cb[i], a.interleaved ? swapped(wp[i]) : wp[i]);
                    }
                }
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (first + g * U * R >= end) break;
            cp_wait_group<G>(g);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = row0 + (g * U + u) * R;
                if (U > 1 && row - sub >= end) break;
                const bool in = row < end;
                const uint4 xv = stage[warp][0][g * U + u][lane];
                if (!BACK && kind == 2) {  // values: copied
                    if (in) *reinterpret_cast<uint4 *>(out + row * head_bytes) = xv;
                    continue;
                }
                float2 x[P], y[P];
                V::unpack(xv, x);
                float r = 1.f;
                if (norm) {
                    float2 ss = twice(0.f);
#pragma unroll
                    for (int i = 0; i < P; ++i) ss = ptx::f2_fma(x[i], x[i], ss);
                    // a row past the last head stays zero also where eps is 0
                    r = row_sum<L>(ss.x + ss.y) * (1.f / D) + a.eps;
                    r = in ? rsqrtf(r) : 0.f;
                }
                const float2 rr = twice(r);
                if (BACK) {
                    const uint4 gv = stage[warp][kArrays - 1][g * U + u][lane];
                    float2 dy[P];
                    V::unpack(gv, dy);
                    partner<T>(gv, dy, a.interleaved, rotated, src, y);
                    float2 dot = twice(0.f);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        dy[i] = ptx::f2_fma(dy[i], ca[i], ptx::f2_mul(y[i], cb[i]));
                        if (norm) {
                            x[i] = ptx::f2_mul(x[i], rr);
                            const float2 p = ptx::f2_mul(dy[i], x[i]);
                            if (kind == 0) dw[0][i] = ptx::f2_add(dw[0][i], p);
                            else dw[1][i] = ptx::f2_add(dw[1][i], p);
                            dot = ptx::f2_fma(w[i], p, dot);
                            dy[i] = ptx::f2_mul(dy[i], w[i]);
                        }
                    }
                    if (norm) {
                        const float2 m = twice(row_sum<L>(dot.x + dot.y) * (-1.f / D));
#pragma unroll
                        for (int i = 0; i < P; ++i)
                            dy[i] = ptx::f2_mul(rr, ptx::f2_fma(x[i], m, dy[i]));
                    }
                    if (in) *reinterpret_cast<uint4 *>(out + row * head_bytes) = V::pack(dy);
                } else {
                    partner<T>(xv, x, a.interleaved, rotated, src, y);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        y[i] = ptx::f2_fma(x[i], ca[i], ptx::f2_mul(y[i], cb[i]));
                        if (norm) y[i] = ptx::f2_mul(y[i], rr);
                    }
                    if (in && s.out_f32) {  // unrounded rows (the queries of a fused step)
                        float *o = static_cast<float *>(s.out) +
                                   ((size_t)token * s.heads + row) * D + j0;
#pragma unroll
                        for (int i = 0; i < P; i += 2)
                            *reinterpret_cast<float4 *>(o + 2 * i) =
                                make_float4(y[i].x, y[i].y, y[i + 1].x, y[i + 1].y);
                    } else if (in) {
                        *reinterpret_cast<uint4 *>(out + row * head_bytes) = V::pack(y);
                    }
                }
            }
        }
        cp_wait<0>();  // also the groups of rows past the last head: none in flight
    }

    if (BACK && a.set[0].weight) {
        // block's sums in a fixed order: rows of a warp, then the warps
        __shared__ float red[kWarps][2][D];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
                float t = i & 1 ? dw[k][i / 2].y : dw[k][i / 2].x;
#pragma unroll
                for (int o = 16; o >= L; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                if (sub == 0) red[warp][k][j0 + i] = t;
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
norm_weight_sum_kernel(const float *__restrict__ partial, int blocks, int D, float *dwq, float *dwk) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float red[kSumSlices][kSumCols + 1];
    const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
    const int c = blockIdx.x * kSumCols + x;
    float t = 0.f;
#pragma unroll 8
    for (int b = y; b < blocks; b += kSumSlices) t += partial[(size_t)b * 2 * D + c];
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
    constexpr int kRows = 32 / (D / (2 * Vec<T>::P)) * U * G;
    long per = 0;
    for (const NormRopeRows &s : a.set) per += (s.heads + kRows - 1) / kRows;
    long grid = (a.num_tokens * per + kWarps - 1) / kWarps;
    // the backward pass keeps its weight sums in registers over a fixed
    // number of blocks, one partial result each
    const long most = BACK ? kNormBackwardBlocks : 0x7fffffffL;
    if (grid > most) grid = most;
    cudaError_t e = launch_dependent(qk_norm_rope_kernel<T, D, U, G, BACK>, (unsigned)grid,
                                     32 * kWarps, 0, a.stream, a);
    if (e == cudaSuccess && BACK && a.set[0].weight)
        e = launch_dependent(norm_weight_sum_kernel, (a.dk_weight ? 2 : 1) * D / kSumCols,
                             kSumCols * kSumSlices, 0, a.stream,
                             static_cast<const float *>(a.partial), (int)grid, D, a.dq_weight,
                             a.dk_weight);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D, bool BACK>
cudaError_t launch(const NormRopeArgs &a) {
    // Few rows: one pass a warp spreads them over many SMs.  Many: the token's
    // cosines, sines and weights are loaded once for up to U * G passes.
    constexpr int kRows = 32 / (D / (2 * Vec<T>::P));
    constexpr int U = BACK ? 2 : 4;
    const long rows = (long)a.num_tokens * (a.set[0].heads + a.set[1].heads + a.set[2].heads);
    if (rows <= 152L * 16 * kRows) return launch_u<T, D, 1, 1, BACK>(a);
    return launch_u<T, D, U, 4, BACK>(a);
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
