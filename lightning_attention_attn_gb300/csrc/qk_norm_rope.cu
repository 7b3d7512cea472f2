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
// write), so the layout serves the loads.  A row is held by L = 16 B-vectors
// lanes (8 to 32), 32 / L rows a warp instruction; a warp takes U such passes
// of one token and one kind (query, key or value heads), so the token's
// cosines and sines and the weights stay in registers for all its rows, and
// U 16-byte loads a lane are in flight at once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_internal.h"

namespace la {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4 &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
}

// One lane's coefficients of its token's rotation: y[e] = n[e] cs[e] +
// partner(n)[e] sn[e], the sign of the partner's term inside sn; the identity
// past rotary_dim.  The transposed rotation has sn negated.
template <int E>
__device__ __forceinline__ void load_rotation(const NormRopeArgs &a, int token, int j0, float sign,
                                              float (&cs)[E], float (&sn)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) cs[e] = 1.f, sn[e] = 0.f;
    if (j0 >= a.rotary_dim) return;
    // positions are checked nowhere on the host: clamped, so every read stays
    // inside the table
    const int pos = min(max(__ldg(a.positions + token), 0), a.rotary_rows - 1);
    const float *row = a.rotary + (size_t)pos * a.rotary_dim;
    const int half = a.rotary_dim >> 1;
    if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const int i = (j0 + e) >> 1;
            const float c = __ldg(row + i), s = sign * __ldg(row + half + i);
            cs[e] = cs[e + 1] = c;
            sn[e] = -s;
            sn[e + 1] = s;
        }
    } else {
        const bool low = j0 < half;
        const float *c = row + (low ? j0 : j0 - half);
        const float sg = low ? -sign : sign;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 cv = __ldg(reinterpret_cast<const float4 *>(c + e));
            const float4 sv = __ldg(reinterpret_cast<const float4 *>(c + half + e));
            cs[e] = cv.x, cs[e + 1] = cv.y, cs[e + 2] = cv.z, cs[e + 3] = cv.w;
            sn[e] = sg * sv.x, sn[e + 1] = sg * sv.y, sn[e + 2] = sg * sv.z,
            sn[e + 3] = sg * sv.w;
        }
    }
}

// x <- rotated x; `src` is the lane that holds the other half's elements.
template <int E>
__device__ __forceinline__ void rotate(float (&x)[E], const float (&cs)[E], const float (&sn)[E],
                                       bool interleaved, int src) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float u = x[e], v = x[e + 1];
            x[e] = fmaf(u, cs[e], v * sn[e]);
            x[e + 1] = fmaf(v, cs[e + 1], u * sn[e + 1]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float p = __shfl_sync(0xffffffffu, x[e], src);
            x[e] = fmaf(x[e], cs[e], p * sn[e]);
        }
    }
}

template <int L> __device__ __forceinline__ float row_sum(float s) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <typename T, int D, int U, bool BACK>
__global__ void __launch_bounds__(32 * kWarps)
qk_norm_rope_kernel(const NormRopeArgs a) {
    constexpr int E = 16 / (int)sizeof(T);  // elements per lane
    constexpr int L = D / E;                // lanes per row
    constexpr int R = 32 / L;               // rows per pass
    constexpr int kRows = R * U;            // rows per work item

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L, col = lane % L, j0 = col * E;
    const int half = a.rotary_dim >> 1;
    // lane of the other half of a rotated pair (itself past rotary_dim)
    const int src = a.interleaved || j0 >= a.rotary_dim ? lane
                    : j0 < half ? lane + half / E : lane - half / E;

    const int nq = (a.set[0].heads + kRows - 1) / kRows, nk = (a.set[1].heads + kRows - 1) / kRows;
    const int nv = (a.set[2].heads + kRows - 1) / kRows;
    const int per = nq + nk + nv;
    const int items = a.num_tokens * per;  // fits: the caller bounds the number of rows

    float dw[2][E];  // this lane's columns of the weights' gradients
    if (BACK) {
#pragma unroll
        for (int e = 0; e < E; ++e) dw[0][e] = dw[1][e] = 0.f;
    }

    for (int item = blockIdx.x * kWarps + warp; item < items; item += gridDim.x * kWarps) {
        const int token = item / per, c = item - token * per;
        const int kind = c < nq ? 0 : c < nq + nk ? 1 : 2;
        const NormRopeRows s = a.set[kind];
        const int row0 = (kind == 0 ? c : kind == 1 ? c - nq : c - nq - nk) * kRows + sub;

        // every load of the item first, so that they overlap
        uint4 xv[U], gv[U];
        const char *xp = static_cast<const char *>(s.x) + (size_t)token * s.x_stride + (size_t)j0 * sizeof(T);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xv[u] = make_uint4(0, 0, 0, 0);
            if (row0 + u * R < s.heads)
                xv[u] = *reinterpret_cast<const uint4 *>(xp + (size_t)(row0 + u * R) * D * sizeof(T));
        }
        if (BACK) {
            const char *gp = static_cast<const char *>(s.dy) + (size_t)token * s.dy_stride +
                             (size_t)j0 * sizeof(T);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                gv[u] = make_uint4(0, 0, 0, 0);
                if (row0 + u * R < s.heads)
                    gv[u] = *reinterpret_cast<const uint4 *>(gp + (size_t)(row0 + u * R) * D * sizeof(T));
            }
        }
        // destination of the token's rows: its row of the output, or its slot
        // of the cache (a slot outside the pool is skipped)
        char *out = static_cast<char *>(s.out);
        size_t head_bytes = D * sizeof(T);
        if (s.cache) {
            const int slot = __ldg(a.slots + token);
            if (slot < 0 || slot >= a.num_slots) continue;
            const int page = slot / a.page_size;
            out += (size_t)page * s.out_stride + (size_t)(slot - page * a.page_size) * D * sizeof(T);
            head_bytes *= a.page_size;
        } else {
            out += (size_t)token * s.out_stride;
        }
        out += (size_t)j0 * sizeof(T);

        if (!BACK && kind == 2) {  // values: copied
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row0 + u * R < s.heads)
                    *reinterpret_cast<uint4 *>(out + (size_t)(row0 + u * R) * head_bytes) = xv[u];
            continue;
        }

        float cs[E], sn[E], w[E];
        load_rotation<E>(a, token, j0, BACK ? -1.f : 1.f, cs, sn);
        if (s.weight) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 t = __ldg(reinterpret_cast<const float4 *>(s.weight + j0 + e));
                w[e] = t.x, w[e + 1] = t.y, w[e + 2] = t.z, w[e + 3] = t.w;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E];
            unpack(xv[u], x);
            float r = 0.f;
            if (s.weight) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
                ss = row_sum<L>(ss);
                // a row past the last head stays zero also where eps is 0
                r = row0 + u * R < s.heads ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;
            }
            if (BACK) {
                float g[E];
                unpack(gv[u], g);
                rotate<E>(g, cs, sn, a.interleaved, src);
                if (s.weight) {
                    float dot = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        x[e] *= r;
                        const float p = g[e] * x[e];
                        if (kind == 0) dw[0][e] += p; else dw[1][e] += p;
                        g[e] *= w[e];
                        dot = fmaf(w[e], p, dot);
                    }
                    dot = row_sum<L>(dot) * (1.f / D);
#pragma unroll
                    for (int e = 0; e < E; ++e) g[e] = r * fmaf(-x[e], dot, g[e]);
                }
                if (row0 + u * R < s.heads)
                    *reinterpret_cast<uint4 *>(out + (size_t)(row0 + u * R) * head_bytes) = pack(g);
            } else {
                if (s.weight) {
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] *= r * w[e];
                }
                rotate<E>(x, cs, sn, a.interleaved, src);
                if (row0 + u * R < s.heads) {
                    if (s.out_f32) {  // unrounded rows (the queries of a fused step)
                        float *o = reinterpret_cast<float *>(s.out) +
                                   ((size_t)token * s.heads + row0 + u * R) * D + j0;
#pragma unroll
                        for (int e = 0; e < E; e += 4)
                            *reinterpret_cast<float4 *>(o + e) =
                                make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                    } else {
                        *reinterpret_cast<uint4 *>(out + (size_t)(row0 + u * R) * head_bytes) = pack(x);
                    }
                }
            }
        }
    }

    if (BACK && a.set[0].weight) {
        // block's sums in a fixed order: rows of a warp, then the warps
        __shared__ float red[kWarps][2][D];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float t = dw[k][e];
#pragma unroll
                for (int o = 16; o >= L; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                if (sub == 0) red[warp][k][j0 + e] = t;
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

// dw[c] = sum over blocks of partial[block][c], in a fixed order: 32 columns
// a block, 32 slices of the blocks' axis.
__global__ void __launch_bounds__(1024)
norm_weight_sum_kernel(const float *__restrict__ partial, int blocks, int D, float *dwq, float *dwk) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float red[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float t = 0.f;
    for (int b = y; b < blocks; b += 32) t += partial[(size_t)b * 2 * D + c];
    red[y][x] = t;
    __syncthreads();
    t = red[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (x == 0) {
        const int col = blockIdx.x * 32 + y;
        if (col < D) dwq[col] = t; else dwk[col - D] = t;
    }
}

template <typename T, int D, int U, bool BACK>
cudaError_t launch_u(const NormRopeArgs &a) {
    constexpr int kRows = 32 / (D / (16 / (int)sizeof(T))) * U;
    long per = 0;
    for (const NormRopeRows &s : a.set) per += (s.heads + kRows - 1) / kRows;
    long grid = (a.num_tokens * per + kWarps - 1) / kWarps;
    // the backward pass keeps its weight sums in registers over a fixed
    // number of blocks, one partial result each
    const long most = BACK ? kNormBackwardBlocks : 0x7fffffffL;
    if (grid > most) grid = most;
    cudaError_t e = launch_dependent(qk_norm_rope_kernel<T, D, U, BACK>, (unsigned)grid,
                                     32 * kWarps, 0, a.stream, a);
    if (e == cudaSuccess && BACK && a.set[0].weight)
        e = launch_dependent(norm_weight_sum_kernel, (a.dk_weight ? 2 : 1) * D / 32, 1024, 0, a.stream,
                             static_cast<const float *>(a.partial), (int)grid, D, a.dq_weight,
                             a.dk_weight);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D, bool BACK>
cudaError_t launch(const NormRopeArgs &a) {
    // One pass a warp spreads a few rows over many SMs; four amortise the
    // token's cosines and sines over its rows.
    constexpr int kRows = 32 / (D / (16 / (int)sizeof(T)));
    const long rows = (long)a.num_tokens * (a.set[0].heads + a.set[1].heads + a.set[2].heads);
    if (rows <= 152L * 16 * kRows) return launch_u<T, D, 1, BACK>(a);
    return launch_u<T, D, 4, BACK>(a);
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
