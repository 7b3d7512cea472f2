// C-ABI front end of the softmax layers' operators: argument checks on the
// host, then the launches.  See include/lightning_attn.h for the contracts.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "la_internal.h"
#include "lightning_attn.h"

namespace {

#define LA_FAIL(status, ...) (la::set_last_error(__VA_ARGS__), (status))
#define LA_INVALID(...) LA_FAIL(LA_ERR_INVALID_ARG, __VA_ARGS__)

la_status from_cuda(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return LA_OK;
    return LA_FAIL(LA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int elem(la_dtype dtype) { return dtype == LA_DTYPE_FP32 ? 4 : 2; }

// One [tokens, heads, head_dim] array with a row stride.
la_status check_rows(const char *name, const void *p, int64_t stride, int heads, int head_dim,
                     la_dtype dtype) {
    if (!p) return LA_INVALID("%s is null", name);
    if (!aligned(p, 16)) return LA_INVALID("%s must be 16-byte aligned", name);
    if (stride < (int64_t)heads * head_dim)
        return LA_INVALID("%s: row stride %lld is less than heads * head_dim", name, (long long)stride);
    if (stride * elem(dtype) % 16 != 0)
        return LA_INVALID("%s: row stride %lld is not a multiple of 16 bytes", name, (long long)stride);
    return LA_OK;
}

la_status check_shape(int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                      int32_t head_dim, la_dtype dtype) {
    if (num_tokens < 0) return LA_INVALID("negative number of tokens (%d)", num_tokens);
    if (num_heads < 1) return LA_INVALID("num_heads < 1 (%d)", num_heads);
    if (num_kv_heads < 0) return LA_INVALID("num_kv_heads < 0 (%d)", num_kv_heads);
    if (head_dim != 64 && head_dim != 128)
        return LA_INVALID("head_dim must be 64 or 128 (got %d)", head_dim);
    if (dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_FP32)
        return LA_INVALID("unknown dtype %d", (int)dtype);
    if ((long long)num_tokens * ((long long)num_heads + 2LL * num_kv_heads) > 0x7fffffffLL)
        return LA_INVALID("too many rows (tokens * heads)");
    return LA_OK;
}

la_status check_rotary(const int32_t *positions, const float *rotary, int32_t rotary_rows,
                       int32_t rotary_dim, int32_t head_dim, const float *q_weight,
                       const float *k_weight, bool has_k, float eps) {
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16 != 0)
        return LA_INVALID("rotary_dim must be a multiple of 16 up to head_dim (got %d)", rotary_dim);
    if (rotary_dim > 0) {
        if (!rotary || !positions) return LA_INVALID("null rotary table or positions");
        if (rotary_rows < 1) return LA_INVALID("rotary_rows < 1 (%d)", rotary_rows);
        if (!aligned(rotary, 16) || !aligned(positions, 4))
            return LA_INVALID("rotary table (16 bytes) or positions (4 bytes) misaligned");
    }
    if (has_k && !q_weight != !k_weight)
        return LA_INVALID("q_weight and k_weight go together");
    if (!has_k && k_weight) return LA_INVALID("k_weight without keys");
    if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)))
        return LA_INVALID("weights must be 16-byte aligned");
    if (q_weight && !(eps >= 0.f && std::isfinite(eps)))
        return LA_INVALID("eps must be finite and not negative");
    return LA_OK;
}

la_status check_pool(int32_t num_pages, int32_t page_size) {
    if (num_pages < 0) return LA_INVALID("num_pages < 0 (%d)", num_pages);
    if (page_size < 1) return LA_INVALID("page_size < 1 (%d)", page_size);
    if ((long long)num_pages * page_size > 0x7fffffffLL)
        return LA_INVALID("num_pages * page_size must be less than 2^31");
    return LA_OK;
}

la_status check_cache(const char *name, const void *p, int64_t page_stride, int32_t num_kv_heads,
                      int32_t page_size, int32_t head_dim, la_dtype dtype) {
    if (!p) return LA_INVALID("%s is null", name);
    if (!aligned(p, 16)) return LA_INVALID("%s must be 16-byte aligned", name);
    if (page_stride < (int64_t)num_kv_heads * page_size * head_dim)
        return LA_INVALID("%s: page stride %lld is less than a page", name, (long long)page_stride);
    if (page_stride * elem(dtype) % 16 != 0)
        return LA_INVALID("%s: page stride is not a multiple of 16 bytes", name);
    return LA_OK;
}

la_status check_table(const int32_t *block_table, int32_t table_stride, int32_t table_width,
                      const int32_t *seq_lens) {
    if (table_width < 0 || table_stride < table_width)
        return LA_INVALID("block table: width %d, stride %d", table_width, table_stride);
    if ((table_width > 0 && !block_table) || !seq_lens) return LA_INVALID("null block_table or seq_lens");
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4))
        return LA_INVALID("block_table and seq_lens must be 4-byte aligned");
    return LA_OK;
}

#define LA_TRY(expr)                       \
    do {                                   \
        const la_status st_ = (expr);      \
        if (st_ != LA_OK) return st_;      \
    } while (0)

la::NormRopeRows rows(const void *x, int64_t x_stride, void *out, int64_t out_stride,
                      const float *weight, int heads, la_dtype dtype) {
    la::NormRopeRows r;
    r.x = x;
    r.x_stride = (size_t)x_stride * elem(dtype);
    r.out = out;
    r.out_stride = (size_t)out_stride * elem(dtype);
    r.weight = weight;
    r.heads = heads;
    return r;
}

la::NormRopeArgs norm_args(const int32_t *positions, const float *rotary, int32_t rotary_rows,
                           int32_t rotary_dim, int32_t interleaved, float eps, int32_t num_tokens,
                           int32_t head_dim, void *stream) {
    la::NormRopeArgs a;
    a.rotary = rotary;
    a.positions = positions;
    a.rotary_rows = rotary_rows;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved != 0;
    a.eps = eps;
    a.num_tokens = num_tokens;
    a.head_dim = head_dim;
    a.stream = static_cast<cudaStream_t>(stream);
    return a;
}

// Sums, maxima and exponential sums of the pieces of split units.
int64_t decode_workspace(int32_t head_dim) {
    return (int64_t)la::kPagedCtas * 2 * la::kPagedMaxRows * (head_dim + 2) * (int64_t)sizeof(float);
}

la_status check_decode(const int32_t *block_table, int32_t table_stride, int32_t table_width,
                       const int32_t *seq_lens, const void *k_cache, int64_t k_page_stride,
                       const void *v_cache, int64_t v_page_stride, int32_t num_pages,
                       int32_t page_size, int32_t batch, int32_t num_heads, int32_t num_kv_heads,
                       int32_t head_dim, la_dtype dtype, float scale, const void *out,
                       const float *lse) {
    if (num_kv_heads < 1 || num_heads % num_kv_heads != 0)
        return LA_INVALID("num_heads (%d) must be a multiple of num_kv_heads (%d)", num_heads,
                          num_kv_heads);
    LA_TRY(check_pool(num_pages, page_size));
    if (!std::isfinite(scale)) return LA_INVALID("scale must be finite");
    if (batch == 0) return LA_OK;
    LA_TRY(check_table(block_table, table_stride, table_width, seq_lens));
    if (num_pages > 0) {
        LA_TRY(check_cache("k_cache", k_cache, k_page_stride, num_kv_heads, page_size, head_dim, dtype));
        LA_TRY(check_cache("v_cache", v_cache, v_page_stride, num_kv_heads, page_size, head_dim, dtype));
    }
    if (!out || !aligned(out, 16)) return LA_INVALID("out must be a 16-byte aligned device array");
    if (!aligned(lse, 4)) return LA_INVALID("lse must be 4-byte aligned");
    return LA_OK;
}

// Queries of an attention, and the output over them.
la_status check_queries(const void *q, int64_t q_stride, int32_t batch, int32_t num_heads, int32_t head_dim,
                        la_dtype dtype, const void *out) {
    LA_TRY(check_rows("q", q, q_stride, num_heads, head_dim, dtype));
    if (out == q && batch > 1 && q_stride != (int64_t)num_heads * head_dim)
        return LA_INVALID("an output in place of its input needs the input's stride");
    return LA_OK;
}

// Tokens that a row of a table can hold.
int capacity(int32_t table_width, int32_t page_size) {
    const long long most = (long long)table_width * page_size;
    return (int)(most < la::kMaxTokens ? most : la::kMaxTokens);
}

la::PagedDecodeArgs decode_args(const void *q, int64_t q_stride, const void *k_cache,
                                int64_t k_page_stride, const void *v_cache, int64_t v_page_stride,
                                const int32_t *block_table, int32_t table_stride,
                                int32_t table_width, const int32_t *seq_lens, int32_t num_pages,
                                int32_t page_size, int32_t batch, int32_t num_heads,
                                int32_t num_kv_heads, int32_t head_dim, float scale, void *out,
                                float *lse, void *workspace, void *stream) {
    la::PagedDecodeArgs a;
    a.q = q;
    a.q_stride = q_stride;
    a.k = k_cache;
    a.v = v_cache;
    a.k_page_stride = k_page_stride;
    a.v_page_stride = v_page_stride;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.table_stride = table_stride;
    a.max_tokens = capacity(table_width, page_size);
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.batch = batch;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = num_heads / num_kv_heads;
    a.head_dim = head_dim;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    a.out = out;
    a.lse = lse;
    a.workspace = static_cast<float *>(workspace);
    a.stream = static_cast<cudaStream_t>(stream);
    return a;
}

la_status check_workspace(const void *workspace, int64_t bytes, int64_t need) {
    if (!workspace || !aligned(workspace, 16))
        return LA_INVALID("workspace must be a 16-byte aligned device array");
    if (bytes < need)
        return LA_INVALID("workspace too small: %lld bytes, %lld needed", (long long)bytes,
                          (long long)need);
    return LA_OK;
}

// Behind the attention's own: the prefix's pieces, the rows' own sums and statistics, the ranges.
int64_t prefix_pieces_floats(const la::PrefixPieces &f, int32_t head_dim) {
    return ((int64_t)f.ctas + f.units) * f.parts * f.stride * (head_dim + 2);
}
int64_t prefix_workspace(const la::PrefixPieces &f, int64_t rows, int32_t head_dim) {
    return decode_workspace(head_dim) +
           (prefix_pieces_floats(f, head_dim) + rows * (head_dim + 2) + 4) * (int64_t)sizeof(float);
}

}  // namespace

extern "C" {

la_status lightning_attn_qk_norm_rope(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
    const float *rotary, int32_t rotary_rows, int32_t rotary_dim, int32_t interleaved,
    const float *q_weight, const float *k_weight, float eps, int32_t num_tokens,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype, void *q_out,
    int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream) {
    LA_TRY(check_shape(num_tokens, num_heads, num_kv_heads, head_dim, dtype));
    if (num_tokens == 0) return LA_OK;
    LA_TRY(check_rotary(positions, rotary, rotary_rows, rotary_dim, head_dim, q_weight, k_weight,
                        num_kv_heads > 0, eps));
    LA_TRY(check_rows("q", q, q_stride, num_heads, head_dim, dtype));
    LA_TRY(check_rows("q_out", q_out, q_out_stride, num_heads, head_dim, dtype));
    if (num_kv_heads > 0) {
        LA_TRY(check_rows("k", k, k_stride, num_kv_heads, head_dim, dtype));
        LA_TRY(check_rows("k_out", k_out, k_out_stride, num_kv_heads, head_dim, dtype));
    }
    if ((q_out == q && q_out_stride != q_stride) ||
        (num_kv_heads > 0 && k_out == k && k_out_stride != k_stride))
        return LA_INVALID("an output in place of its input needs the input's stride");
    if (num_kv_heads > 0 && (q_out == k || k_out == q || k_out == q_out))
        return LA_INVALID("an output is the other input or the other output");
    la::NormRopeArgs a = norm_args(positions, rotary, rotary_rows, rotary_dim, interleaved, eps,
                                   num_tokens, head_dim, stream);
    a.set[0] = rows(q, q_stride, q_out, q_out_stride, q_weight, num_heads, dtype);
    a.set[1] = rows(k, k_stride, k_out, k_out_stride, k_weight, num_kv_heads, dtype);
    return from_cuda(la::qk_norm_rope(a, dtype == LA_DTYPE_BF16), "qk_norm_rope");
}

int64_t lightning_attn_qk_norm_rope_workspace_bytes(int32_t head_dim) {
    if (head_dim != 64 && head_dim != 128) return -1;
    return (int64_t)la::kNormBackwardBlocks * 2 * head_dim * (int64_t)sizeof(float);
}

la_status lightning_attn_qk_norm_rope_backward(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
    const float *rotary, int32_t rotary_rows, int32_t rotary_dim, int32_t interleaved,
    const float *q_weight, const float *k_weight, float eps, int32_t num_tokens,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype,
    const void *d_q_out, int64_t d_q_out_stride, const void *d_k_out, int64_t d_k_out_stride,
    void *d_q, int64_t d_q_stride, void *d_k, int64_t d_k_stride, float *d_q_weight,
    float *d_k_weight, void *workspace, int64_t workspace_bytes, void *stream) {
    LA_TRY(check_shape(num_tokens, num_heads, num_kv_heads, head_dim, dtype));
    LA_TRY(check_rotary(num_tokens ? positions : nullptr, rotary, rotary_rows,
                        num_tokens ? rotary_dim : 0, head_dim, q_weight, k_weight,
                        num_kv_heads > 0, eps));
    if (q_weight) {
        if (!d_q_weight || !aligned(d_q_weight, 4) ||
            (num_kv_heads > 0 && (!d_k_weight || !aligned(d_k_weight, 4))))
            return LA_INVALID("null or misaligned gradient of a weight");
        if (num_kv_heads > 0 && d_q_weight == d_k_weight)
            return LA_INVALID("the two weights' gradients are one array");
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (num_tokens == 0) {  // sums over no rows
        if (!q_weight) return LA_OK;
        LA_TRY(from_cuda(cudaMemsetAsync(d_q_weight, 0, sizeof(float) * head_dim, st),
                         "qk_norm_rope_backward"));
        if (num_kv_heads == 0) return LA_OK;
        return from_cuda(cudaMemsetAsync(d_k_weight, 0, sizeof(float) * head_dim, st),
                         "qk_norm_rope_backward");
    }
    LA_TRY(check_rows("q", q, q_stride, num_heads, head_dim, dtype));
    LA_TRY(check_rows("d_q_out", d_q_out, d_q_out_stride, num_heads, head_dim, dtype));
    LA_TRY(check_rows("d_q", d_q, d_q_stride, num_heads, head_dim, dtype));
    if (num_kv_heads > 0) {
        LA_TRY(check_rows("k", k, k_stride, num_kv_heads, head_dim, dtype));
        LA_TRY(check_rows("d_k_out", d_k_out, d_k_out_stride, num_kv_heads, head_dim, dtype));
        LA_TRY(check_rows("d_k", d_k, d_k_stride, num_kv_heads, head_dim, dtype));
    }
    if (d_q == q || (num_kv_heads > 0 && (d_k == k || d_k == d_q || d_q == k || d_k == q ||
                                          d_q == d_k_out || d_k == d_q_out)))
        return LA_INVALID("a gradient aliases an input or another gradient");
    if ((d_q == d_q_out && d_q_stride != d_q_out_stride) ||
        (num_kv_heads > 0 && d_k == d_k_out && d_k_stride != d_k_out_stride))
        return LA_INVALID("an output in place of its input needs the input's stride");
    if (q_weight)
        LA_TRY(check_workspace(workspace, workspace_bytes,
                               lightning_attn_qk_norm_rope_workspace_bytes(head_dim)));
    la::NormRopeArgs a = norm_args(positions, rotary, rotary_rows, rotary_dim, interleaved, eps,
                                   num_tokens, head_dim, stream);
    a.set[0] = rows(q, q_stride, d_q, d_q_stride, q_weight, num_heads, dtype);
    a.set[0].dy = d_q_out;
    a.set[0].dy_stride = (size_t)d_q_out_stride * elem(dtype);
    a.set[1] = rows(k, k_stride, d_k, d_k_stride, k_weight, num_kv_heads, dtype);
    a.set[1].dy = d_k_out;
    a.set[1].dy_stride = (size_t)d_k_out_stride * elem(dtype);
    a.partial = static_cast<float *>(workspace);
    a.dq_weight = d_q_weight;
    a.dk_weight = num_kv_heads > 0 ? d_k_weight : nullptr;
    return from_cuda(la::qk_norm_rope_backward(a, dtype == LA_DTYPE_BF16), "qk_norm_rope_backward");
}

la_status lightning_attn_paged_append(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
    int64_t v_stride, const int32_t *positions, const float *rotary, int32_t rotary_rows,
    int32_t rotary_dim, int32_t interleaved, const float *q_weight, const float *k_weight,
    float eps, int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    la_dtype dtype, void *q_out, int64_t q_out_stride, void *k_cache, int64_t k_page_stride,
    void *v_cache, int64_t v_page_stride, const int32_t *slots, int32_t num_pages,
    int32_t page_size, void *stream) {
    LA_TRY(check_shape(num_tokens, num_heads, num_kv_heads, head_dim, dtype));
    if (num_kv_heads < 1) return LA_INVALID("num_kv_heads < 1 (%d)", num_kv_heads);
    LA_TRY(check_pool(num_pages, page_size));
    if (num_tokens == 0) return LA_OK;
    LA_TRY(check_rotary(positions, rotary, rotary_rows, rotary_dim, head_dim, q_weight, k_weight,
                        true, eps));
    LA_TRY(check_rows("q", q, q_stride, num_heads, head_dim, dtype));
    LA_TRY(check_rows("k", k, k_stride, num_kv_heads, head_dim, dtype));
    LA_TRY(check_rows("v", v, v_stride, num_kv_heads, head_dim, dtype));
    LA_TRY(check_rows("q_out", q_out, q_out_stride, num_heads, head_dim, dtype));
    if (q_out == q && q_out_stride != q_stride)
        return LA_INVALID("an output in place of its input needs the input's stride");
    if (q_out == k || q_out == v) return LA_INVALID("q_out is k or v");
    if (num_pages > 0 && k_cache == v_cache) return LA_INVALID("k_cache and v_cache are one array");
    if (num_pages > 0) {
        LA_TRY(check_cache("k_cache", k_cache, k_page_stride, num_kv_heads, page_size, head_dim, dtype));
        LA_TRY(check_cache("v_cache", v_cache, v_page_stride, num_kv_heads, page_size, head_dim, dtype));
    }
    if (!slots || !aligned(slots, 4)) return LA_INVALID("slots must be a 4-byte aligned device array");
    la::NormRopeArgs a = norm_args(positions, rotary, rotary_rows, rotary_dim, interleaved, eps,
                                   num_tokens, head_dim, stream);
    a.set[0] = rows(q, q_stride, q_out, q_out_stride, q_weight, num_heads, dtype);
    a.set[1] = rows(k, k_stride, k_cache, k_page_stride, k_weight, num_kv_heads, dtype);
    a.set[2] = rows(v, v_stride, v_cache, v_page_stride, nullptr, num_kv_heads, dtype);
    a.set[1].cache = a.set[2].cache = true;
    a.slots = slots;
    a.num_slots = num_pages * page_size;
    a.page_size = page_size;
    return from_cuda(la::qk_norm_rope(a, dtype == LA_DTYPE_BF16), "paged_append");
}

int64_t lightning_attn_paged_decode_workspace_bytes(int32_t head_dim) {
    if (head_dim != 64 && head_dim != 128) return -1;
    return decode_workspace(head_dim);
}

la_status lightning_attn_paged_decode(
    const void *q, int64_t q_stride, const void *k_cache, int64_t k_page_stride,
    const void *v_cache, int64_t v_page_stride, const int32_t *block_table, int32_t table_stride,
    int32_t table_width, const int32_t *seq_lens, int32_t num_pages, int32_t page_size,
    int32_t batch, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype,
    float scale, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    LA_TRY(check_shape(batch, num_heads, num_kv_heads, head_dim, dtype));
    LA_TRY(check_decode(block_table, table_stride, table_width, seq_lens, k_cache, k_page_stride,
                        v_cache, v_page_stride, num_pages, page_size, batch, num_heads,
                        num_kv_heads, head_dim, dtype, scale, out, lse));
    if (batch == 0) return LA_OK;
    LA_TRY(check_queries(q, q_stride, batch, num_heads, head_dim, dtype, out));
    LA_TRY(check_workspace(workspace, workspace_bytes, decode_workspace(head_dim)));
    const la::PagedDecodeArgs a = decode_args(
        q, q_stride, k_cache, k_page_stride, v_cache, v_page_stride, block_table, table_stride,
        table_width, seq_lens, num_pages, page_size, batch, num_heads, num_kv_heads, head_dim,
        scale, out, lse, workspace, stream);
    return from_cuda(la::paged_decode(a, dtype == LA_DTYPE_BF16, dtype == LA_DTYPE_FP32), "paged_decode");
}

int64_t lightning_attn_paged_step_workspace_bytes(int32_t batch, int32_t num_heads,
                                                  int32_t head_dim) {
    if (batch < 0 || num_heads < 1 || (head_dim != 64 && head_dim != 128)) return -1;
    return decode_workspace(head_dim) + (int64_t)batch * num_heads * head_dim * (int64_t)sizeof(float);
}

la_status lightning_attn_paged_step(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
    int64_t v_stride, const int32_t *positions, const float *rotary, int32_t rotary_rows,
    int32_t rotary_dim, int32_t interleaved, const float *q_weight, const float *k_weight,
    float eps, void *k_cache, int64_t k_page_stride, void *v_cache, int64_t v_page_stride,
    const int32_t *slots, const int32_t *block_table, int32_t table_stride, int32_t table_width,
    const int32_t *seq_lens, int32_t num_pages, int32_t page_size, int32_t batch,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype, float scale,
    void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    LA_TRY(check_shape(batch, num_heads, num_kv_heads, head_dim, dtype));
    LA_TRY(check_decode(block_table, table_stride, table_width, seq_lens, k_cache, k_page_stride,
                        v_cache, v_page_stride, num_pages, page_size, batch, num_heads,
                        num_kv_heads, head_dim, dtype, scale, out, lse));
    if (batch == 0) return LA_OK;
    LA_TRY(check_rotary(positions, rotary, rotary_rows, rotary_dim, head_dim, q_weight, k_weight,
                        true, eps));
    LA_TRY(check_rows("q", q, q_stride, num_heads, head_dim, dtype));
    LA_TRY(check_rows("k", k, k_stride, num_kv_heads, head_dim, dtype));
    LA_TRY(check_rows("v", v, v_stride, num_kv_heads, head_dim, dtype));
    if (!slots || !aligned(slots, 4)) return LA_INVALID("slots must be a 4-byte aligned device array");
    if (num_pages > 0 && k_cache == v_cache) return LA_INVALID("k_cache and v_cache are one array");
    LA_TRY(check_workspace(workspace, workspace_bytes,
                           lightning_attn_paged_step_workspace_bytes(batch, num_heads, head_dim)));
    float *rotated = reinterpret_cast<float *>(static_cast<char *>(workspace) + decode_workspace(head_dim));
    la::NormRopeArgs n = norm_args(positions, rotary, rotary_rows, rotary_dim, interleaved, eps,
                                   batch, head_dim, stream);
    n.set[0] = rows(q, q_stride, rotated, 0, q_weight, num_heads, dtype);
    n.set[0].out_f32 = true;
    n.set[1] = rows(k, k_stride, k_cache, k_page_stride, k_weight, num_kv_heads, dtype);
    n.set[2] = rows(v, v_stride, v_cache, v_page_stride, nullptr, num_kv_heads, dtype);
    n.set[1].cache = n.set[2].cache = true;
    n.slots = slots;
    n.num_slots = num_pages * page_size;
    n.page_size = page_size;
    LA_TRY(from_cuda(la::qk_norm_rope(n, dtype == LA_DTYPE_BF16), "paged_step (append)"));
    const la::PagedDecodeArgs a = decode_args(
        rotated, (int64_t)num_heads * head_dim, k_cache, k_page_stride, v_cache, v_page_stride,
        block_table, table_stride, table_width, seq_lens, num_pages, page_size, batch, num_heads,
        num_kv_heads, head_dim, scale, out, lse, workspace, stream);
    return from_cuda(la::paged_decode(a, dtype == LA_DTYPE_BF16, true), "paged_step (attention)");
}

la_status lightning_attn_paged_bounds(
    const void *k_cache, int64_t k_page_stride, void *bounds, int64_t bounds_page_stride,
    const int32_t *block_table, int32_t table_stride, int32_t table_width, const int32_t *first,
    const int32_t *seq_lens, int32_t num_pages, int32_t page_size, int32_t batch,
    int32_t num_kv_heads, int32_t head_dim, la_dtype dtype, void *stream) {
    if (num_kv_heads < 1) return LA_INVALID("num_kv_heads < 1 (%d)", num_kv_heads);
    LA_TRY(check_shape(batch, num_kv_heads, 0, head_dim, dtype));
    LA_TRY(check_pool(num_pages, page_size));
    if (batch == 0) return LA_OK;
    LA_TRY(check_table(block_table, table_stride, table_width, seq_lens));
    if (!first || !aligned(first, 4)) return LA_INVALID("first must be a 4-byte aligned device array");
    if (num_pages == 0) return LA_OK;
    LA_TRY(check_cache("k_cache", k_cache, k_page_stride, num_kv_heads, page_size, head_dim, dtype));
    LA_TRY(check_cache("bounds", bounds, bounds_page_stride, num_kv_heads, 2, head_dim, dtype));
    if (bounds == k_cache) return LA_INVALID("bounds and k_cache are one array");
    la::PagedBoundsArgs a;
    a.k = k_cache;
    a.bounds = bounds;
    a.k_page_stride = k_page_stride;
    a.bounds_page_stride = bounds_page_stride;
    a.block_table = block_table;
    a.first = first;
    a.seq_lens = seq_lens;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.max_tokens = capacity(table_width, page_size);
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.batch = batch;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(la::paged_bounds(a, dtype == LA_DTYPE_BF16), "paged_bounds");
}

int64_t lightning_attn_paged_select_workspace_bytes(int32_t batch, int32_t num_kv_heads,
                                                    int32_t table_width) {
    if (batch < 0 || num_kv_heads < 1 || table_width < 0) return -1;
    return la::paged_select_workspace(batch, num_kv_heads, table_width);
}

la_status lightning_attn_paged_select(
    const void *q, int64_t q_stride, const void *bounds, int64_t bounds_page_stride,
    const int32_t *block_table, int32_t table_stride, int32_t table_width, const int32_t *seq_lens,
    int32_t num_pages, int32_t page_size, int32_t batch, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, la_dtype dtype, int32_t count, int32_t keep_first, int32_t keep_last,
    int32_t *selected, void *workspace, int64_t workspace_bytes, void *stream) {
    LA_TRY(check_shape(batch, num_heads, num_kv_heads, head_dim, dtype));
    if (num_kv_heads < 1 || num_heads % num_kv_heads != 0)
        return LA_INVALID("num_heads (%d) must be a multiple of num_kv_heads (%d)", num_heads,
                          num_kv_heads);
    LA_TRY(check_pool(num_pages, page_size));
    if (count < 1) return LA_INVALID("count < 1 (%d)", count);
    if (keep_first < 0 || keep_last < 0 || (long long)keep_first + keep_last > count)
        return LA_INVALID("keep_first (%d) and keep_last (%d) must be at least 0 and together at most "
                          "count (%d)", keep_first, keep_last, count);
    if (batch == 0) return LA_OK;
    LA_TRY(check_table(block_table, table_stride, table_width, seq_lens));
    LA_TRY(check_rows("q", q, q_stride, num_heads, head_dim, dtype));
    if (num_pages > 0)
        LA_TRY(check_cache("bounds", bounds, bounds_page_stride, num_kv_heads, 2, head_dim, dtype));
    if (!selected || !aligned(selected, 4))
        return LA_INVALID("selected must be a 4-byte aligned device array");
    if (selected == block_table || selected == seq_lens)
        return LA_INVALID("selected and block_table or seq_lens are one array");
    const int64_t need = la::paged_select_workspace(batch, num_kv_heads, table_width);
    if (need < 0) return LA_INVALID("too many blocks");
    LA_TRY(check_workspace(workspace, workspace_bytes, need));
    la::PagedSelectArgs a;
    a.q = q;
    a.q_stride = q_stride;
    a.bounds = bounds;
    a.bounds_page_stride = bounds_page_stride;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.max_tokens = capacity(table_width, page_size);
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.batch = batch;
    a.num_kv_heads = num_kv_heads;
    a.group = num_heads / num_kv_heads;
    a.head_dim = head_dim;
    a.count = count;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    a.selected = selected;
    a.workspace = workspace;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(la::paged_select(a, dtype == LA_DTYPE_BF16), "paged_select");
}

la_status lightning_attn_paged_sparse_decode(
    const void *q, int64_t q_stride, const void *k_cache, int64_t k_page_stride,
    const void *v_cache, int64_t v_page_stride, const int32_t *block_table, int32_t table_stride,
    int32_t table_width, const int32_t *seq_lens, const int32_t *selected, int32_t count,
    int32_t num_pages, int32_t page_size, int32_t batch, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, la_dtype dtype, float scale, void *out, float *lse, void *workspace,
    int64_t workspace_bytes, void *stream) {
    LA_TRY(check_shape(batch, num_heads, num_kv_heads, head_dim, dtype));
    LA_TRY(check_decode(block_table, table_stride, table_width, seq_lens, k_cache, k_page_stride,
                        v_cache, v_page_stride, num_pages, page_size, batch, num_heads,
                        num_kv_heads, head_dim, dtype, scale, out, lse));
    if (count < 1) return LA_INVALID("count < 1 (%d)", count);
    if (batch == 0) return LA_OK;
    if (!selected || !aligned(selected, 4))
        return LA_INVALID("selected must be a 4-byte aligned device array");
    if ((long long)count * page_size > la::kMaxTokens)
        return LA_FAIL(LA_ERR_UNSUPPORTED, "count * page_size must be at most %d", la::kMaxTokens);
    LA_TRY(check_queries(q, q_stride, batch, num_heads, head_dim, dtype, out));
    LA_TRY(check_workspace(workspace, workspace_bytes, decode_workspace(head_dim)));
    la::PagedDecodeArgs a = decode_args(
        q, q_stride, k_cache, k_page_stride, v_cache, v_page_stride, block_table, table_stride,
        table_width, seq_lens, num_pages, page_size, batch, num_heads, num_kv_heads, head_dim,
        scale, out, lse, workspace, stream);
    a.chosen = selected;
    a.chosen_count = count;
    return from_cuda(la::paged_sparse_decode(a, dtype == LA_DTYPE_BF16), "paged_sparse_decode");
}

int64_t lightning_attn_paged_prefix_decode_workspace_bytes(int32_t batch, int32_t num_heads,
                                                           int32_t num_kv_heads, int32_t head_dim,
                                                           la_dtype dtype) {
    if (batch < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128) || (dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_FP32) ||
        (long long)batch * num_heads > 0x7fffffffLL)
        return -1;
    return prefix_workspace(la::paged_prefix_pieces(batch, num_heads, num_kv_heads, dtype == LA_DTYPE_BF16),
                            (int64_t)batch * num_heads, head_dim);
}

la_status lightning_attn_paged_prefix_decode(
    const void *q, int64_t q_stride, const void *k_cache, int64_t k_page_stride,
    const void *v_cache, int64_t v_page_stride, const int32_t *prefix_table, int32_t prefix_width,
    const int32_t *prefix_len, const int32_t *block_table, int32_t table_stride,
    int32_t table_width, const int32_t *seq_lens, int32_t num_pages, int32_t page_size,
    int32_t batch, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype,
    float scale, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    LA_TRY(check_shape(batch, num_heads, num_kv_heads, head_dim, dtype));
    LA_TRY(check_decode(block_table, table_stride, table_width, seq_lens, k_cache, k_page_stride,
                        v_cache, v_page_stride, num_pages, page_size, batch, num_heads,
                        num_kv_heads, head_dim, dtype, scale, out, lse));
    if (prefix_width < 0) return LA_INVALID("prefix_width < 0 (%d)", prefix_width);
    if (batch == 0) return LA_OK;
    if ((prefix_width > 0 && !prefix_table) || !prefix_len)
        return LA_INVALID("null prefix_table or prefix_len");
    if (!aligned(prefix_table, 4) || !aligned(prefix_len, 4))
        return LA_INVALID("prefix_table and prefix_len must be 4-byte aligned");
    LA_TRY(check_queries(q, q_stride, batch, num_heads, head_dim, dtype, out));
    la::PrefixPieces f = la::paged_prefix_pieces(batch, num_heads, num_kv_heads, dtype == LA_DTYPE_BF16);
    const int64_t rows = (int64_t)batch * num_heads;
    LA_TRY(check_workspace(workspace, workspace_bytes, prefix_workspace(f, rows, head_dim)));
    f.len = prefix_len;
    f.max_tokens = capacity(prefix_width, page_size);
    f.pieces = reinterpret_cast<float *>(static_cast<char *>(workspace) + decode_workspace(head_dim));
    f.own = f.pieces + prefix_pieces_floats(f, head_dim);
    f.own_stat = f.own + rows * head_dim;
    f.ranges = reinterpret_cast<int *>(f.own_stat + 2 * rows);
    la::PagedDecodeArgs a = decode_args(
        q, q_stride, k_cache, k_page_stride, v_cache, v_page_stride, block_table, table_stride,
        table_width, seq_lens, num_pages, page_size, batch, num_heads, num_kv_heads, head_dim,
        scale, out, lse, workspace, stream);
    a.prefix = f;
    return from_cuda(la::paged_prefix_decode(a, prefix_table, dtype == LA_DTYPE_BF16), "paged_prefix_decode");
}

la_status lightning_attn_paged_reserve(
    int32_t *block_table, int32_t table_stride, int32_t table_width, const int32_t *seq_lens,
    const int32_t *new_lens, const uint8_t *finished, int32_t batch, int32_t *free_pages,
    const int32_t *free_count, int32_t num_pages, int32_t page_size, int32_t num_tokens,
    int32_t *slots, int32_t *positions, int32_t *cu_seqlens, uint8_t *served,
    int32_t *seq_lens_out, int32_t *free_count_out, void *stream) {
    if (batch < 0) return LA_INVALID("batch < 0 (%d)", batch);
    if (batch > la::kReserveMaxBatch)
        return LA_FAIL(LA_ERR_UNSUPPORTED, "batch %d: at most %d requests", batch, la::kReserveMaxBatch);
    if (num_tokens < 0) return LA_INVALID("num_tokens < 0 (%d)", num_tokens);
    LA_TRY(check_pool(num_pages, page_size));
    if (batch == 0) return LA_INVALID("batch must be at least 1");
    LA_TRY(check_table(block_table, table_stride, table_width, seq_lens));
    if (!new_lens || !free_count || !cu_seqlens || !served || !seq_lens_out || !free_count_out ||
        (num_pages > 0 && !free_pages) || (num_tokens > 0 && (!slots || !positions)))
        return LA_INVALID("null pointer argument");
    const void *ints[] = {new_lens, free_count, cu_seqlens, seq_lens_out, free_count_out,
                          free_pages, slots, positions};
    for (const void *p : ints)
        if (!aligned(p, 4)) return LA_INVALID("int32 arrays must be 4-byte aligned");
    // a long step reads new_lens again after the other arrays have been written
    if (new_lens == seq_lens_out || new_lens == free_count_out)
        return LA_INVALID("new_lens is an output too");
    la::PagedReserveArgs a;
    a.block_table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.batch = batch;
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.finished = finished;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.num_tokens = num_tokens;
    a.slots = slots;
    a.positions = positions;
    a.cu_seqlens = cu_seqlens;
    a.served = served;
    a.seq_lens_out = seq_lens_out;
    a.free_count_out = free_count_out;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(la::paged_reserve(a), "paged_reserve");
}

}  // extern "C"
