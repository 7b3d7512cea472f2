// Internal interface between the C-ABI front end (api.cu) and the kernels.
// Not installed; the public interface is include/lightning_attn.h.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "lightning_attn.h"

namespace la {

// Launches `kern` with programmatic stream serialization: it may be scheduled
// while the kernel before it in the stream is finishing, and waits
// (grid_dependency_wait) before its first global-memory access, so stream
// order is kept for every memory effect.  Only kernels that begin with that
// wait are launched this way, but for three that read some of the call's arguments before it: the join of the
// paged attention the lengths, through L2, and, behind an acquire, the choice of pages all but the scores and the
// attention behind a shared prefix all but the prefix's pieces.  The first kernel of each of these calls has
// waited, in every CTA, for whatever wrote the arguments, and none of the others is scheduled before that.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kern)(KArgs...), unsigned grid, unsigned block,
                                    size_t smem, cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args &&>(args)...);
}

struct PrefillArgs {
    const void *q, *k, *v;      // [T, H, D]
    const float *decay;         // [H]
    const int32_t *cu_seqlens;  // [nseq + 1], device
    int nseq, total_tokens, num_heads, head_dim, chunk;
    void *out;                  // [T, H, D]
    float *final_state;         // [nseq, H, D, D] or nullptr
    cudaStream_t stream;
    const float *initial_state; // [nseq, H, D, D] or nullptr (zero state)
    bool reverse_out = false;   // write o_t of sequence s to row cu[s] + cu[s+1] - 1 - t
    int min_len = 0;            // sequences shorter than this are left untouched
    // > 0: launch only the work of the rank_limit longest sequences (ranks
    // are in order of length, longest first, for nseq <= kMaxSortedSeqs)
    int rank_limit = 0;
    bool channel_decay = false; // decay is [H, D]: one lambda per key channel
    // Anti-causal sum o_t = sum_{u >= t} lambda^(u-t) (q_t . k_u) v_u (the
    // backward pass's reversed-time products), output rows in place; the
    // final state is then sum_u lambda^(u - t0) k_u^T v_u.  Tensor-core
    // kernel only, zero initial state.
    bool anti_causal = false;
    // Per-block state snapshots (nullptr: none): the state after every
    // snapshot_interval tokens of each sequence, [N, H, D, D] fp32, sequence
    // s's snapshots from index sum_{s' < s} floor(L_s' / snapshot_interval).
    // snapshot_interval is a multiple of the kernel's chunk.
    float *snapshots = nullptr;
    int snapshot_interval = 0;
};

struct DecodeArgs {
    const void *q, *k, *v;      // [B, H, D]
    const float *decay;         // [H]
    float *state;               // [B, H, D, D]
    int batch, num_heads, head_dim;
    void *out;                  // [B, H, D]
    cudaStream_t stream;
    // Packed mode (cu_seqlens != nullptr): entry b is sequence b of a packed
    // batch; its token row is cu_seqlens[b], and only sequences of length
    // exactly 1 are stepped (the others are left untouched).
    const int32_t *cu_seqlens = nullptr;
    int total_tokens = 0;
    bool channel_decay = false; // decay is [H, D]: one lambda per key channel (state row)
};

// Whether a (scalar-decay) call runs on the tensor-core kernel: bf16,
// head_dim 128 and a block size of 16, 32, 64, 128 or 256 (chunk 0 = 128).
inline bool uses_tensor_cores(bool bf16, int head_dim, int chunk) {
    return bf16 && head_dim == 128 &&
           (chunk == 0 || chunk == 16 || chunk == 32 || chunk == 64 || chunk == 128 ||
            chunk == 256);
}

// CUDA-core chunkwise prefill; chunk in {16, 32, 64}, head_dim in {64, 128};
// also the channel-wise decay variant.
cudaError_t prefill_simt_f32(const PrefillArgs &a);
cudaError_t prefill_simt_bf16(const PrefillArgs &a);

// tcgen05 / TMEM / TMA prefill; bf16, head_dim 128, block size 16-256.
// Returns cudaErrorNotSupported when the tensor-map encoder is unavailable.
cudaError_t prefill_tc_bf16(const PrefillArgs &a);

// tcgen05 / TMEM / TMA prefill with the channel-wise decay; bf16, head_dim
// 128, block size 64 (chunk 0 or 64), scalar-decay features (snapshots,
// anti-causal, mixed-step ranks) excluded.
cudaError_t prefill_cw_tc_bf16(const PrefillArgs &a);
// Reads and clears the channel-wise kernel's device error word (the caller
// has synchronised the stream).
cudaError_t take_cw_device_error(unsigned int *err);

// Synchronises `stream`, then reads and clears the device error word.
cudaError_t take_device_error(cudaStream_t stream, unsigned int *err);
// Launches a kernel whose bounded wait must time out after timeout_ns.
cudaError_t selftest_wait_timeout(uint64_t timeout_ns, cudaStream_t stream);

// out row (cu[s] + cu[s+1] - 1 - t) = in row t for every token t of
// sequence s; rows are row_bytes long (a multiple of 16).  in != out.
cudaError_t reverse_sequences(const void *in, void *out, const int32_t *cu_seqlens, int nseq,
                              int total_tokens, size_t row_bytes, cudaStream_t stream);

// Every host-side check of lightning_attn_backward except those of the
// workspace.  Returns an error status, or LA_OK with *work = false when there
// is nothing to compute, or LA_OK with *work = true and *needs_workspace
// telling whether the path that serves the call reads a workspace.
la_status backward_check(const void *q, const void *k, const void *v, const float *decay,
                         const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                         int32_t num_heads, int32_t head_dim, int32_t chunk, la_dtype dtype,
                         const void *d_out, void *d_q, void *d_k, void *d_v, bool *work,
                         bool *needs_workspace);

// Sets the message lightning_attn_last_error() returns on this host thread.
void set_last_error(const char *fmt, ...) __attribute__((format(printf, 1, 2)));

// Memory-bound decode step; head_dim in {64, 128}.
cudaError_t decode_f32(const DecodeArgs &a);
cudaError_t decode_bf16(const DecodeArgs &a);

// ------------------------------------------- softmax layers (paged cache)
// One kind of rows (query, key or value heads) of the norm + rotation pass.
// Strides are in bytes: from one token's rows to the next, or, with `cache`,
// from one page to the next.
struct NormRopeRows {
    const void *x = nullptr;
    size_t x_stride = 0;
    const void *dy = nullptr;      // backward: gradient of the rotated rows
    size_t dy_stride = 0;
    void *out = nullptr;           // rotated rows, or (backward) the gradient of x
    size_t out_stride = 0;
    const float *weight = nullptr; // [D]; nullptr: no norm
    int heads = 0;
    bool cache = false;            // out is a paged cache, written at `slots`
    bool out_f32 = false;          // out is contiguous fp32 [T, heads, D]
};

struct NormRopeArgs {
    NormRopeRows set[3];           // queries, keys, values (copied)
    const float *rotary = nullptr; // [rotary_rows, rotary_dim]: cosines, then sines
    const int32_t *positions = nullptr;
    int rotary_rows = 0, rotary_dim = 0;
    bool interleaved = false;
    float eps = 0.f;
    int num_tokens = 0, head_dim = 0;
    const int32_t *slots = nullptr;
    int num_slots = 0, page_size = 1;
    float *partial = nullptr;      // backward: [kNormBackwardBlocks][2][D]
    float *dq_weight = nullptr, *dk_weight = nullptr;
    cudaStream_t stream = nullptr;
};

// Blocks of the backward pass, each leaving one partial weight gradient.
constexpr int kNormBackwardBlocks = 152 * 5;

cudaError_t qk_norm_rope(const NormRopeArgs &a, bool bf16);
cudaError_t qk_norm_rope_backward(const NormRopeArgs &a, bool bf16);

// Most tokens of a request: room for some tiles past the end in 32-bit token indices.
constexpr int kMaxTokens = 0x7fff0000;

// What the attention over a shared prefix leaves for the requests behind it: the tiles of all units
// (unit_rows query rows of one key-value head; row r is head r % group of the head's group, of request
// r / group), one unit after the other, are cut into `ctas` equal ranges.  CTA c's part of unit u is
// in slots (c + u) * parts .. + parts - 1: along the ranges either c or u grows from one
// part to the next, so c + u is theirs alone.  A slot holds the unnormalised sums [stride][D]
// and (maximum, exponential sum) [stride].
struct PrefixPieces {
    const int32_t *len = nullptr;  // [1] tokens, on the device
    int max_tokens = 0;            // capacity of the prefix's table
    int tile = 1, ctas = 1, units = 1, units_per_head = 1, unit_rows = 1;
    int parts = 1, stride = 0;
    float *pieces = nullptr;
    // A row's sums [B * H][D] and statistics [B * H][2] over its own tokens where one CTA held them all.
    float *own = nullptr, *own_stat = nullptr;
    // [3] ranges that the prefix's kernel has cut its tiles into: ctas, or fewer where that leaves SMs to the
    // own tokens' split kernel (share); the latter's; released by the prefix's kernel once it has waited for
    // whatever wrote the call's arguments, acquired by the own tokens' (its value means nothing).
    int *ranges = nullptr;
    bool share = false;
};

struct PagedDecodeArgs {
    const void *q;                 // [B, H, D] (fp32 where q_f32), q_stride elements a request
    int64_t q_stride;
    const void *k, *v;             // [pages, Hkv, page_size, D]
    int64_t k_page_stride, v_page_stride;  // elements
    const int32_t *block_table;    // [B, table_stride]
    const int32_t *seq_lens;       // [B]
    int table_stride, max_tokens;  // max_tokens: capacity of a table row in tokens
    int num_pages, page_size;
    int batch, num_heads, num_kv_heads, group, head_dim;
    float scale_log2;              // softmax scale times log2(e)
    void *out;                     // [B, H, D]
    float *lse;                    // [B, H] or nullptr
    float *workspace;              // [kPagedCtas][2][rows][D + 2]
    cudaStream_t stream;
    int head_groups = 1;           // units a key-value head is cut into (set by the launcher)
    const int32_t *chosen = nullptr;  // [B, Hkv, chosen_count] blocks of the request
    int chosen_count = 0;
    PrefixPieces prefix;
};

// CTAs the work of the paged attention is divided among (two per SM), and
// the most query heads of one unit.
constexpr int kPagedCtas = 152 * 2;
constexpr int kPagedMaxRows = 16;

cudaError_t paged_decode(const PagedDecodeArgs &a, bool bf16, bool q_f32);

cudaError_t paged_sparse_decode(const PagedDecodeArgs &a, bool bf16);

// Tokens of a tile of a shared prefix on the tensor cores, whose CTAs take an SM each.
constexpr int kPrefixTile = 128;
constexpr int kPrefixCtas = 152;
// The tensor-core kernel over the prefix (bf16): a.block_table is the prefix's, a.prefix as
// paged_prefix_pieces has it.
cudaError_t paged_prefix_tc(const PagedDecodeArgs &a);
// Reads and clears its device error word (the caller has synchronised the stream).
cudaError_t take_prefix_device_error(unsigned int *err);

// The split of a shared prefix (all but len, max_tokens and pieces), and the attention behind it:
// a.prefix is complete.
PrefixPieces paged_prefix_pieces(int64_t batch, int64_t num_heads, int64_t num_kv_heads, bool bf16);
cudaError_t paged_prefix_decode(const PagedDecodeArgs &a, const int32_t *prefix_table, bool bf16);

// Bounds of the pages' keys: [pages, Hkv, 2, D], the minimum of every channel, then the maximum.
struct PagedBoundsArgs {
    const void *k;                 // [pages, Hkv, page_size, D]
    void *bounds;
    int64_t k_page_stride, bounds_page_stride;  // elements
    const int32_t *block_table;    // [B, table_stride]
    const int32_t *first, *seq_lens;  // [B]: the new tokens are first .. seq_lens - 1
    int table_stride, table_width, max_tokens;
    int num_pages, page_size;
    int batch, num_kv_heads, head_dim;
    cudaStream_t stream;
};

cudaError_t paged_bounds(const PagedBoundsArgs &a, bool bf16);

struct PagedSelectArgs {
    const void *q;                 // [B, H, D], q_stride elements a request
    int64_t q_stride;
    const void *bounds;
    int64_t bounds_page_stride;
    const int32_t *block_table;    // [B, table_stride]
    const int32_t *seq_lens;       // [B]
    int table_stride, table_width, max_tokens;
    int num_pages, page_size;
    int batch, num_kv_heads, group, head_dim;
    int count, keep_first, keep_last;
    int32_t *selected;             // [B, Hkv, count]
    void *workspace;
    cudaStream_t stream;
};

// Bytes of its workspace, or -1 where they pass 2^62.
int64_t paged_select_workspace(int64_t batch, int64_t num_kv_heads, int64_t table_width);
cudaError_t paged_select(const PagedSelectArgs &a, bool bf16);

struct PagedReserveArgs {
    int32_t *block_table;          // [B, table_stride]
    int table_stride, table_width, batch;
    const int32_t *seq_lens, *new_lens;
    const uint8_t *finished;       // [B] or nullptr
    int32_t *free_pages;
    const int32_t *free_count;
    int num_pages, page_size, num_tokens;
    int32_t *slots, *positions, *cu_seqlens;
    uint8_t *served;
    int32_t *seq_lens_out, *free_count_out;
    cudaStream_t stream;
};

constexpr int kReserveMaxBatch = 8192;

cudaError_t paged_reserve(const PagedReserveArgs &a);

}  // namespace la
