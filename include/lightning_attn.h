/*
 * lightning_attn.h -- C ABI of the GB300 (sm_103a) lightning-attention library
 * (liblightning_attn.so).
 *
 * The operation (MiniMax-01 technical report, CSDN full translation, §2.2.1
 * "Lightning Attention", eqs. 4-5, with the per-head diagonal decay of the
 * Fig. 12 caption): for every sequence and head h, with lambda = decay[h],
 *
 *     o_t = sum_{u <= t} lambda^(t-u) (q_t . k_u) v_u            (left product)
 *         = q_t kv_t,  kv_t = lambda kv_{t-1} + k_t^T v_t,  kv_{-1} = 0
 *                                                         (right product)
 *
 * computed chunkwise: inside a chunk the masked left product
 * [(Q_i K_i^T) (.) M] V_i, across chunks the right product through a d x d
 * state carried on chip (§2.2.1 "intra-block" / "inter-block").  Packed
 * variable-length batches follow §3.2 ("data packing"): each sequence starts
 * from a zero state.  Decode is the recursion applied to one new token per
 * sequence, updating a cached state in place (§3.3.1 fused decode KV update,
 * §3.3.2 separate prefill and decode kernels).
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     allocates no device memory and keeps no per-call state.
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL means
 *     the legacy default stream).  Calls never synchronise; results are ready
 *     when the stream reaches that point.
 *   - Argument errors are detected on the host before anything is launched
 *     and return LA_ERR_INVALID_ARG / LA_ERR_UNSUPPORTED with nothing written.
 *     A failed launch returns LA_ERR_CUDA.  Errors that only the GPU can see
 *     (e.g. a cu_seqlens array that is not monotone) are not checked: results
 *     are then unspecified but every access stays inside the buffers whose
 *     sizes the arguments state.
 *   - Every pointer must be 16-byte aligned.  Outputs must not alias inputs.
 *   - No C++ exception crosses this boundary.
 *   - lightning_attn_last_error() returns a human-readable reason for the
 *     last non-LA_OK status returned on the calling host thread.
 */
#ifndef LIGHTNING_ATTN_H
#define LIGHTNING_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum la_status {
    LA_OK = 0,
    LA_ERR_INVALID_ARG = 1,   /* null / misaligned pointer, bad size or dtype */
    LA_ERR_UNSUPPORTED = 2,   /* valid request the library has no kernel for */
    LA_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed          */
    LA_ERR_TIMEOUT = 4        /* reserved: a bounded device-side wait gave up  */
} la_status;

typedef enum la_dtype {
    LA_DTYPE_BF16 = 0,        /* q, k, v, out are bf16; fp32 accumulation */
    LA_DTYPE_FP32 = 1         /* q, k, v, out are fp32; fp32 FFMA throughout */
} la_dtype;

/*
 * Chunkwise prefill over a packed batch of sequences.
 *   (MiniMax-01 report §2.2.1 block split; §3.2 data packing; §3.3.1 fused
 *    prefill preprocessing -- here the tile staging and the decay values are
 *    produced inside the kernel.)
 *
 * q, k, v      [total_tokens, num_heads, head_dim], dtype `dtype`, row-major;
 *              token-major packed: sequence s owns rows
 *              [cu_seqlens[s], cu_seqlens[s+1]).
 * decay        [num_heads] fp32, lambda_h, each in (0, 1] (not checked here:
 *              this entry point does not read device memory on the host;
 *              values outside give the formula's value, possibly inf/nan.
 *              The Python binding checks the range before the call).
 * cu_seqlens   [num_seqs + 1] int32 DEVICE array, cu_seqlens[0] = 0,
 *              non-decreasing, cu_seqlens[num_seqs] = total_tokens.  Empty
 *              sequences are allowed (their final state is zero).
 * num_seqs     >= 0 (0: nothing is done).
 * total_tokens >= 0.
 * num_heads    >= 1.
 * head_dim     64 or 128.
 * chunk        block size B: 0 picks the default for the path
 *              (128 on the tensor-core path, 64 otherwise).  The
 *              tensor-core path (bf16, head_dim 128) takes 16, 32, 64, 128
 *              or 256 (its tiles are 128 tokens; a smaller block runs as
 *              masked tiles advancing B tokens, at 128 / B times the
 *              tensor-core work; a 256-token block as two tiles whose
 *              coupling term goes through the state after the first, the
 *              same sum regrouped); the fp32 / head_dim 64 CUDA-core path
 *              takes 16, 32 or 64 (128 and 256: LA_ERR_UNSUPPORTED).  The
 *              result does
 *              not depend on B beyond rounding (K3 report reading notes, CP
 *              for linear attention: any chunk split is mathematically
 *              equivalent).
 * dtype        LA_DTYPE_BF16 or LA_DTYPE_FP32.
 * out          [total_tokens, num_heads, head_dim], dtype `dtype`: o_t.
 * final_state  nullable; [num_seqs, num_heads, head_dim, head_dim] fp32:
 *              final_state[s][h][i][j] = sum_u lambda_h^(L_s-1-u) k_u[i] v_u[j]
 *              (the state after the last token of sequence s, i.e. the prefix
 *              cache a following decode step continues from).
 * stream       cudaStream_t as void*.
 */
la_status lightning_attn_prefill(const void *q, const void *k, const void *v,
                                 const float *decay, const int32_t *cu_seqlens,
                                 int32_t num_seqs, int32_t total_tokens,
                                 int32_t num_heads, int32_t head_dim,
                                 int32_t chunk, la_dtype dtype, void *out,
                                 float *final_state, void *stream);

/*
 * Prefill that continues every sequence from a cached state (the prefix KV
 * cache of MiniMax-01 report §3.3.1: a new segment of a sequence whose
 * earlier tokens were already consumed into a d x d state).  With S0 =
 * initial_state[s][h] the recursion starts at kv_{-1} = S0, so
 *
 *     o_t = sum_{u <= t} lambda^(t-u) (q_t . k_u) v_u + lambda^(t+1) q_t S0
 *     final_state = lambda^L S0 + sum_u lambda^(L-1-u) k_u^T v_u
 *
 * (the result of one prefill over the earlier tokens and this segment
 * together).  Arguments are those of lightning_attn_prefill plus
 *
 * initial_state  nullable; [num_seqs, num_heads, head_dim, head_dim] fp32,
 *                same layout as final_state; NULL means zero states (then
 *                the call equals lightning_attn_prefill).  It may be the
 *                same array as final_state (the cache is updated in place:
 *                every state is read before it is overwritten); any other
 *                overlap of the two is rejected with LA_ERR_INVALID_ARG.  An
 *                empty sequence's final state is its initial state.
 */
la_status lightning_attn_prefill_with_state(const void *q, const void *k, const void *v,
                                            const float *decay, const int32_t *cu_seqlens,
                                            int32_t num_seqs, int32_t total_tokens,
                                            int32_t num_heads, int32_t head_dim,
                                            int32_t chunk, la_dtype dtype,
                                            const float *initial_state, void *out,
                                            float *final_state, void *stream);

/*
 * Prefill that also keeps the state at every block boundary: the prefix cache
 * of a linear-attention layer kept once per block of tokens (K3 report notes
 * on the inference engine: storing every step's state would give up linear
 * attention's advantage, storing none gives no prefix reuse, so one cache
 * entry per block).  Arguments and results are those of
 * lightning_attn_prefill_with_state, plus
 *
 * snapshot_interval  tokens per block, > 0 and a multiple of the block the
 *                    call computes with (the chunk; for chunk 0, 128 on the
 *                    tensor-core path -- bf16, head_dim 128 -- and 64
 *                    otherwise); LA_ERR_INVALID_ARG otherwise.
 * snapshots          [N, num_heads, head_dim, head_dim] fp32 device array,
 *                    16-byte aligned, N = lightning_attn_snapshot_count(...)
 *                    of the same cu_seqlens (host copy).  Sequence s owns
 *                    entries [b_s, b_s + floor(L_s / snapshot_interval)) with
 *                    b_s = sum_{s' < s} floor(L_s' / snapshot_interval); entry
 *                    b_s + j holds the state after the first
 *                    (j + 1) * snapshot_interval tokens of s -- the final_state
 *                    a prefill of those tokens alone (from the same initial
 *                    state) returns.  A trailing partial block gets none.
 */
la_status lightning_attn_prefill_snapshots(const void *q, const void *k, const void *v,
                                           const float *decay, const int32_t *cu_seqlens,
                                           int32_t num_seqs, int32_t total_tokens,
                                           int32_t num_heads, int32_t head_dim, int32_t chunk,
                                           la_dtype dtype, const float *initial_state, void *out,
                                           float *final_state, int32_t snapshot_interval,
                                           float *snapshots, void *stream);

/* Number of snapshots lightning_attn_prefill_snapshots writes for these
 * sequences (host copy of cu_seqlens, num_seqs + 1 entries): the sum of
 * floor(L_s / snapshot_interval).  -1 for invalid arguments. */
int64_t lightning_attn_snapshot_count(const int32_t *cu_seqlens_host, int32_t num_seqs,
                                      int32_t snapshot_interval);

/*
 * Prefill with a channel-wise decay: one lambda per head and KEY channel
 * (K3 report reading notes: the scalar decay generalised to a channel-wise
 * one that can fall back to the uniform decay; it acts on the channels Q and
 * K share).  With lam_i = decay[h * head_dim + i] the state recursion is
 *     kv_t[i][j] = lam_i kv_{t-1}[i][j] + k_t[i] v_t[j],   o_t = q_t kv_t
 * i.e. o_t = sum_{u <= t} (sum_i q_t[i] k_u[i] lam_i^(t-u)) v_u
 *            + sum_i q_t[i] lam_i^(t+1) S0[i][:]  (from a cached state S0).
 * Arguments as for lightning_attn_prefill_with_state, except
 *   decay  [num_heads, head_dim] fp32, each in (0, 1].
 * Kernels: bf16 with head_dim 128 and chunk 0 or 64 runs the tensor-core
 * kernel (64-token blocks; intra-block scores from 16-token sub-blocks whose
 * decay factors are split between the query and key sides, every operand a
 * hi/lo bf16 pair but the key side of the off-diagonal scores).  For its
 * diagonal sub-blocks lambda is raised to 2^-12 where smaller: a score term
 * at distance 1..15 then moves by less than 2^-12 |q_t[i] k_u[i]|.  Those
 * factors reach mu_i^-8 on the query side and mu_i^-7 on the key side, with
 * mu_i = max(lambda_i, 2^-12), so the kernel needs |q_t[i]| mu_i^-8 and
 * |k_u[i]| mu_i^-7 below the bf16 maximum (about 3.4e38): always true for
 * |q| < 2^32 and |k| < 2^44.  Every other case
 * runs the CUDA-core (FFMA) kernel: chunk 0 (= 64), 16, 32 or 64 (fp32, or
 * head_dim 64); 128 and 256 return LA_ERR_UNSUPPORTED.
 */
la_status lightning_attn_prefill_channel_decay(const void *q, const void *k, const void *v,
                                               const float *decay, const int32_t *cu_seqlens,
                                               int32_t num_seqs, int32_t total_tokens,
                                               int32_t num_heads, int32_t head_dim, int32_t chunk,
                                               la_dtype dtype, const float *initial_state,
                                               void *out, float *final_state, void *stream);

/*
 * Decode step with a channel-wise decay (decay [num_heads, head_dim]):
 *     state[b][h][i][j] <- lam_i state[b][h][i][j] + k[i] v[j],  out = q state.
 * Other arguments as for lightning_attn_decode.
 */
la_status lightning_attn_decode_channel_decay(const void *q, const void *k, const void *v,
                                              const float *decay, float *state, int32_t batch,
                                              int32_t num_heads, int32_t head_dim,
                                              la_dtype dtype, void *out, void *stream);

/*
 * One decode step for a batch of sequences, each with one new token.
 *   (MiniMax-01 report §3.3.2: length-1 inputs get their own memory-bound
 *    kernel; §3.3.1: the KV computation and the prefix-KV-cache update are
 *    fused into one kernel.)
 *
 * For every b < batch, h < num_heads, with lambda = decay[h]:
 *     state[b][h] <- lambda * state[b][h] + k[b][h]^T v[b][h]     (in place)
 *     out[b][h]    = q[b][h] . state[b][h]                 (after the update)
 *
 * q, k, v, out [batch, num_heads, head_dim], dtype `dtype`.
 * decay        [num_heads] fp32.
 * state        [batch, num_heads, head_dim, head_dim] fp32, read and written.
 * batch >= 0 (0: nothing is done), num_heads >= 1, head_dim 64 or 128.
 */
la_status lightning_attn_decode(const void *q, const void *k, const void *v,
                                const float *decay, float *state,
                                int32_t batch, int32_t num_heads,
                                int32_t head_dim, la_dtype dtype, void *out,
                                void *stream);

/*
 * Gradients for training (MiniMax-01 report §2.2.1; §2.2.2 measures the
 * training speed of lightning attention): given dout = dL/do for the outputs
 * of lightning_attn_prefill on the same arguments (zero initial states),
 *
 *     dq_t = sum_{u <= t} lambda^(t-u) (dout_t . v_u) k_u
 *     dk_u = sum_{t >= u} lambda^(t-u) (dout_t . v_u) q_t
 *     dv_u = sum_{t >= u} lambda^(t-u) (q_t . k_u) dout_t
 *
 * per sequence and head.  dq is the forward form applied to (dout, v, k);
 * dk and dv are anti-causal forms (sums over t >= u).  On the tensor-core
 * path (bf16, head_dim 128, chunk 0-128) the call makes three launches of
 * the prefill kernel, one causal and two anti-causal, and does not touch
 * `workspace`; on the CUDA-core path it runs the forward form in reversed
 * time, with four time-reversal copies through `workspace`.  Same dtype /
 * head_dim / chunk rules and precision as lightning_attn_prefill.
 *
 * q, k, v, d_out          [total_tokens, num_heads, head_dim], dtype `dtype`
 * d_q, d_k, d_v           outputs, same shape and dtype; distinct arrays,
 *                         none of them equal to an input
 * workspace               caller-owned device memory, 256-byte aligned, of at
 *                         least lightning_attn_backward_workspace_bytes(...)
 *                         bytes; its contents are scratch (overwritten).  Not
 *                         used on the tensor-core path, where it may be NULL
 *                         with workspace_bytes 0.
 * other arguments         as for lightning_attn_prefill.
 * Gradients with respect to decay, to a cached initial state or from a
 * final-state loss are not computed.
 */
la_status lightning_attn_backward(const void *q, const void *k, const void *v,
                                  const float *decay, const int32_t *cu_seqlens,
                                  int32_t num_seqs, int32_t total_tokens, int32_t num_heads,
                                  int32_t head_dim, int32_t chunk, la_dtype dtype,
                                  const void *d_out, void *d_q, void *d_k, void *d_v,
                                  void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace lightning_attn_backward needs (three [T, H, d] arrays,
 * each rounded up to 256 bytes); -1 for invalid arguments. */
int64_t lightning_attn_backward_workspace_bytes(int32_t total_tokens, int32_t num_heads,
                                                int32_t head_dim, la_dtype dtype);

/*
 * lightning_attn_backward without a caller workspace (the paper has no
 * counterpart; this is a convenience of this library).  For callers that
 * cannot allocate device memory at call time -- code under another
 * framework's memory manager that forbids raw cudaMalloc, or a loop that
 * must not call cudaMalloc because it can synchronise the device -- the
 * scratch comes from one fixed array of lightning_attn_backward_noalloc_max_bytes()
 * bytes (64 MiB) that every GPU loading the library holds until the process
 * exits.  Arguments and results are those of lightning_attn_backward.  On the
 * tensor-core path (bf16, head_dim 128, chunk 0-128) no scratch is used
 * and no size limit applies; otherwise a call whose
 * lightning_attn_backward_workspace_bytes() exceeds the array returns
 * LA_ERR_INVALID_ARG before touching the GPU (argument errors, empty calls
 * and unsupported block sizes are reported first, exactly as by
 * lightning_attn_backward).  The first call on a device looks up the array's
 * device address (cudaGetSymbolAddress) with that device current, and so does
 * the first call after the device's context has been destroyed and made
 * again (cudaDeviceReset); make such a call before any stream capture.  The
 * array is shared by all calls: calls that overlap on the GPU race on it;
 * calls ordered on one stream do not.  Nothing is allocated.
 */
la_status lightning_attn_backward_noalloc(const void *q, const void *k, const void *v,
                                          const float *decay, const int32_t *cu_seqlens,
                                          int32_t num_seqs, int32_t total_tokens,
                                          int32_t num_heads, int32_t head_dim, int32_t chunk,
                                          la_dtype dtype, const void *d_out, void *d_q,
                                          void *d_k, void *d_v, void *stream);

/* Size in bytes of the fixed scratch array of lightning_attn_backward_noalloc. */
int64_t lightning_attn_backward_noalloc_max_bytes(void);

/*
 * One serving step over a packed batch in which every sequence continues from
 * its cached state (MiniMax-01 report §3.3.2: inputs of length 1 and of
 * length > 1 get separate kernels on separate CUDA streams; §3.3.1 prefix KV
 * cache).  For every sequence s with L_s = cu_seqlens[s+1] - cu_seqlens[s]
 * new tokens, the result is that of lightning_attn_prefill_with_state with
 * initial_state = final_state = state:
 *   L_s == 1: the decode step (kv <- lambda kv + k^T v, o = q kv) on
 *             decode_stream;
 *   L_s >= 2: the chunkwise prefill on prefill_stream, state updated in place;
 *   L_s == 0: nothing (the state is unchanged).
 * Both launches read cu_seqlens on the device, so no host copy of the lengths
 * is needed.  The decode launch waits for the work already queued on
 * prefill_stream and prefill_stream waits for the decode launch before its
 * next work, so the whole step is ordered on prefill_stream (two events per
 * device are created on first use for this fork and join; calls from
 * several host threads are serialised while they enqueue).  With
 * decode_stream == prefill_stream the two launches simply run one after the
 * other.  A decode_stream of higher priority than prefill_stream lets the
 * decode kernel's small blocks start before the prefill's large ones occupy
 * the SMs (measured: 20 sequences x 64 heads, 2 with 50 new tokens, 45 ->
 * 37 us).  chunk is the path's default; dtype rules as for prefill.
 *
 * q, k, v, out    [total_tokens, num_heads, head_dim], dtype `dtype`
 * state           [num_seqs, num_heads, head_dim, head_dim] fp32, read and written
 * cu_seqlens_host nullable HOST copy of cu_seqlens.  When given (and
 *                 num_seqs <= 128) the prefill launch covers only the
 *                 sequences with >= 2 new tokens; without it every sequence
 *                 gets prefill CTAs that exit at once for the short ones.
 */
la_status lightning_attn_mixed_step(const void *q, const void *k, const void *v,
                                    const float *decay, const int32_t *cu_seqlens,
                                    int32_t num_seqs, int32_t total_tokens, int32_t num_heads,
                                    int32_t head_dim, la_dtype dtype, float *state, void *out,
                                    const int32_t *cu_seqlens_host, void *prefill_stream,
                                    void *decode_stream);

/* ------------------------------------------------------------------------
 * Softmax layers of a hybrid stack (one such layer after every seven lightning
 * layers in MiniMax-01): the operators a serving step needs around their paged
 * key-value cache, and the per-head norm with the position rotation that
 * precedes either kind of attention, with its gradients.
 *
 * Common to these calls
 *   - Row strides (q_stride, ...) are in ELEMENTS, from one token's heads to
 *     the next; a token's [heads, head_dim] block is contiguous.  Slices of one
 *     fused projection output are therefore taken as they are.  Strides and
 *     pointers of floating-point arrays are multiples of 16 bytes; int32 and
 *     byte arrays need their natural alignment only.
 *   - rotary  [rotary_rows, rotary_dim] fp32: row p holds the rotary_dim / 2
 *             cosines and then the rotary_dim / 2 sines of position p.
 *             rotary_dim is a multiple of 16 up to head_dim; 0 (rotary and
 *             positions NULL) means no rotation.
 *   - interleaved  0: element i is rotated with element i + rotary_dim / 2;
 *             1: element 2 i with element 2 i + 1.  Elements from rotary_dim on
 *             are not rotated.
 *   - positions [num_tokens] int32; values outside the table are clamped to it.
 *   - q_weight, k_weight [head_dim] fp32, shared by the heads; both NULL: no norm.
 *   - A key-value cache is two arrays [num_pages, num_kv_heads, page_size,
 *             head_dim]; k_page_stride and v_page_stride are the elements from
 *             one page to the next (>= num_kv_heads * page_size * head_dim), so
 *             the two may be halves of one array.  Slot s is row s % page_size
 *             of page s / page_size; num_pages * page_size < 2^31.  page_size
 *             is any number >= 1.
 *   - dtype of q, k, v, the cache and the outputs is LA_DTYPE_BF16 or
 *             LA_DTYPE_FP32; head_dim 64 or 128.  Arithmetic and sums are fp32
 *             (squares too: a norm's elements up to about 10^19), rounded once
 *             into an output.  One exception: over a bf16 cache the softmax
 *             weights, and the queries of lightning_attn_paged_step, enter the
 *             products as two bf16 numbers, off by at most 2^-16 of each.
 * ------------------------------------------------------------------------ */

/*
 * RMS norm over each query and key head and the position rotation, in one pass:
 *     n = x (mean(x^2) + eps)^-1/2 weight,   y = R(position) n
 *
 * q [num_tokens, num_heads, head_dim], k [num_tokens, num_kv_heads, head_dim];
 * q_out, k_out likewise (contiguous, or strided).  q_out may be q and k_out may
 * be k (with the same stride); no other overlap is allowed.  num_kv_heads = 0
 * (k and k_out NULL) processes the queries alone.
 */
la_status lightning_attn_qk_norm_rope(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
    const float *rotary, int32_t rotary_rows, int32_t rotary_dim, int32_t interleaved,
    const float *q_weight, const float *k_weight, float eps, int32_t num_tokens,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype, void *q_out,
    int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream);

/*
 * Gradients of lightning_attn_qk_norm_rope: given d_q_out and d_k_out (gradients
 * of its outputs) and its inputs, with g = R^T dy and r = (mean(x^2) + eps)^-1/2
 *     dx = r (weight g - x r mean(weight g x r)),   d_weight = sum_rows g x r
 * d_q and d_k (dtype `dtype`) may be the arrays of d_q_out and d_k_out.
 * d_q_weight, d_k_weight [head_dim] fp32 (overwritten; NULL when there are no
 * weights).  workspace: lightning_attn_qk_norm_rope_workspace_bytes(head_dim)
 * bytes, 16-byte aligned, not shared by calls that may overlap (not used, and may
 * be NULL, without weights).  The sums are taken in a fixed order: the same
 * call gives the same bits.
 */
la_status lightning_attn_qk_norm_rope_backward(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
    const float *rotary, int32_t rotary_rows, int32_t rotary_dim, int32_t interleaved,
    const float *q_weight, const float *k_weight, float eps, int32_t num_tokens,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype,
    const void *d_q_out, int64_t d_q_out_stride, const void *d_k_out, int64_t d_k_out_stride,
    void *d_q, int64_t d_q_stride, void *d_k, int64_t d_k_stride, float *d_q_weight,
    float *d_k_weight, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lightning_attn_qk_norm_rope_backward; -1 for an
 * invalid head_dim. */
int64_t lightning_attn_qk_norm_rope_workspace_bytes(int32_t head_dim);

/*
 * lightning_attn_qk_norm_rope whose keys, and the values as they are, go into
 * the cache: row t of k (normed and rotated) and v into slot slots[t].  A slot
 * outside [0, num_pages * page_size) (e.g. -1, a padding token) writes no
 * cache row; the slots of one call are otherwise distinct.
 */
la_status lightning_attn_paged_append(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
    int64_t v_stride, const int32_t *positions, const float *rotary, int32_t rotary_rows,
    int32_t rotary_dim, int32_t interleaved, const float *q_weight, const float *k_weight,
    float eps, int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    la_dtype dtype, void *q_out, int64_t q_out_stride, void *k_cache, int64_t k_page_stride,
    void *v_cache, int64_t v_page_stride, const int32_t *slots, int32_t num_pages,
    int32_t page_size, void *stream);

/*
 * Softmax attention of one new token per request over the paged cache:
 *     out[b][h] = sum_t p_t v_t,  p = softmax_t(scale q[b][h] . k_t),
 * over the first seq_lens[b] tokens of request b (its new token among them), keys
 * and values of head h / (num_heads / num_kv_heads).
 *
 * q            [batch, num_heads, head_dim] (row stride q_stride).
 * block_table  [batch, table_width] int32, table_stride elements a row: token t of
 *              request b is row t % page_size of page block_table[b][t / page_size].
 *              Entries past a request's last block are not read; a page outside
 *              [0, num_pages) leaves its tokens out of the softmax.
 * seq_lens     [batch] int32; negative counts as 0, more than table_width *
 *              page_size as that.  A request with no token (or none left) gets
 *              zeros, and -infinity as its lse; one whose scores are all -infinity
 *              NaN, with the same lse.
 * scale        softmax scale (e.g. head_dim^-1/2).
 * out          [batch, num_heads, head_dim], contiguous; may be q where that is, too.
 * lse          nullable; [batch, num_heads] fp32: log sum_t e^(scale q . k_t).
 * workspace    lightning_attn_paged_decode_workspace_bytes(head_dim) bytes,
 *              16-byte aligned; scratch, not shared by calls that may overlap
 *              (two captured graphs that may run at once need one each).
 * num_heads is a multiple of num_kv_heads.  What lies in the cache past a
 * request's last token is not used, whatever it holds.  Infinities that are
 * attended to count as the formula has it: a score of -infinity has weight 0, one
 * of +infinity (or NaN) makes the head's row and lse NaN, an infinite value makes its
 * column that infinity, or NaN where both signs meet or where its weight is 0 or
 * less than 2^-100 of the largest.
 */
la_status lightning_attn_paged_decode(
    const void *q, int64_t q_stride, const void *k_cache, int64_t k_page_stride,
    const void *v_cache, int64_t v_page_stride, const int32_t *block_table, int32_t table_stride,
    int32_t table_width, const int32_t *seq_lens, int32_t num_pages, int32_t page_size,
    int32_t batch, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype,
    float scale, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lightning_attn_paged_decode; -1 for an invalid
 * head_dim. */
int64_t lightning_attn_paged_decode_workspace_bytes(int32_t head_dim);

/*
 * One serving step of a softmax layer: lightning_attn_paged_append of each
 * request's new token (row b of q, k, v), then lightning_attn_paged_decode over
 * the cache that now holds it.  The normed and rotated queries pass between the
 * two in fp32 (in the workspace; see above for their products), so out is rounded
 * once.  seq_lens counts the
 * new tokens.  workspace: lightning_attn_paged_step_workspace_bytes(...) bytes,
 * 16-byte aligned.
 */
la_status lightning_attn_paged_step(
    const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
    int64_t v_stride, const int32_t *positions, const float *rotary, int32_t rotary_rows,
    int32_t rotary_dim, int32_t interleaved, const float *q_weight, const float *k_weight,
    float eps, void *k_cache, int64_t k_page_stride, void *v_cache, int64_t v_page_stride,
    const int32_t *slots, const int32_t *block_table, int32_t table_stride, int32_t table_width,
    const int32_t *seq_lens, int32_t num_pages, int32_t page_size, int32_t batch,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype, float scale,
    void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lightning_attn_paged_step; -1 for invalid sizes. */
int64_t lightning_attn_paged_step_workspace_bytes(int32_t batch, int32_t num_heads,
                                                  int32_t head_dim);

/*
 * Long contexts: attention over a few pages of the cache that are chosen by a cheap score.
 *
 * lightning_attn_paged_bounds keeps, for every page and key-value head, the smallest and the
 * largest value of each channel of the page's keys, as they enter the cache.
 * bounds is [num_pages, num_kv_heads, 2, head_dim], minima then maxima, in the cache's dtype (and so
 * exact; bounds_page_stride elements from one page to the next).  Tokens
 * first[b] .. seq_lens[b] - 1 of request b are new: bounds of a block that begins among them are
 * written, those of the block that begins before them (first[b] inside it) are extended, all others stay.
 * After tokens of a block have been replaced, its bounds are taken anew with first[b]
 * at its beginning.  Values outside [0, table_width * page_size] are clamped to it; nothing is
 * done for a request without new tokens, nor for a block whose page is outside [0, num_pages).  The
 * blocks with new tokens lie in distinct pages.  A NaN key makes both bounds of its channel NaN.
 */
la_status lightning_attn_paged_bounds(
    const void *k_cache, int64_t k_page_stride, void *bounds, int64_t bounds_page_stride,
    const int32_t *block_table, int32_t table_stride, int32_t table_width, const int32_t *first,
    const int32_t *seq_lens, int32_t num_pages, int32_t page_size, int32_t batch,
    int32_t num_kv_heads, int32_t head_dim, la_dtype dtype, void *stream);

/*
 * Chooses `count` blocks of every request and key-value head.  The score of a block is
 *     max over the heads h that share the key-value head of  sum_d max(q_hd lo_d, q_hd hi_d),
 * which no q_h . k of the block exceeds; as by arithmetic in 64 bits on these inputs, however
 * near two scores are.  Equal scores go to the lower block, NaN counts as infinity.
 *
 * q            [batch, num_heads, head_dim] (row stride q_stride), as for the attention.
 * bounds       as lightning_attn_paged_bounds keeps them, for all blocks of the requests.
 * keep_first, keep_last  the first and the last blocks of a request that are chosen whatever their
 *              scores; together at most count.
 * selected     [batch, num_kv_heads, count] int32: the chosen blocks (indices into the request's
 *              row of block_table) in ascending order, then -1 where the request has fewer.  No other
 *              argument's array.
 *              Blocks whose page is outside [0, num_pages) are not chosen.
 * workspace    lightning_attn_paged_select_workspace_bytes(...) bytes, 16-byte aligned; scratch, not
 *              shared by calls that may overlap.
 */
la_status lightning_attn_paged_select(
    const void *q, int64_t q_stride, const void *bounds, int64_t bounds_page_stride,
    const int32_t *block_table, int32_t table_stride, int32_t table_width, const int32_t *seq_lens,
    int32_t num_pages, int32_t page_size, int32_t batch, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, la_dtype dtype, int32_t count, int32_t keep_first, int32_t keep_last,
    int32_t *selected, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lightning_attn_paged_select; -1 for invalid sizes. */
int64_t lightning_attn_paged_select_workspace_bytes(int32_t batch, int32_t num_kv_heads,
                                                    int32_t table_width);

/*
 * lightning_attn_paged_decode over the tokens of chosen blocks alone.
 *
 * selected     [batch, num_kv_heads, count] int32, blocks of the request (in any order); of a row the
 *              first min(count, ceil(seq_lens[b] / page_size)) entries count.  An entry outside
 *              the request's blocks stands for no tokens, one that is there twice for its tokens twice.
 * The rest is as for lightning_attn_paged_decode (the workspace too); a head whose choice holds no token
 * gets zeros and an lse of -infinity.  count * page_size is at most 2^31 - 2^16 (LA_ERR_UNSUPPORTED).
 */
la_status lightning_attn_paged_sparse_decode(
    const void *q, int64_t q_stride, const void *k_cache, int64_t k_page_stride,
    const void *v_cache, int64_t v_page_stride, const int32_t *block_table, int32_t table_stride,
    int32_t table_width, const int32_t *seq_lens, const int32_t *selected, int32_t count,
    int32_t num_pages, int32_t page_size, int32_t batch, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, la_dtype dtype, float scale, void *out, float *lse, void *workspace,
    int64_t workspace_bytes, void *stream);

/*
 * lightning_attn_paged_decode where the requests share a prefix (a system prompt, a document):
 * request b attends to the first prefix_len[0] tokens of the prefix's pages and to the first
 * seq_lens[b] tokens of its own, and the prefix's keys and values are read for the batch as a whole.
 * With 64 query and 8 key-value heads of 128 in bf16 that is faster than lightning_attn_paged_decode over tables
 * that name the prefix's pages (its length a multiple of page_size) from 16 requests behind 2K tokens, 8 behind
 * 8K, 4 behind 32K or 2 behind 128K; for fewer it is slower (4 behind 2K 17 us instead of 10).
 *
 * prefix_table [prefix_width] int32, prefix_len [1] int32: as a row of block_table and its length.
 * block_table, seq_lens  the requests' own tokens behind the prefix, which begin with a
 *              page of their own; 0 tokens are allowed.  (Both kinds of pages are of one pool;
 *              pages outside [0, num_pages) leave their tokens out.)
 * workspace    lightning_attn_paged_prefix_decode_workspace_bytes(...) bytes, 16-byte aligned;
 *              scratch, not shared by calls that may overlap.
 * The rest, infinities included, is as for lightning_attn_paged_decode; lse is that of all tokens.
 * In bf16 the waits of its pipeline are bounded: lightning_attn_device_status reports one that gave up.
 */
la_status lightning_attn_paged_prefix_decode(
    const void *q, int64_t q_stride, const void *k_cache, int64_t k_page_stride,
    const void *v_cache, int64_t v_page_stride, const int32_t *prefix_table, int32_t prefix_width,
    const int32_t *prefix_len, const int32_t *block_table, int32_t table_stride,
    int32_t table_width, const int32_t *seq_lens, int32_t num_pages, int32_t page_size,
    int32_t batch, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, la_dtype dtype,
    float scale, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lightning_attn_paged_prefix_decode; -1 for invalid sizes. */
int64_t lightning_attn_paged_prefix_decode_workspace_bytes(int32_t batch, int32_t num_heads,
                                                           int32_t num_kv_heads, int32_t head_dim,
                                                           la_dtype dtype);

/*
 * Page bookkeeping of one serving step, from the requests' lengths, on the GPU.
 * In this order:
 *   1. A finished request (finished[b] != 0; finished may be NULL) pushes the
 *      pages of its ceil(seq_lens[b] / page_size) first blocks onto the free
 *      stack, requests and blocks in ascending order, and has length 0 from there on.
 *      The table's entries go as they are, so they have to be pages here.
 *   2. Request b asks for the pages that new_lens[b] more tokens need beyond
 *      those it has.  Requests are served in ascending order: b is served if its
 *      tokens fit its table row, and if it needs no page or the pages needed by
 *      the requests up to b (those that do not fit their row left out) are on the stack.
 *      A served request's new blocks get the pages popped from the top, one
 *      after the other.
 *   3. The new tokens are numbered in the order of the requests, served or not.
 *
 * block_table  [batch, table_width] int32 (table_stride elements a row), updated:
 *              new blocks of served requests.
 * seq_lens     [batch] int32, new_lens [batch] int32 (negative counts as 0).
 * free_pages   [num_pages] int32 stack, free_count [1] its height (entries below
 *              it are free pages); entries pushed in step 1 are written, popped
 *              ones left in place.
 * slots, positions [num_tokens] int32: slot and position (length so far + index)
 *              of every new token; slot -1, position 0 for tokens of requests
 *              not served and for entries past the last new token.  num_tokens is
 *              the arrays' size: tokens past it are not written.
 * cu_seqlens   [batch + 1] int32: first new token of every request, and the total;
 *              2^31 - 1 where that or more come before (past num_tokens: the
 *              other outputs do not depend on it).
 * served       [batch] bytes, 1 or 0.
 * seq_lens_out [batch], free_count_out [1] int32: lengths after the step (a request
 *              not served keeps its length, 0 if it finished) and the stack's
 *              height.  They may be seq_lens and free_count (not new_lens).
 * batch <= 8192 (LA_ERR_UNSUPPORTED above).  Other overlaps are not allowed.
 */
la_status lightning_attn_paged_reserve(
    int32_t *block_table, int32_t table_stride, int32_t table_width, const int32_t *seq_lens,
    const int32_t *new_lens, const uint8_t *finished, int32_t batch, int32_t *free_pages,
    const int32_t *free_count, int32_t num_pages, int32_t page_size, int32_t num_tokens,
    int32_t *slots, int32_t *positions, int32_t *cu_seqlens, uint8_t *served,
    int32_t *seq_lens_out, int32_t *free_count_out, void *stream);

/*
 * Synchronises `stream`, then reports whether a kernel of this library raised
 * its device error word since the last call (and clears it).  The
 * tensor-core kernels (prefill, attention behind a shared prefix) bound every wait of
 * their pipelines (about 2 s); a wait
 * that gives up ends the kernel cleanly (the context stays usable), leaves the
 * outputs of that launch unspecified and makes this call return
 * LA_ERR_TIMEOUT.  Returns LA_ERR_CUDA if the synchronisation fails.
 */
la_status lightning_attn_device_status(void *stream);

/*
 * Failure-detection self test: launches one CTA that waits on a barrier
 * nothing will ever complete, with the same bounded wait the prefill
 * pipeline uses, giving up after timeout_ns.  A following
 * lightning_attn_device_status() must return LA_ERR_TIMEOUT.
 */
la_status lightning_attn_selftest_wait_timeout(uint64_t timeout_ns, void *stream);

/* Static English name of a status code; never NULL. */
const char *lightning_attn_status_string(la_status status);

/* Reason for the last non-OK status on this host thread ("" if none). */
const char *lightning_attn_last_error(void);

/* ABI version of this header: (major << 16) | minor. */
int32_t lightning_attn_version(void);

#define LIGHTNING_ATTN_VERSION ((1 << 16) | 5)

#ifdef __cplusplus
}
#endif

#endif /* LIGHTNING_ATTN_H */
