/*
 * llama_ops.h -- per-step entry points of the decoder block (same kernels the
 * block forward launches), for unit-level parity checks and for callers that
 * compose the steps themselves.  Conventions as in llama_block.h: device
 * pointers, 16-byte alignment, row-major, asynchronous on `stream`, errors
 * returned (nothing enqueued on error).  dtype is LLAMA_F32 or LLAMA_BF16.
 * These entry points allocate nothing and, but for those that take a status
 * pointer, report device-side wait expiry only through their return of later
 * calls' CUDA errors (no status word).
 */
#ifndef LLAMA_OPS_H
#define LLAMA_OPS_H

#include "llama_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* RMSNorm of T rows of width d ("The Evolving Transformer 04 · LLaMA", §03):
 * out[t] = x[t] / sqrt(mean(x[t]^2) + eps) * g.  x, out: [T][d]; g: [d].
 * d must be a multiple of 8 (bf16) or 4 (fp32).  out may alias x. */
llama_status llama_op_rmsnorm(int32_t dtype, const void *x, const void *g, void *out, int32_t T, int32_t d,
                              float eps, llama_stream stream);

/* Linear layer without bias ("The Evolving Transformer 04 · LLaMA", §05: nn.Linear(bias=False)):
 *   epilogue 0: C = A W^T            C [M][N], dtype
 *   epilogue 1: C = R + A W^T        R, C [M][N], dtype (C may alias R)
 *   epilogue 2: C = A W^T            C [M][N], fp32
 * A: [M][K]; W: [N][K].  K must be a multiple of 8.  bf16 runs on the tcgen05
 * tensor cores with fp32 accumulation; fp32 runs on CUDA cores. */
llama_status llama_op_linear(int32_t dtype, const void *A, const void *W, const void *R, void *C, int32_t M,
                             int32_t N, int32_t K, int32_t epilogue, llama_stream stream);

/* Causal grouped-query attention over a KV cache ("The Evolving Transformer 04
 * · LLaMA", §05 GQA; "Full Llama 3 transformer block", How it works):
 * o[b][s][h] = sum_{j <= start_pos + s} softmax_j(q[b][s][h] . K[b][h / (H/G)][j] / sqrt(D)) V[b][h / (H/G)][j].
 * q, o: [B][S][H][D] (q already rotated); kv->k, kv->v: [max_batch][G][max_seq_len][D].
 * Requirements as for llama_block_forward; D in {16, 32, 64, 128}.
 * workspace: caller-owned device scratch of at least
 * llama_op_attention_workspace_bytes(dtype, B, S, start_pos, H, D) bytes
 * (the split-KV partials of the decode path); may be NULL when that is 0. */
size_t llama_op_attention_workspace_bytes(int32_t dtype, int32_t B, int32_t S, int32_t start_pos, int32_t H,
                                          int32_t D);
llama_status llama_op_attention(int32_t dtype, const void *q, const llama_kv_cache *kv, void *o, int32_t B,
                                int32_t S, int32_t start_pos, int32_t H, int32_t G, int32_t D, void *workspace,
                                size_t workspace_bytes, llama_stream stream);

/* RoPE cos/sin table: table[p][i] = {cos(p f_i), sin(p f_i)}, f_i = theta^(-2i/D),
 * p in [0, max_seq), i in [0, D/2), fp32 pairs computed in fp64 ("Mini Llama 2
 * Implementation", Rotary positional embeddings).  table: float[max_seq][D/2][2].
 * scaling_factor > 1 applies the Llama 3.1 stretch to f_i with low_freq_factor,
 * high_freq_factor and original_max_pos exactly as the llama_config fields of the
 * same names describe; scaling_factor <= 1 leaves f_i unscaled (the other three
 * are then ignored). */
llama_status llama_op_rope_table(float *table, int32_t max_seq, int32_t D, float theta, float scaling_factor,
                                 float low_freq_factor, float high_freq_factor, int32_t original_max_pos,
                                 llama_stream stream);

/* RoPE + KV-cache write: qkv [B*S][(H + 2G) D] holds, per token, q (H heads),
 * k (G heads), v (G heads).  Writes q rotated at position start_pos + s to
 * q_out [B*S][H][D], k rotated to kv->k[b][g][start_pos + s], v unrotated to
 * kv->v[b][g][start_pos + s]; nothing else in the cache changes.  layout
 * (llama_rope_layout) picks the pairs rotated together; the vectors keep their
 * natural component order in both layouts.
 * table from llama_op_rope_table with max_seq >= start_pos + S. */
llama_status llama_op_rope_kv_write(int32_t dtype, const void *qkv, void *q_out, const llama_kv_cache *kv,
                                    const float *table, int32_t table_max_seq, int32_t B, int32_t S,
                                    int32_t start_pos, int32_t H, int32_t G, int32_t D, int32_t layout,
                                    llama_stream stream);

/* Decode-step attention that allocates nothing.  The method's pages have no
 * counterpart: this entry point exists for callers that cannot allocate device
 * memory when they run attention (a serving engine whose pool already owns
 * the device memory, an embedded runtime with a fixed budget, code that must
 * not synchronise the device the way cudaMalloc can).
 *
 * Computes the same as llama_op_attention with dtype LLAMA_BF16 and S = 1:
 * q, o: [B][H][D] bf16, kv: bf16 [max_batch][G][max_seq_len][D], keys
 * 0 .. start_pos visible.  The split-KV partial results live in one array of
 * LLAMA_NOALLOC_SCRATCH_BYTES that is part of the library image on every GPU
 * that loads it, held until the process exits; no cudaMalloc / cudaFree or
 * allocating library routine is called.
 *   - Limit: one sequence's partials, H * ceil((start_pos + 1) / 256) *
 *     (D + 2) * 4 bytes, must fit in LLAMA_NOALLOC_SCRATCH_BYTES, else
 *     LLAMA_ERR_RANGE (nothing runs); a single chunk (start_pos < 256) needs
 *     none.  Batches whose partials do not fit run in groups of sequences, one
 *     group after another on the stream, each reusing the array.  With
 *     H = 32 and D = 128 a sequence needs 16,640 bytes per 256 positions:
 *     32 MiB holds one sequence of up to 516,096 cached positions, and B = 64
 *     sequences of 4096 positions in one group.
 *   - D in {64, 128}, n_heads / n_kv_heads <= 8 (LLAMA_ERR_UNSUPPORTED otherwise).
 *   - The first call on a device looks up the array's device address (a
 *     one-time set-up per CUDA context, done with that device current, and
 *     done again after the device's context was reset); make that first call
 *     before any stream capture.
 *   - All calls share the array and every call overwrites the partials it
 *     reads, so nothing needs clearing; calls that may run at the same time on
 *     the GPU (unordered streams) race on the array and must be avoided.
 *   - The kernel's bounded waits (2 s, never reached in normal operation)
 *     have no status word to report to here: if one ran out, the call still
 *     returns LLAMA_OK and o is undefined. */
#define LLAMA_NOALLOC_SCRATCH_BYTES (32u << 20)
llama_status llama_op_attention_decode_noalloc(const void *q, const llama_kv_cache *kv, void *o, int32_t B,
                                               int32_t start_pos, int32_t H, int32_t G, int32_t D,
                                               llama_stream stream);

/* ------------------------------------------------------------------------
 * Batches of sequences of different lengths, over a paged key-value cache.
 *
 * The method's pages run every sequence of a batch at one start_pos over a
 * contiguous cache ("Full Llama 3 transformer block", How it works); the entry
 * points below compute the same RoPE, cache write and grouped-query attention
 * when each sequence has its own length and its keys and values lie in pages.
 * The order of a step is llama_op_rope_kv_write_paged, then
 * llama_op_attention_packed (prompts, continued prompts, mixed batches) or
 * llama_op_attention_paged_decode (one new token per sequence).
 *
 * Device status: lengths, offsets and page ids live on the device, where the
 * host cannot check them before the launch.  Each of these entry points takes
 * status, a device int32 that the caller has set to 0 (or NULL): the first
 * problem that a kernel meets is stored there as a llama_status and the call
 * goes on as described below; nothing is read or written out of range.
 *
 * Every pointer belongs to the device that is current (LLAMA_ERR_INVALID_ARG
 * otherwise).  q_offsets, kv_lens, page_table and status need the alignment of
 * their elements only, the rest 16 bytes (LLAMA_ERR_ALIGN).  Calls allocate nothing, keep nothing between calls and can be
 * captured into a CUDA graph; a replay reads the lengths, offsets and page ids
 * as they are then, within the bounds given on the host at capture.  A
 * workspace may hold anything before a call and is scratch after it: calls that
 * are ordered (one stream, one graph after another) can share one, calls that
 * may run at the same time need one each. */

/* Pages of one layer's keys and values: k and v are each
 * [n_pages][n_kv_heads][page_size][d_head] of the call's dtype, consecutive
 * pages page_stride elements apart (0: dense; a larger stride lets the pages of
 * k and v, or of several layers, interleave).  Position p of sequence i lies in
 * row p % page_size of page page_table[i * table_stride + p / page_size].
 * page_table is a device array; entries past the last page in use may hold
 * anything.  Sequences may share pages that they only read (a common prefix).
 * page_size: 16, 32, 64, 128 or 256 (LLAMA_ERR_UNSUPPORTED otherwise).
 * page_stride: 0 or >= n_kv_heads * page_size * d_head, a multiple of 16 bytes.
 * A page id outside [0, n_pages) reads as a page of zeros, is not written, and
 * records LLAMA_ERR_RANGE. */
typedef struct {
    void *k;
    void *v;
    const int32_t *page_table;
    int32_t n_pages;
    int32_t page_size;
    int32_t max_pages;    /* entries of a page_table row that may be used */
    int32_t table_stride; /* entries from one row to the next, >= max_pages */
    int64_t page_stride;  /* elements from one page to the next, 0: dense */
} llama_paged_kv_cache;

/* Most sequences of one call, the largest max_kv_len, most query heads, and most
 * (token, query head) pairs, n_tokens * H (LLAMA_ERR_UNSUPPORTED above). */
#define LLAMA_PACKED_MAX_SEQS 4096
#define LLAMA_PACKED_MAX_KV 8388480
#define LLAMA_PACKED_MAX_HEADS 65535
#define LLAMA_PACKED_MAX_ROWS 1073741824

/* n_seqs sequences packed one after another: the new tokens of sequence i are
 * rows [q_offsets[i], q_offsets[i + 1]) of the token-major arrays of the call
 * (q_offsets: device, n_seqs + 1 entries, non-decreasing, within [0,
 * n_tokens]); kv_lens[i] (device, n_seqs entries) counts its positions with
 * those tokens included, so that its new tokens are the last ones:  token t is
 * at position kv_lens[i] - (q_offsets[i + 1] - t).  Sequences without new
 * tokens are allowed.  Rows outside all sequences (padding behind the last one)
 * are not written, and what they hold has no effect.
 * max_kv_len: no kv_lens entry is larger (host value; it may be larger than any).
 * A sequence with bad offsets is left out (offsets that descend make others
 * overlap: the rows of o and q_out may then hold anything); a length that is
 * negative, above max_kv_len or above max_pages * page_size counts as 0.  Both
 * record LLAMA_ERR_RANGE. */
typedef struct {
    const int32_t *q_offsets;
    const int32_t *kv_lens;
    int32_t n_seqs;
    int32_t n_tokens; /* rows of the token-major arrays */
    int32_t max_kv_len;
} llama_packed_batch;

/* RoPE and the write of keys and values into their pages.  qkv [n_tokens]
 * [(H + 2G) D], q_out [n_tokens][H][D], table, layout and the rotation as for
 * llama_op_rope_kv_write; token t turns at its position, rotated k and raw v go
 * to that position's row of its page, nothing else in the cache changes.  No two
 * tokens of a call may share a position's row.  A token whose position is
 * negative or >= table_max_seq gets a row of zeros in q_out, is not written to
 * the cache, and records LLAMA_ERR_RANGE. */
llama_status llama_op_rope_kv_write_paged(int32_t dtype, const void *qkv, void *q_out,
                                          const llama_paged_kv_cache *kv, const llama_packed_batch *batch,
                                          const float *table, int32_t table_max_seq, int32_t H, int32_t G,
                                          int32_t D, int32_t layout, int32_t *status, llama_stream stream);

/* Causal grouped-query attention of a packed batch: for token t of sequence i
 * at position p,
 *   o[t][h] = sum_{j <= p} softmax_j(q[t][h] . K_i[h / (H/G)][j] / sqrt(D)) V_i[h / (H/G)][j]
 * over the sequence's pages (its own new keys included: write them first).
 * q, o: [n_tokens][H][D], q already rotated.  A token that sees no key (p < 0:
 * kv_lens[i] is less than the sequence's tokens) gets zeros.  Rows of the pages
 * at or behind kv_lens[i] may hold anything, NaN included; the keys and values
 * before it have to be finite.  A query row that holds NaN or an infinity gives
 * NaN for its head where it sees a key; other rows and heads are as without it.
 * D in {16, 32, 64, 128}.  Scores, statistics and sums are fp32; with LLAMA_BF16
 * each softmax weight is rounded to bf16 for its product with V, here and in the
 * decode call (here a second time where a later key of the same 128 outweighs it
 * and all keys before by more than 2^8).
 * workspace: caller-owned device scratch of at least
 * llama_op_attention_packed_workspace_bytes bytes (which reads only n_seqs,
 * n_tokens and max_kv_len of batch; 0 for arguments that the call refuses); may
 * be NULL when that is 0. */
size_t llama_op_attention_packed_workspace_bytes(int32_t dtype, const llama_packed_batch *batch, int32_t H,
                                                 int32_t G, int32_t D);
llama_status llama_op_attention_packed(int32_t dtype, const void *q, const llama_paged_kv_cache *kv,
                                       const llama_packed_batch *batch, void *o, int32_t H, int32_t G, int32_t D,
                                       void *workspace, size_t workspace_bytes, int32_t *status,
                                       llama_stream stream);

/* The same for one new token per sequence: q, o: [n_seqs][H][D], row i at
 * position kv_lens[i] - 1.  A sequence of length 0 gets zeros.  The cache's
 * length is split over the GPU and the parts joined by their log-sum-exp.  The
 * split follows from the sizes, max_kv_len (an upper bound, as in
 * llama_packed_batch) and the lengths of all sequences of the call, so the last
 * bits of a result depend on them, but not from run to run. */
size_t llama_op_attention_paged_decode_workspace_bytes(int32_t dtype, int32_t n_seqs, int32_t max_kv_len,
                                                       int32_t H, int32_t G, int32_t D);
llama_status llama_op_attention_paged_decode(int32_t dtype, const void *q, const llama_paged_kv_cache *kv,
                                             const int32_t *kv_lens, int32_t n_seqs, int32_t max_kv_len, void *o,
                                             int32_t H, int32_t G, int32_t D, void *workspace,
                                             size_t workspace_bytes, int32_t *status, llama_stream stream);

/* Bound, in SM clock cycles, on every wait of the bf16 kernels of
 * llama_op_attention_packed and llama_op_attention_paged_decode that gives up,
 * for later calls (and captures) of the process; 0 restores the default, about
 * 4e9 cycles (2 s at 2 GHz), which no legitimate wait reaches.  As
 * llama_block_set_wait_budget: a wait that runs out records
 * LLAMA_ERR_DEVICE_TIMEOUT in the call's status, the kernel returns once its
 * copies and MMAs in flight have completed (those waits keep the default) with
 * its tensor memory freed, o is undefined and the next call starts afresh.  A
 * diagnosis knob; the library itself never sets it.  LLAMA_ERR_INVALID_ARG for
 * a negative budget. */
llama_status llama_op_set_wait_budget(int64_t cycles);

/* Log-probabilities of given tokens, with the entropy of each distribution and
 * its likeliest tokens.  logits: [T][V] of dtype, rows row_stride elements
 * apart (>= V; columns at and behind V are not read).  Every array of this call
 * needs the alignment of its elements only.
 * With p = softmax(logits[t]):
 *   logprobs[t]        = ln p[targets[t]]          (fp32)
 *   entropy[t]         = -sum_v p[v] ln p[v]       (fp32; NULL: not computed)
 *   top_ids[t][j]      = id of the j-th largest logit, the lowest id among equals
 *   top_logprobs[t][j] = ln p[top_ids[t][j]]       (fp32, [T][top_k])
 * targets: int32 [T].  A target of -1 (a position without a next token) gives
 * logprobs[t] = 0; any other target outside [0, V) gives NaN and records
 * LLAMA_ERR_RANGE.  targets and logprobs may both be NULL.
 * 0 <= top_k <= min(V, LLAMA_LOGPROBS_MAX_TOP); with top_k = 0 the two arrays
 * are ignored.
 * A logit of -inf has probability 0 (ln p = -inf) and adds nothing to the
 * entropy; a row of nothing but -inf has ln p = -inf throughout and entropy 0.
 * NaN or +inf anywhere in a row makes its logprobs, top_logprobs and entropy NaN;
 * NaN is never among the top (ids that cannot be filled are -1). */
llama_status llama_op_token_logprobs(int32_t dtype, const void *logits, int64_t row_stride, const int32_t *targets,
                                     int32_t T, int32_t V, float *logprobs, float *entropy, int32_t top_k,
                                     int32_t *top_ids, float *top_logprobs, int32_t *status, llama_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* LLAMA_OPS_H */
