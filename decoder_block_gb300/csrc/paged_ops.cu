// C entry points of the packed / paged operators, over 4-bit pages too, of the token
// log-probabilities and of the verification of drafts (llama_ops.h): validation, then
// the launch.
#include <atomic>
#include <initializer_list>

#include "kernels.h"
#include "kv4.cuh"
#include "paged_kernels.h"

using namespace llama;

namespace {

std::atomic<long long> wait_cycles{0};  // 0: the default

// Device memory of the current device, aligned to `align` bytes: 16 where vectors or TMA
// boxes are read or written, the size of an element where those come one at a time.
llama_status check(const void *p, unsigned align) {
  if (p == nullptr) return LLAMA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % align != 0) return LLAMA_ERR_ALIGN;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return LLAMA_ERR_INVALID_ARG;
  }
  if (a.type == cudaMemoryTypeManaged) return LLAMA_OK;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return LLAMA_ERR_INVALID_ARG;
  }
  return a.type == cudaMemoryTypeDevice && a.device == dev ? LLAMA_OK : LLAMA_ERR_INVALID_ARG;
}

llama_status check_all(std::initializer_list<const void *> ptrs, unsigned align) {
  for (const void *p : ptrs) {
    const llama_status s = check(p, align);
    if (s != LLAMA_OK) return s;
  }
  return LLAMA_OK;
}

llama_status check_status(const int32_t *status) { return status == nullptr ? LLAMA_OK : check(status, 4); }

llama_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return LLAMA_OK;
  note_cuda_error(e);
  return LLAMA_ERR_CUDA;
}

bool dtype_ok(int32_t dtype) { return dtype == LLAMA_F32 || dtype == LLAMA_BF16; }
int esize(int32_t dtype) { return dtype == LLAMA_BF16 ? 2 : 4; }

// Head shape, in the order the other operators check it.
llama_status check_heads(int32_t H, int32_t G, int32_t D) {
  if (H <= 0 || G <= 0 || D <= 0) return LLAMA_ERR_INVALID_ARG;
  if (H % G != 0) return LLAMA_ERR_SHAPE;
  if ((D != 16 && D != 32 && D != 64 && D != 128) || H > LLAMA_PACKED_MAX_HEADS) return LLAMA_ERR_UNSUPPORTED;
  return LLAMA_OK;
}

// Everything about the cache struct but its pointers.  dtype: of its elements, or KV4_PAGES.
constexpr int32_t KV4_PAGES = -1;
llama_status view_of(const llama_paged_kv_cache *kv, int32_t dtype, int32_t G, int32_t D, PagedView *out) {
  if (kv->n_pages <= 0 || kv->page_size <= 0 || kv->max_pages <= 0 || kv->table_stride < kv->max_pages)
    return LLAMA_ERR_INVALID_ARG;
  PagedView v;
  for (v.page_log2 = 4; v.page_log2 <= 8 && (1 << v.page_log2) != kv->page_size; ++v.page_log2) {
  }
  if (v.page_log2 > 8) return LLAMA_ERR_UNSUPPORTED;
  const long long dense =
      dtype == KV4_PAGES ? (long long)G * kv4_block_bytes(kv->page_size, D) : (long long)G * kv->page_size * D;
  const int unit = dtype == KV4_PAGES ? 1 : esize(dtype);
  v.page_stride = kv->page_stride == 0 ? dense : kv->page_stride;
  if (v.page_stride < dense) return LLAMA_ERR_INVALID_ARG;
  if (v.page_stride * unit % 16 != 0) return LLAMA_ERR_ALIGN;
  if (v.page_stride >= (dtype == KV4_PAGES ? 1LL << 32 : (1LL << 39) / unit)) return LLAMA_ERR_UNSUPPORTED;
  v.table = kv->page_table;
  v.n_pages = kv->n_pages;
  v.max_pages = kv->max_pages;
  v.table_stride = kv->table_stride;
  *out = v;
  return LLAMA_OK;
}

llama_status check_batch(const llama_packed_batch *b, int32_t H) {
  if (b->n_seqs < 0 || b->n_tokens < 0 || b->max_kv_len < 0) return LLAMA_ERR_INVALID_ARG;
  if (b->n_seqs > LLAMA_PACKED_MAX_SEQS || b->max_kv_len > LLAMA_PACKED_MAX_KV ||
      (long long)b->n_tokens * H > LLAMA_PACKED_MAX_ROWS)
    return LLAMA_ERR_UNSUPPORTED;
  return LLAMA_OK;
}

PackedView view_of(const llama_packed_batch *b) {
  PackedView v;
  v.q_offsets = b->q_offsets;
  v.kv_lens = b->kv_lens;
  v.n_seqs = b->n_seqs;
  v.n_tokens = b->n_tokens;
  v.max_kv_len = b->max_kv_len;
  return v;
}

bool decode_sizes_ok(int32_t n_seqs, int32_t max_kv_len, int32_t H, int32_t G, int32_t D) {
  return n_seqs > 0 && n_seqs <= LLAMA_PACKED_MAX_SEQS && max_kv_len >= 0 && max_kv_len <= LLAMA_PACKED_MAX_KV &&
         check_heads(H, G, D) == LLAMA_OK;
}

// The checks of a write, of packed and of decode attention; pages: dtype, or KV4_PAGES.
llama_status check_write(int32_t dtype, int32_t pages, const void *qkv, const void *q_out,
                         const llama_paged_kv_cache *kv, const llama_packed_batch *batch, const float *table,
                         int32_t table_max_seq, int32_t H, int32_t G, int32_t D, int32_t layout, const int32_t *status,
                         PagedView *pv) {
  if (!dtype_ok(dtype)) return LLAMA_ERR_INVALID_ARG;
  if (layout != LLAMA_ROPE_INTERLEAVED && layout != LLAMA_ROPE_HALVES) return LLAMA_ERR_INVALID_ARG;
  if (kv == nullptr || batch == nullptr || table_max_seq <= 0) return LLAMA_ERR_INVALID_ARG;
  llama_status s = check_heads(H, G, D);
  if (s == LLAMA_OK) s = check_batch(batch, H);
  if (s == LLAMA_OK) s = view_of(kv, pages, G, D, pv);
  if (s != LLAMA_OK) return s;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return LLAMA_OK;
  s = check_all({qkv, q_out, kv->k, kv->v, table}, 16);
  if (s == LLAMA_OK) s = check_all({kv->page_table, batch->q_offsets, batch->kv_lens}, 4);
  return s == LLAMA_OK ? check_status(status) : s;
}

llama_status check_workspace(const void *workspace, size_t workspace_bytes, size_t need) {
  if (need == 0) return LLAMA_OK;
  if (workspace_bytes < need) return LLAMA_ERR_RANGE;
  return check(workspace, 16);
}

llama_status check_packed(int32_t dtype, int32_t pages, const void *q, const llama_paged_kv_cache *kv,
                          const llama_packed_batch *batch, const void *o, int32_t H, int32_t G, int32_t D,
                          const void *workspace, size_t workspace_bytes, const int32_t *status, PagedView *pv) {
  if (!dtype_ok(dtype) || kv == nullptr || batch == nullptr) return LLAMA_ERR_INVALID_ARG;
  llama_status s = check_heads(H, G, D);
  if (s == LLAMA_OK) s = check_batch(batch, H);
  if (s == LLAMA_OK) s = view_of(kv, pages, G, D, pv);
  if (s != LLAMA_OK) return s;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return LLAMA_OK;
  s = check_all({q, o, kv->k, kv->v}, 16);
  if (s == LLAMA_OK) s = check_all({kv->page_table, batch->q_offsets, batch->kv_lens}, 4);
  if (s == LLAMA_OK) s = check_status(status);
  if (s != LLAMA_OK) return s;
  return check_workspace(workspace, workspace_bytes,
                         pages == KV4_PAGES ? llama_op_attention_packed_kv4_workspace_bytes(dtype, batch, H, G, D)
                                            : llama_op_attention_packed_workspace_bytes(dtype, batch, H, G, D));
}

llama_status check_decode(int32_t dtype, int32_t pages, const void *q, const llama_paged_kv_cache *kv,
                          const int32_t *kv_lens, int32_t n_seqs, int32_t max_kv_len, const void *o, int32_t H,
                          int32_t G, int32_t D, const void *workspace, size_t workspace_bytes, const int32_t *status,
                          PagedView *pv) {
  if (!dtype_ok(dtype) || kv == nullptr || n_seqs < 0 || max_kv_len < 0) return LLAMA_ERR_INVALID_ARG;
  llama_status s = check_heads(H, G, D);
  if (s == LLAMA_OK && (n_seqs > LLAMA_PACKED_MAX_SEQS || max_kv_len > LLAMA_PACKED_MAX_KV)) s = LLAMA_ERR_UNSUPPORTED;
  if (s == LLAMA_OK && pages == KV4_PAGES && !kv4_decode_fits(n_seqs, max_kv_len, H, G)) s = LLAMA_ERR_UNSUPPORTED;
  if (s == LLAMA_OK) s = view_of(kv, pages, G, D, pv);
  if (s != LLAMA_OK) return s;
  if (n_seqs == 0) return LLAMA_OK;
  s = check_all({q, o, kv->k, kv->v}, 16);
  if (s == LLAMA_OK) s = check_all({kv->page_table, kv_lens}, 4);
  if (s == LLAMA_OK) s = check_status(status);
  if (s != LLAMA_OK) return s;
  return check_workspace(workspace, workspace_bytes,
                         pages == KV4_PAGES
                             ? llama_op_attention_paged_decode_kv4_workspace_bytes(dtype, n_seqs, max_kv_len, H, G, D)
                             : llama_op_attention_paged_decode_workspace_bytes(dtype, n_seqs, max_kv_len, H, G, D));
}

llama_status check_drafts(const llama_draft_batch *b, int32_t V) {
  if (b == nullptr || b->n_seqs < 0 || b->n_rows < 0 || b->max_drafts < 0 || V <= 0) return LLAMA_ERR_INVALID_ARG;
  if (b->n_seqs > LLAMA_PACKED_MAX_SEQS || b->max_drafts > LLAMA_MAX_DRAFTS ||
      b->n_rows > LLAMA_PACKED_MAX_SEQS * (LLAMA_MAX_DRAFTS + 1))
    return LLAMA_ERR_UNSUPPORTED;
  return LLAMA_OK;
}

}  // namespace

long long llama::op_wait_cycles() {
  const long long c = wait_cycles.load(std::memory_order_relaxed);
  return c > 0 ? c : kWaitBudgetCycles;
}

extern "C" {

llama_status llama_op_set_wait_budget(int64_t cycles) {
  if (cycles < 0) return LLAMA_ERR_INVALID_ARG;
  wait_cycles.store(cycles, std::memory_order_relaxed);
  return LLAMA_OK;
}

llama_status llama_op_rope_kv_write_paged(int32_t dtype, const void *qkv, void *q_out,
                                          const llama_paged_kv_cache *kv, const llama_packed_batch *batch,
                                          const float *table, int32_t table_max_seq, int32_t H, int32_t G,
                                          int32_t D, int32_t layout, int32_t *status, llama_stream stream) {
  PagedView pv;
  const llama_status s = check_write(dtype, dtype, qkv, q_out, kv, batch, table, table_max_seq, H, G, D, layout, status, &pv);
  if (s != LLAMA_OK || batch->n_seqs == 0 || batch->n_tokens == 0) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const float2 *t2 = reinterpret_cast<const float2 *>(table);
  const PackedView b = view_of(batch);
  if (dtype == LLAMA_BF16)
    return status_of(launch_rope_kv_paged<bf16>((const bf16 *)qkv, (bf16 *)q_out, (bf16 *)kv->k, (bf16 *)kv->v, pv, b,
                                                t2, table_max_seq, H, G, D, layout, status, st));
  return status_of(launch_rope_kv_paged<float>((const float *)qkv, (float *)q_out, (float *)kv->k, (float *)kv->v, pv,
                                               b, t2, table_max_seq, H, G, D, layout, status, st));
}

llama_status llama_op_rope_kv4_write_paged(int32_t dtype, const void *qkv, void *q_out,
                                           const llama_paged_kv_cache *kv, const llama_packed_batch *batch,
                                           const float *table, int32_t table_max_seq, int32_t H, int32_t G,
                                           int32_t D, int32_t layout, int32_t *status, llama_stream stream) {
  PagedView pv;
  const llama_status s = check_write(dtype, KV4_PAGES, qkv, q_out, kv, batch, table, table_max_seq, H, G, D, layout, status, &pv);
  if (s != LLAMA_OK || batch->n_seqs == 0 || batch->n_tokens == 0) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const float2 *t2 = reinterpret_cast<const float2 *>(table);
  const PackedView b = view_of(batch);
  uint8_t *k = (uint8_t *)kv->k, *v = (uint8_t *)kv->v;
  if (dtype == LLAMA_BF16)
    return status_of(launch_rope_kv4<bf16>((const bf16 *)qkv, (bf16 *)q_out, k, v, pv, b, t2, table_max_seq, H, G, D,
                                           layout, status, st));
  return status_of(launch_rope_kv4<float>((const float *)qkv, (float *)q_out, k, v, pv, b, t2, table_max_seq, H, G, D,
                                          layout, status, st));
}

size_t llama_kv4_block_bytes(int32_t page_size, int32_t d_head) {
  const bool page_ok = page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 || page_size == 256;
  return page_ok && check_heads(1, 1, d_head) == LLAMA_OK ? (size_t)kv4_block_bytes(page_size, d_head) : 0;
}

llama_status llama_op_kv4_read_paged(int32_t dtype, const llama_paged_kv_cache *kv, const llama_packed_batch *batch,
                                     void *k_out, void *v_out, int32_t G, int32_t D, int32_t *status,
                                     llama_stream stream) {
  if (!dtype_ok(dtype) || kv == nullptr || batch == nullptr) return LLAMA_ERR_INVALID_ARG;
  llama_status s = check_heads(G, G, D);
  if (s == LLAMA_OK) s = check_batch(batch, G);
  PagedView pv;
  if (s == LLAMA_OK) s = view_of(kv, KV4_PAGES, G, D, &pv);
  if (s != LLAMA_OK) return s;
  if (batch->n_seqs == 0 || batch->n_tokens == 0 || (k_out == nullptr && v_out == nullptr)) return LLAMA_OK;
  if (k_out != nullptr) s = check(k_out, 16);
  if (s == LLAMA_OK && v_out != nullptr) s = check(v_out, 16);
  if (s == LLAMA_OK) s = check_all({kv->k, kv->v}, 16);
  if (s == LLAMA_OK) s = check_all({kv->page_table, batch->q_offsets, batch->kv_lens}, 4);
  if (s == LLAMA_OK) s = check_status(status);
  if (s != LLAMA_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const PackedView b = view_of(batch);
  const uint8_t *k = (const uint8_t *)kv->k, *v = (const uint8_t *)kv->v;
  if (dtype == LLAMA_BF16)
    return status_of(launch_kv4_read<bf16>(k, v, (bf16 *)k_out, (bf16 *)v_out, pv, b, G, D, status, st));
  return status_of(launch_kv4_read<float>(k, v, (float *)k_out, (float *)v_out, pv, b, G, D, status, st));
}

size_t llama_op_attention_packed_workspace_bytes(int32_t dtype, const llama_packed_batch *batch, int32_t H,
                                                 int32_t G, int32_t D) {
  if (!dtype_ok(dtype) || batch == nullptr || check_heads(H, G, D) != LLAMA_OK || check_batch(batch, H) != LLAMA_OK)
    return 0;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return 0;
  const PackedView b = view_of(batch);
  return dtype == LLAMA_BF16 ? packed_tc_workspace_bytes(b, H, G, D) : packed_simt_workspace_bytes(b, H, G, D);
}

llama_status llama_op_attention_packed(int32_t dtype, const void *q, const llama_paged_kv_cache *kv,
                                       const llama_packed_batch *batch, void *o, int32_t H, int32_t G, int32_t D,
                                       void *workspace, size_t workspace_bytes, int32_t *status,
                                       llama_stream stream) {
  PagedView pv;
  const llama_status s = check_packed(dtype, dtype, q, kv, batch, o, H, G, D, workspace, workspace_bytes, status, &pv);
  if (s != LLAMA_OK || batch->n_seqs == 0 || batch->n_tokens == 0) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const PackedView b = view_of(batch);
  if (dtype == LLAMA_BF16)
    return status_of(launch_packed_tc((const bf16 *)q, (const bf16 *)kv->k, (const bf16 *)kv->v, (bf16 *)o, pv, b, H,
                                      G, D, workspace, status, st));
  return status_of(launch_packed_simt((const float *)q, (const float *)kv->k, (const float *)kv->v, (float *)o, pv, b, H,
                                      G, D, (float *)workspace, status, st));
}

size_t llama_op_attention_packed_kv4_workspace_bytes(int32_t dtype, const llama_packed_batch *batch, int32_t H,
                                                     int32_t G, int32_t D) {
  const size_t need = llama_op_attention_packed_workspace_bytes(dtype, batch, H, G, D);
  if (dtype != LLAMA_BF16 || batch == nullptr || check_heads(H, G, D) != LLAMA_OK ||
      check_batch(batch, H) != LLAMA_OK || batch->n_seqs == 0 || batch->n_tokens == 0)
    return need;
  return packed_kv4_workspace_bytes(view_of(batch), H, G, D);
}

llama_status llama_op_attention_packed_kv4(int32_t dtype, const void *q, const llama_paged_kv_cache *kv,
                                           const llama_packed_batch *batch, void *o, int32_t H, int32_t G, int32_t D,
                                           void *workspace, size_t workspace_bytes, int32_t *status,
                                           llama_stream stream) {
  PagedView pv;
  const llama_status s = check_packed(dtype, KV4_PAGES, q, kv, batch, o, H, G, D, workspace, workspace_bytes, status, &pv);
  if (s != LLAMA_OK || batch->n_seqs == 0 || batch->n_tokens == 0) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const PackedView b = view_of(batch);
  const uint8_t *k = (const uint8_t *)kv->k, *v = (const uint8_t *)kv->v;
  if (dtype == LLAMA_BF16)
    return status_of(launch_packed_kv4((const bf16 *)q, k, v, (bf16 *)o, pv, b, H, G, D, workspace, status, st));
  return status_of(launch_packed_simt((const float *)q, k, v, (float *)o, pv, b, H, G, D, (float *)workspace, status, st));
}

size_t llama_op_attention_paged_decode_workspace_bytes(int32_t dtype, int32_t n_seqs, int32_t max_kv_len,
                                                       int32_t H, int32_t G, int32_t D) {
  if (!dtype_ok(dtype) || !decode_sizes_ok(n_seqs, max_kv_len, H, G, D)) return 0;
  if (dtype == LLAMA_BF16)
    return paged_decode_tc_workspace_bytes(n_seqs, max_kv_len, H, G, D);
  return paged_decode_simt_workspace_bytes(n_seqs, max_kv_len, H, G, D);
}

llama_status llama_op_attention_paged_decode(int32_t dtype, const void *q, const llama_paged_kv_cache *kv,
                                             const int32_t *kv_lens, int32_t n_seqs, int32_t max_kv_len, void *o,
                                             int32_t H, int32_t G, int32_t D, void *workspace,
                                             size_t workspace_bytes, int32_t *status, llama_stream stream) {
  PagedView pv;
  const llama_status s = check_decode(dtype, dtype, q, kv, kv_lens, n_seqs, max_kv_len, o, H, G, D, workspace,
                                      workspace_bytes, status, &pv);
  if (s != LLAMA_OK || n_seqs == 0) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == LLAMA_BF16)
    return status_of(launch_paged_decode_tc((const bf16 *)q, (const bf16 *)kv->k, (const bf16 *)kv->v, (bf16 *)o, pv,
                                            kv_lens, n_seqs, max_kv_len, H, G, D, workspace, status, st));
  return status_of(launch_paged_decode_simt((const float *)q, (const float *)kv->k, (const float *)kv->v, (float *)o, pv,
                                            kv_lens, n_seqs, max_kv_len, H, G, D, (float *)workspace, status, st));
}

size_t llama_op_attention_paged_decode_kv4_workspace_bytes(int32_t dtype, int32_t n_seqs, int32_t max_kv_len,
                                                           int32_t H, int32_t G, int32_t D) {
  if (decode_sizes_ok(n_seqs, max_kv_len, H, G, D) && !kv4_decode_fits(n_seqs, max_kv_len, H, G)) return 0;
  if (dtype != LLAMA_BF16 || !decode_sizes_ok(n_seqs, max_kv_len, H, G, D))
    return llama_op_attention_paged_decode_workspace_bytes(dtype, n_seqs, max_kv_len, H, G, D);
  return kv4_decode_workspace_bytes(n_seqs, max_kv_len, H, G, D);
}

llama_status llama_op_attention_paged_decode_kv4(int32_t dtype, const void *q, const llama_paged_kv_cache *kv,
                                                 const int32_t *kv_lens, int32_t n_seqs, int32_t max_kv_len, void *o,
                                                 int32_t H, int32_t G, int32_t D, void *workspace,
                                                 size_t workspace_bytes, int32_t *status, llama_stream stream) {
  PagedView pv;
  const llama_status s = check_decode(dtype, KV4_PAGES, q, kv, kv_lens, n_seqs, max_kv_len, o, H, G, D, workspace,
                                      workspace_bytes, status, &pv);
  if (s != LLAMA_OK || n_seqs == 0) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const uint8_t *k = (const uint8_t *)kv->k, *v = (const uint8_t *)kv->v;
  if (dtype == LLAMA_BF16)
    return status_of(launch_kv4_decode((const bf16 *)q, k, v, (bf16 *)o, pv, kv_lens, n_seqs, max_kv_len, H, G, D,
                                       workspace, status, st));
  return status_of(launch_paged_decode_simt((const float *)q, k, v, (float *)o, pv, kv_lens, n_seqs, max_kv_len, H, G, D,
                                            (float *)workspace, status, st));
}

llama_status llama_op_token_logprobs(int32_t dtype, const void *logits, int64_t row_stride, const int32_t *targets,
                                     int32_t T, int32_t V, float *logprobs, float *entropy, int32_t top_k,
                                     int32_t *top_ids, float *top_logprobs, int32_t *status, llama_stream stream) {
  if (!dtype_ok(dtype) || T < 0 || V <= 0 || row_stride < V || top_k < 0) return LLAMA_ERR_INVALID_ARG;
  if ((targets == nullptr) != (logprobs == nullptr)) return LLAMA_ERR_INVALID_ARG;
  if (top_k > V) return LLAMA_ERR_RANGE;
  if (top_k > LLAMA_LOGPROBS_MAX_TOP) return LLAMA_ERR_UNSUPPORTED;
  if (T == 0) return LLAMA_OK;
  llama_status s = check(logits, (unsigned)esize(dtype));
  if (s == LLAMA_OK && logprobs != nullptr) s = check_all({targets, logprobs}, 4);
  if (s == LLAMA_OK && entropy != nullptr) s = check(entropy, 4);
  if (s == LLAMA_OK && top_k > 0) s = check_all({top_ids, top_logprobs}, 4);
  if (s == LLAMA_OK) s = check_status(status);
  if (s != LLAMA_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == LLAMA_BF16)
    return status_of(launch_token_logprobs<bf16>((const bf16 *)logits, row_stride, targets, T, V, logprobs, entropy,
                                                 top_k, top_ids, top_logprobs, status, LLAMA_ERR_RANGE, st));
  return status_of(launch_token_logprobs<float>((const float *)logits, row_stride, targets, T, V, logprobs, entropy,
                                                top_k, top_ids, top_logprobs, status, LLAMA_ERR_RANGE, st));
}

size_t llama_op_verify_drafts_workspace_bytes(const llama_draft_batch *batch, int32_t V) {
  return check_drafts(batch, V) == LLAMA_OK ? verify_drafts_workspace_bytes(batch->n_rows, V) : 0;
}

llama_status llama_op_verify_drafts(int32_t dtype, const void *target_logits, int64_t target_stride,
                                    const void *draft_logits, int64_t draft_seq_stride, int64_t draft_step_stride,
                                    int32_t V, const llama_draft_batch *batch, int32_t *out_tokens,
                                    int32_t *n_accepted, float *logprobs, void *workspace, size_t workspace_bytes,
                                    int32_t *status, llama_stream stream) {
  if (!dtype_ok(dtype)) return LLAMA_ERR_INVALID_ARG;
  llama_status s = check_drafts(batch, V);
  if (s != LLAMA_OK) return s;
  if (target_stride < V || (draft_logits != nullptr && (draft_seq_stride < 0 || draft_step_stride < 0)))
    return LLAMA_ERR_INVALID_ARG;
  if (batch->max_drafts > 0 && (batch->uniforms == nullptr) != (batch->noise == nullptr)) return LLAMA_ERR_INVALID_ARG;
  if (batch->noise != nullptr && batch->noise_stride < V) return LLAMA_ERR_INVALID_ARG;
  if (batch->n_seqs == 0) return LLAMA_OK;
  if (batch->n_rows > 0) {
    s = check(target_logits, (unsigned)esize(dtype));
    if (s == LLAMA_OK && draft_logits != nullptr) s = check(draft_logits, (unsigned)esize(dtype));
    if (s == LLAMA_OK) s = check(batch->tokens, 4);
  }
  if (s == LLAMA_OK) s = check_all({batch->q_offsets, out_tokens, n_accepted}, 4);
  if (s == LLAMA_OK && batch->temperatures != nullptr) s = check(batch->temperatures, 4);
  if (s == LLAMA_OK && batch->noise != nullptr) s = check(batch->noise, 4);
  if (s == LLAMA_OK && batch->noise != nullptr && batch->max_drafts > 0) s = check(batch->uniforms, 4);
  if (s == LLAMA_OK && logprobs != nullptr) s = check(logprobs, 4);
  if (s == LLAMA_OK) s = check_status(status);
  if (s == LLAMA_OK)
    s = check_workspace(workspace, workspace_bytes, llama_op_verify_drafts_workspace_bytes(batch, V));
  if (s != LLAMA_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == LLAMA_BF16)
    return status_of(launch_verify_drafts<bf16>((const bf16 *)target_logits, target_stride, (const bf16 *)draft_logits,
                                                draft_seq_stride, draft_step_stride, V, *batch, out_tokens, n_accepted,
                                                logprobs, workspace, status, st));
  return status_of(launch_verify_drafts<float>((const float *)target_logits, target_stride, (const float *)draft_logits,
                                               draft_seq_stride, draft_step_stride, V, *batch, out_tokens, n_accepted,
                                               logprobs, workspace, status, st));
}

}  // extern "C"
