// Packed batches over a paged KV cache: the device-side views and lookups that
// the paged kernels share (llama_ops.h describes the layout and what happens to
// lengths, offsets and page ids that are out of range).
#pragma once

#include "common.cuh"
#include "llama_ops.h"

namespace llama {

struct PagedView {
  const int *table = nullptr;
  int n_pages = 0, page_log2 = 0, max_pages = 0, table_stride = 0;
  long long page_stride = 0;  // elements

  // Page of index `idx` of sequence i, -1 when its id is out of range.
  __device__ __forceinline__ int page(int i, int idx) const {
    const int id = ld_after_wait(table + (size_t)i * table_stride + idx);
    return (unsigned)id < (unsigned)n_pages ? id : -1;
  }
  __device__ __forceinline__ long long capacity() const { return (long long)max_pages << page_log2; }
};

struct PackedView {
  const int *q_offsets = nullptr, *kv_lens = nullptr;
  int n_seqs = 0, n_tokens = 0, max_kv_len = 0;
};

// Length of a sequence as the kernels use it: 0 when it is out of range.
__device__ __forceinline__ int checked_len(int len, int max_kv_len, const PagedView &pv) {
  return (len < 0 || len > max_kv_len || len > pv.capacity()) ? 0 : len;
}

// Rows [first, first + count) and length of sequence i; count = 0 when its
// offsets are out of range.
struct SeqSpan {
  int first, count, kv_len;
};
__device__ __forceinline__ SeqSpan seq_span(const PackedView &b, const PagedView &pv, int i) {
  const int a = ld_after_wait(b.q_offsets + i), e = ld_after_wait(b.q_offsets + i + 1);
  SeqSpan s;
  s.first = a;
  s.count = (a >= 0 && e >= a && e <= b.n_tokens) ? e - a : 0;
  s.kv_len = checked_len(ld_after_wait(b.kv_lens + i), b.max_kv_len, pv);
  return s;
}

// Records LLAMA_ERR_RANGE when sequence i's offsets or length are out of range.
__device__ __forceinline__ void check_seq(const PackedView &b, const PagedView &pv, int i, int *status) {
  const int a = ld_after_wait(b.q_offsets + i), e = ld_after_wait(b.q_offsets + i + 1), len = ld_after_wait(b.kv_lens + i);
  if (a < 0 || e < a || e > b.n_tokens || len < 0 || len > b.max_kv_len || len > pv.capacity())
    report_status(status, LLAMA_ERR_RANGE);
}

// Sequence that owns row t, found by the whole warp: the last i with
// q_offsets[i] <= t, 32 probes a round (one round for up to 32 sequences, two
// for up to 1024); -1 when no sequence owns the row.  Offsets that do not rise
// end the search all the same, and the span found is checked.
__device__ __forceinline__ int find_seq(const PackedView &b, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = b.n_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int probe = lo + lane * step;
    const bool le = lane * step < n && ld_after_wait(b.q_offsets + probe) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return -1;
    const int k = 31 - __clz(m);
    n = min(step, n - k * step);
    lo += k * step;
  }
  const int a = ld_after_wait(b.q_offsets + lo), e = ld_after_wait(b.q_offsets + lo + 1);
  return (a >= 0 && a <= t && t < e && e <= b.n_tokens) ? lo : -1;
}

// Sum of two counts, at most INT_MAX: offsets that descend make sequences overlap, and
// their blocks may number more than an int holds.
__device__ __forceinline__ int add_counts(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); }

// Inclusive sum of counts over the threads of a CTA of 1024; warp_sums: 32 shared ints.
__device__ __forceinline__ int cta_scan(int v, int *warp_sums) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = add_counts(v, x);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = add_counts(s, x);
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int out = add_counts(v, warp > 0 ? warp_sums[warp - 1] : 0);
  __syncthreads();
  return out;
}

}  // namespace llama
