// RoPE and the write of keys and values into cache pages for packed rows
// ("Mini Llama 2 Implementation", Rotary positional embeddings; "Full Llama 3
// transformer block", How it works: rotate, then write at the position).
// Pure data movement: every row is read once and written once.
#include "paged_kernels.h"

namespace llama {
namespace {

// Grid: x over the 16-byte vectors of one row, y over rows t0 + blockIdx.y.
template <typename T>
__global__ void __launch_bounds__(256) rope_kv_paged_kernel(const T *__restrict__ qkv, T *__restrict__ q_out,
                                                            T *__restrict__ kc, T *__restrict__ vc, PagedView pv,
                                                            PackedView b, const float2 *__restrict__ table,
                                                            int table_max_seq, int t0, int H, int G, int D, int halves,
                                                            int *status) {
  constexpr int V = Vec16<T>::N;
  const int t = t0 + blockIdx.y;
  if (t0 == 0 && blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < b.n_seqs; i += blockDim.x) check_seq(b, pv, i, status);
  const int i = find_seq(b, t);
  if (i < 0) return;
  const SeqSpan s = seq_span(b, pv, i);
  const int p = s.kv_len - (s.first + s.count - t);
  const bool in_range = p >= 0 && p < table_max_seq;
  const int page = in_range ? pv.page(i, p >> pv.page_log2) : -1;
  if (page < 0 && blockIdx.x == 0 && threadIdx.x == 0) report_status(status, LLAMA_ERR_RANGE);

  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= (H + 2 * G) * D / V) return;
  const int col = c * V;
  const int head = col / D, e = col % D;
  const T *src = qkv + (size_t)t * (H + 2 * G) * D + col;
  const int slot = p & ((1 << pv.page_log2) - 1);
  if (head >= H + G) {
    if (page >= 0)
      store16(vc + page * pv.page_stride + (((long long)(head - H - G) << pv.page_log2) + slot) * D + e, load16(src));
    return;
  }
  if (head >= H && page < 0) return;
  T *dst = head < H ? q_out + ((size_t)t * H + head) * D
                    : kc + page * pv.page_stride + (((long long)(head - H) << pv.page_log2) + slot) * D;
  if (halves && e >= D / 2) return;  // the thread of the lower half moves both
  if (!in_range) {
    Vec16<T> z;
    z.raw = make_uint4(0, 0, 0, 0);
    store16(dst + e, z);
    if (halves) store16(dst + e + D / 2, z);
    return;
  }
  const Vec16<T> x = load16(src);
  if (!halves) {
    const float4 *cs = reinterpret_cast<const float4 *>(table + (size_t)p * (D / 2) + e / 2);
    Vec16<T> o;
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const float4 c4 = cs[k];
      float a = x.get(4 * k), y = x.get(4 * k + 1);
      o.set(4 * k, a * c4.x - y * c4.y);
      o.set(4 * k + 1, a * c4.y + y * c4.x);
      a = x.get(4 * k + 2);
      y = x.get(4 * k + 3);
      o.set(4 * k + 2, a * c4.z - y * c4.w);
      o.set(4 * k + 3, a * c4.w + y * c4.z);
    }
    store16(dst + e, o);
  } else {
    const float2 *cs = table + (size_t)p * (D / 2) + e;
    const Vec16<T> y = load16(src + D / 2);
    Vec16<T> lo, hi;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float2 cv = cs[k];
      const float a = x.get(k), bb = y.get(k);
      lo.set(k, a * cv.x - bb * cv.y);
      hi.set(k, a * cv.y + bb * cv.x);
    }
    store16(dst + e, lo);
    store16(dst + e + D / 2, hi);
  }
}

}  // namespace

template <typename T>
cudaError_t launch_rope_kv_paged(const T *qkv, T *q_out, T *k, T *v, const PagedView &pv, const PackedView &b,
                                 const float2 *table, int table_max_seq, int H, int G, int D, int halves, int *status,
                                 cudaStream_t st) {
  const int vecs = (H + 2 * G) * D / Vec16<T>::N;
  const unsigned gx = (unsigned)((vecs + 255) / 256);
  for (int t0 = 0; t0 < b.n_tokens; t0 += 65535) {  // grid y is at most 65535 rows per launch
    const int n = b.n_tokens - t0 < 65535 ? b.n_tokens - t0 : 65535;
    count_launch();
    rope_kv_paged_kernel<T><<<dim3(gx, (unsigned)n), 256, 0, st>>>(qkv, q_out, k, v, pv, b, table, table_max_seq, t0,
                                                                   H, G, D, halves, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template cudaError_t launch_rope_kv_paged<float>(const float *, float *, float *, float *, const PagedView &,
                                                 const PackedView &, const float2 *, int, int, int, int, int, int *,
                                                 cudaStream_t);
template cudaError_t launch_rope_kv_paged<bf16>(const bf16 *, bf16 *, bf16 *, bf16 *, const PagedView &,
                                                const PackedView &, const float2 *, int, int, int, int, int, int *,
                                                cudaStream_t);

}  // namespace llama
