// RoPE and the write of keys and values into cache pages for packed rows
// ("Mini Llama 2 Implementation", Rotary positional embeddings; "Full Llama 3
// transformer block", How it works: rotate, then write at the position).
//
// Pure data movement: every row is read once and written once.  A CTA takes one to
// four consecutive rows; one warp per row finds its sequence, position and page, and
// all threads then move the rows in units of two 16-byte vectors of a head, D / 2
// apart (the two that rotate together in the halves layout), with two units of each
// thread's loads in flight.  (One CTA per 256 vectors, each warp looking its row up
// for itself, took 50 us at 8192 rows of 32 + 2 x 8 heads of 128, bf16; this takes
// 38.5, 5.3 TB/s or 0.78 of the measured rate of one long copy; a plain copy of as many
// bytes takes 35.5 to 37.5.)
#include "paged_kernels.h"

namespace llama {
namespace {

constexpr int PW_THREADS = 256;
constexpr int PW_CTAS = 3;   // CTAs of an SM (a fourth: 41 us for the 38.5 above)
constexpr int PW_ROWS = 4;   // rows of a CTA, at most
constexpr int PW_UNITS = 2;  // units of a thread in flight

struct PwArgs {
  PagedView pv;
  PackedView b;
  const float2 *table;
  int table_max_seq;
  int H, G, D, rows;  // rows of a CTA
  int unit_log2;      // units of a head: 1 << unit_log2
  int halves;
  int *status;
};

template <typename T>
__global__ void __launch_bounds__(PW_THREADS, PW_CTAS)
    rope_kv_paged_kernel(const T *qkv, T *q_out, T *kc, T *vc, const __grid_constant__ PwArgs a) {
  constexpr int V = Vec16<T>::N;
  __shared__ int s_pos[PW_ROWS], s_page[PW_ROWS];  // position: -1 out of range, -2 no such row
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int t0 = (int)blockIdx.x * a.rows;
  const int heads = a.H + 2 * a.G, units = heads << a.unit_log2;
  const int slot_mask = (1 << a.pv.page_log2) - 1;
  allow_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.b.n_seqs; i += PW_THREADS) check_seq(a.b, a.pv, i, a.status);
  if (warp < a.rows) {
    const int t = t0 + warp;
    const int i = t < a.b.n_tokens ? find_seq(a.b, t) : -1;
    int pos = -2, page = -1;
    if (i >= 0) {
      const SeqSpan s = seq_span(a.b, a.pv, i);
      pos = s.kv_len - (s.first + s.count - t);
      if (pos < 0 || pos >= a.table_max_seq) pos = -1;
      else page = a.pv.page(i, pos >> a.pv.page_log2);
      if (page < 0 && lane == 0) report_status(a.status, LLAMA_ERR_RANGE);
    }
    if (lane == 0) {
      s_pos[warp] = pos;
      s_page[warp] = page;
    }
  }
  __syncthreads();

  // units of the CTA's rows, one row after another
  int row = 0, u = threadIdx.x;
  auto settle = [&] {
    while (u >= units && row < a.rows) {
      u -= units;
      ++row;
    }
  };
  settle();
  while (row < a.rows) {
    Vec16<T> x[PW_UNITS], y[PW_UNITS];
    float4 cs[PW_UNITS][V / 2];
    int r_[PW_UNITS], u_[PW_UNITS];
#pragma unroll
    for (int k = 0; k < PW_UNITS; ++k) {
      r_[k] = row < a.rows && s_pos[row] != -2 ? row : -1;
      u_[k] = u;
      if (r_[k] >= 0) {
        const int head = u >> a.unit_log2, e = (u & ((1 << a.unit_log2) - 1)) * V;
        const T *src = qkv + ((size_t)(t0 + row) * heads + head) * a.D + e;
        x[k].raw = ld_once_after_wait(src);
        y[k].raw = ld_once_after_wait(src + a.D / 2);
        // the unit's V pairs: (e + j, e + j + D/2); or (e + 2j, e + 2j + 1), then those D/2 further
        if (head < a.H + a.G && s_pos[row] >= 0) {  // (the table is made once: a constant here)
          const float4 *c = reinterpret_cast<const float4 *>(a.table + (size_t)s_pos[row] * (a.D / 2) +
                                                             (a.halves ? e : e / 2));
          const float4 *c2 = a.halves ? c + V / 4 : c + a.D / 8;
#pragma unroll
          for (int j = 0; j < V / 4; ++j) {
            cs[k][j] = __ldg(c + j);
            cs[k][V / 4 + j] = __ldg(c2 + j);
          }
        }
      }
      u += PW_THREADS;
      settle();
    }
#pragma unroll
    for (int k = 0; k < PW_UNITS; ++k) {
      if (r_[k] < 0) continue;
      const int head = u_[k] >> a.unit_log2, e = (u_[k] & ((1 << a.unit_log2) - 1)) * V, e2 = e + a.D / 2;
      const int pos = s_pos[r_[k]], page = s_page[r_[k]];
      if (head >= a.H && page < 0) continue;
      T *dst;
      if (head < a.H) {
        dst = q_out + ((size_t)(t0 + r_[k]) * a.H + head) * a.D;
      } else {
        const int g = head < a.H + a.G ? head - a.H : head - a.H - a.G;
        dst = (head < a.H + a.G ? kc : vc) + page * a.pv.page_stride +
              (((long long)g << a.pv.page_log2) + (pos & slot_mask)) * a.D;
      }
      Vec16<T> p = x[k], q = y[k];
      if (pos < 0) {
        p.raw = q.raw = make_uint4(0, 0, 0, 0);
      } else if (head < a.H + a.G) {
        const float2 *c = reinterpret_cast<const float2 *>(cs[k]);
        if (a.halves) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float f = x[k].get(j), g = y[k].get(j);
            p.set(j, f * c[j].x - g * c[j].y);
            q.set(j, f * c[j].y + g * c[j].x);
          }
        } else {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            float f = x[k].get(2 * j), g = x[k].get(2 * j + 1);
            p.set(2 * j, f * c[j].x - g * c[j].y);
            p.set(2 * j + 1, f * c[j].y + g * c[j].x);
            f = y[k].get(2 * j);
            g = y[k].get(2 * j + 1);
            q.set(2 * j, f * c[V / 2 + j].x - g * c[V / 2 + j].y);
            q.set(2 * j + 1, f * c[V / 2 + j].y + g * c[V / 2 + j].x);
          }
        }
      }
      store16(dst + e, p);
      store16(dst + e2, q);
    }
  }
}

}  // namespace

template <typename T>
cudaError_t launch_rope_kv_paged(const T *qkv, T *q_out, T *k, T *v, const PagedView &pv, const PackedView &b,
                                 const float2 *table, int table_max_seq, int H, int G, int D, int halves, int *status,
                                 cudaStream_t st) {
  constexpr int V = Vec16<T>::N;
  PwArgs a;
  a.pv = pv;
  a.b = b;
  a.table = table;
  a.table_max_seq = table_max_seq;
  a.H = H;
  a.G = G;
  a.D = D;
  a.halves = halves;
  a.status = status;
  for (a.unit_log2 = 0; (2 * V) << a.unit_log2 < D; ++a.unit_log2) {
  }
  // few rows: one per CTA, many: enough per CTA that a thread has several units to move
  const int sms = sm_count();
  a.rows = 1;
  while (a.rows < PW_ROWS && b.n_tokens / (2 * a.rows) >= 4 * sms) a.rows *= 2;
  count_launch();
  return launch_pdl(rope_kv_paged_kernel<T>, dim3((unsigned)((b.n_tokens + a.rows - 1) / a.rows)), dim3(PW_THREADS), 0,
                    st, qkv, q_out, k, v, a);
}

template cudaError_t launch_rope_kv_paged<float>(const float *, float *, float *, float *, const PagedView &,
                                                 const PackedView &, const float2 *, int, int, int, int, int, int *,
                                                 cudaStream_t);
template cudaError_t launch_rope_kv_paged<bf16>(const bf16 *, bf16 *, bf16 *, bf16 *, const PagedView &,
                                                const PackedView &, const float2 *, int, int, int, int, int, int *,
                                                cudaStream_t);

}  // namespace llama
