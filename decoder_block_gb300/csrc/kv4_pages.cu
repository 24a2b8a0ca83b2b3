// RoPE and the write of keys and values into 4-bit cache pages, and the way back
// ("Mini Llama 2 Implementation", Rotary positional embeddings; "Full Llama 3
// transformer block", How it works: rotate, then write at the position).
//
// Both are data movement.  A CTA takes a few consecutive rows; one warp per row finds
// its sequence, position and page.
//   write  query heads move in units of two 16-byte vectors D / 2 apart, the two that
//          turn together in the halves layout.  Of keys and values a thread takes 32
//          elements, 16 and 16 more D / 2 further: whole blocks, so that a scale is
//          found without asking another thread.
//   read   a thread turns four bytes of codes into eight elements.
#include "kv4.cuh"
#include "paged_kernels.h"

namespace llama {
namespace {

constexpr int KW_THREADS = 256;
constexpr int KW_CTAS = 3;   // CTAs of an SM
constexpr int KW_ROWS = 4;   // rows of a CTA, at most
constexpr int KW_UNITS = 2;  // units of a thread in flight
constexpr int KR_UNITS = 4;

struct KwArgs {
  PagedView pv;
  PackedView b;
  const float2 *table;
  int table_max_seq;
  int H, G, D, rows;  // rows of a CTA
  int halves;
  int *status;
};

// Position and page of the CTA's rows, one warp each: position -1 out of range, -2 no such row.
__device__ __forceinline__ void find_rows(const PagedView &pv, const PackedView &b, int t0, int rows, int max_pos,
                                          bool early_is_bad, int *s_pos, int *s_page, int *status) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (warp >= rows) return;
  const int t = t0 + warp;
  const int i = t < b.n_tokens ? find_seq(b, t) : -1;
  int pos = -2, page = -1;
  if (i >= 0) {
    const SeqSpan s = seq_span(b, pv, i);
    pos = s.kv_len - (s.first + s.count - t);
    if (pos < 0 || pos >= max_pos) {
      if ((pos >= 0 || early_is_bad) && lane == 0) report_status(status, LLAMA_ERR_RANGE);
      pos = -1;
    } else {
      page = pv.page(i, pos >> pv.page_log2);
      if (page < 0 && lane == 0) report_status(status, LLAMA_ERR_RANGE);
    }
  }
  if (lane == 0) {
    s_pos[warp] = pos;
    s_page[warp] = page;
  }
}

// The rotation, every product, difference and sum rounded to fp32 by itself: what is stored
// in 4 bits then follows from the inputs alone, not from which of them the compiler fuses.
__device__ __forceinline__ void turn(float a, float b, float2 c, float &p, float &q) {
  p = __fsub_rn(__fmul_rn(a, c.x), __fmul_rn(b, c.y));
  q = __fadd_rn(__fmul_rn(a, c.y), __fmul_rn(b, c.x));
}

// N: elements of a thread's unit of keys and values, 32, or 16 where a head has no more.
template <typename T, int N>
__global__ void __launch_bounds__(KW_THREADS, KW_CTAS)
    rope_kv4_kernel(const T *qkv, T *q_out, uint8_t *kc, uint8_t *vc, const __grid_constant__ KwArgs a) {
  constexpr int V = Vec16<T>::N;
  __shared__ int s_pos[KW_ROWS], s_page[KW_ROWS];
  const int t0 = (int)blockIdx.x * a.rows;
  const int heads = a.H + 2 * a.G, per_head = a.D / (2 * V);
  allow_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.b.n_seqs; i += KW_THREADS) check_seq(a.b, a.pv, i, a.status);
  find_rows(a.pv, a.b, t0, a.rows, a.table_max_seq, true, s_pos, s_page, a.status);
  __syncthreads();

  // (the table is made once: a constant here)
  auto angles = [&](int pos, int at) { return a.table + (size_t)pos * (a.D / 2) + at; };

  // Keys and values first: theirs is the longer way.
  const int kv_units = 2 * a.G * (a.D / N);
  for (int u0 = threadIdx.x; u0 < a.rows * kv_units; u0 += KW_THREADS) {
    const int row = u0 / kv_units, u = u0 % kv_units;
    const int pos = s_pos[row], page = s_page[row];
    if (pos < 0 || page < 0) continue;
    const int head = u / (a.D / N), e = u % (a.D / N) * (N / 2);  // elements e .., and those D / 2 further
    const bool key = head < a.G;
    const T *src = qkv + ((size_t)(t0 + row) * heads + a.H + head) * a.D;
    float x[N];
#pragma unroll
    for (int j = 0; j < N; j += V) {
      Vec16<T> v;
      v.raw = ld_once_after_wait(src + (j < N / 2 ? e + j : a.D / 2 + e + j - N / 2));
#pragma unroll
      for (int k = 0; k < V; ++k) x[j + k] = v.get(k);
    }
    if (key && a.halves) {
      const float4 *c = reinterpret_cast<const float4 *>(angles(pos, e));
#pragma unroll
      for (int j = 0; j < N / 2; j += 2) {
        const float4 f = __ldg(c + j / 2);
        turn(x[j], x[N / 2 + j], make_float2(f.x, f.y), x[j], x[N / 2 + j]);
        turn(x[j + 1], x[N / 2 + j + 1], make_float2(f.z, f.w), x[j + 1], x[N / 2 + j + 1]);
      }
    } else if (key) {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(
            angles(pos, j < N / 2 ? (e + j) / 2 : (a.D / 2 + e + j - N / 2) / 2)));
        turn(x[j], x[j + 1], make_float2(f.x, f.y), x[j], x[j + 1]);
        turn(x[j + 2], x[j + 3], make_float2(f.z, f.w), x[j + 2], x[j + 3]);
      }
    }
    const int g = key ? head : head - a.G, slot = pos & ((1 << a.pv.page_log2) - 1);
    const Kv4Row r = kv4_row(key ? kc : vc, a.pv, page, g, a.D, slot);
    bool bad = false;
    // blocks of 16: at e and, with N = 32, at e + D / 2
#pragma unroll
    for (int j = 0; j < N / KV4_BLOCK; ++j) {
      const int at = N == 32 ? e + j * (a.D / 2) : 0;
      uint32_t w[2];
      const uint32_t byte = kv4_quantise(x + j * KV4_BLOCK, w, bad);
      *reinterpret_cast<uint2 *>(const_cast<uint8_t *>(r.codes) + at / 2) = make_uint2(w[0], w[1]);
      const_cast<uint8_t *>(r.scales)[at / KV4_BLOCK] = (uint8_t)byte;
    }
    if (bad) report_status(a.status, LLAMA_ERR_RANGE);
  }

  const int q_units = a.H * per_head;
  for (int u0 = threadIdx.x; u0 < a.rows * q_units; u0 += KW_THREADS * KW_UNITS) {
    Vec16<T> x[KW_UNITS], y[KW_UNITS];
    float4 cs[KW_UNITS][V / 2];
    int pos[KW_UNITS];
    size_t at[KW_UNITS];
#pragma unroll
    for (int k = 0; k < KW_UNITS; ++k) {
      const int uu = u0 + k * KW_THREADS;
      pos[k] = -2;
      if (uu >= a.rows * q_units) continue;
      const int row = uu / q_units, u = uu % q_units;
      pos[k] = s_pos[row];
      if (pos[k] == -2) continue;
      const int head = u / per_head, e = u % per_head * V;
      const T *src = qkv + ((size_t)(t0 + row) * heads + head) * a.D + e;
      at[k] = ((size_t)(t0 + row) * a.H + head) * a.D + e;
      x[k].raw = ld_once_after_wait(src);
      y[k].raw = ld_once_after_wait(src + a.D / 2);
      if (pos[k] >= 0) {
        // the unit's V pairs: (e + j, e + j + D/2); or (e + 2j, e + 2j + 1), then those D/2 further
        const float4 *c = reinterpret_cast<const float4 *>(angles(pos[k], a.halves ? e : e / 2));
        const float4 *c2 = a.halves ? c + V / 4 : c + a.D / 8;
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
          cs[k][j] = __ldg(c + j);
          cs[k][V / 4 + j] = __ldg(c2 + j);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < KW_UNITS; ++k) {
      if (pos[k] == -2) continue;
      Vec16<T> p, q;
      if (pos[k] < 0) {
        p.raw = q.raw = make_uint4(0, 0, 0, 0);
      } else {
        const float2 *c = reinterpret_cast<const float2 *>(cs[k]);
        float f, g;
        if (a.halves) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            turn(x[k].get(j), y[k].get(j), c[j], f, g);
            p.set(j, f);
            q.set(j, g);
          }
        } else {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            turn(x[k].get(2 * j), x[k].get(2 * j + 1), c[j], f, g);
            p.set(2 * j, f);
            p.set(2 * j + 1, g);
            turn(y[k].get(2 * j), y[k].get(2 * j + 1), c[V / 2 + j], f, g);
            q.set(2 * j, f);
            q.set(2 * j + 1, g);
          }
        }
      }
      store16(q_out + at[k], p);
      store16(q_out + at[k] + a.D / 2, q);
    }
  }
}

struct KrArgs {
  PagedView pv;
  PackedView b;
  const uint8_t *k, *v;
  int G, D, rows, word_log2;  // words of eight elements of a head: 1 << word_log2
  int *status;
};

template <typename T>
__global__ void __launch_bounds__(KW_THREADS) kv4_read_kernel(T *k_out, T *v_out, const __grid_constant__ KrArgs a) {
  __shared__ int s_pos[KW_ROWS], s_page[KW_ROWS];
  const int t0 = (int)blockIdx.x * a.rows;
  allow_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.b.n_seqs; i += KW_THREADS) check_seq(a.b, a.pv, i, a.status);
  find_rows(a.pv, a.b, t0, a.rows, INT_MAX, false, s_pos, s_page, a.status);
  __syncthreads();
  const int head_units = a.G << a.word_log2, units = 2 * head_units;  // of a row: k's, then v's
  for (int u0 = threadIdx.x; u0 < a.rows * units; u0 += KW_THREADS * KR_UNITS) {
    uint32_t w[KR_UNITS], byte[KR_UNITS];
    T *dst[KR_UNITS];
#pragma unroll
    for (int i = 0; i < KR_UNITS; ++i) {
      const int uu = u0 + i * KW_THREADS;
      dst[i] = nullptr;
      w[i] = 0x88888888u;  // zeros
      byte[i] = 0;
      if (uu >= a.rows * units) continue;
      const int row = uu / units, u = uu % units;
      if (s_pos[row] == -2) continue;
      const bool value = u >= head_units;
      T *out = value ? v_out : k_out;
      if (out == nullptr) continue;
      const int g = (value ? u - head_units : u) >> a.word_log2, e = u & ((1 << a.word_log2) - 1);
      dst[i] = out + ((size_t)(t0 + row) * a.G + g) * a.D + e * 8;
      if (s_page[row] < 0) continue;
      const Kv4Row r = kv4_row(value ? a.v : a.k, a.pv, s_page[row], g, a.D, s_pos[row] & ((1 << a.pv.page_log2) - 1));
      w[i] = (uint32_t)ld_after_wait(reinterpret_cast<const int *>(r.codes) + e);
      asm volatile("ld.global.u8 %0, [%1];" : "=r"(byte[i]) : "l"(r.scales + e / 2));
    }
#pragma unroll
    for (int i = 0; i < KR_UNITS; ++i) {
      if (dst[i] == nullptr) continue;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(dst[i]) = kv4_eight(w[i], kv4_scales(byte[i]));
      } else {
        const float s = kv4_scale(byte[i]);
        reinterpret_cast<float4 *>(dst[i])[0] = kv4_four(w[i], 0, s);
        reinterpret_cast<float4 *>(dst[i])[1] = kv4_four(w[i], 1, s);
      }
    }
  }
}

// Rows of a CTA: one where rows are few, else enough that a thread has several units to move.
int rows_of(int n_tokens) {
  const int sms = sm_count();
  int rows = 1;
  while (rows < KW_ROWS && n_tokens / (2 * rows) >= 4 * sms) rows *= 2;
  return rows;
}

}  // namespace

template <typename T>
cudaError_t launch_rope_kv4(const T *qkv, T *q_out, uint8_t *k, uint8_t *v, const PagedView &pv, const PackedView &b,
                            const float2 *table, int table_max_seq, int H, int G, int D, int halves, int *status,
                            cudaStream_t st) {
  KwArgs a;
  a.pv = pv;
  a.b = b;
  a.table = table;
  a.table_max_seq = table_max_seq;
  a.H = H;
  a.G = G;
  a.D = D;
  a.halves = halves;
  a.status = status;
  a.rows = rows_of(b.n_tokens);
  count_launch();
  return launch_pdl(D == 16 ? rope_kv4_kernel<T, 16> : rope_kv4_kernel<T, 32>,
                    dim3((unsigned)((b.n_tokens + a.rows - 1) / a.rows)), dim3(KW_THREADS), 0, st, qkv, q_out, k, v, a);
}

template <typename T>
cudaError_t launch_kv4_read(const uint8_t *k, const uint8_t *v, T *k_out, T *v_out, const PagedView &pv,
                            const PackedView &b, int G, int D, int *status, cudaStream_t st) {
  KrArgs a;
  a.pv = pv;
  a.b = b;
  a.k = k;
  a.v = v;
  a.G = G;
  a.D = D;
  for (a.word_log2 = 0; 8 << a.word_log2 < D; ++a.word_log2) {
  }
  a.status = status;
  a.rows = rows_of(b.n_tokens);
  count_launch();
  return launch_pdl(kv4_read_kernel<T>, dim3((unsigned)((b.n_tokens + a.rows - 1) / a.rows)), dim3(KW_THREADS), 0, st,
                    k_out, v_out, a);
}

template cudaError_t launch_rope_kv4<float>(const float *, float *, uint8_t *, uint8_t *, const PagedView &,
                                            const PackedView &, const float2 *, int, int, int, int, int, int *,
                                            cudaStream_t);
template cudaError_t launch_rope_kv4<bf16>(const bf16 *, bf16 *, uint8_t *, uint8_t *, const PagedView &,
                                           const PackedView &, const float2 *, int, int, int, int, int, int *,
                                           cudaStream_t);
template cudaError_t launch_kv4_read<float>(const uint8_t *, const uint8_t *, float *, float *, const PagedView &,
                                            const PackedView &, int, int, int *, cudaStream_t);
template cudaError_t launch_kv4_read<bf16>(const uint8_t *, const uint8_t *, bf16 *, bf16 *, const PagedView &,
                                           const PackedView &, int, int, int *, cudaStream_t);

}  // namespace llama
