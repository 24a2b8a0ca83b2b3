// RoPE and the write of keys and values into 4-bit cache pages, and the way back
// ("Mini Llama 2 Implementation", Rotary positional embeddings; "Full Llama 3
// transformer block", How it works: rotate, then write at the position).
//
// Both are data movement.  A CTA takes a few consecutive rows; one warp per row finds
// its sequence, position and page.  A thread keeps its place in a row (which head, which
// elements) and goes through the rows, so that the place is worked out once.
//   write  query heads move in units of two 16-byte vectors D / 2 apart, the two that
//          turn together in the halves layout.  Of keys and values a thread takes 32
//          elements, 16 and 16 more D / 2 further: whole blocks, so that a scale is
//          found without asking another thread.
//   read   a thread turns four bytes of codes into eight elements.
// What bounds them is a CTA's chain of look-up, load, arithmetic and store: 8192 rows of
// 4096 + 2 * 1024 bf16 are written in 38 us (4.7 TB/s, 0.69 of the copy rate) and read back
// in 13; 39778 rows of 2 * 1024 are read from memory in 41 (5.1 TB/s, 0.74).  fp32: written in 61 us,
// read back in 23.  (80 registers, of which bf16 spills 12 bytes and fp32 16.)
#include "kv4.cuh"
#include "paged_kernels.h"

namespace llama {
namespace {

constexpr int KW_THREADS = 256;
constexpr int KW_CTAS = 3;   // CTAs of an SM
constexpr int KW_ROWS = 8;   // places for a CTA's rows
constexpr int KW_UNITS = 2;  // rows of a thread in flight
constexpr int KR_UNITS = 4;
// Rows of a CTA at most, written and read: finding their places is shared, but the last CTAs are
// longer.  (8192 rows of 4096 + 2 * 1024 bf16 written: 92, 61, 52, 54 and 54 us at 1, 2, 4, 8 and
// 16, with less arithmetic 51 and 53 at 4 and 8; 40000 rows of 2 * 1024 read: 100, 63, 46, 41 and 41.  Asking for the rows to be written
// before their places are known gains nothing: 53.)
constexpr int KW_MOST = 4, KR_MOST = 8;

struct KwArgs {
  PagedView pv;
  PackedView b;
  const float2 *table;
  int table_max_seq;
  int H, G, D, rows;  // rows of a CTA
  int halves;
  int q_lanes, kv_lanes;  // threads side by side in a row (powers of two)
  int q_log2, kv_log2;    // units of a head: 1 << these
  int *status;
};

// Position and page of the CTA's rows, one warp each: position -1 out of range, -2 no such row.
// Also where the page begins in a pool, in bytes.
__device__ __forceinline__ void find_rows(const PagedView &pv, const PackedView &b, int t0, int rows, int max_pos,
                                          bool early_is_bad, int *s_pos, long long *s_page, int *status) {
  const int lane = threadIdx.x & 31;
  for (int row = threadIdx.x / 32; row < rows; row += KW_THREADS / 32) {
    const int t = t0 + row;
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
      s_pos[row] = pos;
      s_page[row] = page < 0 ? -1 : page * pv.page_stride;
    }
  }
}

// The rotation, every product, difference and sum rounded to fp32 by itself: what is stored
// in 4 bits then follows from the inputs alone, not from which of them the compiler fuses.
__device__ __forceinline__ void turn(float a, float b, float2 c, float &p, float &q) {
  p = __fsub_rn(__fmul_rn(a, c.x), __fmul_rn(b, c.y));
  q = __fadd_rn(__fmul_rn(a, c.y), __fmul_rn(b, c.x));
}

__device__ __forceinline__ void set_two(Vec16<float> &v, int i, float a, float b) {
  v.set(i, a);
  v.set(i + 1, b);
}
__device__ __forceinline__ void set_two(Vec16<bf16> &v, int i, float a, float b) {
  reinterpret_cast<__nv_bfloat162 *>(&v.raw)[i / 2] = __floats2bfloat162_rn(a, b);
}

// N: elements of a thread's unit of keys and values, 32, or 16 where a head has no more.
template <typename T, int N>
__global__ void __launch_bounds__(KW_THREADS, KW_CTAS)
    rope_kv4_kernel(const T *qkv, T *q_out, uint8_t *kc, uint8_t *vc, const __grid_constant__ KwArgs a) {
  constexpr int V = Vec16<T>::N;
  __shared__ int s_pos[KW_ROWS];
  __shared__ long long s_page[KW_ROWS];
  const int t0 = (int)blockIdx.x * a.rows;
  const int heads = a.H + 2 * a.G;
  allow_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.b.n_seqs; i += KW_THREADS) check_seq(a.b, a.pv, i, a.status);
  find_rows(a.pv, a.b, t0, a.rows, a.table_max_seq, true, s_pos, s_page, a.status);
  __syncthreads();

  // (the table is made once: a constant here)
  auto angles = [&](int pos, int at) { return a.table + (size_t)pos * (a.D / 2) + at; };

  // Keys and values first: theirs is the longer way.
  const int kv_units = 2 * a.G << a.kv_log2, kv_rows = KW_THREADS / a.kv_lanes;
  for (int u = threadIdx.x & (a.kv_lanes - 1); u < kv_units; u += a.kv_lanes) {
    // elements e .., and those D / 2 further
    const int head = u >> a.kv_log2, e = (u & ((1 << a.kv_log2) - 1)) * (N / 2);
    const bool key = head < a.G;
    uint8_t *const block =
        (key ? kc : vc) + (long long)(key ? head : head - a.G) * kv4_block_bytes(1 << a.pv.page_log2, a.D);
    const T *const first = qkv + ((size_t)t0 * heads + a.H + head) * a.D;
    for (int row = threadIdx.x / a.kv_lanes; row < a.rows; row += kv_rows) {
      const int pos = s_pos[row];
      const long long page = s_page[row];
      if (pos < 0 || page < 0) continue;
      const T *src = first + (size_t)row * (heads * a.D);
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
      const int slot = pos & ((1 << a.pv.page_log2) - 1);
      uint8_t *codes = block + page + slot * kv4_code_bytes(a.D);
      uint8_t *scales = block + page + (kv4_code_bytes(a.D) << a.pv.page_log2) + slot * kv4_scale_bytes(a.D);
      bool bad = false;
      // blocks of 16: at e and, with N = 32, at e + D / 2
#pragma unroll
      for (int j = 0; j < N / KV4_BLOCK; ++j) {
        const int at = N == 32 ? e + j * (a.D / 2) : 0;
        uint32_t w[2];
        const uint32_t byte = kv4_quantise(reinterpret_cast<float(&)[KV4_BLOCK]>(x[j * KV4_BLOCK]), w, bad);
        *reinterpret_cast<uint2 *>(codes + at / 2) = make_uint2(w[0], w[1]);
        scales[at / KV4_BLOCK] = (uint8_t)byte;
      }
      if (bad) report_status(a.status, LLAMA_ERR_RANGE);
    }
  }

  const int q_units = a.H << a.q_log2, q_rows = KW_THREADS / a.q_lanes;
  for (int u = threadIdx.x & (a.q_lanes - 1); u < q_units; u += a.q_lanes) {
    const int head = u >> a.q_log2, e = (u & ((1 << a.q_log2) - 1)) * V;
    const T *const q_first = qkv + ((size_t)t0 * heads + head) * a.D + e;
    T *const out = q_out + ((size_t)t0 * a.H + head) * a.D + e;
    for (int r0 = threadIdx.x / a.q_lanes; r0 < a.rows; r0 += KW_UNITS * q_rows) {
      Vec16<T> x[KW_UNITS], y[KW_UNITS];
      float4 cs[KW_UNITS][V / 2];
      int pos[KW_UNITS];
      size_t at[KW_UNITS];
#pragma unroll
      for (int k = 0; k < KW_UNITS; ++k) {
        const int row = r0 + k * q_rows;
        pos[k] = row < a.rows ? s_pos[row] : -2;
        if (pos[k] == -2) continue;
        const T *src = q_first + (size_t)row * (heads * a.D);
        at[k] = (size_t)row * (a.H * a.D);
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
          float f, g, f2, g2;
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            if (a.halves) {
              turn(x[k].get(j), y[k].get(j), c[j], f, g);
              turn(x[k].get(j + 1), y[k].get(j + 1), c[j + 1], f2, g2);
            } else {
              turn(x[k].get(j), x[k].get(j + 1), c[j / 2], f, f2);
              turn(y[k].get(j), y[k].get(j + 1), c[V / 2 + j / 2], g, g2);
            }
            set_two(p, j, f, f2);
            set_two(q, j, g, g2);
          }
        }
        store16(out + at[k], p);
        store16(out + at[k] + a.D / 2, q);
      }
    }
  }
}

struct KrArgs {
  PagedView pv;
  PackedView b;
  const uint8_t *k, *v;
  int G, D, rows, word_log2;  // words of eight elements of a head: 1 << word_log2
  int lanes;
  int *status;
};

template <typename T>
__global__ void __launch_bounds__(KW_THREADS) kv4_read_kernel(T *k_out, T *v_out, const __grid_constant__ KrArgs a) {
  __shared__ int s_pos[KW_ROWS];
  __shared__ long long s_page[KW_ROWS];
  const int t0 = (int)blockIdx.x * a.rows;
  allow_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.b.n_seqs; i += KW_THREADS) check_seq(a.b, a.pv, i, a.status);
  find_rows(a.pv, a.b, t0, a.rows, INT_MAX, false, s_pos, s_page, a.status);
  __syncthreads();
  const int head_units = a.G << a.word_log2, units = 2 * head_units;  // of a row: k's, then v's
  const int slot_mask = (1 << a.pv.page_log2) - 1, step = KW_THREADS / a.lanes;
  for (int u = threadIdx.x & (a.lanes - 1); u < units; u += a.lanes) {
    const bool value = u >= head_units;
    T *const out = value ? v_out : k_out;
    if (out == nullptr) continue;
    const int g = (value ? u - head_units : u) >> a.word_log2, e = u & ((1 << a.word_log2) - 1);
    const Kv4Row first = kv4_row(value ? a.v : a.k, a.pv, 0, g, a.D, 0);
    const uint8_t *const codes = first.codes + 4 * e, *const scales = first.scales + e / 2;
    T *const dst0 = out + ((size_t)t0 * a.G + g) * a.D + e * 8;
    for (int r0 = threadIdx.x / a.lanes; r0 < a.rows; r0 += KR_UNITS * step) {
      uint32_t w[KR_UNITS], byte[KR_UNITS];
      T *dst[KR_UNITS];
#pragma unroll
      for (int i = 0; i < KR_UNITS; ++i) {
        const int row = r0 + i * step;
        dst[i] = nullptr;
        w[i] = 0x88888888u;  // zeros
        byte[i] = 0;
        const int pos = row < a.rows ? s_pos[row] : -2;
        if (pos == -2) continue;
        dst[i] = dst0 + (size_t)row * (a.G * a.D);
        const long long page = s_page[row];
        if (page < 0) continue;
        const int slot = pos & slot_mask;
        w[i] = (uint32_t)ld_after_wait(reinterpret_cast<const int *>(codes + page + slot * kv4_code_bytes(a.D)));
        asm volatile("ld.global.u8 %0, [%1];" : "=r"(byte[i]) : "l"(scales + page + slot * kv4_scale_bytes(a.D)));
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
}

// Rows of a CTA: one where rows are few, else enough that a thread has several to go through.
int rows_of(int n_tokens, int most) {
  const int sms = sm_count();
  int rows = 1;
  while (rows < most && n_tokens / (2 * rows) >= 4 * sms) rows *= 2;
  return rows;
}
int log2_of(int n) {  // of a power of two
  int k = 0;
  while (1 << k < n) ++k;
  return k;
}
// Threads side by side in a row of `units`.
int lanes_of(int units) {
  int n = 1;
  while (n < KW_THREADS && n < units) n *= 2;
  return n;
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
  a.rows = rows_of(b.n_tokens, KW_MOST);
  a.q_log2 = log2_of(D / (2 * Vec16<T>::N));
  a.kv_log2 = log2_of(D == 16 ? 1 : D / 32);
  a.q_lanes = lanes_of(H << a.q_log2);
  a.kv_lanes = lanes_of(2 * G << a.kv_log2);
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
  a.word_log2 = log2_of(D / 8);
  a.status = status;
  a.rows = rows_of(b.n_tokens, KR_MOST);
  a.lanes = lanes_of(2 * G * D / 8);
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
