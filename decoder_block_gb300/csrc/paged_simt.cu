// fp32 attention over cache pages on CUDA cores ("The Evolving Transformer 04 ·
// LLaMA", §05 GQA; "Full Llama 3 transformer block", How it works: keys
// j <= position).  One pass over the keys with the running maximum and sum of the
// softmax; fp32 products and sums throughout.
#include <float.h>
#include <math.h>

#include "paged_kernels.h"
#include "ptx.cuh"

namespace llama {
namespace {

// ---------------------------------------------------------------- packed ---
// CTA = (sequence, KV head g, 64 rows of the flattened (position, head of the
// group) index R = position * r + hh): the r heads of a group share every K/V
// tile, and no row is padding but in a sequence's last tile.  256 threads, 4 x 4
// scores and 4 x (D / 16) outputs per thread.
constexpr int PS_ROWS = 64, PS_KEYS = 64, PS_THREADS = 256;

template <int D>
struct PsLayout {
  static constexpr int LDQ = D + 4, LDP = PS_KEYS + 4;  // rows 16 bytes apart in banks
  static constexpr int OFF_K = PS_ROWS * LDQ;
  static constexpr int OFF_V = OFF_K + PS_KEYS * LDQ;
  static constexpr int OFF_P = OFF_V + PS_KEYS * LDQ;
  static constexpr int BYTES = (OFF_P + PS_ROWS * LDP) * 4;
};

// Stages rows of 16-byte vectors as fp32; `row_ptr(i)` null gives zeros.
template <int D, typename F>
__device__ __forceinline__ void stage_rows(float *dst, int rows, F &&row_ptr) {
  constexpr int V = Vec16<float>::N, RV = D / V;
  for (int u = threadIdx.x; u < rows * RV; u += blockDim.x) {
    const int i = u / RV, c = (u % RV) * V;
    const float *p = row_ptr(i);
    Vec16<float> x;
    x.raw = make_uint4(0, 0, 0, 0);
    if (p != nullptr) x = load16(p + c);
    float *d = dst + i * (D + 4) + c;
#pragma unroll
    for (int k = 0; k < V; k += 4)
      *reinterpret_cast<float4 *>(d + k) = make_float4(x.get(k), x.get(k + 1), x.get(k + 2), x.get(k + 3));
  }
}

template <int D>
__global__ void __launch_bounds__(PS_THREADS) packed_simt_kernel(const float *__restrict__ q, const float *__restrict__ kc,
                                                                 const float *__restrict__ vc, float *__restrict__ o,
                                                                 PagedView pv, PackedView b, int H, int G, float scale,
                                                                 int *status) {
  using L = PsLayout<D>;
  extern __shared__ __align__(16) float smem_f[];
  float *sq = smem_f, *sk = smem_f + L::OFF_K, *sv = smem_f + L::OFF_V, *sp = smem_f + L::OFF_P;
  const int r = H / G, g = blockIdx.y;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  if (blockIdx.x == 0 && g == 0)
    for (int i = threadIdx.x; i < b.n_seqs; i += blockDim.x) check_seq(b, pv, i, status);
  // block -> (sequence, tile): the grid holds at least one block for every tile
  __shared__ int found[2];
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  if (threadIdx.x < 32) {
    int base = 0;
    for (int i0 = 0; i0 < b.n_seqs; i0 += 32) {
      const int i = i0 + threadIdx.x;
      const int n = i < b.n_seqs ? (int)(((long long)seq_span(b, pv, i).count * r + PS_ROWS - 1) / PS_ROWS) : 0;
      int end = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, end, off);
        if (threadIdx.x >= off) end += x;
      }
      const int mine = (int)blockIdx.x - base - (end - n);
      if (mine >= 0 && mine < n) {
        found[0] = i;
        found[1] = mine;
      }
      base += __shfl_sync(0xffffffffu, end, 31);
      if (base > (int)blockIdx.x) break;
    }
  }
  __syncthreads();
  const int seq = found[0], tile = found[1];
  if (seq < 0) return;
  const SeqSpan s = seq_span(b, pv, seq);
  const int row0 = tile * PS_ROWS;
  const int rows = min(PS_ROWS, s.count * r - row0);
  const int shift = s.kv_len - s.count;  // position of the sequence's first new token

  stage_rows<D>(sq, PS_ROWS, [&](int i) -> const float * {
    if (i >= rows) return nullptr;
    const int R = row0 + i;
    return q + ((size_t)(s.first + R / r) * H + g * r + R % r) * D;
  });
  int pos[4];
  float m[4], l[4], acc[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int R = row0 + min(ty * 4 + i, rows - 1);
    pos[i] = shift + R / r;
    m[i] = -FLT_MAX;  // finite: a row that sees no key keeps weights of 0 instead of NaN
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
  }
  const int n_keys = min(s.kv_len, shift + (row0 + rows - 1) / r + 1);
  for (int k0 = 0; k0 < n_keys; k0 += PS_KEYS) {
    __syncthreads();
    auto row_of = [&](const float *pool, int j) -> const float * {
      const int p = k0 + j;
      if (p >= s.kv_len) return nullptr;
      const int page = pv.page(seq, p >> pv.page_log2);
      if (page < 0) return nullptr;
      return pool + page * pv.page_stride +
             (((long long)g << pv.page_log2) + (p & ((1 << pv.page_log2) - 1))) * D;
    };
    stage_rows<D>(sk, PS_KEYS, [&](int j) { return row_of(kc, j); });
    stage_rows<D>(sv, PS_KEYS, [&](int j) { return row_of(vc, j); });
    if (threadIdx.x < PS_KEYS) {
      const int p = k0 + (int)threadIdx.x;
      if (p < s.kv_len && pv.page(seq, p >> pv.page_log2) < 0) report_status(status, LLAMA_ERR_RANGE);
    }
    __syncthreads();
    // scores of rows ty*4 + i against keys tx + 16 j
    float sc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 a[4], c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (ty * 4 + i) * L::LDQ + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * L::LDQ + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sc[i][j] = fmaf(a[i].x, c[j].x, fmaf(a[i].y, c[j].y, fmaf(a[i].z, c[j].z, fmaf(a[i].w, c[j].w, sc[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sc[i][j] = k0 + tx + 16 * j <= pos[i] ? sc[i][j] * scale : -INFINITY;
        mt = fmaxf(mt, sc[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
      const float mn = fmaxf(m[i], mt);
      const float corr = expf(m[i] - mn);
      m[i] = mn;
      float ls = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(sc[i][j] - mn);
        ls += p;
        sp[(ty * 4 + i) * L::LDP + tx + 16 * j] = p;
      }
      l[i] = l[i] * corr + ls;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) acc[i][c] *= corr;
    }
    __syncwarp();  // a row's 16 threads are half a warp: only they read its weights
    // outputs of rows ty*4 + i, columns tx + 16 c
#pragma unroll 4
    for (int j = 0; j < PS_KEYS; j += 4) {
      float4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(sp + (ty * 4 + i) * L::LDP + j);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const float *vp = sv + j * L::LDQ + tx + 16 * c;
        const float v0 = vp[0], v1 = vp[L::LDQ], v2 = vp[2 * L::LDQ], v3 = vp[3 * L::LDQ];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[i][c] = fmaf(w[i].x, v0, fmaf(w[i].y, v1, fmaf(w[i].z, v2, fmaf(w[i].w, v3, acc[i][c]))));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float ls = l[i];
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
    const int R = row0 + ty * 4 + i;
    if (ty * 4 + i >= rows) continue;
    const float inv = ls > 0.f ? 1.f / ls : 0.f;
    float *dst = o + ((size_t)(s.first + R / r) * H + g * r + R % r) * D;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) dst[tx + 16 * c] = (acc[i][c] * inv);
  }
}

template <int D>
cudaError_t packed_simt(const float *q, const float *k, const float *v, float *o, const PagedView &pv, const PackedView &b, int H,
                        int G, int *status, cudaStream_t st) {
  static PerContextOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(packed_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                PsLayout<D>::BYTES);
  });
  if (e != cudaSuccess) return e;
  // every sequence ends in at most one tile that is not full
  const long long tiles = (long long)b.n_tokens * (H / G) / PS_ROWS + b.n_seqs;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  count_launch();
  packed_simt_kernel<D><<<dim3((unsigned)tiles, (unsigned)G), PS_THREADS, PsLayout<D>::BYTES, st>>>(
      q, k, v, o, pv, b, H, G, 1.0f / sqrtf((float)D), status);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- decode ---
// CTA = (part of the keys, sequence, KV head and block of up to 8 of its query
// heads); 64 keys at a time staged as fp32.
constexpr int PD_KEYS = 64, PD_THREADS = 256, PD_HEADS = 8;

// Split of one sequence's keys over CTAs: parts of `chunk` keys, `n` of them at the
// longest length the call allows.
struct DecodeSplit {
  int chunk = 0, n = 1;
};
DecodeSplit decode_split(int n_seqs, int max_kv_len, int H, int G) {
  // About four CTAs per SM when the batch alone does not give them, parts of at
  // least 128 keys (two tiles) so that the join stays small beside them.
  const long long ctas = (long long)n_seqs * G * ((H / G + PD_HEADS - 1) / PD_HEADS);
  const long long want = (4 * 152 + ctas - 1) / ctas, most = (max_kv_len + 127) / 128;
  const int n = (int)(want < most ? want : most > 1 ? most : 1);
  DecodeSplit s;
  s.chunk = ((max_kv_len + n - 1) / n + PD_KEYS - 1) / PD_KEYS * PD_KEYS;
  if (s.chunk < PD_KEYS) s.chunk = PD_KEYS;
  s.n = (max_kv_len + s.chunk - 1) / s.chunk;
  if (s.n < 1) s.n = 1;
  return s;
}

template <int D>
__global__ void __launch_bounds__(PD_THREADS) paged_decode_simt_kernel(const float *__restrict__ q,
                                                                       const float *__restrict__ kc,
                                                                       const float *__restrict__ vc, float *__restrict__ o,
                                                                       float *__restrict__ part, PagedView pv,
                                                                       const int *__restrict__ kv_lens, int max_kv_len,
                                                                       int H, int G, DecodeSplit split, float scale,
                                                                       int *status) {
  constexpr int LDQ = D + 4, SLICES = PD_THREADS / D;
  constexpr int RED = SLICES * PD_HEADS * D, TILE = PD_KEYS * LDQ;
  __shared__ __align__(16) float sk[TILE > RED ? TILE : RED];  // K, then V, of one tile; at the end the slices
  __shared__ __align__(16) float sq[PD_HEADS * D];
  __shared__ float sp[PD_HEADS][PD_KEYS + 1];
  __shared__ float sm[PD_HEADS], sl[PD_HEADS], sc[PD_HEADS];
  const int r = H / G, blocks = (r + PD_HEADS - 1) / PD_HEADS;
  const int g = blockIdx.z / blocks, h0 = (blockIdx.z % blocks) * PD_HEADS;
  const int nh = min(PD_HEADS, r - h0), seq = blockIdx.y;
  const int raw_len = __ldg(kv_lens + seq);
  const int len = checked_len(raw_len, max_kv_len, pv);
  if (len != raw_len && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) report_status(status, LLAMA_ERR_RANGE);
  const int k0 = blockIdx.x * split.chunk, k1 = min(len, k0 + split.chunk);
  if (k0 >= len && !(blockIdx.x == 0 && split.n == 1)) return;
  const size_t bh = (size_t)seq * H + g * r + h0;

  for (int u = threadIdx.x; u < nh * D; u += PD_THREADS) sq[u] = (q[bh * D + u]) * scale;
  if (threadIdx.x < PD_HEADS) {
    sm[threadIdx.x] = -INFINITY;
    sl[threadIdx.x] = 0.f;
  }
  const int d = threadIdx.x % D, slice = threadIdx.x / D;
  float acc[PD_HEADS];
#pragma unroll
  for (int h = 0; h < PD_HEADS; ++h) acc[h] = 0.f;
  for (int t0 = k0; t0 < k1; t0 += PD_KEYS) {
    const int n = min(PD_KEYS, k1 - t0);
    auto row_of = [&](const float *pool, int j) -> const float * {
      if (j >= n) return nullptr;
      const int p = t0 + j;
      const int page = pv.page(seq, p >> pv.page_log2);
      if (page < 0) return nullptr;
      return pool + page * pv.page_stride + (((long long)g << pv.page_log2) + (p & ((1 << pv.page_log2) - 1))) * D;
    };
    __syncthreads();
    stage_rows<D>(sk, PD_KEYS, [&](int j) { return row_of(kc, j); });
    if (threadIdx.x < n && pv.page(seq, (t0 + (int)threadIdx.x) >> pv.page_log2) < 0)
      report_status(status, LLAMA_ERR_RANGE);
    __syncthreads();
    {
      const int key = threadIdx.x % PD_KEYS;
      for (int h = threadIdx.x / PD_KEYS; h < nh; h += PD_THREADS / PD_KEYS) {
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < D; e += 4) {
          const float4 a = *reinterpret_cast<const float4 *>(sq + h * D + e);
          const float4 c = *reinterpret_cast<const float4 *>(sk + key * LDQ + e);
          x = fmaf(a.x, c.x, fmaf(a.y, c.y, fmaf(a.z, c.z, fmaf(a.w, c.w, x))));
        }
        sp[h][key] = key < n ? x : -INFINITY;
      }
    }
    __syncthreads();
    // warp h: the running maximum and sum of head h; every tile holds a key, so the maximum is one
    const int h = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (h < nh) {
      const float a = sp[h][lane], c = sp[h][lane + 32];
      const float mn = fmaxf(sm[h], warp_max(fmaxf(a, c)));
      const float pa = expf(a - mn), pc = expf(c - mn);
      const float ls = warp_sum(pa + pc);
      sp[h][lane] = pa;
      sp[h][lane + 32] = pc;
      __syncwarp();
      if (lane == 0) {
        const float corr = expf(sm[h] - mn);
        sc[h] = corr;
        sl[h] = sl[h] * corr + ls;
        sm[h] = mn;
      }
    }
    stage_rows<D>(sk, PD_KEYS, [&](int j) { return row_of(vc, j); });
    __syncthreads();
#pragma unroll
    for (int hh = 0; hh < PD_HEADS; ++hh)
      if (hh < nh) {
        float a = acc[hh] * sc[hh];
        for (int j = slice; j < n; j += SLICES) a = fmaf(sp[hh][j], sk[j * LDQ + d], a);
        acc[hh] = a;
      }
  }
  // join the slices of the keys
  __syncthreads();
  float *red = sk;  // [SLICES][PD_HEADS][D]
#pragma unroll
  for (int hh = 0; hh < PD_HEADS; ++hh)
    if (hh < nh) red[(slice * PD_HEADS + hh) * D + d] = acc[hh];
  __syncthreads();
  for (int u = threadIdx.x; u < nh * D; u += PD_THREADS) {
    const int hh = u / D, e = u % D;
    float x = 0.f;
#pragma unroll
    for (int s = 0; s < SLICES; ++s) x += red[(s * PD_HEADS + hh) * D + e];
    if (split.n == 1) {
      o[bh * D + u] = (sl[hh] > 0.f ? x / sl[hh] : 0.f);
    } else {
      float *pp = part + ((bh + hh) * split.n + blockIdx.x) * (D + 2);
      pp[e] = x;
      if (e == 0) {
        pp[D] = sm[hh] * 1.4426950408889634f;  // the join works in powers of two
        pp[D + 1] = sl[hh];
      }
    }
  }
}

// One warp-wide column of threads per output: o = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.
__global__ void __launch_bounds__(128) paged_combine_kernel(const float *__restrict__ part, float *__restrict__ o,
                                                            PagedView pv, const int *__restrict__ kv_lens,
                                                            int max_kv_len, int H, int D, DecodeSplit split) {
  const int bh = blockIdx.x, d = threadIdx.x;
  const int len = checked_len(__ldg(kv_lens + bh / H), max_kv_len, pv);
  const int n = (len + split.chunk - 1) / split.chunk;
  const float *p = part + (size_t)bh * split.n * (D + 2);
  float m = -INFINITY;
#pragma unroll 8
  for (int s = 0; s < n; ++s) m = fmaxf(m, p[s * (D + 2) + D]);
  float ov = 0.f, lv = 0.f;
#pragma unroll 8
  for (int s = 0; s < n; ++s) {
    const float f = ptx::ex2_approx(p[s * (D + 2) + D] - m);
    ov = fmaf(f, p[s * (D + 2) + d], ov);
    lv = fmaf(f, p[s * (D + 2) + D + 1], lv);
  }
  o[(size_t)bh * D + d] = (n > 0 ? ov / lv : 0.f);
}

template <int D>
cudaError_t decode_simt(const float *q, const float *k, const float *v, float *o, const PagedView &pv, const int *kv_lens, int n_seqs,
                        int max_kv_len, int H, int G, float *part, int *status, cudaStream_t st) {
  const DecodeSplit split = decode_split(n_seqs, max_kv_len, H, G);
  const int blocks = (H / G + PD_HEADS - 1) / PD_HEADS;
  if ((long long)G * blocks > 65535 || (long long)n_seqs * H > 0x7fffffffLL) return cudaErrorInvalidValue;
  count_launch();
  paged_decode_simt_kernel<D><<<dim3((unsigned)split.n, (unsigned)n_seqs, (unsigned)(G * blocks)), PD_THREADS, 0,
                                   st>>>(q, k, v, o, part, pv, kv_lens, max_kv_len, H, G, split,
                                         1.0f / sqrtf((float)D), status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || split.n == 1) return e;
  count_launch();
  paged_combine_kernel<<<(unsigned)(n_seqs * H), (unsigned)D, 0, st>>>(part, o, pv, kv_lens, max_kv_len, H, D, split);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_simt(const float *q, const float *k, const float *v, float *o, const PagedView &pv, const PackedView &b,
                               int H, int G, int D, int *status, cudaStream_t st) {
  switch (D) {
    case 16: return packed_simt<16>(q, k, v, o, pv, b, H, G, status, st);
    case 32: return packed_simt<32>(q, k, v, o, pv, b, H, G, status, st);
    case 64: return packed_simt<64>(q, k, v, o, pv, b, H, G, status, st);
    case 128: return packed_simt<128>(q, k, v, o, pv, b, H, G, status, st);
  }
  return cudaErrorInvalidValue;
}

size_t paged_decode_simt_workspace_bytes(int n_seqs, int max_kv_len, int H, int G, int D) {
  const DecodeSplit split = decode_split(n_seqs, max_kv_len, H, G);
  return split.n > 1 ? (size_t)n_seqs * H * split.n * (D + 2) * sizeof(float) : 0;
}

cudaError_t launch_paged_decode_simt(const float *q, const float *k, const float *v, float *o, const PagedView &pv,
                                     const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int D, float *part,
                                     int *status, cudaStream_t st) {
  switch (D) {
    case 16: return decode_simt<16>(q, k, v, o, pv, kv_lens, n_seqs, max_kv_len, H, G, part, status, st);
    case 32: return decode_simt<32>(q, k, v, o, pv, kv_lens, n_seqs, max_kv_len, H, G, part, status, st);
    case 64: return decode_simt<64>(q, k, v, o, pv, kv_lens, n_seqs, max_kv_len, H, G, part, status, st);
    case 128: return decode_simt<128>(q, k, v, o, pv, kv_lens, n_seqs, max_kv_len, H, G, part, status, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace llama
