// fp32 attention over cache pages on CUDA cores ("The Evolving Transformer 04 ·
// LLaMA", §05 GQA; "Full Llama 3 transformer block", How it works: keys
// j <= position).  One pass over the keys with the running maximum and sum of the
// softmax; fp32 products and sums throughout (the tensor cores round fp32 operands).
// Keys are split over CTAs when the rows alone are too few to fill the SMs, and the
// parts joined in order: o = sum e^(m_c - M) o_c / sum e^(m_c - M) l_c.  Pages of fp32 and
// pages held in 4 bits differ in how a tile's vectors are loaded alone.
#include <float.h>
#include <math.h>

#include "kv4.cuh"
#include "paged_kernels.h"

namespace llama {
namespace {

constexpr int KEYS = 64;        // keys of a tile
constexpr int THREADS = 256;
// CTAs per SM that the splits aim at.  max_kv_len stands for every sequence, so in a
// ragged batch most of them find no keys (16 against 4 per SM: 147 us for 266).
constexpr int SM_CTAS = 16;

// Split of the keys over CTAs: parts of `chunk` keys, `n` of them at the longest
// length that the call allows.
struct Split {
  int chunk = KEYS, n = 1;
};
Split split_of(long long ctas, int max_kv_len, int least) {
  const long long aim = (long long)SM_CTAS * sm_count();
  const long long want = (aim + ctas - 1) / ctas, most = (max_kv_len + least - 1) / least;
  const int n = (int)(want < most ? want : most > 1 ? most : 1);
  Split s;
  s.chunk = ((max_kv_len + n - 1) / n + KEYS - 1) / KEYS * KEYS;
  if (s.chunk < KEYS) s.chunk = KEYS;
  s.n = (max_kv_len + s.chunk - 1) / s.chunk;
  if (s.n < 1) s.n = 1;
  return s;
}

// Vector c of a row.
__device__ __forceinline__ float4 four(const float *row, int c) { return *reinterpret_cast<const float4 *>(row + c * 4); }
__device__ __forceinline__ float4 four(const Kv4Row &row, int c) {
  return kv4_four(reinterpret_cast<const uint32_t *>(row.codes)[c / 2], c & 1, kv4_scale(row.scales[c / 4]));
}

// A thread's vectors of a tile of KEYS rows of D floats: vector u = i * THREADS + tid
// is column u % (D / 4) of row u / (D / 4).
template <int D>
struct TileRegs {
  static constexpr int RV = D / 4, PER = KEYS * RV / THREADS;
  float4 x[PER];
  // row_ptr(i): row i in memory (a float * or Kv4Row), null for zeros
  template <typename F>
  __device__ __forceinline__ void load(F &&row_ptr) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = i * THREADS + threadIdx.x;
      const auto p = row_ptr(u / RV);
      x[i] = p != nullptr ? four(p, u % RV) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(float *dst) const {  // rows 16 bytes apart in banks
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = i * THREADS + threadIdx.x;
      *reinterpret_cast<float4 *>(dst + u / RV * (D + 4) + u % RV * 4) = x[i];
    }
  }
};

// Row of position p of a sequence in a pool, null when its page id is out of range.
__device__ __forceinline__ const float *page_row(const float *pool, const PagedView &pv, int seq, int g, int D, int p) {
  const int page = pv.page(seq, p >> pv.page_log2);
  if (page < 0) return nullptr;
  return pool + page * pv.page_stride + (((long long)g << pv.page_log2) + (p & ((1 << pv.page_log2) - 1))) * D;
}
__device__ __forceinline__ Kv4Row page_row(const uint8_t *pool, const PagedView &pv, int seq, int g, int D, int p) {
  const int page = pv.page(seq, p >> pv.page_log2);
  return page < 0 ? Kv4Row() : kv4_row(pool, pv, page, g, D, p & ((1 << pv.page_log2) - 1));
}

// ---------------------------------------------------------------- packed ---
// CTA = (sequence, KV head g, 64 rows of the flattened (position, head of the
// group) index R = position * r + hh, part of the keys): the r heads of a group share
// every K/V tile, and no row is padding but in a sequence's last tile.  4 x 4 scores
// and 4 x (D / 16) outputs per thread.
constexpr int ROWS = 64;

template <int D>
struct PsLayout {
  static constexpr int LDQ = D + 4, LDP = KEYS + 4;
  static constexpr int OFF_K = ROWS * LDQ;
  static constexpr int OFF_V = OFF_K + KEYS * LDQ;
  static constexpr int OFF_P = OFF_V + KEYS * LDQ;
  static constexpr int BYTES = (OFF_P + ROWS * LDP) * 4;
};

// Keys that the tile of rows R in [row0, row0 + rows) of a sequence sees.
__device__ __forceinline__ int tile_keys(const SeqSpan &s, int r, int row0) {
  const int rows = min(ROWS, s.count * r - row0);
  return max(0, s.kv_len - s.count + (row0 + rows - 1) / r + 1);
}

template <typename P>  // of a pool's elements: float, or uint8_t for 4-bit blocks
struct PsArgs {
  const float *q;
  const P *k, *v;
  float *o, *part;  // part [split.n][n_tokens][H][D + 2]
  PagedView pv;
  PackedView b;
  int H, G;
  Split split;
  float scale;
  int *status;
};

template <int D, typename P>
__global__ void __launch_bounds__(THREADS) packed_simt_kernel(const __grid_constant__ PsArgs<P> a) {
  using L = PsLayout<D>;
  using Row = decltype(page_row((const P *)nullptr, PagedView(), 0, 0, 0, 0));
  extern __shared__ __align__(16) float smem_f[];
  float *sq = smem_f, *sk = smem_f + L::OFF_K, *sv = smem_f + L::OFF_V, *sp = smem_f + L::OFF_P;
  const int r = a.H / a.G, g = blockIdx.y;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  allow_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x == 0 && g == 0 && blockIdx.z == 0)
    for (int i = threadIdx.x; i < a.b.n_seqs; i += THREADS) check_seq(a.b, a.pv, i, a.status);
  // block -> (sequence, tile): the grid holds at least one block for every tile
  __shared__ int found[2];
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  if (threadIdx.x < 32) {
    int base = 0;
    for (int i0 = 0; i0 < a.b.n_seqs; i0 += 32) {
      const int i = i0 + threadIdx.x;
      const int n =
          i < a.b.n_seqs ? (int)(((long long)seq_span(a.b, a.pv, i).count * r + ROWS - 1) / ROWS) : 0;
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
  const int seq = found[0], row0 = found[1] * ROWS;
  if (seq < 0) return;
  const SeqSpan s = seq_span(a.b, a.pv, seq);
  const int rows = min(ROWS, s.count * r - row0);
  const int shift = s.kv_len - s.count;  // position of the sequence's first new token
  const int n_keys = tile_keys(s, r, row0);
  const int k_begin = blockIdx.z * a.split.chunk, k_end = min(n_keys, k_begin + a.split.chunk);
  if (blockIdx.z > 0 && k_begin >= n_keys) return;
  const bool whole = n_keys <= a.split.chunk;  // one part: no join

  for (int u = threadIdx.x; u < ROWS * (D / 4); u += THREADS) {
    const int i = u / (D / 4), c = u % (D / 4) * 4, R = row0 + i;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < rows)
      x = *reinterpret_cast<const float4 *>(a.q + ((size_t)(s.first + R / r) * a.H + g * r + R % r) * D + c);
    *reinterpret_cast<float4 *>(sq + i * L::LDQ + c) = x;
  }
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
  for (int k0 = k_begin; k0 < k_end; k0 += KEYS) {
    {
      TileRegs<D> kr, vr;
      kr.load([&](int j) { return k0 + j < s.kv_len ? page_row(a.k, a.pv, seq, g, D, k0 + j) : Row(); });
      vr.load([&](int j) { return k0 + j < s.kv_len ? page_row(a.v, a.pv, seq, g, D, k0 + j) : Row(); });
      if (threadIdx.x < KEYS) {
        const int p = k0 + (int)threadIdx.x;
        if (p < s.kv_len && a.pv.page(seq, p >> a.pv.page_log2) < 0) report_status(a.status, LLAMA_ERR_RANGE);
      }
      __syncthreads();
      kr.store(sk);
      vr.store(sv);
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
      float4 x[4], c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(sq + (ty * 4 + i) * L::LDQ + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * L::LDQ + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sc[i][j] = fmaf(x[i].x, c[j].x, fmaf(x[i].y, c[j].y, fmaf(x[i].z, c[j].z, fmaf(x[i].w, c[j].w, sc[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sc[i][j] = k0 + tx + 16 * j <= pos[i] ? sc[i][j] * a.scale : -INFINITY;
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
    for (int j = 0; j < KEYS; j += 4) {
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
    const size_t row = (size_t)(s.first + R / r) * a.H + g * r + R % r;
    if (whole) {
      const float inv = pos[i] < 0 ? 0.f : 1.f / ls;  // no key: zeros; scores of NaN or -inf alone: NaN
#pragma unroll
      for (int c = 0; c < D / 16; ++c) a.o[row * D + tx + 16 * c] = acc[i][c] * inv;
    } else {
      float *pp = a.part + ((size_t)blockIdx.z * a.b.n_tokens * a.H + row) * (D + 2);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) pp[tx + 16 * c] = acc[i][c];
      if (tx == 0) {
        pp[D] = m[i];
        pp[D + 1] = ls;
      }
    }
  }
}

// Joins the parts c0, c0 + by, ... below n, `step` floats apart, of one row of D floats
// (then m and l): one warp, to its (m, l) and unscaled sums.
template <int D>
struct RowParts {
  static constexpr int PER = D > 32 ? D / 32 : 1;
  float m = -INFINITY, l = 0.f, acc[PER];
  __device__ __forceinline__ RowParts(const float *p, size_t step, int n, int c0, int by) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int c = c0 + by * lane; c < n; c += by * 32) m = fmaxf(m, p[c * step + D]);
    m = warp_max(m);
#pragma unroll 4
    for (int c = c0; c < n; c += by) {
      const float f = expf(p[c * step + D] - m);
      l = fmaf(f, p[c * step + D + 1], l);
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (lane + 32 * e < D) acc[e] = fmaf(f, p[c * step + lane + 32 * e], acc[e]);
    }
  }
};

template <int D, typename P>
__global__ void __launch_bounds__(THREADS) packed_join_simt_kernel(const __grid_constant__ PsArgs<P> a) {
  const long long row = (long long)blockIdx.x * (THREADS / 32) + threadIdx.x / 32;  // token, head
  grid_dependency_wait();
  if (row >= (long long)a.b.n_tokens * a.H) return;
  const int t = (int)(row / a.H), r = a.H / a.G, hh = (int)(row % a.H) % r;
  const int seq = find_seq(a.b, t);
  if (seq < 0) return;
  const SeqSpan s = seq_span(a.b, a.pv, seq);
  const int n_keys = tile_keys(s, r, ((t - s.first) * r + hh) / ROWS * ROWS);
  if (n_keys <= a.split.chunk) return;
  const RowParts<D> x(a.part + row * (D + 2), (size_t)a.b.n_tokens * a.H * (D + 2),
                      (n_keys + a.split.chunk - 1) / a.split.chunk, 0, 1);
  const int lane = threadIdx.x & 31;
  const bool sees = s.kv_len - (s.first + s.count - t) >= 0;
#pragma unroll
  for (int e = 0; e < RowParts<D>::PER; ++e)
    if (lane + 32 * e < D) a.o[row * D + lane + 32 * e] = sees ? x.acc[e] / x.l : 0.f;
}

// every sequence ends in at most one tile that is not full
long long packed_tiles(const PackedView &b, int H, int G) { return (long long)b.n_tokens * (H / G) / ROWS + b.n_seqs; }
Split packed_split(const PackedView &b, int H, int G) {
  return split_of(packed_tiles(b, H, G) * G, b.max_kv_len, 2 * KEYS);
}

template <int D, typename P>
cudaError_t packed_simt(PsArgs<P> a, cudaStream_t st) {
  static PerContextOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(packed_simt_kernel<D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                PsLayout<D>::BYTES);
  });
  if (e != cudaSuccess) return e;
  a.scale = 1.0f / sqrtf((float)D);
  const long long tiles = packed_tiles(a.b, a.H, a.G);
  if (tiles > 0x7fffffffLL || a.G > 65535) return cudaErrorInvalidValue;
  count_launch();
  const cudaError_t r = launch_pdl(packed_simt_kernel<D, P>, dim3((unsigned)tiles, (unsigned)a.G, (unsigned)a.split.n),
                                   dim3(THREADS), PsLayout<D>::BYTES, st, a);
  if (r != cudaSuccess || a.split.n == 1) return r;
  count_launch();
  const long long rows = (long long)a.b.n_tokens * a.H;
  return launch_pdl(packed_join_simt_kernel<D, P>, dim3((unsigned)((rows + THREADS / 32 - 1) / (THREADS / 32))),
                    dim3(THREADS), 0, st, a);
}

// ---------------------------------------------------------------- decode ---
// CTA = (part of the keys, sequence, KV head and block of up to 8 of its query
// heads); the next tile's K and V are on their way while this one is worked on.
constexpr int HEADS = 8;

template <int D>
struct DsLayout {
  static constexpr int LD = D + 4, SLICES = THREADS / D;
  static constexpr int RED = SLICES * HEADS * D;  // the slices' sums, over K and V at the end
  static constexpr int OFF_V = KEYS * LD;
  static constexpr int KV = 2 * KEYS * LD > RED ? 2 * KEYS * LD : RED;
  static constexpr int OFF_Q = KV;
  static constexpr int OFF_S = OFF_Q + HEADS * D;       // scores [HEADS][KEYS + 1]
  static constexpr int OFF_W = OFF_S + HEADS * (KEYS + 1) / 4 * 4 + 4;  // weights [KEYS][HEADS]
  static constexpr int BYTES = (OFF_W + KEYS * HEADS) * 4;
};

template <typename P>  // of a pool's elements: float, or uint8_t for 4-bit blocks
struct DsArgs {
  const float *q;
  const P *k, *v;
  float *o, *part;  // part [n_seqs][H][split.n][D + 2]
  PagedView pv;
  const int *kv_lens;
  int n_seqs, max_kv_len, H, G;
  Split split;
  float scale;
  int *status;
};

template <int D, typename P>
__global__ void __launch_bounds__(THREADS) paged_decode_simt_kernel(const __grid_constant__ DsArgs<P> a) {
  using L = DsLayout<D>;
  using Row = decltype(page_row((const P *)nullptr, PagedView(), 0, 0, 0, 0));
  extern __shared__ __align__(16) float smem_f[];
  float *sk = smem_f, *sv = smem_f + L::OFF_V, *sq = smem_f + L::OFF_Q, *ss = smem_f + L::OFF_S,
        *sw = smem_f + L::OFF_W;
  __shared__ float sm[HEADS], sl[HEADS], sc[HEADS];
  const int r = a.H / a.G, blocks = (r + HEADS - 1) / HEADS;
  const int g = blockIdx.z / blocks, h0 = (blockIdx.z % blocks) * HEADS;
  const int nh = min(HEADS, r - h0), seq = blockIdx.y;
  allow_dependents_launch();
  grid_dependency_wait();
  const int raw_len = ld_after_wait(a.kv_lens + seq);
  const int len = checked_len(raw_len, a.max_kv_len, a.pv);
  if (len != raw_len && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
    report_status(a.status, LLAMA_ERR_RANGE);
  const int k0 = blockIdx.x * a.split.chunk, k1 = min(len, k0 + a.split.chunk);
  if (k0 >= len && blockIdx.x > 0) return;
  const size_t bh = (size_t)seq * a.H + g * r + h0;

  TileRegs<D> kr, vr;
  auto load = [&](int t0) {
    kr.load([&](int j) { return t0 + j < k1 ? page_row(a.k, a.pv, seq, g, D, t0 + j) : Row(); });
    vr.load([&](int j) { return t0 + j < k1 ? page_row(a.v, a.pv, seq, g, D, t0 + j) : Row(); });
    const int p = t0 + (int)threadIdx.x;
    if (threadIdx.x < KEYS && p < k1 && a.pv.page(seq, p >> a.pv.page_log2) < 0)
      report_status(a.status, LLAMA_ERR_RANGE);
  };
  load(k0);
  for (int u = threadIdx.x; u < HEADS * D; u += THREADS) sq[u] = u < nh * D ? a.q[bh * D + u] * a.scale : 0.f;
  if (threadIdx.x < HEADS) {
    sm[threadIdx.x] = -INFINITY;
    sl[threadIdx.x] = 0.f;
  }
  const int d = threadIdx.x % D, slice = threadIdx.x / D;
  const int h = threadIdx.x / 32, lane = threadIdx.x & 31;
  float acc[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) acc[i] = 0.f;
  for (int t0 = k0; t0 < k1; t0 += KEYS) {
    const int n = min(KEYS, k1 - t0);
    __syncthreads();
    kr.store(sk);
    vr.store(sv);
    __syncthreads();
    if (t0 + KEYS < k1) load(t0 + KEYS);
    {  // scores of key tid % 64 for heads tid / 64 and tid / 64 + 4
      const int key = threadIdx.x % KEYS, ha = threadIdx.x / KEYS, hb = ha + HEADS / 2;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int e = 0; e < D; e += 4) {
        const float4 c = *reinterpret_cast<const float4 *>(sk + key * L::LD + e);
        const float4 p = *reinterpret_cast<const float4 *>(sq + ha * D + e);
        const float4 q = *reinterpret_cast<const float4 *>(sq + hb * D + e);
        x = fmaf(p.x, c.x, fmaf(p.y, c.y, fmaf(p.z, c.z, fmaf(p.w, c.w, x))));
        y = fmaf(q.x, c.x, fmaf(q.y, c.y, fmaf(q.z, c.z, fmaf(q.w, c.w, y))));
      }
      ss[ha * (KEYS + 1) + key] = key < n ? x : -INFINITY;
      ss[hb * (KEYS + 1) + key] = key < n ? y : -INFINITY;
    }
    __syncthreads();
    {  // warp h: the running maximum and sum of head h; every tile holds a key, so the maximum is one
      const float x = ss[h * (KEYS + 1) + lane], y = ss[h * (KEYS + 1) + lane + 32];
      const float mn = fmaxf(sm[h], warp_max(fmaxf(x, y)));
      const float px = expf(x - mn), py = expf(y - mn);
      const float ls = warp_sum(px + py);
      sw[lane * HEADS + h] = px;
      sw[(lane + 32) * HEADS + h] = py;
      __syncwarp();
      if (lane == 0) {
        const float corr = expf(sm[h] - mn);
        sc[h] = corr;
        sl[h] = sl[h] * corr + ls;
        sm[h] = mn;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HEADS; ++i) acc[i] *= sc[i];
    for (int j = slice; j < n; j += L::SLICES) {
      const float v = sv[j * L::LD + d];
      const float4 w0 = *reinterpret_cast<const float4 *>(sw + j * HEADS);
      const float4 w1 = *reinterpret_cast<const float4 *>(sw + j * HEADS + 4);
      acc[0] = fmaf(w0.x, v, acc[0]);
      acc[1] = fmaf(w0.y, v, acc[1]);
      acc[2] = fmaf(w0.z, v, acc[2]);
      acc[3] = fmaf(w0.w, v, acc[3]);
      acc[4] = fmaf(w1.x, v, acc[4]);
      acc[5] = fmaf(w1.y, v, acc[5]);
      acc[6] = fmaf(w1.z, v, acc[6]);
      acc[7] = fmaf(w1.w, v, acc[7]);
    }
  }
  __syncthreads();
  float *red = smem_f;  // [SLICES][HEADS][D]
#pragma unroll
  for (int i = 0; i < HEADS; ++i) red[(slice * HEADS + i) * D + d] = acc[i];
  __syncthreads();
  for (int u = threadIdx.x; u < nh * D; u += THREADS) {
    const int i = u / D, e = u % D;
    float x = 0.f;
#pragma unroll
    for (int s = 0; s < L::SLICES; ++s) x += red[(s * HEADS + i) * D + e];
    if (len <= a.split.chunk) {
      a.o[bh * D + u] = len > 0 ? x / sl[i] : 0.f;
    } else {
      float *pp = a.part + ((bh + i) * a.split.n + blockIdx.x) * (D + 2);
      pp[e] = x;
      if (e == 0) {
        pp[D] = sm[i];
        pp[D + 1] = sl[i];
      }
    }
  }
}

// A CTA per row: the parts are many and the rows few, so its warps share them.
template <int D, typename P>
__global__ void __launch_bounds__(THREADS) decode_join_simt_kernel(const __grid_constant__ DsArgs<P> a) {
  constexpr int WARPS = THREADS / 32;
  __shared__ float sm[WARPS], sl[WARPS], so[WARPS][D];
  const int row = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x & 31;  // sequence, head
  grid_dependency_wait();
  const int len = checked_len(ld_after_wait(a.kv_lens + row / a.H), a.max_kv_len, a.pv);
  if (len <= a.split.chunk) return;
  const RowParts<D> x(a.part + (size_t)row * a.split.n * (D + 2), D + 2, (len + a.split.chunk - 1) / a.split.chunk,
                      warp, WARPS);
  if (lane == 0) {
    sm[warp] = x.m;
    sl[warp] = x.l;
  }
#pragma unroll
  for (int e = 0; e < RowParts<D>::PER; ++e)
    if (lane + 32 * e < D) so[warp][lane + 32 * e] = x.acc[e];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = fmaxf(m, sm[w]);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float f = expf(sm[w] - m);  // a warp without parts: e^-inf
    l = fmaf(f, sl[w], l);
    o = fmaf(f, so[w][threadIdx.x], o);
  }
  a.o[(size_t)row * D + threadIdx.x] = o / l;
}

Split decode_split(int n_seqs, int max_kv_len, int H, int G) {
  return split_of((long long)n_seqs * G * ((H / G + HEADS - 1) / HEADS), max_kv_len, KEYS);
}

template <int D, typename P>
cudaError_t decode_simt(DsArgs<P> a, cudaStream_t st) {
  static PerContextOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(paged_decode_simt_kernel<D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                DsLayout<D>::BYTES);
  });
  if (e != cudaSuccess) return e;
  a.scale = 1.0f / sqrtf((float)D);
  const long long units = (long long)a.G * ((a.H / a.G + HEADS - 1) / HEADS), rows = (long long)a.n_seqs * a.H;
  if (units > 65535 || rows > 0x7fffffffLL) return cudaErrorInvalidValue;
  count_launch();
  const cudaError_t r = launch_pdl(paged_decode_simt_kernel<D, P>,
                                   dim3((unsigned)a.split.n, (unsigned)a.n_seqs, (unsigned)units), dim3(THREADS),
                                   DsLayout<D>::BYTES, st, a);
  if (r != cudaSuccess || a.split.n == 1) return r;
  count_launch();
  return launch_pdl(decode_join_simt_kernel<D, P>, dim3((unsigned)rows), dim3(THREADS), 0, st, a);
}

}  // namespace

size_t packed_simt_workspace_bytes(const PackedView &b, int H, int G, int D) {
  const Split s = packed_split(b, H, G);
  return s.n > 1 ? (size_t)s.n * b.n_tokens * H * (D + 2) * sizeof(float) : 0;
}

template <typename P>
cudaError_t launch_packed_simt(const float *q, const P *k, const P *v, float *o, const PagedView &pv,
                               const PackedView &b, int H, int G, int D, float *part, int *status, cudaStream_t st) {
  PsArgs<P> a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.part = part;
  a.pv = pv;
  a.b = b;
  a.H = H;
  a.G = G;
  a.split = packed_split(b, H, G);
  a.status = status;
  switch (D) {
    case 16: return packed_simt<16>(a, st);
    case 32: return packed_simt<32>(a, st);
    case 64: return packed_simt<64>(a, st);
    case 128: return packed_simt<128>(a, st);
  }
  return cudaErrorInvalidValue;
}

size_t paged_decode_simt_workspace_bytes(int n_seqs, int max_kv_len, int H, int G, int D) {
  const Split s = decode_split(n_seqs, max_kv_len, H, G);
  return s.n > 1 ? (size_t)n_seqs * H * s.n * (D + 2) * sizeof(float) : 0;
}

template <typename P>
cudaError_t launch_paged_decode_simt(const float *q, const P *k, const P *v, float *o, const PagedView &pv,
                                     const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int D, float *part,
                                     int *status, cudaStream_t st) {
  DsArgs<P> a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.part = part;
  a.pv = pv;
  a.kv_lens = kv_lens;
  a.n_seqs = n_seqs;
  a.max_kv_len = max_kv_len;
  a.H = H;
  a.G = G;
  a.split = decode_split(n_seqs, max_kv_len, H, G);
  a.status = status;
  switch (D) {
    case 16: return decode_simt<16>(a, st);
    case 32: return decode_simt<32>(a, st);
    case 64: return decode_simt<64>(a, st);
    case 128: return decode_simt<128>(a, st);
  }
  return cudaErrorInvalidValue;
}

template cudaError_t launch_packed_simt<float>(const float *, const float *, const float *, float *, const PagedView &,
                                               const PackedView &, int, int, int, float *, int *, cudaStream_t);
template cudaError_t launch_packed_simt<uint8_t>(const float *, const uint8_t *, const uint8_t *, float *,
                                                 const PagedView &, const PackedView &, int, int, int, float *, int *,
                                                 cudaStream_t);
template cudaError_t launch_paged_decode_simt<float>(const float *, const float *, const float *, float *,
                                                     const PagedView &, const int *, int, int, int, int, int, float *,
                                                     int *, cudaStream_t);
template cudaError_t launch_paged_decode_simt<uint8_t>(const float *, const uint8_t *, const uint8_t *, float *,
                                                       const PagedView &, const int *, int, int, int, int, int, float *,
                                                       int *, cudaStream_t);

}  // namespace llama
