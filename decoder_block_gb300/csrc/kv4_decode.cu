// One new token per sequence over cache pages held in 4 bits, q and o bf16 ("Full Llama 3
// transformer block", How it works: cached keys 0 .. kv_len - 1; "The Evolving Transformer
// 04 · LLaMA", §05 GQA).
//   o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),  x_j = q.k_j log2(e) / sqrt(D),
// in one pass over the keys, the running maximum m and the sum in fp32.
//
// The cache is read once, and a byte of it is nearly two elements: what has to be kept small
// is the work per element.  A warp takes 32 keys at a time for the 8 (or 16) heads of an
// item, codes go from shared memory into registers and from there straight into the
// operands of mma.sync, keys and columns of the values on its 16-row side:
//   S^T[16 keys x 8 heads] = K Q^T,     O^T[16 columns x 8 heads] += V^T P^T.
// The order of d within K and Q, and of the columns in V and O, is free: it is the one that
// leaves every thread whole words of codes.  Two codes become two bf16 with a shift, a
// masked or and an fma (kv4.cuh); V's products run over keys, so the words of two keys are
// interleaved first, half a word at a time.  P^T comes from S^T by movmatrix.  (tcgen05 takes
// its operands from shared memory: the bf16 written there and read back are four times the
// codes, more than the SM's shared memory moves in the time that the codes take to come.)
// Each warp copies its own tiles into its own shared memory, a few tiles ahead, and waits
// for nothing but those copies.
//
// All tiles of the call in one row -- sequence by sequence, head block by head block -- are
// dealt out to the CTAs, and a CTA's to its warps, in even runs.  A run that begins or ends
// inside an item leaves its (O, m, l); the CTA joins those of its warps, in order, and
// what begins or ends inside the CTA's run goes to the workspace, where a second kernel
// joins it, in order.  With short sequences (direct) a CTA takes one item instead, and there
// is no second kernel.
#include <cuda_fp16.h>
#include <float.h>

#include "kv4.cuh"
#include "paged_kernels.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int KD_KEYS = 32;  // keys of a warp's tile
constexpr float KD_RESCALE = 8.0f;  // log2 units: the running maximum is raised when it grows by > 2^8
// Weights are fp16 for their product with V: 2^7 times what they are, so that the largest,
// 2^15, has room above, and what is less than 2^-31 of the running maximum's, not 2^-24, is
// lost (120000 keys of such weights: 2^-14 of the sum).
constexpr float KD_WEIGHT = 7.0f;
constexpr float KD_VALUE = 2.0f;  // V's operand is half of V
// Key tiles of a CTA's item in the direct form, at most.
constexpr int KD_DIRECT_TILES = 64;

// NB: blocks of 8 heads of an item.
template <int D, int NB>
struct KdLayout {
  static constexpr int WARPS = NB == 1 ? 16 : 8;
  static constexpr int RB = kv4_code_bytes(D), SB = kv4_scale_bytes(D);
  static constexpr int HALF = KD_KEYS * (RB + SB), STAGE = 2 * HALF;  // K, then V: codes, then scales
  static constexpr int PART = 8 * NB * (D + 2) * 4;  // (O, m, l) of an item
  static constexpr int FIT = (NB == 1 ? 9216 : 13824) / STAGE;
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr int RING = STAGES * STAGE > PART ? STAGES * STAGE : PART;  // of a warp; its last part at the end
  static constexpr int OFF_PART = WARPS * RING;   // of each warp, its first
  static constexpr int OFF_META = OFF_PART + WARPS * PART;
  static constexpr int OFF_SUMS = OFF_META + WARPS * 2 * 16;
  static constexpr int OFF_FIRST = OFF_SUMS + 128;  // tiles before sequence i
  static int bytes(int n_seqs) { return OFF_FIRST + (n_seqs + 1) * 4; }
};
static_assert(KdLayout<128, 1>::OFF_FIRST + (LLAMA_PACKED_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits an SM");
static_assert(KdLayout<128, 2>::OFF_FIRST + (LLAMA_PACKED_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits an SM");

struct KdArgs {
  const bf16 *q;
  const uint8_t *k, *v;
  bf16 *o;
  PagedView pv;
  const int *kv_lens;
  int n_seqs, max_kv_len;
  int H, G, r, subs, units;  // r: heads of a group; subs: head blocks of a group; units = G * subs
  int direct;
  float scale_log2;
  float *part;  // [CTA][2][8 NB][D + 2]
  int4 *spans;  // of each CTA: sequence, unit and last CTA of the item that it begins and leaves (-1: none)
  int *status;
};

// A piece of an item that a warp leaves for its CTA to join.
struct KdMeta {
  int seq, unit;  // seq -1: none
  int j0, j1;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_half(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t kd_pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t kd_pack_half2(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// N words (or, N = 0, one that is not whole) from shared memory.
template <int N>
__device__ __forceinline__ void ld_words(uint32_t at, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}
__device__ __forceinline__ uint32_t ld_byte(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// A place in the row of tiles.
struct KdCursor {
  int seq, unit, g, j, n, len;  // n: tiles of the sequence, len: its keys
  __device__ __forceinline__ void seek(const KdArgs &a, const int *first, long long at) {
    int lo = 0, hi = a.n_seqs;  // the last sequence that begins at or before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if ((long long)first[mid] * a.units <= at) lo = mid;
      else hi = mid;
    }
    n = first[lo + 1] - first[lo];
    const long long rest = at - (long long)first[lo] * a.units;
    set(a, lo, (int)(rest / n), (int)(rest % n), n);
  }
  __device__ __forceinline__ void set(const KdArgs &a, int s, int u, int at, int tiles) {
    seq = s;
    unit = u;
    g = u / a.subs;
    j = at;
    n = tiles;
    len = ld_after_wait(a.kv_lens + s);
  }
  __device__ __forceinline__ void next(const KdArgs &a, const int *first) {
    if (++j < n || a.direct) return;
    int s = seq, u = unit + 1;
    if (u == a.units) {
      u = 0;
      for (++s; s < a.n_seqs; ++s) {
        n = first[s + 1] - first[s];
        if (n > 0) break;
      }
      if (s == a.n_seqs) return;  // the end of the row
    }
    set(a, s, u, 0, n);
  }
};

template <int D, int NB>
__global__ void __launch_bounds__(KdLayout<D, NB>::WARPS * 32, 1) kv4_decode_kernel(const __grid_constant__ KdArgs a) {
  using L = KdLayout<D, NB>;
  constexpr int THREADS = L::WARPS * 32;
  constexpr int KW = D / 32 > 0 ? D / 32 : 1;  // words of a key's codes that a thread takes (of 8 elements)
  constexpr int VW = D / 64 > 0 ? D / 64 : 1;  // of a value's
  constexpr int STEPS = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, gi = lane / 4, ti = lane & 3;
  const uint32_t s0 = ptx::smem_u32(smem);
  int *first = reinterpret_cast<int *>(smem + L::OFF_FIRST);
  int *sums = reinterpret_cast<int *>(smem + L::OFF_SUMS);
  KdMeta *meta = reinterpret_cast<KdMeta *>(smem + L::OFF_META);
  allow_dependents_launch();
  grid_dependency_wait();

  // ------------------------------------------------------------- lengths ---
  if (lane < 2) meta[warp * 2 + lane].seq = -1;
  auto no_keys = [&](int i, int from, int step) {  // sequence i: zeros
    uint4 *dst = reinterpret_cast<uint4 *>(a.o + (size_t)i * a.H * D);
    for (int e = from; e < a.H * D / 8; e += step) dst[e] = make_uint4(0, 0, 0, 0);
  };
  KdCursor at = {0, 0, 0, 0, 0, 0};
  long long begin = 0, each = 1;
  int n_run;  // tiles of this CTA's run
  if (a.direct) {
    const int seq = blockIdx.x / a.units, unit = blockIdx.x % a.units;
    const int raw = ld_after_wait(a.kv_lens + seq), len = checked_len(raw, a.max_kv_len, a.pv);
    if (raw != len && unit == 0 && threadIdx.x == 0) report_status(a.status, LLAMA_ERR_RANGE);
    n_run = (len + KD_KEYS - 1) / KD_KEYS;
    if (n_run == 0) {
      if (unit == 0) no_keys(seq, threadIdx.x, THREADS);
      return;
    }
    at.set(a, seq, unit, 0, n_run);
  } else {
    // (4096 sequences: 8 or 16 each)
    const int per = (a.n_seqs + THREADS - 1) / THREADS;
    int mine = 0;
    for (int k = 0; k < per; ++k) {
      const int i = threadIdx.x * per + k;
      if (i >= a.n_seqs) break;
      const int raw = ld_after_wait(a.kv_lens + i), len = checked_len(raw, a.max_kv_len, a.pv);
      if (raw != len && blockIdx.x == 0) report_status(a.status, LLAMA_ERR_RANGE);
      const int n = (len + KD_KEYS - 1) / KD_KEYS;
      first[i] = n;
      mine += n;
      if (n == 0 && i % (int)gridDim.x == (int)blockIdx.x) no_keys(i, 0, 1);
    }
    int end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    if (lane == 31) sums[warp] = end;
    __syncthreads();
    int before = end - mine;
    for (int w = 0; w < warp; ++w) before += sums[w];
    for (int k = 0; k < per; ++k) {
      const int i = threadIdx.x * per + k;
      if (i >= a.n_seqs) break;
      const int n = first[i];
      first[i] = before;
      before += n;
    }
    if (threadIdx.x == THREADS - 1) first[a.n_seqs] = before;
    __syncthreads();
    const long long total = (long long)first[a.n_seqs] * a.units;
    each = (total + gridDim.x - 1) / gridDim.x;
    each = each > L::WARPS ? each : L::WARPS;
    begin = min(total, each * blockIdx.x);
    n_run = (int)(min(total, begin + each) - begin);
  }
  const int w0 = (int)((long long)n_run * warp / L::WARPS), w1 = (int)((long long)n_run * (warp + 1) / L::WARPS);
  const uint32_t ring = s0 + warp * L::RING;

  // -------------------------------------------------------------- copies ---
  // Lanes 0 to 7 look up where a tile's rows lie: bit 0 says which 16 rows, bit 1 K or V, bit
  // 2 codes or scales.  A half behind the last key is given the first half's rows, which may
  // be read; its scores are replaced.
  KdCursor ahead = at;  // the tile whose pages are known and that is copied next
  int left = w1 - w0, id = 0, slot = 0;
  const int rows_mask = (1 << a.pv.page_log2) - 1;
  const uint8_t *const pool = lane & 2 ? a.v : a.k;
  const int row_bytes = lane & 4 ? L::SB : L::RB, to_scales = lane & 4 ? L::RB << a.pv.page_log2 : 0;
  const int block = kv4_block_bytes(1 << a.pv.page_log2, D);
  auto look_up = [&] {
    if (left > 0 && lane < 8) {
      int p = ahead.j * KD_KEYS + (lane & 1) * 16;
      p = p < ahead.len ? p : ahead.j * KD_KEYS;
      slot = p & rows_mask;
      id = ld_after_wait(a.pv.table + (size_t)ahead.seq * a.pv.table_stride + (p >> a.pv.page_log2));
    }
  };
  auto request = [&](int n) {
    if (left > 0) {
      const uint32_t stage = ring + n % L::STAGES * L::STAGE;
      constexpr int CHUNK = L::RB < 16 ? L::RB : 16, PER_ROW = L::RB / CHUNK;
      const bool bad = lane < 8 && (unsigned)id >= (unsigned)a.pv.n_pages;
      const unsigned bads = __ballot_sync(0xffffffffu, bad);
      const uint8_t *ptr = pool;
      if (!bad) ptr += id * a.pv.page_stride + (ahead.g * block + to_scales + slot * row_bytes);
      auto rows_at = [&](int from) {
        return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(ptr), from));
      };
      auto copies = [&](bool all_good) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
          for (int i = 0; i < PER_ROW; ++i) {
            const int byte = (i * 32 + lane) * CHUNK, half = D >= 64 ? i * 32 / PER_ROW / 16 : lane / 16;
            const uint32_t to = stage + which * L::HALF + byte;
            const uint8_t *from = rows_at(which * 2 + half) + (byte - half * 16 * L::RB);
            if (all_good || !(bads >> (which * 2 + half) & 1)) {
              copy_async<CHUNK>(to, from);
            } else {  // a page of zeros
              asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(to), "r"(0x88888888u) : "memory");
              if (CHUNK == 16)
                asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(to + 8), "r"(0x88888888u) : "memory");
            }
          }
        // scales: K's by lanes 0 .., V's by lanes 16 ..
        const int which = lane / 16, l = lane % 16, half = l / L::SB & 1, src = 4 + which * 2 + half;
        const uint8_t *from = rows_at(src) + l % L::SB * 16;
        if (l < 2 * L::SB && (all_good || !(bads >> src & 1)))
          copy_async<16>(stage + which * L::HALF + KD_KEYS * L::RB + l * 16, from);
      };
      if (bads == 0) {
        copies(true);
      } else {
        if (lane == 0) report_status(a.status, LLAMA_ERR_RANGE);
        copies(false);
      }
      ahead.next(a, first);
      --left;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  if (left > 0) {
    if (a.direct) at.j = w0;
    else at.seek(a, first, begin + w0);
    ahead = at;
    look_up();
#pragma unroll 1
    for (int n = 0; n < L::STAGES - 1; ++n) {
      request(n);
      look_up();
    }
    const int todo = w1 - w0;
    int done = 0;
    while (done < todo) {
      // ----------------------------------------------------------- a piece ---
      const int seq = at.seq, unit = at.unit, j0 = at.j, n_tiles = at.n;
      const int j1 = min(n_tiles, j0 + todo - done);
      const int len = at.len, g = at.g;
      const int h_in = (unit - g * a.subs) * (8 * NB), nh = min(8 * NB, a.r - h_in);
      const size_t row0 = (size_t)seq * a.H + g * a.r + h_in;
      uint32_t qf[NB][STEPS][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int h = b * 8 + gi;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(a.q + (row0 + h) * D + ti * (D / 4));
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qf[b][s][e] = 0;
            if (h < nh) qf[b][s][e] = (uint32_t)ld_after_wait(reinterpret_cast<const int *>(src) + 2 * s + e);
          }
      }
      float acc[NB][STEPS][4], m[NB][2], l[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[b][i][e] = 0.f;
        m[b][0] = m[b][1] = -FLT_MAX;  // finite: a row whose scores are all -inf keeps weights of 0
        l[b][0] = l[b][1] = 0.f;
      }
#pragma unroll 1
      for (int j = j0; j < j1; ++j, ++done) {
        request(done + L::STAGES - 1);
        look_up();
        asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 1) : "memory");
        __syncwarp();
        const uint32_t sk = ring + done % L::STAGES * L::STAGE, sv = sk + L::HALF;
        // scores: keys gi and gi + 8 of both halves of the tile
        float sc[2][NB][4];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mb][b][e] = 0.f;
          uint32_t w[2][KW];
          Kv4Scale sa[2], sb[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = mb * 16 + e * 8 + gi;
            const uint32_t scales = sk + KD_KEYS * L::RB + row * L::SB;
            if constexpr (D >= 32) ld_words<KW>(sk + row * L::RB + ti * (D / 8), w[e]);
            else ld_words<KW>(sk + row * L::RB + ti / 2 * 4, w[e]);
            if constexpr (D == 16) w[e][0] >>= 8 * (ti & 1);
            if constexpr (D == 128) {
              uint16_t x;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(scales + ti * 2));
              sa[e] = kv4_scales((uint32_t)x & 255);
              sb[e] = kv4_scales((uint32_t)x >> 8);
            } else {
              sa[e] = kv4_scales(ld_byte(scales + (D == 64 ? ti : D == 32 ? ti / 2 : 0)));
              sb[e] = sa[e];
            }
          }
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            // elements 4 s .. 4 s + 3 of the thread's; 16 of them share a scale
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t word = w[e][s / 2];
              const Kv4Scale &k = s < 4 ? sa[e] : sb[e];
              f[e] = s % 2 == 0 ? kv4_pair<0>(word, k) : kv4_pair<2>(word, k);
              f[2 + e] = s % 2 == 0 ? kv4_pair<1>(word, k) : kv4_pair<3>(word, k);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816(sc[mb][b], f, qf[b][s][0], qf[b][s][1]);
          }
        }
        if ((j + 1) * KD_KEYS > len) {
          const int key = j * KD_KEYS + gi;
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key + mb * 16 + (e / 2) * 8 >= len) sc[mb][b][e] = -INFINITY;
        }
        // weights: heads 8 b + 2 ti and the next
        uint32_t pf[2][NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float mx[2];
          bool need = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(fmaxf(sc[0][b][e], sc[0][b][e + 2]), fmaxf(sc[1][b][e], sc[1][b][e + 2])) * a.scale_log2;
            need |= mx[e] > m[b][e] + KD_RESCALE;
          }
          if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
              const float up = fmaxf(m[b][e], mx[e]), f = ptx::ex2_approx(m[b][e] - up);
              m[b][e] = up;
              l[b][e] *= f;
#pragma unroll
              for (int i = 0; i < STEPS; ++i) {
                acc[b][i][e] *= f;
                acc[b][i][e + 2] *= f;
              }
            }
          }
          const float less[2] = {KD_WEIGHT - m[b][0], KD_WEIGHT - m[b][1]};
#pragma unroll
          for (int mb = 0; mb < 2; ++mb) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = ptx::ex2_approx(fmaf(sc[mb][b][e], a.scale_log2, less[e & 1]));
              l[b][e & 1] += p[e];
            }
            pf[mb][b][0] = transpose8x8(kd_pack_half2(p[0], p[1]));
            pf[mb][b][1] = transpose8x8(kd_pack_half2(p[2], p[3]));
          }
        }
        // outputs: columns gi (D / 8) .. of the values, keys 2 ti, 2 ti + 1, and 8 more
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          uint32_t even[2][VW], odd[2][VW];
          Kv4Half sv2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = mb * 16 + e * 8 + 2 * ti;
            uint32_t x[VW], y[VW];
            const uint32_t at = sv + row * L::RB + (D >= 64 ? gi * (D / 16) : D == 32 ? gi / 2 * 4 : gi / 4 * 4);
            ld_words<VW>(at, x);
            ld_words<VW>(at + L::RB, y);
            const uint32_t sat = sv + KD_KEYS * L::RB + row * L::SB + gi * L::SB / 8;
            sv2[e] = kv4_halves(ld_byte(sat), ld_byte(sat + L::SB));
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              if constexpr (D == 32) {
                x[w] >>= 8 * (gi & 1);
                y[w] >>= 8 * (gi & 1);
              } else if constexpr (D == 16) {
                x[w] >>= 4 * (gi & 3);
                y[w] >>= 4 * (gi & 3);
              }
              even[e][w] = __byte_perm(x[w], y[w], 0x5410);
              odd[e][w] = __byte_perm(x[w], y[w], 0x7632);
            }
          }
#pragma unroll
          for (int i = 0; i < STEPS; ++i) {
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t ev = even[e][i / 4], od = odd[e][i / 4];
              const Kv4Half &k = sv2[e];
              f[2 * e] = i % 4 == 0 ? kv4_half_pair<0>(ev, k) : i % 4 == 1 ? kv4_half_pair<1>(ev, k)
                         : i % 4 == 2 ? kv4_half_pair<2>(ev, k) : kv4_half_pair<3>(ev, k);
              f[2 * e + 1] = i % 4 == 0 ? kv4_half_pair<0>(od, k) : i % 4 == 1 ? kv4_half_pair<1>(od, k)
                             : i % 4 == 2 ? kv4_half_pair<2>(od, k) : kv4_half_pair<3>(od, k);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816_half(acc[b][i], f, pf[mb][b][0], pf[mb][b][1]);
          }
        }
        __syncwarp();  // the stage may be filled again
        at.next(a, first);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], o);
      // column of step i: gi (D / 8) + 2 i, and the next
      if (j0 == 0 && j1 == n_tiles) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = b * 8 + ti * 2 + e;
            if (h >= nh) continue;
            const float inv = KD_VALUE / l[b][e];  // scores of NaN or -inf alone: NaN
            uint32_t *dst = reinterpret_cast<uint32_t *>(a.o + (row0 + h) * D + gi * (D / 8));
#pragma unroll
            for (int i = 0; i < STEPS; ++i) dst[i] = kd_pack2(acc[b][i][e] * inv, acc[b][i][e + 2] * inv);
          }
      } else {
        // the last piece goes over this warp's tiles, which are all used up
        const int which = j0 == 0 ? 1 : 0;
        if (which) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
        }
        float *p = reinterpret_cast<float *>(smem + (which ? warp * L::RING : L::OFF_PART + warp * L::PART));
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = b * 8 + ti * 2 + e;
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
              *reinterpret_cast<float2 *>(p + h * D + gi * (D / 8) + 2 * i) = make_float2(acc[b][i][e], acc[b][i][e + 2]);
            if (gi == 0) {
              p[8 * NB * D + h] = m[b][e];
              p[8 * NB * (D + 1) + h] = l[b][e];
            }
          }
        if (lane == 0) meta[warp * 2 + which] = KdMeta{seq, unit, j0, j1};
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  // ---------------------------------------------------------------- joins ---
  // Pieces in order: each warp's first, then its last; a lane for each.  A chain of one item's
  // pieces begins where the piece before belongs to another.
  __syncthreads();
  static_assert(2 * L::WARPS <= 32, "a lane for every piece");
  auto piece = [&](int s) {
    return reinterpret_cast<const float *>(smem + (s & 1 ? s / 2 * L::RING : L::OFF_PART + s / 2 * L::PART));
  };
  KdMeta mine = {-1, 0, 0, 0};
  if (lane < 2 * L::WARPS) mine = meta[lane];
  const unsigned there = __ballot_sync(0xffffffffu, mine.seq >= 0);
  const unsigned below = there & ((1u << lane) - 1u);
  const int prev = below != 0 ? 31 - __clz(below) : lane;
  const int prev_seq = __shfl_sync(0xffffffffu, mine.seq, prev), prev_unit = __shfl_sync(0xffffffffu, mine.unit, prev);
  const bool joined = prev != lane && prev_seq == mine.seq && prev_unit == mine.unit;
  unsigned starts = __ballot_sync(0xffffffffu, mine.seq >= 0 && !joined);
  int4 span = make_int4(-1, 0, 0, 0);
  while (starts != 0) {
    const int c = __ffs(starts) - 1;
    starts &= starts - 1;
    const unsigned chain = there & (starts != 0 ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu) & ~((1u << c) - 1u);
    const int last = 31 - __clz(chain);
    KdMeta head;
    head.seq = __shfl_sync(0xffffffffu, mine.seq, c);
    head.unit = __shfl_sync(0xffffffffu, mine.unit, c);
    head.j0 = __shfl_sync(0xffffffffu, mine.j0, c);
    const int end = __shfl_sync(0xffffffffu, mine.j1, last);
    const int n_tiles = a.direct ? n_run : first[head.seq + 1] - first[head.seq];
    const bool whole = head.j0 == 0 && end == n_tiles;
    if (!whole && head.j0 == 0) {
      const long long item_end = (long long)first[head.seq] * a.units + (long long)(head.unit + 1) * n_tiles;
      span = make_int4(head.seq, head.unit, (int)((item_end - 1) / each), 0);
    }
    const int g = head.unit / a.subs, h_in = head.unit % a.subs * (8 * NB), nh = min(8 * NB, a.r - h_in);
    float *out = whole ? nullptr : a.part + ((size_t)blockIdx.x * 2 + (head.j0 == 0 ? 1 : 0)) * (8 * NB * (D + 2));
    for (int u = threadIdx.x; u < nh * (D / 2); u += THREADS) {
      const int h = u / (D / 2), d = u % (D / 2) * 2;
      float mm = -FLT_MAX, ll = 0.f, x = 0.f, y = 0.f;
      for (unsigned left = chain; left != 0; left &= left - 1) mm = fmaxf(mm, piece(__ffs(left) - 1)[8 * NB * D + h]);
      for (unsigned left = chain; left != 0; left &= left - 1) {
        const float *p = piece(__ffs(left) - 1);
        const float f = ptx::ex2_approx(p[8 * NB * D + h] - mm);
        const float2 v = *reinterpret_cast<const float2 *>(p + h * D + d);
        ll = fmaf(f, p[8 * NB * (D + 1) + h], ll);
        x = fmaf(f, v.x, x);
        y = fmaf(f, v.y, y);
      }
      if (whole) {
        const float inv = KD_VALUE / ll;
        *reinterpret_cast<uint32_t *>(a.o + ((size_t)head.seq * a.H + g * a.r + h_in + h) * D + d) =
            kd_pack2(x * inv, y * inv);
      } else {
        *reinterpret_cast<float2 *>(out + h * D + d) = make_float2(x, y);
        if (d == 0) {
          out[8 * NB * D + h] = mm;
          out[8 * NB * (D + 1) + h] = ll;
        }
      }
    }
  }
  if (a.spans != nullptr && threadIdx.x == 0) a.spans[blockIdx.x] = span;
}

// Joins the parts of the items that several CTAs had: a CTA of D / 2 threads for each CTA that
// may have begun one, and head.
template <int D, int NB>
__global__ void __launch_bounds__(D / 2) kv4_decode_join_kernel(const __grid_constant__ KdArgs a) {
  grid_dependency_wait();
  const int c0 = blockIdx.x, h = blockIdx.y;
  const int4 span = ld_after_wait(a.spans + c0);
  if (span.x < 0) return;
  const int g = span.y / a.subs, h_in = span.y % a.subs * (8 * NB);
  if (h >= a.r - h_in) return;
  auto part = [&](int c) { return a.part + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * (8 * NB * (D + 2)); };
  const int d = threadIdx.x * 2;
  float m = -FLT_MAX, l = 0.f, x = 0.f, y = 0.f;
#pragma unroll 4
  for (int c = c0; c <= span.z; ++c) m = fmaxf(m, part(c)[8 * NB * D + h]);
#pragma unroll 4
  for (int c = c0; c <= span.z; ++c) {
    const float *p = part(c);
    const float f = ptx::ex2_approx(p[8 * NB * D + h] - m);
    const float2 v = *reinterpret_cast<const float2 *>(p + h * D + d);
    l = fmaf(f, p[8 * NB * (D + 1) + h], l);
    x = fmaf(f, v.x, x);
    y = fmaf(f, v.y, y);
  }
  const float inv = KD_VALUE / l;
  *reinterpret_cast<uint32_t *>(a.o + ((size_t)span.x * a.H + g * a.r + h_in + h) * D + d) = kd_pack2(x * inv, y * inv);
}

// Form and grid of a call.
struct KdPlan {
  int nb = 1, subs = 1, units = 1;
  bool direct = true;
  int ctas = 1;
  size_t off_part = 0, bytes = 0;
};
KdPlan plan_of(int n_seqs, int max_kv_len, int H, int G, int D) {
  KdPlan p;
  const int r = H / G, sms = sm_count();
  p.nb = r > 8 ? 2 : 1;
  p.subs = (r + 8 * p.nb - 1) / (8 * p.nb);
  p.units = G * p.subs;
  const long long items = (long long)n_seqs * p.units;
  p.direct = (max_kv_len + KD_KEYS - 1) / KD_KEYS <= KD_DIRECT_TILES && items <= 0x7fffffffLL;
  p.ctas = p.direct ? (int)items : sms > 2 ? sms : 2;
  if (!p.direct) {
    p.off_part = ((size_t)p.ctas * 16 + 127) / 128 * 128;
    p.bytes = p.off_part + (size_t)p.ctas * 2 * 8 * p.nb * (D + 2) * 4;
  }
  return p;
}

template <int D, int NB>
cudaError_t launch(KdArgs a, const KdPlan &p, cudaStream_t st) {
  using L = KdLayout<D, NB>;
  static PerContextOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(kv4_decode_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::bytes(LLAMA_PACKED_MAX_SEQS));
  });
  if (e != cudaSuccess) return e;
  count_launch();
  const cudaError_t r =
      launch_pdl(kv4_decode_kernel<D, NB>, dim3((unsigned)p.ctas), dim3(L::WARPS * 32), L::bytes(a.n_seqs), st, a);
  if (r != cudaSuccess || p.direct) return r;
  count_launch();
  return launch_pdl(kv4_decode_join_kernel<D, NB>, dim3((unsigned)(p.ctas - 1), 8 * NB), dim3(D / 2), 0, st, a);
}

}  // namespace

size_t kv4_decode_workspace_bytes(int n_seqs, int max_kv_len, int H, int G, int D) {
  return plan_of(n_seqs, max_kv_len, H, G, D).bytes;
}

cudaError_t launch_kv4_decode(const bf16 *q, const uint8_t *k, const uint8_t *v, bf16 *o, const PagedView &pv,
                              const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int D, void *workspace,
                              int *status, cudaStream_t st) {
  const KdPlan p = plan_of(n_seqs, max_kv_len, H, G, D);
  KdArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.pv = pv;
  a.kv_lens = kv_lens;
  a.n_seqs = n_seqs;
  a.max_kv_len = max_kv_len;
  a.H = H;
  a.G = G;
  a.r = H / G;
  a.subs = p.subs;
  a.units = p.units;
  a.direct = p.direct;
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)D);
  a.part = p.direct ? nullptr : reinterpret_cast<float *>((char *)workspace + p.off_part);
  a.spans = p.direct ? nullptr : reinterpret_cast<int4 *>(workspace);
  a.status = status;
#define KD_CASE(d) \
  case d: return p.nb == 1 ? launch<d, 1>(a, p, st) : launch<d, 2>(a, p, st);
  switch (D) {
    KD_CASE(16)
    KD_CASE(32)
    KD_CASE(64)
    KD_CASE(128)
  }
#undef KD_CASE
  return cudaErrorInvalidValue;
}

}  // namespace llama
