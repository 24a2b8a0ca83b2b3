// Attention of few query rows a sequence over cache pages held in 4 bits, q and o bf16: one
// new token of each sequence, or the last confirmed one and its drafts ("Full Llama 3
// transformer block", How it works: keys j <= position; "The Evolving Transformer 04 ·
// LLaMA", §05 GQA).  For token t at position p
//   o = sum_{j<=p} 2^(x_j - m) v_j / sum_{j<=p} 2^(x_j - m),  x_j = q.k_j log2(e) / sqrt(D),
// in one pass over the keys, the running maximum m and the sum in fp32.
//
// The cache is read once, and a byte of it is nearly two elements: what has to be kept small
// is the work per element.  A warp takes 64 or 32 keys at a time for 8, 16 or 24 rows (head of the
// group, token) of a sequence; codes go from shared memory into registers and from there
// straight into the operands of mma.sync, keys and columns of the values on its 16-row side:
//   S^T[16 keys x 8 rows] = K Q^T,     O^T[16 columns x 8 rows] += V^T P^T.
// The order of d within K and Q, and of the columns in V and O, is free: it is the one that
// leaves every thread whole words of codes.  Two codes become two 16-bit numbers with a
// shift, a masked or and an fma (kv4.cuh): K bf16 as Q is, V fp16, and P^T, which comes from
// S^T by movmatrix, fp16 too.  V's products run over keys, so the words of two keys are
// interleaved first, half a word at a time.  (With the rows on tcgen05's side of 128, as in
// packed_tc.cu, the 16-bit numbers go through shared memory, four times the codes, and the side is
// mostly padding: 64 sequences of 5 rows on 8 KV heads 104 us.  Keys on that side, from tensor
// memory for one of the two products, were not tried.)
// Each warp copies its own tiles into its own shared memory, a few tiles ahead, and waits
// for nothing but those copies.
//
// All tiles of the call in one row -- sequence by sequence, block of rows by block of rows --
// are dealt out to the CTAs, and a CTA's to its warps, in even runs.  A run that begins or
// ends inside an item leaves its (O, m, l); the CTA joins those of its warps, in order,
// and what begins or ends inside the CTA's run goes to the workspace, where a second kernel
// joins it, in order.  With short sequences (direct: one token each) a CTA takes one item
// instead, and there is no second kernel.
//
// Measured, D = 128 and 8 KV heads of four: 64 sequences of 253 to 4096 keys 41.5 us, of which
// about 11 are the kernels' beginnings and joins; between, 5.3 TB/s (0.78 of the copy rate),
// instructions issued in two cycles of three.  One sequence of 120001 keys 40.5 us.  64
// sequences of five rows 71 us: three times the products on the same unpacked numbers,
// bound by their latency (255 registers, with 64 bytes of them spilled, leave two warps to a
// scheduler).  The page ids of a tile are looked up by an index of run time, which puts them in
// 16 to 32 bytes of local memory in every form.
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>

#include <type_traits>

#include "kv4.cuh"
#include "paged_kernels.h"
#include "ptx.cuh"

namespace llama {
namespace {

// Keys of a warp's tile: as many as the registers have room for, what is done once a tile is a
// third of a tile of 32 keys.  (64 sequences of one and of three rows, four heads to a group: 41.6
// and 51.6 us at 64 keys, 46.7 and 55.6 at 32.)
constexpr int kd_keys(int NB) { return NB <= 2 ? 64 : 32; }
// Places before an item's first tile in the row that is dealt out: an item's beginning and end
// (its queries, its output) take as long as 64 keys.  (64 sequences of 253 to 4096 keys, 8 KV
// heads of 4 rows: 43.7, 41.2, 42.6 us with 0, 1, 2 tiles of 64 keys; of 20 rows, tiles of 32:
// 75.5, 72.7, 71.4, 71.8 with 0, 1, 2, 3.)
constexpr int kd_start(int NB) { return 64 / kd_keys(NB); }
constexpr float KD_RESCALE = 8.0f;  // log2 units: the running maximum is raised when it grows by > 2^8
// Weights are fp16 for their product with V: 2^7 times what they are, so that the largest,
// 2^15, has room above, and what is less than 2^-31 of the running maximum's, not 2^-24, is
// lost (120000 keys of such weights: 2^-14 of the sum).
constexpr float KD_WEIGHT = 7.0f;
constexpr float KD_VALUE = 2.0f;  // V's operand is half of V
// Keys of a CTA's item in the direct form, at most; elements of them where the items leave three
// of four SMs idle.  (Direct / planned, D = 128, 8 KV heads: one sequence of 1000 keys 8.6 / 8.9 us,
// of 1500 10.7 / 9.1; four of 1500 11.2 / 10.2; 16 of 1000 9.1 / 12.9, of 2048 14.5 / 18.3.  D = 64,
// 3 KV heads: four of 1500 7.9 / 8.5, of 2048 9.1 / 8.7; 16 of 2048 9.2 / 9.8.)
constexpr int KD_DIRECT_KEYS = 2048, KD_DIRECT_FEW = 1024 * 128;
constexpr int KD_MAX_NB = 3;
constexpr int KD_ROUNDS = 10, KD_FEW_KEYS = 384;  // of packed calls: see kv4_rows_fit
constexpr int KD_FEW_ROWS = 48, KD_MIXED_ROUNDS = 96;  // see kv4_rows_few
constexpr int KD_BATCH = 2;  // pieces that a join within a CTA reads at a time
constexpr int KD_LEAST = 4;  // tiles of a CTA's run, at least: a warp on each scheduler

// NB: blocks of 8 rows of an item.
template <int D, int NB>
struct KdLayout {
  static constexpr int WARPS = 8, KEYS = kd_keys(NB);
  static constexpr int RB = kv4_code_bytes(D), SB = kv4_scale_bytes(D);
  static constexpr int HALF = KEYS * (RB + SB), STAGE = 2 * HALF;  // K, then V: codes, then scales
  static constexpr int PART = 8 * NB * (D + 2) * 4;  // (O, m, l) of an item
  static constexpr int FIT = (NB <= 2 ? 18432 : 13824) / STAGE;
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr int RING = STAGES * STAGE > PART ? STAGES * STAGE : PART;  // of a warp; its last part at the end
  static constexpr int OFF_PART = WARPS * RING;   // of each warp, its first
  static constexpr int OFF_META = OFF_PART + WARPS * PART;
  static constexpr int OFF_SUMS = OFF_META + WARPS * 2 * 48;
  // tiles before sequence i: of one item with a row each, else of its items for one KV head
  static constexpr int OFF_FIRST = OFF_SUMS + 128;
  static int bytes(int n_seqs) { return OFF_FIRST + (n_seqs + 1) * 4; }
};
static_assert(KdLayout<128, 1>::OFF_FIRST + (LLAMA_PACKED_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits an SM");
static_assert(KdLayout<128, 2>::OFF_FIRST + (LLAMA_PACKED_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits an SM");
static_assert(KdLayout<128, 3>::OFF_FIRST + (LLAMA_PACKED_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits an SM");

struct KdArgs {
  const bf16 *q;
  const uint8_t *k, *v;
  bf16 *o;
  PagedView pv;
  PackedView b;  // q_offsets null: one row of q and o per sequence
  int H, G, r;   // r: heads of a group
  int few;       // tokens of a sequence that this kernel takes; those of others are another's
  int times;     // items of a sequence for each of the tiles that `first` counts
  int most;      // tiles that `first` may count: offsets that descend make sequences overlap
  int direct;
  float scale_log2;
  float *part;  // [CTA][2][8 NB][D + 2]
  int4 *spans;  // of each CTA, the item that it begins and leaves: two, its last CTA (-1: none) and as KdOut has it
  int *status;
};

__device__ __forceinline__ uint32_t kd_pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
// N words side by side.
template <int N>
__device__ __forceinline__ void kd_store(uint32_t *dst, const uint32_t (&w)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4 *>(dst + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
  } else {
    dst[0] = w[0];
  }
}
// A piece of an item that a warp leaves for its CTA to join.
struct __align__(16) KdMeta {
  int seq, unit;  // seq -1: none
  int j0, j1, n;  // its key tiles, and all of the item's
  int first, count, kv_len;  // of the sequence
  int g, r0;
  int pad[2];
};

// An item as its join has it: its rows in o, and the keys that the sequence's first token sees.
struct KdOut {
  int first, g, r0, nr, before;
  __device__ __forceinline__ KdOut(const KdArgs &a, int first_, int count, int kv_len, int g_, int r0_, int most)
      : first(first_), g(g_), r0(r0_), nr(min(most, count * a.r - r0_)), before(kv_len - count + 1) {}
};

// Sums of a fragment's columns -- steps i of rows 8 b + 2 ti + e, a float2 of each lane -- over
// the pieces piece(0) .. piece(n - 1), in that order, BATCH of them read at a time.  SPLIT:
// warps that share the steps.
template <int D, int NB, int SPLIT, int BATCH>
struct KdSum {
  static constexpr int STEPS = D / 16 / SPLIT;
  int i0;  // the first of the steps
  float2 x[STEPS];
  float top = -FLT_MAX, l = 0.f;
  template <typename F>
  __device__ __forceinline__ KdSum(int be, int part, int n, F &&piece) : i0(part * STEPS) {
    const int lane = threadIdx.x & 31, h = be / 2 * 8 + (lane & 3) * 2 + (be & 1);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) x[i] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int s = 0; s < n; s += BATCH) {
      float m[BATCH], w[BATCH];
      float2 v[BATCH][STEPS];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        m[k] = -FLT_MAX;
        w[k] = 0.f;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) v[k][i] = make_float2(0.f, 0.f);
        if (s + k < n) {
          const float *p = piece(s + k);
          m[k] = p[8 * NB * D + h];
          w[k] = p[8 * NB * (D + 1) + h];
#pragma unroll
          for (int i = 0; i < STEPS; ++i)
            v[k][i] = *reinterpret_cast<const float2 *>(p + (be * (D / 16) + i0 + i) * 64 + lane * 2);
        }
      }
      float up = top;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) up = fmaxf(up, m[k]);
      const float less = ptx::ex2_approx(top - up);
      top = up;
      l *= less;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        x[i].x *= less;
        x[i].y *= less;
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const float f = ptx::ex2_approx(m[k] - up);
        l = fmaf(f, w[k], l);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          x[i].x = fmaf(f, v[k][i].x, x[i].x);
          x[i].y = fmaf(f, v[k][i].y, x[i].y);
        }
      }
    }
  }
  // The rows' outputs: a lane has D / 8 columns of its own.
  __device__ __forceinline__ void store(const KdArgs &a, const KdOut &k, int be) const {
    const int lane = threadIdx.x & 31, h = be / 2 * 8 + (lane & 3) * 2 + (be & 1);
    if (h >= k.nr) return;
    const int i = (k.r0 + h) / a.r;
    if (k.before + i <= 0) return;  // it sees nothing
    const float inv = KD_VALUE / l;
    uint32_t *dst = reinterpret_cast<uint32_t *>(
        a.o + ((size_t)(k.first + i) * a.H + k.g * a.r + (k.r0 + h - i * a.r)) * D + lane / 4 * (D / 8) + 2 * i0);
    uint32_t w[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) w[i] = kd_pack2(x[i].x * inv, x[i].y * inv);
    kd_store<STEPS>(dst, w);
  }
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

// The rows and keys of a sequence as its items have them; no rows where they are out of range
// or another kernel's.
__device__ __forceinline__ SeqSpan kd_span(const KdArgs &a, int i) {
  if (a.b.q_offsets != nullptr) {
    const SeqSpan s = seq_span(a.b, a.pv, i);
    return s.count <= a.few ? s : SeqSpan{s.first, 0, 0};
  }
  return SeqSpan{i, 1, checked_len(ld_after_wait(a.b.kv_lens + i), a.b.max_kv_len, a.pv)};
}
template <int NB>
__host__ __device__ __forceinline__ int kd_tiles(int keys) { return (keys + kd_keys(NB) - 1) / kd_keys(NB); }

// Token and head in the group of an item's row, without a division for each: the item's first
// row has been divided, and what is left is small (fp32 is exact to half a step there).
struct KdRows {
  int token0, head0;
  float inv;
  __device__ __forceinline__ KdRows(int r0, int r) : token0(r0 / r), head0(r0 - r0 / r * r), inv(1.f / (float)r) {}
  __device__ __forceinline__ int token(int h) const { return token0 + (int)(((float)(head0 + h) + 0.5f) * inv); }
  __device__ __forceinline__ int head(int h, int r) const { return head0 + h - (token(h) - token0) * r; }
};

// A place in the row of tiles.  A unit is a KV head and a block of 8 NB rows.
template <int NB>
struct KdCursor {
  int seq, unit, units, g, sub, j, n;  // units, n: of the sequence, n its key tiles
  SeqSpan s;
  __device__ __forceinline__ void set(const KdArgs &a, int i, int u, int at) {
    seq = i;
    s = kd_span(a, i);
    n = kd_tiles<NB>(s.kv_len);
    const int subs = (s.count * a.r + 8 * NB - 1) / (8 * NB);
    units = a.G * subs;
    unit = u;
    g = u / subs;
    sub = u - g * subs;
    j = at;
  }
  __device__ __forceinline__ void seek(const KdArgs &a, const int *first, long long at) {
    int lo = 0, hi = a.b.n_seqs;  // the last sequence that begins at or before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if ((long long)first[mid] * a.times <= at) lo = mid;
      else hi = mid;
    }
    const long long rest = at - (long long)first[lo] * a.times;
    set(a, lo, 0, 0);
    // (a 64-bit division takes some hundred cycles)
    const int slots = n + kd_start(NB), u = rest <= 0x7fffffffLL ? (int)rest / slots : (int)(rest / slots);
    const int subs = units / a.G;
    unit = u;
    g = u / subs;
    sub = u - g * subs;
    j = (int)(rest - (long long)u * slots) - kd_start(NB);
  }
  __device__ __forceinline__ bool next(const KdArgs &a, const int *first) {  // true: it is another item's
    if (++j < n || a.direct) return false;
    int i = seq, u = unit + 1;
    if (u == units) {
      u = 0;
      for (++i; i < a.b.n_seqs && first[i + 1] == first[i]; ++i) {
      }
      if (i == a.b.n_seqs) return false;  // the end of the row
    }
    set(a, i, u, -kd_start(NB));
    return true;
  }
};

template <int D, int NB>
__global__ void __launch_bounds__(KdLayout<D, NB>::WARPS * 32, 1) kv4_rows_kernel(const __grid_constant__ KdArgs a) {
  using L = KdLayout<D, NB>;
  constexpr int THREADS = L::WARPS * 32;
  constexpr int KW = D / 32 > 0 ? D / 32 : 1;  // words of a key's codes that a thread takes (of 8 elements)
  constexpr int VW = D / 64 > 0 ? D / 64 : 1;  // of a value's
  constexpr int STEPS = D / 16, MB = L::KEYS / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, gi = lane / 4, ti = lane & 3;
  const uint32_t s0 = ptx::smem_u32(smem);
  int *first = reinterpret_cast<int *>(smem + L::OFF_FIRST);
  int *sums = reinterpret_cast<int *>(smem + L::OFF_SUMS);
  KdMeta *meta = reinterpret_cast<KdMeta *>(smem + L::OFF_META);
  static_assert(sizeof(KdMeta) == 48, "a piece's place");
  const uint32_t ring = s0 + warp * L::RING;
  allow_dependents_launch();
  if (lane < 2) meta[warp * 2 + lane].seq = -1;
  grid_dependency_wait();

  // ------------------------------------------------------------- lengths ---
  KdCursor<NB> at;
  long long begin = 0, each = 1;
  int n_run;  // tiles of this CTA's run
  if (a.direct) {
    const int units = a.G * ((a.r + 8 * NB - 1) / (8 * NB));
    const int seq = blockIdx.x / units, unit = blockIdx.x % units;
    at.set(a, seq, unit, 0);
    n_run = at.n;
    if (unit == 0 && threadIdx.x == 0 && ld_after_wait(a.b.kv_lens + seq) != at.s.kv_len)
      report_status(a.status, LLAMA_ERR_RANGE);
    if (n_run == 0) {  // no keys: zeros
      uint4 *dst = reinterpret_cast<uint4 *>(a.o + (size_t)seq * a.H * D);
      if (unit == 0)
        for (int e = threadIdx.x; e < a.H * D / 8; e += THREADS) dst[e] = make_uint4(0, 0, 0, 0);
      return;
    }
  } else {
    // (4096 sequences: 16 each)
    const int per = (a.b.n_seqs + THREADS - 1) / THREADS;
    auto add = [&](int x, int y) { return (int)min((unsigned)x + (unsigned)y, (unsigned)a.most); };
    int mine = 0;
    bool blind = false;  // rows before their sequence's first key
    for (int k = 0; k < per; ++k) {
      const int i = threadIdx.x * per + k;
      if (i >= a.b.n_seqs) break;
      const SeqSpan s = kd_span(a, i);
      if (blockIdx.x == 0) {
        if (a.b.q_offsets != nullptr) check_seq(a.b, a.pv, i, a.status);
        else if (ld_after_wait(a.b.kv_lens + i) != s.kv_len) report_status(a.status, LLAMA_ERR_RANGE);
      }
      int n = kd_tiles<NB>(s.kv_len);
      if (n > 0) n += kd_start(NB);
      if (a.b.q_offsets != nullptr) n = min((long long)n * ((s.count * a.r + 8 * NB - 1) / (8 * NB)), (long long)a.most);
      blind |= s.kv_len < s.count;
      first[i] = n;
      mine = add(mine, n);
    }
    int end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end = add(end, x);
    }
    if (lane == 31) sums[warp] = end;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, end, 1);  // (not end - mine: the sums may be cut off)
    if (lane == 0) before = 0;
    for (int w = 0; w < warp; ++w) before = add(before, sums[w]);
    for (int k = 0; k < per; ++k) {
      const int i = threadIdx.x * per + k;
      if (i >= a.b.n_seqs) break;
      const int n = first[i];
      first[i] = before;
      before = add(before, n);
    }
    if (threadIdx.x == THREADS - 1) first[a.b.n_seqs] = before;
    if (__syncthreads_or(blind))  // those rows are zeros
      for (int i = 0; i < a.b.n_seqs; ++i) {
        const SeqSpan s = kd_span(a, i);
        const long long n = (long long)max(0, s.count - s.kv_len) * (a.H * D / 8);
        uint4 *dst = reinterpret_cast<uint4 *>(a.o + (size_t)s.first * a.H * D);
        for (long long e = (long long)blockIdx.x * THREADS + threadIdx.x; e < n; e += (long long)gridDim.x * THREADS)
          dst[e] = make_uint4(0, 0, 0, 0);
      }
    const long long total = (long long)first[a.b.n_seqs] * a.times;
    each = (total + gridDim.x - 1) / gridDim.x;
    each = each > KD_LEAST ? each : KD_LEAST;
    begin = min(total, each * blockIdx.x);
    n_run = (int)(min(total, begin + each) - begin);
  }
  const int share = n_run / L::WARPS, more = n_run % L::WARPS;  // the first `more` warps take one more
  const int w0 = warp * share + min(warp, more), todo = share + (warp < more ? 1 : 0);

  if (todo > 0) {
    if (a.direct) at.j = w0;
    else at.seek(a, first, begin + w0);
    // ------------------------------------------------------------ copies ---
    // A tile's rows are runs of 16, which no page splits; a run behind the last key is given the
    // first one's rows, which may be read, and its scores are replaced.  Every lane knows the
    // page ids and adds to pointers of its own (by bulk copies, whose operands have to be made
    // uniform, a tile of 32 keys took 893 instructions for the 838 of lanes asking one another
    // and the 823 of this).
    KdCursor<NB> ahead = at;  // the tile whose pages are known and that is copied next
    constexpr int RUNS = L::KEYS / 16;
    constexpr int CHUNK = L::RB < 16 ? L::RB : 16;             // bytes of a lane's copy
    constexpr int COPIES = D >= 64 ? L::RB / 32 : 1;           // of 32 lanes for a run; D < 64: for two
    constexpr int S_PIECES = L::KEYS * L::SB / 16;             // of 16 bytes: K's scales, and V's
    constexpr int S_COPIES = S_PIECES > 16 ? S_PIECES / 16 : 1;
    int left = todo, fill = 0, id[RUNS], slot[RUNS], s_id = 0, s_slot = 0;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) id[r] = slot[r] = 0;
    const int rows_mask = (1 << a.pv.page_log2) - 1;
    const bool wide = 1 << a.pv.page_log2 >= L::KEYS;  // a tile lies in one page
    const uint32_t stride = (uint32_t)a.pv.page_stride;
    // scales: pieces lane + 32 i, K's first; S_PIECES is 32 at most, then i says K or V
    const int s_piece = lane % S_PIECES, s_run = s_piece / L::SB;
    const bool s_mine = lane < 2 * S_PIECES;
    const uint8_t *from_k, *from_v, *from_s[S_COPIES];
    auto aim = [&] {  // this lane's bytes of page 0
      const int block = kv4_block_bytes(1 << a.pv.page_log2, D) * ahead.g;
      const int off = D >= 64 ? lane * 16 : lane % 16 * CHUNK;
      from_k = a.k + block + off;
      from_v = a.v + block + off;
      // the item's queries, a line each: they are loaded when its first tile is there
      const int r0 = ahead.sub * (8 * NB), nr = min(8 * NB, ahead.s.count * a.r - r0);
      constexpr int LINES = D >= 64 ? D / 64 : 1;
      const KdRows rows(r0, a.r);
      for (int i = lane; i < nr * LINES; i += 32) {
        const int h = i / LINES;
        const bf16 *row = a.q + ((size_t)(ahead.s.first + rows.token(h)) * a.H + ahead.g * a.r + rows.head(h, a.r)) * D;
        asm volatile("prefetch.global.L1 [%0];" ::"l"(row + i % LINES * 64));
      }
#pragma unroll
      for (int i = 0; i < S_COPIES; ++i)
        from_s[i] = ((S_COPIES > 1 ? i : lane / S_PIECES) == 0 ? a.k : a.v) + block + (L::RB << a.pv.page_log2) +
                    s_piece % L::SB * 16;
    };
    auto look_up = [&] {
      if (left <= 0) return;
      const int p = ahead.j * L::KEYS;
      const int *table = a.pv.table + (size_t)ahead.seq * a.pv.table_stride;
      id[0] = ld_after_wait(table + (p >> a.pv.page_log2));
      slot[0] = p & rows_mask;
      if (wide) {
        s_id = id[0];
        s_slot = slot[0] + s_run * 16;
        return;
      }
#pragma unroll
      for (int r = 1; r < RUNS; ++r) {
        const int pr = p + 16 * r < ahead.s.kv_len ? p + 16 * r : p;
        id[r] = ld_after_wait(table + (pr >> a.pv.page_log2));
        slot[r] = pr & rows_mask;
      }
      const int ps = p + 16 * s_run < ahead.s.kv_len ? p + 16 * s_run : p;
      s_id = ld_after_wait(table + (ps >> a.pv.page_log2));
      s_slot = ps & rows_mask;
    };
    auto to_tile = [](KdCursor<NB> &c, int rest) {  // over the places before an item's first tile
      const int step = min(max(-c.j, 0), rest);
      c.j += step;
      return step;
    };
    auto request = [&] {
      if (left > 0) {
        const uint32_t stage = ring + fill * L::STAGE, to = stage + lane * CHUNK;
        bool bad = (unsigned)id[0] >= (unsigned)a.pv.n_pages;  // a page is out of range
        if (wide && !bad) {
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            // (with D < 64 lanes 16 .. have another row in each of their runs)
            const uint8_t *p = (which ? from_v : from_k) + (uint64_t)(uint32_t)id[0] * stride + slot[0] * L::RB +
                               (D >= 64 ? 0 : lane / 16 * 16 * L::RB);
#pragma unroll
            for (int i = 0; i < L::KEYS * L::RB / (32 * CHUNK); ++i)
              copy_async<CHUNK>(to + which * L::HALF + i * 32 * CHUNK, p + i * 32 * CHUNK);
          }
        } else {
          if (!wide)
#pragma unroll
            for (int r = 1; r < RUNS; ++r) bad |= (unsigned)id[r] >= (unsigned)a.pv.n_pages;
          if (bad && lane == 0) report_status(a.status, LLAMA_ERR_RANGE);
#pragma unroll
          for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int r = 0; r < RUNS; r += D >= 64 ? 1 : 2) {
              const int in = wide ? 0 : r, r1 = D >= 64 ? in : wide ? 0 : r + 1;
              const int my_id = D >= 64 || lane < 16 ? id[in] : id[r1];
              const int my_slot = (D >= 64 || lane < 16 ? slot[in] : slot[r1]) +
                                  (wide ? (r + (D >= 64 ? 0 : lane / 16)) * 16 : 0);
              const uint8_t *p = (which ? from_v : from_k) + (uint64_t)(uint32_t)my_id * stride + my_slot * L::RB;
              const uint32_t dst = to + which * L::HALF + r * 16 * L::RB;
#pragma unroll
              for (int i = 0; i < COPIES; ++i) {
                if ((unsigned)my_id < (unsigned)a.pv.n_pages) {
                  copy_async<CHUNK>(dst + i * 512, p + i * 512);
                } else {  // zeros
                  asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(dst + i * 512), "r"(0x88888888u) : "memory");
                  if (CHUNK == 16)
                    asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(dst + i * 512 + 8), "r"(0x88888888u) : "memory");
                }
              }
            }
        }
        if (s_mine && (unsigned)s_id < (unsigned)a.pv.n_pages) {
          const uint64_t off = (uint64_t)(uint32_t)s_id * stride + (uint32_t)(s_slot * L::SB);
#pragma unroll
          for (int i = 0; i < S_COPIES; ++i)
            copy_async<16>(stage + (S_COPIES > 1 ? i : lane / S_PIECES) * L::HALF + L::KEYS * L::RB + s_piece * 16,
                           from_s[i] + off);
        }
        --left;
        if (ahead.next(a, first)) {
          aim();
          left -= to_tile(ahead, left);
        }
        fill = fill + 1 == L::STAGES ? 0 : fill + 1;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    left -= to_tile(ahead, left);
    aim();
    look_up();
#pragma unroll 1
    for (int n = 0; n < L::STAGES - 1; ++n) {
      request();
      look_up();
    }
    int done = 0, use = 0;
    while ((done += to_tile(at, todo - done)) < todo) {
      // ----------------------------------------------------------- a piece ---
      const int seq = at.seq, unit = at.unit, j0 = at.j, n_tiles = at.n, g = at.g;
      const int j1 = min(n_tiles, j0 + todo - done);
      const int r0 = at.sub * (8 * NB), nr = min(8 * NB, at.s.count * a.r - r0);
      const int before = at.s.kv_len - at.s.count + 1;  // keys that the sequence's first new token sees
      const KdRows rows(r0, a.r);
      // row h of the item in q and o
      auto row_at = [&](int h) { return (size_t)(at.s.first + rows.token(h)) * a.H + g * a.r + rows.head(h, a.r); };
      uint32_t qf[NB][STEPS][2];
      int sees[NB][2];  // keys that this thread's columns of S^T see
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int h = b * 8 + gi;
        const int *src = reinterpret_cast<const int *>(a.q + row_at(min(h, nr - 1)) * D + ti * (D / 4));
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          if constexpr (STEPS >= 2) {
            if (s % 2 == 0) {
              const int4 x = ld_after_wait(reinterpret_cast<const int4 *>(src + 2 * s));
              qf[b][s][0] = (uint32_t)x.x;
              qf[b][s][1] = (uint32_t)x.y;
              qf[b][s + 1 < STEPS ? s + 1 : s][0] = (uint32_t)x.z;
              qf[b][s + 1 < STEPS ? s + 1 : s][1] = (uint32_t)x.w;
            }
          } else {
            qf[b][s][0] = (uint32_t)ld_after_wait(src);
            qf[b][s][1] = (uint32_t)ld_after_wait(src + 1);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) sees[b][e] = before + rows.token(min(b * 8 + ti * 2 + e, nr - 1));
      }
      const int all_see = before + rows.token0;
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
        request();
        look_up();
        asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 1) : "memory");
        __syncwarp();
        const uint32_t sk = ring + use * L::STAGE, sv = sk + L::HALF;
        // scores: keys gi and gi + 8 of every 16, 32 keys at a time
        float sc[MB][NB][4];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mb][b][e] = 0.f;
#pragma unroll
        for (int m0 = 0; m0 < MB; m0 += 2) {
          uint32_t w[4][KW];
          Kv4Scale sa[4], sb[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = m0 * 16 + e * 8 + gi;
            const uint32_t scales = sk + L::KEYS * L::RB + row * L::SB;
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
          for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
              uint32_t f[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t word = w[2 * mb + e][s / 2];
                const Kv4Scale &k = s < 4 ? sa[2 * mb + e] : sb[2 * mb + e];
                f[e] = s % 2 == 0 ? kv4_pair<0>(word, k) : kv4_pair<2>(word, k);
                f[2 + e] = s % 2 == 0 ? kv4_pair<1>(word, k) : kv4_pair<3>(word, k);
              }
#pragma unroll
              for (int b = 0; b < NB; ++b) mma16816(sc[m0 + mb][b], f, qf[b][s][0], qf[b][s][1]);
            }
        }
        if ((j + 1) * L::KEYS > all_see) {
          const int key = j * L::KEYS + gi;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key + mb * 16 + (e / 2) * 8 >= sees[b][e & 1]) sc[mb][b][e] = -INFINITY;
        }
        // weights: rows 8 b + 2 ti and the next
        uint32_t pf[MB][NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float mx[2];
          bool need = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(sc[0][b][e], sc[0][b][e + 2]);
#pragma unroll
            for (int mb = 1; mb < MB; ++mb) mx[e] = fmaxf(mx[e], fmaxf(sc[mb][b][e], sc[mb][b][e + 2]));
            mx[e] *= a.scale_log2;
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
          for (int mb = 0; mb < MB; ++mb) {
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
        for (int mb = 0; mb < MB; ++mb) {
          uint32_t even[2][VW], odd[2][VW];
          Kv4Half sv2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = mb * 16 + e * 8 + 2 * ti;
            uint32_t x[VW], y[VW];
            const uint32_t from = sv + row * L::RB + (D >= 64 ? gi * (D / 16) : D == 32 ? gi / 2 * 4 : gi / 4 * 4);
            ld_words<VW>(from, x);
            ld_words<VW>(from + L::RB, y);
            const uint32_t scales = sv + L::KEYS * L::RB + row * L::SB + gi * L::SB / 8;
            sv2[e] = kv4_halves(ld_byte(scales), ld_byte(scales + L::SB));
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
        use = use + 1 == L::STAGES ? 0 : use + 1;
        if (j + 1 < j1) ++at.j;  // (the piece is looked at below)
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
            if (h >= nr || sees[b][e] <= 0) continue;
            const float inv = KD_VALUE / l[b][e];  // scores of NaN or -inf alone: NaN
            uint32_t w[STEPS];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) w[i] = kd_pack2(acc[b][i][e] * inv, acc[b][i][e + 2] * inv);
            kd_store<STEPS>(reinterpret_cast<uint32_t *>(a.o + row_at(h) * D + gi * (D / 8)), w);
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
            // in the order of the fragments: a warp's stores are whole
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
              *reinterpret_cast<float2 *>(p + ((b * 2 + e) * STEPS + i) * 64 + lane * 2) =
                  make_float2(acc[b][i][e], acc[b][i][e + 2]);
            if (gi == 0) {
              p[8 * NB * D + b * 8 + ti * 2 + e] = m[b][e];
              p[8 * NB * (D + 1) + b * 8 + ti * 2 + e] = l[b][e];
            }
          }
        if (lane == 0)
          meta[warp * 2 + which] =
              KdMeta{seq, unit, j0, j1, n_tiles, at.s.first, at.s.count, at.s.kv_len, g, r0, {0, 0}};
      }
      at.next(a, first);
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
  int my_seq = -1, my_unit = 0;
  if (lane < 2 * L::WARPS) {
    my_seq = meta[lane].seq;
    my_unit = meta[lane].unit;
  }
  const unsigned there = __ballot_sync(0xffffffffu, my_seq >= 0);
  const unsigned below = there & ((1u << lane) - 1u);
  const int prev = below != 0 ? 31 - __clz(below) : lane;
  const int prev_seq = __shfl_sync(0xffffffffu, my_seq, prev), prev_unit = __shfl_sync(0xffffffffu, my_unit, prev);
  const bool joined = prev != lane && prev_seq == my_seq && prev_unit == my_unit;
  unsigned starts = __ballot_sync(0xffffffffu, my_seq >= 0 && !joined);
  if (a.spans != nullptr && threadIdx.x == 0) {  // the CTA's last item: it may begin it and not end it
    int4 span = make_int4(-1, 0, 0, 0), item = span;
    if (starts != 0) {
      const KdMeta &x = meta[31 - __clz(starts)];
      if (x.j0 == 0 && meta[31 - __clz(there)].j1 < x.n) {
        const long long item_end = (long long)first[x.seq] * a.times + (long long)(x.unit + 1) * (x.n + kd_start(NB));
        span = make_int4((int)min((item_end - 1) / each, (long long)gridDim.x - 1), x.first, x.count, x.kv_len);
        item = make_int4(x.g, x.r0, 0, 0);
      }
    }
    a.spans[2 * blockIdx.x] = span;
    a.spans[2 * blockIdx.x + 1] = item;
  }
  // A warp for each chain and two blocks' worth of fragments (rows 8 b + e, + 2, + 4, + 6).
  int u = 0;
  while (starts != 0) {
    const int c = __ffs(starts) - 1;
    starts &= starts - 1;
    const unsigned chain = there & (starts != 0 ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu) & ~((1u << c) - 1u);
    const KdMeta &x = meta[c];
    const KdOut k(a, x.first, x.count, x.kv_len, x.g, x.r0, 8 * NB);
    const bool whole = x.j0 == 0 && meta[31 - __clz(chain)].j1 == x.n;
    float *out = whole ? nullptr : a.part + ((size_t)blockIdx.x * 2 + (x.j0 == 0 ? 1 : 0)) * (8 * NB * (D + 2));
    for (int be = 0; be < 2 * NB; ++be) {
      if (be / 2 * 8 + (be & 1) >= k.nr) continue;  // no rows
      if (u++ % L::WARPS != warp) continue;
      // (behind its first piece a chain goes on with the first one of each warp that follows)
      const KdSum<D, NB, 1, KD_BATCH> sum(be, 0, __popc(chain), [&](int s) { return piece(s == 0 ? c : (c / 2 + s) * 2); });
      if (whole) {
        sum.store(a, k, be);
        continue;
      }
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        *reinterpret_cast<float2 *>(out + (be * STEPS + i) * 64 + lane * 2) = sum.x[i];
      if (gi == 0) {
        const int h = be / 2 * 8 + ti * 2 + (be & 1);
        out[8 * NB * D + h] = sum.top;
        out[8 * NB * (D + 1) + h] = sum.l;
      }
    }
  }
}

// Joins the parts of the items that several CTAs had: KD_JOIN warps for each CTA that may have
// begun one and fragment.
template <int D>
constexpr int KD_JOIN = D >= 64 ? 4 : D / 16;
template <int D, int NB>
__global__ void __launch_bounds__(64 * NB * KD_JOIN<D>) kv4_rows_join_kernel(const __grid_constant__ KdArgs a) {
  grid_dependency_wait();
  const int c0 = blockIdx.x, be = threadIdx.x / 32 / KD_JOIN<D>, part = threadIdx.x / 32 % KD_JOIN<D>;
  const int4 span = ld_after_wait(a.spans + 2 * c0), item = ld_after_wait(a.spans + 2 * c0 + 1);
  if (span.x < 0) return;
  const KdOut k(a, span.y, span.z, span.w, item.x, item.y, 8 * NB);
  const KdSum<D, NB, KD_JOIN<D>, NB == 1 ? 16 : 8> sum(be, part, span.x - c0 + 1, [&](int s) {
    return a.part + ((size_t)(c0 + s) * 2 + (s == 0 ? 1 : 0)) * (8 * NB * (D + 2));
  });
  sum.store(a, k, be);
}

// Form and grid of a call; rows: of a sequence and KV head, on average.
struct KdPlan {
  int nb = 1, ctas = 1;
  bool direct = false;
  size_t off_part = 0, bytes = 0;
};
KdPlan plan_of(const PackedView &b, long long rows, int H, int G, int D, bool decode) {
  KdPlan p;
  const int sms = sm_count();
  p.nb = rows <= 8 ? 1 : rows <= 16 || decode ? 2 : KD_MAX_NB;
  const long long items = (long long)b.n_seqs * G * ((H / G + 8 * p.nb - 1) / (8 * p.nb));
  p.direct = decode && b.max_kv_len <= KD_DIRECT_KEYS && items <= sms &&
             (4 * items > sms || b.max_kv_len * D <= KD_DIRECT_FEW);
  p.ctas = p.direct ? (int)items : sms > 2 ? sms : 2;
  if (!p.direct) {
    p.off_part = ((size_t)p.ctas * 32 + 127) / 128 * 128;
    p.bytes = p.off_part + (size_t)p.ctas * 2 * 8 * p.nb * (D + 2) * 4;
  }
  return p;
}

template <int D, int NB>
cudaError_t launch(KdArgs a, const KdPlan &p, cudaStream_t st) {
  using L = KdLayout<D, NB>;
  static PerContextOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(kv4_rows_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::bytes(LLAMA_PACKED_MAX_SEQS));
  });
  if (e != cudaSuccess) return e;
  count_launch();
  const cudaError_t r =
      launch_pdl(kv4_rows_kernel<D, NB>, dim3((unsigned)p.ctas), dim3(L::WARPS * 32), L::bytes(a.b.n_seqs), st, a);
  if (r != cudaSuccess || p.direct) return r;
  count_launch();
  return launch_pdl(kv4_rows_join_kernel<D, NB>, dim3((unsigned)(p.ctas - 1)), dim3(64 * NB * KD_JOIN<D>), 0, st, a);
}

// Tiles of a KV head's items over all sequences, at most.
long long most_tiles(const PackedView &b, int H, int G) {
  return (long long)(kd_tiles<KD_MAX_NB>(b.max_kv_len) + kd_start(KD_MAX_NB)) * ((long long)b.n_tokens * (H / G) / 8 + b.n_seqs);
}

cudaError_t launch_rows(const bf16 *q, const uint8_t *k, const uint8_t *v, bf16 *o, const PagedView &pv,
                        const PackedView &b, int H, int G, int D, int few, void *workspace, const KdPlan &p,
                        int *status, cudaStream_t st) {
  KdArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.pv = pv;
  a.b = b;
  a.H = H;
  a.G = G;
  a.r = H / G;
  a.few = few;
  a.direct = p.direct;
  a.times = b.q_offsets != nullptr ? G : G * ((a.r + 8 * p.nb - 1) / (8 * p.nb));
  a.most = b.q_offsets != nullptr ? (int)most_tiles(b, H, G) : 0x7fffffff;
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)D);
  a.part = p.direct ? nullptr : reinterpret_cast<float *>((char *)workspace + p.off_part);
  a.spans = p.direct ? nullptr : reinterpret_cast<int4 *>(workspace);
  a.status = status;
#define KD_CASE(d)                                     \
  case d:                                              \
    return p.nb == 1 ? launch<d, 1>(a, p, st) : p.nb == 2 ? launch<d, 2>(a, p, st) : launch<d, KD_MAX_NB>(a, p, st);
  switch (D) {
    KD_CASE(16)
    KD_CASE(32)
    KD_CASE(64)
    KD_CASE(128)
  }
#undef KD_CASE
  return cudaErrorInvalidValue;
}

PackedView decode_view(const int *kv_lens, int n_seqs, int max_kv_len) {
  PackedView b;
  b.kv_lens = kv_lens;
  b.n_seqs = n_seqs;
  b.n_tokens = n_seqs;
  b.max_kv_len = max_kv_len;
  return b;
}

long long rows_of(const PackedView &b, int H, int G) {
  return ((long long)b.n_tokens * (H / G) + b.n_seqs - 1) / b.n_seqs;
}

}  // namespace

// The tiles of a KV head, and those of a CTA, are counted in ints.
bool kv4_decode_fits(int n_seqs, int max_kv_len, int H, int G) {
  const long long subs = (H / G + 15) / 16;
  const long long keys = (long long)n_seqs * max_kv_len;
  return keys <= 1LL << 35 && keys <= (1LL << 42) / (G * subs);
}

size_t kv4_decode_workspace_bytes(int n_seqs, int max_kv_len, int H, int G, int D) {
  return plan_of(decode_view(nullptr, n_seqs, max_kv_len), H / G, H, G, D, true).bytes;
}

cudaError_t launch_kv4_decode(const bf16 *q, const uint8_t *k, const uint8_t *v, bf16 *o, const PagedView &pv,
                              const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int D, void *workspace,
                              int *status, cudaStream_t st) {
  const PackedView b = decode_view(kv_lens, n_seqs, max_kv_len);
  return launch_rows(q, k, v, o, pv, b, H, G, D, INT_MAX, workspace, plan_of(b, H / G, H, G, D, true), status, st);
}

// Few rows, which tcgen05's 128-row tiles would mostly pad: those of one item on average, or
// of so many that the warps take KD_ROUNDS of their tiles each at the longest length (64
// sequences of 20 rows behind 2200 keys, 8 KV heads: 77 us for 104; 26 of 73 rows behind up to
// 3300 keys, one KV head: 20 for 31; at 15 rounds 17 for 24, but 30 for 25).  Over a few keys
// tcgen05 takes a single kernel, and is better while its items are fewer than its CTAs (5 rows
// behind 300 keys, 90 items 9.3 us for 10.3, 150 items 13.3 for 9.2; 64 sequences of 5 on 8 KV
// heads 33.5 for 23.6, 1000 of 2 behind 10 keys 202 for 37) or have more rows (100 sequences of
// 60 behind 300 keys, 3 KV heads 19 for 23).  (The counts of tiles are ints.)
bool kv4_rows_fit(const PackedView &b, int H, int G) {
  const long long most = most_tiles(b, H, G);
  if (most > 0x7fffffffLL || most * G > (1LL << 30) * sm_count()) return false;
  const bool few_keys = b.max_kv_len <= KD_FEW_KEYS;
  if (rows_of(b, H, G) <= 8 * KD_MAX_NB) return !few_keys || 3LL * b.n_seqs * G > 2LL * sm_count();
  const long long tiles = (long long)G * kd_tiles<KD_MAX_NB>(b.max_kv_len) *
                          ((long long)b.n_tokens * (H / G) / (8 * KD_MAX_NB) + b.n_seqs);
  return !few_keys && tiles <= (long long)KD_ROUNDS * sm_count() * 8;
}
// The average says nothing of a prompt among single tokens, whose keys would be unpacked again for
// every 24 of its rows.  Where one sequence may bring so many that a warp has KD_MIXED_ROUNDS of
// their tiles, at the longest length, sequences of more than KD_FEW_ROWS rows are left to tcgen05
// (64 sequences of 40 rows: 128 us here, 110 there).  8 KV heads of four, single tokens and a
// prompt, all here / shared out: 255 behind up to 300 keys and 1024 behind 6000 490 / 181 us, 500
// behind 100 and 2000 behind 100 318 / 94.  Where there is no such sequence the other's three
// kernels cost 5 to 7 us: 64 sequences of five rows behind 300 keys 24 / 29, behind 2000 66 / 73, 256
// behind up to 4096 236 / 243.  Below the limit batches stay here, mixed ones for longer than they
// had to (128 and 512 behind 3000, 62 rounds, 164 / 111; 64 and 300 behind 8000, 86 rounds, 176 / 104),
// the drafts of 64 users under a bound of 8192 keys (72 rounds) without those kernels.
int kv4_rows_few(const PackedView &b, int H, int G) {
  const long long rows = ((long long)b.n_tokens - b.n_seqs + 1) * (H / G);
  const int few = H / G < KD_FEW_ROWS ? KD_FEW_ROWS / (H / G) : 1;
  if (rows <= KD_FEW_ROWS) return INT_MAX;
  const long long tiles =
      (long long)G * kd_tiles<KD_MAX_NB>(b.max_kv_len) * ((rows + 8 * KD_MAX_NB - 1) / (8 * KD_MAX_NB));
  return tiles > (long long)KD_MIXED_ROUNDS * sm_count() * 8 ? few : INT_MAX;
}
size_t kv4_rows_workspace_bytes(const PackedView &b, int H, int G, int D) {
  return plan_of(b, rows_of(b, H, G), H, G, D, false).bytes;
}
cudaError_t launch_kv4_rows(const bf16 *q, const uint8_t *k, const uint8_t *v, bf16 *o, const PagedView &pv,
                            const PackedView &b, int H, int G, int D, int few, void *workspace, int *status,
                            cudaStream_t st) {
  return launch_rows(q, k, v, o, pv, b, H, G, D, few, workspace, plan_of(b, rows_of(b, H, G), H, G, D, false), status,
                     st);
}

}  // namespace llama
