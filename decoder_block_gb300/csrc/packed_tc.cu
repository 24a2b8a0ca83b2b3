// Causal grouped-query attention of a packed batch over cache pages, bf16, on
// tcgen05 tensor cores ("The Evolving Transformer 04 · LLaMA", §05 GQA; "Full Llama 3
// transformer block", How it works: keys j <= position).  d_head 64 or 128; 16 and 32
// run as 64, their tiles filled up with zeros by the copies.  For token t at position p and its KV head's keys and values
//   o = sum_{j<=p} 2^(x_j - m) v_j / sum_{j<=p} 2^(x_j - m),  x_j = q.k_j log2(e) / sqrt(D),
// in one pass over the keys with the running maximum m and sum in fp32.
//
// A work item is (sequence, KV head, block of 2 * Mq query positions, range of
// 128-key tiles).  Its 128-row query tile t holds the rb heads of the group (all r, or
// 128 of more) at Mq = 128 / rb positions, row i * rb + hh: one TMA box, so that every
// K/V tile in shared memory serves the whole group.  Keys and values arrive page by
// page: one box per page (at most 128 rows) and 64 columns, in the 128-byte swizzle
// the MMAs read, so a tile is the same whatever the page size (at S = 8192 pages of 16
// and of 256 differ by 5 %).  Rows behind the sequence's last key may hold
// anything: their scores are replaced, not added to, and the V rows are cleared in
// shared memory before the product reads them (0 * NaN is not 0).
//   warp 0      takes items, loads Q, then V and the next K tiles into two-stage rings;
//               each lane issues one page's box and holds the next tile's id.  Lanes
//               issue one after another (about 65 ns each), so the 32 boxes that pages
//               of 16 rows make of a stage are issued by four more warps (S = 8192:
//               379 us for 456); larger pages do better without them (364 us for 373)
//   warp 1      one thread issues S_t = Q_t K^T and O_t += P_t V (fp32 in tensor
//               memory, P from tensor memory)
//   warps 2-9   softmax of tile 0 / 1, one thread per row; the output
// Work is dealt out in one of two ways:
//   * direct: one item per CTA, found by the CTA itself from the offsets (few
//     items, short keys: no kernel but this one runs);
//   * planned: a one-CTA kernel lists the items longest first and zeroes a
//     counter that persistent CTAs take them from.  When the longest items would
//     outlast the rest (few query rows against many keys) it splits their keys
//     into pieces; a piece leaves fp32 (O, m, l) per row in the workspace, and a
//     third kernel joins them in piece order, so results do not depend on timing.
// Every wait is bounded (llama_op_set_wait_budget).  A CTA that gives up records
// LLAMA_ERR_DEVICE_TIMEOUT and leaves once its copies, MMAs and tensor memory stores in
// flight are done; the four loading warps each arm the bytes they are about to ask for.
#include <cudaTypedefs.h>
#include <float.h>

#include "paged_kernels.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int PT_THREADS = 320;
constexpr int PT_KEYS = 128;    // keys of a tile
constexpr int PT_STAGES = 2;
constexpr float PT_RESCALE = 8.0f;  // log2 units: the running maximum is raised when it grows by > 2^8
constexpr int PT_MIN_PIECE = 4;     // key tiles that a split item's pieces may have, at least (9 make 3 + 3 + 3)
constexpr int PT_SPLIT_COST = 4;    // what a split costs, in key tiles of time
constexpr int PT_PLAN_THREADS = 1024;
constexpr int PT_BUCKETS = 1024;    // item lengths the planner tells apart

template <int D>
struct PtLayout {
  static constexpr int ATOM = 128 * 128;  // 128 rows x 64 columns
  static constexpr int TILE = (D / 64) * ATOM;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + PT_STAGES * TILE;
  static constexpr int OFF_ITEM = OFF_V + PT_STAGES * TILE;  // PtItem
  static constexpr int OFF_BAR = OFF_ITEM + 64;
  // q_full, q_empty, fin, kv_full[2], kv_empty[2], s_full[3], p_full[3], o_done[2],
  // i_full, near_end (16-row pages)
  static constexpr int NBAR = 3 + 2 * PT_STAGES + 8 + 2;
  // S buffers of 128 columns in tensor memory, then O of both query tiles.  With D = 64
  // there is room for a third: a query tile's next S is ready when its softmax is done
  // with this one (S = 8192, 32 heads: 306 us for 324).  With D = 128 the next S goes where
  // this one's P was.
  static constexpr int S_BUFS = D == 64 ? 3 : 2;
  static constexpr int BYTES_MIN = 1024 + OFF_BAR + NBAR * 8 + 16;
  // one CTA per SM: two would need all of tensor memory each
  static constexpr int BYTES = BYTES_MIN > 116 * 1024 ? BYTES_MIN : 116 * 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t O_COL = S_BUFS * 128;
};

// A work item as the producer hands it to the other roles.
struct PtItem {
  int seq, q0;        // sequence (-1: no more items), first query position of the block
  int g, h0, nh;      // KV head, first query head and number of them
  int unit;           // KV head and block of query heads
  int first, count, kv_len;
  int j0, j1;         // key tiles
  int slot;           // a piece of a split item: where its partial goes (-1: not split)
};
static_assert(sizeof(PtItem) <= 64, "PtItem fits its slot");

// Planner's output, in the workspace.
struct PtPlan {
  int n_entries;  // items are entries x units
  int next;       // item counter, past the CTAs' first items
  int n_split, pad;
};
struct __align__(16) PtEntry {
  int seq, blk;
  int range;  // first key tile | last + 1 << 16
  int slot;
  int first, count, kv_len, pad;  // the sequence's rows and length
};
static_assert(LLAMA_PACKED_MAX_KV / PT_KEYS <= 65535, "key tiles fit 16 bits");
struct __align__(16) PtSplit {  // a split block: its pieces' partials are slots slot .. slot + n - 1
  int q0, slot, n;
  int first, count, kv_len, pad[2];  // the sequence's rows and length
};

struct PtArgs {
  bf16 *o;
  PagedView pv;
  PackedView b;
  int H, G, D, r;        // D: the heads' width (the kernel's or less); r: heads of a group
  int rb, subs;          // heads of a work item (at most 128), items of a group
  int Mq, box;           // query positions of a tile; rows of a page's TMA box
  float scale_log2;
  PtPlan *plan;          // null: direct
  PtEntry *entries;
  float *part;           // [slot][unit][2 tiles][4 warps][D + 2][32 rows]
  int *status;
  long long wait_cycles;  // a wait's budget
};

__device__ __forceinline__ uint32_t pt_pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}

// The MMA thread paces the kernel, so it forms its operands with few instructions: the
// upper word of every shared-memory descriptor here is the same (128-byte swizzle, 8-row
// groups 1024 bytes apart), and offsets are added to the lower one.
constexpr uint32_t PT_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
// ACC 1: add to D; 0: overwrite it; -1: as `acc` says.
template <int ACC>
__device__ __forceinline__ void pt_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(PT_DESC_HI), "r"(idesc), "n"(ACC)
      : "memory");
}
template <int ACC>
__device__ __forceinline__ void pt_mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  if constexpr (ACC < 0)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(PT_DESC_HI), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(PT_DESC_HI), "r"(idesc), "n"(ACC)
        : "memory");
}

// Key tiles that the rows [lo, hi) of a sequence's new tokens see.
__device__ __forceinline__ int tiles_of(int shift, int lo, int hi) {
  if (hi <= lo || shift + hi <= 0) return 0;
  return (shift + hi - 1) / PT_KEYS + 1;
}
// The key tiles [j0, end) that query tile t of an item works on.
__device__ __forceinline__ int item_end(const PtItem &it, int Mq, int t) {
  const int lo = it.q0 + t * Mq, hi = min(it.count, lo + Mq);
  return min(it.j1, tiles_of(it.kv_len - it.count, lo, hi));
}

// ------------------------------------------------------------------ plan ---
// A block's sequence and key tiles are looked up twice (to count, to place); a thread
// keeps those of its first blocks, so a batch of up to 4096 blocks is looked up once.
constexpr int PT_KEEP = 4;

__global__ void __launch_bounds__(PT_PLAN_THREADS) packed_plan_kernel(PagedView pv, PackedView b, int units, int Mq,
                                                                      int sms, int max_blocks, int max_entries,
                                                                      PtPlan *plan, PtEntry *entries, PtSplit *splits,
                                                                      int *status) {
  __shared__ int first_blk[LLAMA_PACKED_MAX_SEQS + 1];  // blocks before sequence i
  __shared__ SeqSpan seqs[PT_PLAN_THREADS];             // the first sequences
  __shared__ int hist[PT_BUCKETS];
  __shared__ int warp_sums[32];
  __shared__ unsigned long long work_sum;
  __shared__ int n_split, n_slots;
  const int tid = threadIdx.x;
  allow_dependents_launch();
  hist[tid] = 0;
  if (tid == 0) {
    work_sum = 0;
    n_split = n_slots = 0;
    first_blk[0] = 0;
  }
  grid_dependency_wait();
  // blocks of every sequence, as sums: 1024 sequences a round
  int base = 0;
  for (int i0 = 0; i0 < b.n_seqs; i0 += PT_PLAN_THREADS) {
    const int i = i0 + tid;
    int n = 0;
    if (i < b.n_seqs) {
      check_seq(b, pv, i, status);
      const SeqSpan s = seq_span(b, pv, i);
      n = (s.count + 2 * Mq - 1) / (2 * Mq);
      if (i0 == 0) seqs[tid] = s;
    }
    const int end = add_counts(base, cta_scan(n, warp_sums));
    if (i < b.n_seqs) first_blk[i + 1] = end;
    if (tid == PT_PLAN_THREADS - 1) warp_sums[0] = end;
    __syncthreads();
    base = warp_sums[0];
    __syncthreads();
  }
  // (more blocks than well-formed offsets can make: see add_counts)
  const int n_blk = min(base, max_blocks);
  auto span_of = [&](int i) { return i < PT_PLAN_THREADS ? seqs[i] : seq_span(b, pv, i); };
  // sequence (the last i with first_blk[i] <= u), block and key tiles of block u
  auto look_up = [&](int u, int &seq, int &blk) {
    int lo = 0, hi = b.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first_blk[mid] <= u) lo = mid;
      else hi = mid;
    }
    seq = lo;
    blk = u - first_blk[lo];
    const SeqSpan s = span_of(lo);
    return tiles_of(s.kv_len - s.count, blk * 2 * Mq, min(s.count, (blk + 1) * 2 * Mq));
  };
  int seq[PT_KEEP], blk[PT_KEEP], len[PT_KEEP];
  unsigned long long mine = 0;
#pragma unroll
  for (int k = 0; k < PT_KEEP; ++k) {
    const int u = k * PT_PLAN_THREADS + tid;
    len[k] = u < n_blk ? look_up(u, seq[k], blk[k]) : 0;
    mine += (unsigned)len[k];
  }
  for (int u = PT_KEEP * PT_PLAN_THREADS + tid; u < n_blk; u += PT_PLAN_THREADS) {
    int s, x;
    mine += (unsigned)look_up(u, s, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if ((tid & 31) == 0 && mine != 0) atomicAdd(&work_sum, mine);
  __syncthreads();
  // An SM's even share of the key tiles.  An item that is longer by more than a split
  // costs is what the others would wait for: it is cut into pieces of at most a share.  An
  // item of n > share tiles makes fewer than n / share + 1 < 2 n / share pieces and the n of
  // all blocks add up to share * sms / units at most, so pieces number less than 2 * sms /
  // units, which sizes the workspace (packed_sizes).
  const unsigned long long even = (work_sum * units + sms - 1) / sms;
  const int share = even > 65535 ? 65535 : even > PT_MIN_PIECE ? (int)even : PT_MIN_PIECE;  // no item is longer
  auto pieces_of = [&](int n) { return n > share + PT_SPLIT_COST ? (n + share - 1) / share : 1; };
  // longest piece first: counting sort
  auto bucket = [&](int n, int pieces) { return PT_BUCKETS - 1 - min((n + pieces - 1) / pieces, PT_BUCKETS - 1); };
#pragma unroll
  for (int k = 0; k < PT_KEEP; ++k)
    if (k * PT_PLAN_THREADS + tid < n_blk) {
      const int p = pieces_of(len[k]);
      atomicAdd(&hist[bucket(len[k], p)], p);
    }
  for (int u = PT_KEEP * PT_PLAN_THREADS + tid; u < n_blk; u += PT_PLAN_THREADS) {
    int s, x;
    const int n = look_up(u, s, x), p = pieces_of(n);
    atomicAdd(&hist[bucket(n, p)], p);
  }
  __syncthreads();
  const int v = hist[tid], end = cta_scan(v, warp_sums);
  hist[tid] = end - v;
  __syncthreads();
  auto place = [&](int s, int x, int n) {
    PtEntry e;
    e.seq = s;
    e.blk = x;
    const SeqSpan span = span_of(s);
    e.first = span.first;
    e.count = span.count;
    e.kv_len = span.kv_len;
    e.pad = 0;
    const int p = pieces_of(n), each = (n + p - 1) / p;
    int slot = -1;
    if (p > 1) {
      slot = atomicAdd(&n_slots, p);
      splits[atomicAdd(&n_split, 1)] = PtSplit{x * 2 * Mq, slot, p, span.first, span.count, span.kv_len, {0, 0}};
    }
    const int at = atomicAdd(&hist[bucket(n, p)], p);
    for (int i = 0; i < p; ++i) {
      e.range = min(n, i * each) | min(n, (i + 1) * each) << 16;
      e.slot = slot < 0 ? -1 : slot + i;
      if (at + i < max_entries) entries[at + i] = e;
    }
  };
#pragma unroll
  for (int k = 0; k < PT_KEEP; ++k)
    if (k * PT_PLAN_THREADS + tid < n_blk) place(seq[k], blk[k], len[k]);
  for (int u = PT_KEEP * PT_PLAN_THREADS + tid; u < n_blk; u += PT_PLAN_THREADS) {
    int s, x;
    const int n = look_up(u, s, x);
    place(s, x, n);
  }
  if (tid == PT_PLAN_THREADS - 1) {
    plan->n_entries = min(end, max_entries);
    plan->next = 0;
  }
  __syncthreads();
  if (tid == 0) plan->n_split = n_split;
}

// ----------------------------------------------------------------- loads ---
// One warp's part of filling stage jj % 2 with V of key tile j and K of tile j + 1 (when
// the item has it).  A tile comes in boxes of a page's rows (at most 128) and 64 columns;
// the WARPS warps' lanes share the stage's 16 boxes of V and 16 of K at most.
template <int D, int WARPS>
struct StageLoads {
  using L = PtLayout<D>;
  static constexpr int ATOMS = D / 64, MINE = 32 / WARPS;
  const PtArgs &a;
  const CUtensorMap *map;
  uint32_t dst;
  int box, at, ahead;  // this lane's box and 64-column atom; 1: of K, one tile ahead
  int page = -1;       // of this lane's box in the coming stage

  __device__ __forceinline__ StageLoads(const PtArgs &args, const CUtensorMap *tmK, const CUtensorMap *tmV,
                                        uint32_t smem, int warp)
      : a(args) {
    const int lane = threadIdx.x & 31, slot = warp * MINE + lane;
    ahead = slot >= 16 ? 1 : 0;
    map = ahead ? tmK : tmV;
    box = lane < MINE ? (slot & 15) / ATOMS : PT_KEYS;  // past the tile: no box
    at = (slot & 15) % ATOMS;
    dst = smem + (ahead ? L::OFF_K : L::OFF_V) + at * L::ATOM + box * a.box * 128;
  }
  __device__ __forceinline__ int boxes_of(const PtItem &it, int j) const {
    return j < it.j1 ? min(PT_KEYS / a.box, (it.kv_len - j * PT_KEYS + a.box - 1) / a.box) : 0;
  }
  __device__ __forceinline__ uint32_t bytes(const PtItem &it, int j) const {
    return boxes_of(it, j) * a.box * 128u * ATOMS;
  }
  // First row of a tile's boxes in their pages.
  __device__ __forceinline__ int row_of(int j) const {
    return (j * PT_KEYS) & ((1 << a.pv.page_log2) - 1) & ~(a.box - 1);
  }
  // Page of a box of tile j: its id, n_pages (a page of zeros) when the id is out of
  // range, -1 when the tile has no such box.
  __device__ __forceinline__ int page_of(const PtItem &it, int j, int b) const {
    if (b >= boxes_of(it, j)) return -1;
    const int id = a.pv.page(it.seq, (j * PT_KEYS + b * a.box) >> a.pv.page_log2);
    if (id < 0) report_status(a.status, LLAMA_ERR_RANGE);
    return id < 0 ? a.pv.n_pages : id;
  }
  __device__ __forceinline__ void begin(const PtItem &it) { page = page_of(it, it.j0 + ahead, box); }
  // The page for tile j's stage; looks the next stage's up.
  __device__ __forceinline__ int advance(const PtItem &it, int j) {
    const int now = page;
    page = page_of(it, j + 1 + ahead, box);
    return now;
  }
  // Parity of kv_empty to wait for before stage jj is filled.  Stage 1 is released once
  // more than it was filled: its first K overwrites no earlier stage's but the first
  // item's first tile.
  __device__ __forceinline__ uint32_t parity(int jj) const {
    return ((jj / PT_STAGES) & 1) ^ (jj % PT_STAGES == 0 ? 1 : 0);
  }
  // Every loading warp arrives at the stage's barrier, with the bytes of its own boxes.
  __device__ __forceinline__ void issue(const PtItem &it, int j, int jj, int pg, uint32_t bar) const {
    const unsigned boxes = __ballot_sync(0xffffffffu, pg >= 0);
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive_expect_tx(bar, __popc(boxes) * a.box * 128u);
    __syncwarp();
    if (pg >= 0)
      ptx::tma_load_4d(dst + ((jj + ahead) % PT_STAGES) * L::TILE, map, at * 64, row_of(j + ahead), it.g, pg, bar);
  }
};

// ------------------------------------------------------------- attention ---
// ISSUERS: warps from PT_THREADS on that load the stages (0: warp 0 does).
template <int D, int ISSUERS>
__global__ void __launch_bounds__(PT_THREADS + ISSUERS * 32, 1)
    packed_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PtArgs a) {
  using L = PtLayout<D>;
  constexpr int ATOMS = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::NBAR);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  PtItem *item_slot = reinterpret_cast<PtItem *>(smem + L::OFF_ITEM);

  __shared__ int s_loaded[4];

  const uint32_t s0 = ptx::smem_u32(smem);
  const uint32_t bar0 = ptx::smem_u32(bars);
  const uint32_t q_full = bar0, q_empty = bar0 + 8, fin = bar0 + 16;
  // Stage jj % 2 of the rings: V of tile jj and K of the item's next tile, which one
  // step of the MMA thread needs together (an item's first K comes with its Q).
  auto kv_full = [&](int s) { return bar0 + 8u * (3 + s); };
  auto kv_empty = [&](int s) { return bar0 + 8u * (3 + PT_STAGES + s); };
  auto s_full = [&](int buf) { return bar0 + 8u * (3 + 2 * PT_STAGES + buf); };
  auto p_full = [&](int buf) { return bar0 + 8u * (6 + 2 * PT_STAGES + buf); };
  auto o_done = [&](int t) { return bar0 + 8u * (9 + 2 * PT_STAGES + t); };

  // with issuers: an item has been handed over; their loads have come to its last tile
  const uint32_t i_full = bar0 + 8u * (11 + 2 * PT_STAGES), near_end = i_full + 8;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (ptx::mbar_wait_within(bar, parity, abort_flag, a.wait_cycles)) return true;
    report_status(a.status, LLAMA_ERR_DEVICE_TIMEOUT);
    return false;
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

  if (threadIdx.x == 0) {
    ptx::mbar_init(q_full, 1);
    // the MMAs reading Q are done; each softmax and issuing warp has read the item
    ptx::mbar_init(q_empty, 9 + ISSUERS);
    ptx::mbar_init(i_full, 1);
    ptx::mbar_init(near_end, 1);
    ptx::mbar_init(fin, 1);
    for (int s = 0; s < PT_STAGES; ++s) {
      ptx::mbar_init(kv_full(s), ISSUERS > 0 ? ISSUERS : 1);
      ptx::mbar_init(kv_empty(s), 1);
    }
    for (int i = 0; i < 3; ++i) {
      ptx::mbar_init(s_full(i), 1);
      ptx::mbar_init(p_full(i), 128);
    }
    ptx::mbar_init(o_done(0), 1);
    ptx::mbar_init(o_done(1), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  // Query rows behind rb * Mq are never loaded: zero them.
  if (warp >= 2 && warp < 10 && a.rb * a.Mq < 128) {
    const int first = a.rb * a.Mq;
    for (int t = 0; t < 2; ++t)
      for (int at = 0; at < ATOMS; ++at) {
        uint4 *p = reinterpret_cast<uint4 *>(smem + L::OFF_Q + t * L::TILE + at * L::ATOM + first * 128);
        for (int i = threadIdx.x - 64; i < (128 - first) * 8; i += PT_THREADS - 64) p[i] = make_uint4(0, 0, 0, 0);
      }
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), L::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  allow_dependents_launch();
  grid_dependency_wait();

  if (warp == 0) {
    // ---------------------------------------------------------- producer ---
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tmQ);
      ptx::tma_prefetch_desc(&tmK);
      ptx::tma_prefetch_desc(&tmV);
    }
    const int units = a.G * a.subs;
    const int n_items = a.plan != nullptr ? *reinterpret_cast<volatile int *>(&a.plan->n_entries) * units : 0;
    // The CTA's next item (all lanes); seq = -1 when there is none.
    auto fetch = [&](int k) {
      PtItem it;
      it.seq = -1;
      if (a.plan != nullptr) {
        int u = blockIdx.x;
        if (k > 0) {
          if (lane == 0) u = gridDim.x + atomicAdd(&a.plan->next, 1);
          u = __shfl_sync(0xffffffffu, u, 0);
          if (u >= n_items) return it;
        }
        const int4 *e = reinterpret_cast<const int4 *>(a.entries + u / units);
        const int4 x = ld_after_wait(e), y = ld_after_wait(e + 1);  // the first: there is room, if not an entry
        if (u >= n_items) return it;
        it.seq = x.x;
        it.unit = u % units;
        it.q0 = x.y * 2 * a.Mq;
        it.j0 = x.z & 0xffff;
        it.j1 = (unsigned)x.z >> 16;
        it.slot = x.w;
        it.first = y.x;
        it.count = y.y;
        it.kv_len = y.z;
      } else {
        if (k > 0) return it;
        const int want = blockIdx.x / units;
        int base = 0;
        for (int i0 = 0; i0 < a.b.n_seqs; i0 += 32) {
          const int i = i0 + lane;
          const int n = i < a.b.n_seqs ? (seq_span(a.b, a.pv, i).count + 2 * a.Mq - 1) / (2 * a.Mq) : 0;
          int end = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += x;
          }
          const int mine = want - base - (end - n);
          const unsigned m = __ballot_sync(0xffffffffu, mine >= 0 && mine < n);
          if (m != 0) {
            const int src = __ffs(m) - 1;
            it.seq = i0 + src;
            it.q0 = __shfl_sync(0xffffffffu, mine, src) * 2 * a.Mq;
            break;
          }
          base += __shfl_sync(0xffffffffu, end, 31);
          if (base > want) break;
        }
        if (it.seq < 0) return it;
        it.unit = blockIdx.x % units;
        it.slot = -1;
      }
      it.g = it.unit / a.subs;
      it.h0 = it.g * a.r + it.unit % a.subs * a.rb;
      it.nh = min(a.rb, (it.g + 1) * a.r - it.h0);
      if (a.plan == nullptr) {
        const SeqSpan s = seq_span(a.b, a.pv, it.seq);
        it.first = s.first;
        it.count = s.count;
        it.kv_len = s.kv_len;
        it.j0 = 0;
        it.j1 = tiles_of(s.kv_len - s.count, it.q0, min(s.count, it.q0 + 2 * a.Mq));
      }
      return it;
    };
    StageLoads<D, 1> loads(a, &tmK, &tmV, s0, 0);
    const int my_box = lane / ATOMS, my_at = lane % ATOMS;  // this lane's box of an item's first K
    int items = 0, tiles = 0;  // Q loads issued; key tiles of earlier items and of this one
    bool ended = false;        // the end was handed over: the last Q has landed
    bool ok = true;
    PtItem it = fetch(0);
    for (int k = 0; ok; ++k) {
      const int first_page = it.seq >= 0 ? loads.page_of(it, it.j0, my_box) : -1;
      if (ISSUERS == 0 && it.seq >= 0) loads.begin(it);
      if (k > 0 && !wait_warp(q_empty, (k - 1) & 1)) break;
      if (lane == 0) {
        *item_slot = it;  // published by the arrivals
        if (ISSUERS > 0) ptx::mbar_arrive(i_full);
      }
      __syncwarp();
      if (it.seq < 0) {
        if (lane == 0) ptx::mbar_arrive(q_full);
        ended = true;
        break;
      }
      const int n_t = it.q0 + a.Mq < it.count ? 2 : 1;  // query tiles that hold rows
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(q_full, n_t * ATOMS * a.rb * a.Mq * 128u + loads.bytes(it, it.j0));
        for (int t = 0; t < n_t; ++t)
          for (int at = 0; at < ATOMS; ++at)
            ptx::tma_load_3d(s0 + L::OFF_Q + t * L::TILE + at * L::ATOM, &tmQ, at * 64, it.h0,
                             it.first + it.q0 + t * a.Mq, q_full);
      }
      __syncwarp();
      if (first_page >= 0)
        ptx::tma_load_4d(s0 + L::OFF_K + (tiles % PT_STAGES) * L::TILE + my_at * L::ATOM + my_box * a.box * 128, &tmK,
                         my_at * 64, loads.row_of(it.j0), it.g, first_page, q_full);
      ++items;
      // The next item's look-ups are hidden behind the last tiles of this one; any earlier and
      // items are dealt out before it shows which CTAs run late (S = 2048: 58 us for 39).
      if (ISSUERS > 0) {
        if (!wait_warp(near_end, k & 1)) break;
        tiles += max(0, it.j1 - it.j0);
        it = fetch(k + 1);
        continue;
      }
      PtItem next;
      bool fetched = false;
      for (int j = it.j0; j < it.j1; ++j, ++tiles) {
        if (j + 1 == it.j1) {
          next = fetch(k + 1);
          fetched = true;
        }
        const int page = loads.advance(it, j);
        if (!wait_warp(kv_empty(tiles % PT_STAGES), loads.parity(tiles))) {
          ok = false;
          break;
        }
        loads.issue(it, j, tiles, page, kv_full(tiles % PT_STAGES));
      }
      if (!ok) break;
      if (!fetched) next = fetch(k + 1);
      it = next;
    }
    // every issued copy lands before the CTA exits
    __syncwarp();
    if (lane == 0) {
      if (items > 0 && !ended) ptx::mbar_drain(q_full, (items - 1) & 1, nullptr, 0);
      if (ISSUERS == 0)
        for (int j = max(0, tiles - PT_STAGES); j < tiles; ++j)
          ptx::mbar_drain(kv_full(j % PT_STAGES), (j / PT_STAGES) & 1, nullptr, 0);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA ---
    if (lane == 0) {
      constexpr uint32_t idesc_qk = ptx::idesc_bf16_f32(128, PT_KEYS, false);
      constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(128, D, true);
      const uint32_t q_lo = desc_lo(s0 + L::OFF_Q, 16), k_lo = desc_lo(s0 + L::OFF_K, 16);
      const uint32_t v_lo = desc_lo(s0 + L::OFF_V, L::ATOM);  // V: MN-major, 64-column blocks an atom apart
      auto issue_s = [&](int jj, int t, int buf) {
        const uint32_t kb = k_lo + (jj % PT_STAGES) * (L::TILE >> 4), qb = q_lo + t * (L::TILE >> 4);
        const uint32_t d = tmem + buf * 128;
        pt_mma_ss<0>(d, qb, kb, idesc_qk);
#pragma unroll
        for (int kk = 1; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * L::ATOM + (kk % 4) * 32) >> 4;
          pt_mma_ss<1>(d, qb + off, kb + off, idesc_qk);
        }
        ptx::mma_commit(s_full(buf));
      };
      auto issue_pv = [&](int jj, bool first, bool last, int t, int buf) {
        const uint32_t vb = v_lo + (jj % PT_STAGES) * (L::TILE >> 4);
        const uint32_t d = tmem + L::O_COL + t * D, p = tmem + buf * 128;
        pt_mma_ts<-1>(d, p, vb, idesc_pv, first ? 0u : 1u);
#pragma unroll
        for (int kk = 1; kk < PT_KEYS / 16; ++kk)  // 16 keys: two 8-row groups
          pt_mma_ts<1>(d, p + kk * 8, vb + kk * (16 * 128 >> 4), idesc_pv, 1u);
        if (last) ptx::mma_commit(o_done(t));
      };
      // S_0(j+1) goes out right after PV_0(j): the softmax of tile 0 for the next keys
      // overlaps that of tile 1, and the next item's first S products the output of this one.
      bool ok = true;
      int jg = 0, n0 = 0, n1 = 0;  // key tiles over all items: of the ring, of query tiles 0 and 1
      // With three buffers the S products take them in turn (key tile by key tile, query tile
      // 0 first), and so do the P products; with two, query tile t keeps buffer t.
      int s_buf = 0, p_buf = 0, p_phase = 0;
      auto next_s = [&](int jj, int t) {
        issue_s(jj, t, L::S_BUFS == 3 ? s_buf : t);
        s_buf = s_buf == 2 ? 0 : s_buf + 1;
      };
      auto next_pv = [&](int jj, bool first, bool last, int t) -> bool {
        const int buf = L::S_BUFS == 3 ? p_buf : t;
        if (!wait(p_full(buf), L::S_BUFS == 3 ? p_phase : (t == 0 ? n0 : n1) & 1)) return false;
        if (t == 0) ++n0;
        else ++n1;
        if (p_buf == 2) p_phase ^= 1;
        p_buf = p_buf == 2 ? 0 : p_buf + 1;
        ptx::tc_fence_after();
        issue_pv(jj, first, last, t, buf);
        return true;
      };
      int owed = 1;                // stage whose release is still to come (1: see StageLoads)
      static_assert(PT_STAGES == 2, "K of tile jj + 1 lies in the other stage");
      for (int k = 0; ok; ++k) {
        if (!wait(q_full, k & 1)) break;
        const PtItem it = *item_slot;
        if (it.seq < 0) break;
        const int e0 = item_end(it, a.Mq, 0), e1 = item_end(it, a.Mq, 1);
        const int n = it.j1 - it.j0;
        if (n <= 0) {  // no row of the block sees a key
          ptx::mbar_arrive(q_empty);
          continue;
        }
        ptx::tc_fence_after();
        if (it.j0 < e0) next_s(jg, 0);
        if (it.j0 < e1) next_s(jg, 1);
        if (owed >= 0) ptx::mma_commit(kv_empty(owed));
        owed = -1;
        if (n == 1) ptx::mma_commit(q_empty);
        // One key tile: t0, t1 say which query tiles work on it, s0, s1 on the next one.
        auto step = [&](int i, bool t0, bool t1, bool s0, bool s1) -> bool {
          const int jj = jg + i, st = jj % PT_STAGES;
          if (!wait(kv_full(st), (jj / PT_STAGES) & 1)) return false;
          if constexpr (L::S_BUFS == 3) {
            ptx::tc_fence_after();
            if (s0) next_s(jj + 1, 0);
            if (t0 && !next_pv(jj, i == 0, true, 0)) return false;
            if (s1) next_s(jj + 1, 1);
            if (t1 && !next_pv(jj, i == 0, true, 1)) return false;
          } else {
            if (t0 && !next_pv(jj, i == 0, !s0, 0)) return false;
            if (s0) {
              ptx::tc_fence_after();
              next_s(jj + 1, 0);
            }
            if (t1 && !next_pv(jj, i == 0, !s1, 1)) return false;
            if (s1) next_s(jj + 1, 1);
          }
          // The stage may be filled again when the next tile's K has been used too; behind an
          // item's last tile that is the next item's first.
          if (i + 1 < n) ptx::mma_commit(kv_empty(st));
          else owed = st;
          if (i + 2 == n) ptx::mma_commit(q_empty);
          return true;
        };
        // This thread paces the kernel, so the tiles that both query tiles see, and whose
        // successors they see too, go without the questions of the last ones.
        const int plain = min(min(e0, e1) - 1 - it.j0, n - 1);
        int i = 0;
        for (; ok && i < plain; ++i) ok = step(i, true, true, true, true);
        for (; ok && i < n; ++i) {
          const int j = it.j0 + i;
          ok = step(i, j < e0, j < e1, j + 1 < e0, j + 1 < e1);
        }
        jg += n;
      }
      ptx::mma_commit(fin);
      ptx::mbar_drain(fin, 0, nullptr, 0);
    }
  } else if (ISSUERS > 0 && warp >= 10) {
    // ------------------------------------------------------------ issuers ---
    StageLoads<D, ISSUERS == 0 ? 1 : ISSUERS> loads(a, &tmK, &tmV, s0, warp - 10);
    int tiles = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!wait_warp(i_full, k & 1)) break;
      const PtItem it = *item_slot;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_empty);
      if (it.seq < 0) break;
      if (it.j0 >= it.j1 && warp == 10 && lane == 0) ptx::mbar_arrive(near_end);
      loads.begin(it);
      for (int j = it.j0; j < it.j1; ++j, ++tiles) {
        const int page = loads.advance(it, j);
        if (!wait_warp(kv_empty(tiles % PT_STAGES), loads.parity(tiles))) {
          ok = false;
          break;
        }
        if (j + 1 == it.j1 && warp == 10 && lane == 0) ptx::mbar_arrive(near_end);
        loads.issue(it, j, tiles, page, kv_full(tiles % PT_STAGES));
      }
    }
    __syncwarp();
    ptx::settle_loads<ISSUERS == 0 ? 1 : ISSUERS, PT_STAGES>(tiles, warp - 10, s_loaded, kv_full);
  } else {
    // ----------------------------------------------------------- softmax ---
    const int t = (warp - 2) / 4;
    const int qq = warp & 3;
    const int row = qq * 32 + lane;
    const int hh = row % a.rb, i = row / a.rb;
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    const uint32_t o_col = lane_base + L::O_COL + t * D;
    const uint64_t scale2 = ptx::f2pack(a.scale_log2, a.scale_log2);
    if (a.plan == nullptr && blockIdx.x == 0)
      for (int u = threadIdx.x - 64; u < a.b.n_seqs; u += PT_THREADS - 64) check_seq(a.b, a.pv, u, a.status);
    bool ok = true;
    int jg = 0, jt = 0;  // key tiles of earlier items: of the ring, of this query tile
    int done = 0;        // o_done phases: of every tile (three S buffers), of every item (two)
    int mg = 0;          // S products of earlier items
    for (int k = 0; ok; ++k) {
      if (!wait_warp(q_full, k & 1)) break;
      const PtItem it = *item_slot;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_empty);
      if (it.seq < 0) break;
      const int shift = it.kv_len - it.count;
      const int e0 = item_end(it, a.Mq, 0), e1 = item_end(it, a.Mq, 1);
      const int my_end = t == 0 ? e0 : e1;
      const int n_kv = max(0, my_end - it.j0);
      const int rel = it.q0 + t * a.Mq + i;
      const bool valid = i < a.Mq && rel < it.count && hh < it.nh;
      const int pos = shift + min(rel, it.count - 1);
      // finite: rows that see no key of a tile keep weights of 0 instead of NaN
      float m_run = -FLT_MAX;
      uint64_t l2 = ptx::f2pack(0.f, 0.f);  // running row sum, two partial halves
      const int a0 = max(0, e0 - it.j0), a1 = max(0, e1 - it.j0);
      for (int jl = 0; jl < n_kv; ++jl) {
        const int j = it.j0 + jl;
        // this tile's place among all S products
        const int m = mg + min(jl, a0) + min(jl, a1) + (t == 1 && jl < a0 ? 1 : 0);
        const int buf = L::S_BUFS == 3 ? m % 3 : t;
        const uint32_t s_col = lane_base + buf * 128;
        if (!wait_warp(s_full(buf), (L::S_BUFS == 3 ? m / 3 : jt + jl) & 1)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const int key0 = j * PT_KEYS;
        // The last tile of a sequence: clear the V rows behind its last key.  The first
        // query tile that works on the tile does it, before its P is handed over.
        if (key0 + PT_KEYS > it.kv_len && t == (j < e0 ? 0 : 1)) {
          const int st = (jg + jl) % PT_STAGES;
          if (!wait_warp(kv_full(st), ((jg + jl) / PT_STAGES) & 1)) {
            ok = false;
            break;
          }
          if (key0 + row >= it.kv_len) {
            uint4 *vr = reinterpret_cast<uint4 *>(smem + L::OFF_V + st * L::TILE + row * 128);
#pragma unroll
            for (int at = 0; at < ATOMS; ++at)
#pragma unroll
              for (int c = 0; c < 8; ++c) vr[at * (L::ATOM / 16) + c] = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
        }
        // One pass over the tile, 32 columns at a time.  p = 2^(s*scale - m_run)
        // uses the running maximum as it stands; a chunk whose own maximum exceeds
        // it by more than 2^8 first raises it, scaling the row sum, the P chunks
        // already written for this tile and, once the tile is done, O.  P (bf16)
        // lands over S columns already read.  Those chunks' P are rounded a second time
        // by it; each is then below 2^-8 of the largest, 96 of them 0.27 of the row's sum at
        // most.  (Raised by whole powers of two, which change no bit of P, the largest
        // weight is no longer 1 and rounds too: 0.0019-0.0023 for 0.0011-0.0021 relative
        // to 64-bit results on 18 batches.)
        const bool masked = __any_sync(0xffffffffu, key0 + PT_KEYS - 1 > pos);
        float alpha_tile = 1.f;
        bool rescaled = false;  // warp-uniform
        // (rolled up beside the issuers: 379 us for 383 over 16-row pages, ragged 151 for 157;
        // without them 375 for 364)
#pragma unroll(ISSUERS > 0 ? 1 : 4)
        for (int c = 0; c < PT_KEYS; c += 32) {
          float sv[32];
          float cm;
          if (masked) {
            ptx::tmem_ld32(s_col + c, sv);
            cm = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (key0 + c + e > pos) sv[e] = -INFINITY;
              cm = fmaxf(cm, sv[e]);
            }
          } else {
            ptx::tmem_ld32_max(s_col + c, sv, cm);
          }
          const float cms = cm * a.scale_log2;
          const bool need = cms > m_run + PT_RESCALE;
          if (__any_sync(0xffffffffu, need)) {
            float alpha = 1.f;
            if (need) {
              alpha = ptx::ex2_approx(m_run - cms);
              m_run = cms;
            }
            l2 = ptx::fmul2(l2, ptx::f2pack(alpha, alpha));
            alpha_tile *= alpha;
            rescaled = true;
            if (c > 0) {
              ptx::tmem_st_wait();
#pragma unroll 1
              for (int pc = 0; pc < c / 2; pc += 16) {
                float pv[16];
                ptx::tmem_ld16(s_col + pc, pv);
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const uint32_t u = __float_as_uint(pv[e]);
                  w[e] = pt_pack2(__uint_as_float(u << 16) * alpha, __uint_as_float(u & 0xffff0000u) * alpha);
                }
                ptx::tmem_st16(s_col + pc, w);
              }
            }
          }
          const uint64_t negm2 = ptx::f2pack(-m_run, -m_run);
          uint32_t pk[16];
          uint64_t lc = ptx::f2pack(0.f, 0.f);  // a second, independent add chain
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            ptx::f2unpack(ptx::ffma2(ptx::f2pack(sv[e], sv[e + 1]), scale2, negm2), x0, x1);
            const float p0 = ptx::ex2_approx(x0), p1 = ptx::ex2_approx(x1);
            if ((e & 2) == 0)
              l2 = ptx::fadd2(l2, ptx::f2pack(p0, p1));
            else
              lc = ptx::fadd2(lc, ptx::f2pack(p0, p1));
            // bf16 P: the tensor cores' operand; the row sum keeps the unrounded values
            pk[e / 2] = pt_pack2(p0, p1);
          }
          l2 = ptx::fadd2(l2, lc);
          ptx::tmem_st16(s_col + c / 2, pk);
        }
        // The last product into O has to be done before O is scaled.  With two buffers it is: it
        // was issued before this tile's S, whose commit covers it.  With three it may still run;
        // its phase is waited for at every tile, so that none is passed over.
        if (L::S_BUFS == 3 && jl > 0) {
          if (!wait_warp(o_done(t), (done + jl - 1) & 1)) {
            ptx::tmem_st_wait();  // of this tile's P: nothing of this CTA may be in flight when it leaves
            ok = false;
            break;
          }
          ptx::tc_fence_after();
        }
        if (jl > 0 && rescaled) {  // O holds the earlier key tiles
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            float ov[16];
            ptx::tmem_ld16(o_col + c, ov);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(ov[e] * alpha_tile);
            ptx::tmem_st16(o_col + c, w);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(p_full(buf));
      }
      if (!ok) break;
      if (n_kv > 0) {
        done += L::S_BUFS == 3 ? n_kv : 1;
        if (!wait_warp(o_done(t), (done - 1) & 1)) break;
        ptx::tc_fence_after();
      }
      float la, lb;
      ptx::f2unpack(l2, la, lb);
      float l = la + lb;
      bf16 *dst = a.o + ((size_t)(it.first + rel) * a.H + it.h0 + hh) * a.D;
      if (it.slot < 0) {
        // a row that sees no key is zeros; one whose scores are all NaN or -inf is NaN (0 / 0)
        const float inv = pos < 0 ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float ov[16];
          if (n_kv > 0) {
            ptx::tmem_ld16(o_col + c, ov);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = 0.f;
          }
          if (valid && c < a.D) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pt_pack2(ov[2 * e] * inv, ov[2 * e + 1] * inv);
            *reinterpret_cast<uint4 *>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      } else if (__any_sync(0xffffffffu, valid)) {
        // a piece: the partial (O, m, l) of these 32 rows, one column after another
        float *mine = a.part + ((((size_t)it.slot * (a.G * a.subs) + it.unit) * 2 + t) * 4 + qq) * ((D + 2) * 32) + lane;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float ov[16];
          if (n_kv > 0) {
            ptx::tmem_ld16(o_col + c, ov);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) mine[(c + e) * 32] = ov[e];
        }
        mine[D * 32] = m_run;
        mine[(D + 1) * 32] = l;
      }
      // the next item's first PV product overwrites O only after this warp's next P
      ptx::tc_fence_before();
      jg += max(0, it.j1 - it.j0);
      jt += n_kv;
      mg += a0 + a1;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Joins the pieces of split items, o = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p in
// piece order.  A CTA takes 32 rows of one block and unit at a time, a warp JOIN_COLS
// columns of them; four pieces are on their way at a time.  Most calls split nothing, and
// this kernel ends them: JOIN_CTAS per SM that loop, instead of a CTA for everything that
// there could be (8 KV heads: 1280), take 4 us off such a call.
constexpr int JOIN_COLS = 8;
constexpr int JOIN_CTAS = 4;

template <int D>
__global__ void __launch_bounds__(D / JOIN_COLS * 32) packed_join_kernel(const __grid_constant__ PtArgs a,
                                                                         const PtSplit *splits) {
  grid_dependency_wait();
  const int units = a.G * a.subs;
  const int n_split = *reinterpret_cast<volatile int *>(&a.plan->n_split);
  const int lane = threadIdx.x & 31, c0 = threadIdx.x / 32 * JOIN_COLS;
  for (int w = blockIdx.x; w < n_split * units * 8; w += gridDim.x) {
    const int qq = w % 4, t = w / 4 % 2, unit = w / 8 % units;
    const PtSplit s = splits[w / 8 / units];
    const int row = qq * 32 + lane, hh = row % a.rb, i = row / a.rb;
    const int rel = s.q0 + t * a.Mq + i;
    const int g = unit / a.subs, h = g * a.r + unit % a.subs * a.rb + hh;
    const bool valid = i < a.Mq && rel < s.count && h < (g + 1) * a.r;
    if (!__any_sync(0xffffffffu, valid)) continue;  // nothing was written
    const float *p = a.part + ((((size_t)s.slot * units + unit) * 2 + t) * 4 + qq) * ((D + 2) * 32) + lane;
    const size_t step = (size_t)units * 8 * (D + 2) * 32;
    float m = -FLT_MAX;
#pragma unroll 8
    for (int x = 0; x < s.n; ++x) m = fmaxf(m, p[x * step + D * 32]);
    float l = 0.f, o[JOIN_COLS];
#pragma unroll
    for (int e = 0; e < JOIN_COLS; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int x = 0; x < s.n; ++x) {
      const float *px = p + x * step;
      const float f = ptx::ex2_approx(px[D * 32] - m);
      l = fmaf(f, px[(D + 1) * 32], l);
#pragma unroll
      for (int e = 0; e < JOIN_COLS; ++e) o[e] = fmaf(f, px[(c0 + e) * 32], o[e]);
    }
    if (!valid || c0 >= a.D) continue;
    const float inv = s.kv_len - s.count + rel < 0 ? 0.f : 1.f / l;
    uint32_t v[JOIN_COLS / 2];
#pragma unroll
    for (int e = 0; e < JOIN_COLS / 2; ++e) v[e] = pt_pack2(o[2 * e] * inv, o[2 * e + 1] * inv);
    *reinterpret_cast<uint4 *>(a.o + ((size_t)(s.first + rel) * a.H + h) * a.D + c0) =
        make_uint4(v[0], v[1], v[2], v[3]);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

}  // namespace

bool make_paged_map(CUtensorMap *map, const bf16 *pool, const PagedView &pv, int G, int D, int box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t ps = (cuuint64_t)1 << pv.page_log2;
  cuuint64_t dims[4] = {(cuuint64_t)D, ps, (cuuint64_t)G, (cuuint64_t)pv.n_pages};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, ps * D * 2, (cuuint64_t)pv.page_stride * 2};
  cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1}, es[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<bf16 *>(pool), dims, strides, bx, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_heads_map(CUtensorMap *map, const bf16 *q, int rows, int H, int D, int box_heads, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
  cuuint32_t bx[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16 *>(q), dims, strides, bx, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// Sizes of one call: items, and the workspace they need (0 bytes: direct).
struct PtSizes {
  int rb = 0, subs = 0, units = 0, Mq = 0;
  long long max_blocks = 0;  // (sequence, block) pairs, at most
  int max_split = 0, max_slots = 0;
  long long max_entries = 0;
  size_t off_entries = 0, off_splits = 0, off_part = 0, bytes = 0;
};

PtSizes packed_sizes(const PackedView &b, int H, int G, int D, int sms) {
  PtSizes z;
  const int r = H / G;
  z.rb = r < 128 ? r : 128;
  z.subs = (r + z.rb - 1) / z.rb;
  z.units = G * z.subs;
  z.Mq = 128 / z.rb;
  z.max_blocks = (long long)b.n_tokens / (2 * z.Mq) + (b.n_seqs < b.n_tokens ? b.n_seqs : b.n_tokens);
  // Direct: no more than one item per SM, and so few key tiles that the planned form, which
  // costs about 8 us more to start and join, cannot win them back by splitting items for
  // the idle SMs (planned / direct: 8B-shaped, 512 tokens behind 600 29 / 21 us, 1100
  // behind 900 39 / 33, but three tokens, the longest behind 1900, 20 / 28).
  const long long items = z.max_blocks * z.units, tiles = (b.max_kv_len + PT_KEYS - 1) / PT_KEYS;
  if (items <= sms && tiles <= 16 && tiles * (sms - items) <= 8LL * sms) return z;
  // Split items: none where no sequence is long enough (no share is below PT_MIN_PIECE) or
  // every SM has an item anyway; see the planner.
  z.max_slots = b.max_kv_len > (PT_MIN_PIECE + PT_SPLIT_COST) * PT_KEYS && z.units < sms ? 2 * sms / z.units : 0;
  z.max_split = z.max_slots / 2;
  z.max_entries = z.max_blocks + z.max_slots;
  z.off_entries = sizeof(PtPlan);
  z.off_splits = z.off_entries + (size_t)z.max_entries * sizeof(PtEntry);
  z.off_part = z.off_splits + (size_t)z.max_split * sizeof(PtSplit);
  z.off_part = (z.off_part + 127) / 128 * 128;
  z.bytes = z.off_part + (size_t)z.max_slots * z.units * 8 * (D + 2) * 32 * sizeof(float);
  return z;
}

template <int D>
cudaError_t launch_tc(const bf16 *q, const bf16 *k, const bf16 *v, bf16 *o, const PagedView &pv, const PackedView &b,
                      int H, int G, int width, void *workspace, int *status, cudaStream_t st) {
  using L = PtLayout<D>;
  static PerContextOnce attr;
  cudaError_t e = attr.run([] {
    const cudaError_t e =
        cudaFuncSetAttribute(packed_tc_kernel<D, 0>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(packed_tc_kernel<D, 4>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  });
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  const PtSizes z = packed_sizes(b, H, G, D, sms);
  PtArgs a;
  a.o = o;
  a.pv = pv;
  a.b = b;
  a.H = H;
  a.G = G;
  a.D = width;
  a.r = H / G;
  a.rb = z.rb;
  a.subs = z.subs;
  a.Mq = z.Mq;
  a.box = 1 << (pv.page_log2 < 7 ? pv.page_log2 : 7);
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)width);
  a.plan = nullptr;
  a.entries = nullptr;
  a.part = nullptr;
  a.status = status;
  a.wait_cycles = op_wait_cycles();
  CUtensorMap mq, mk, mv;
  if (!make_heads_map(&mq, q, b.n_tokens, H, width, a.rb, a.Mq) || !make_paged_map(&mk, k, pv, G, width, a.box) ||
      !make_paged_map(&mv, v, pv, G, width, a.box))
    return cudaErrorInvalidValue;
  auto kernel = a.box == 16 ? packed_tc_kernel<D, 4> : packed_tc_kernel<D, 0>;
  const dim3 threads(PT_THREADS + (a.box == 16 ? 128 : 0));
  if (z.bytes == 0) {
    count_launch();
    return launch_pdl(kernel, dim3((unsigned)(z.max_blocks * z.units)), threads, L::BYTES, st, mq,
                      mk, mv, a);
  }
  char *w = reinterpret_cast<char *>(workspace);
  a.plan = reinterpret_cast<PtPlan *>(w);
  a.entries = reinterpret_cast<PtEntry *>(w + z.off_entries);
  PtSplit *splits = reinterpret_cast<PtSplit *>(w + z.off_splits);
  a.part = reinterpret_cast<float *>(w + z.off_part);
  count_launch();
  e = launch_pdl(packed_plan_kernel, dim3(1), dim3(PT_PLAN_THREADS), 0, st, pv, b, z.units, a.Mq, sms,
                 (int)z.max_blocks, (int)z.max_entries, a.plan, a.entries, splits, status);
  if (e != cudaSuccess) return e;
  const long long items = z.max_entries * z.units;
  count_launch();
  e = launch_pdl(kernel, dim3((unsigned)(items < sms ? items : sms)), threads, L::BYTES, st, mq,
                 mk, mv, a);
  if (e != cudaSuccess || z.max_split == 0) return e;
  count_launch();
  const long long joins = (long long)z.max_split * z.units * 8, ctas = (long long)JOIN_CTAS * sms;
  return launch_pdl(packed_join_kernel<D>, dim3((unsigned)(joins < ctas ? joins : ctas)), dim3(D / JOIN_COLS * 32), 0,
                    st, a, (const PtSplit *)splits);
}

}  // namespace

size_t packed_tc_workspace_bytes(const PackedView &b, int H, int G, int D) {
  return packed_sizes(b, H, G, D < 64 ? 64 : D, sm_count()).bytes;
}

cudaError_t launch_packed_tc(const bf16 *q, const bf16 *k, const bf16 *v, bf16 *o, const PagedView &pv,
                             const PackedView &b, int H, int G, int D, void *workspace, int *status, cudaStream_t st) {
  if (D == 128) return launch_tc<128>(q, k, v, o, pv, b, H, G, D, workspace, status, st);
  return launch_tc<64>(q, k, v, o, pv, b, H, G, D, workspace, status, st);
}

}  // namespace llama
