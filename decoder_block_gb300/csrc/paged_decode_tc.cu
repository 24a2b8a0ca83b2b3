// One new token per sequence over cache pages, bf16, on tcgen05 tensor cores ("Full
// Llama 3 transformer block", How it works: cached keys 0 .. kv_len - 1; "The Evolving
// Transformer 04 · LLaMA", §05 GQA).  d_head 64 or 128; 16 and 32 run as 64, their
// tiles filled up with zeros by the copies.
//
// The cache is read once and that is what bounds the step; the tensor cores keep
// the CUDA cores free enough for the loads to set the pace.  Keys are the
// 128-row side of both products (the heads of a group, at most 16, the columns):
//   S^T[128 keys x 16] = K_tile Q^T,      O^T[D x 16] += V_tile^T P^T,
// with p = 2^(s log2(e)/sqrt(D) - m), one running maximum m and sum l per head in
// fp32 over one pass.  Pages arrive as TMA boxes of their own, so a tile in shared
// memory is the same whatever the page size; V rows behind the last key, which
// may hold anything, are cleared in shared memory (0 * NaN is not 0).  l is 0 for a
// sequence without keys alone, whose row is zeros; a query that holds NaN or an infinity
// makes it NaN (m stays -inf where every score is NaN or -inf).
//   warp 0     takes items and loads Q
//   warp 1     one thread issues the MMAs
//   warps 2-5  softmax, one thread per key; the output, one thread per column
//   warps 6-9  load K and V: each lane issues one box and holds the next tile's page id.
//              Lanes of a warp issue one after another, about 65 ns each, and pages of 16
//              rows make 32 boxes of a tile (64 sequences over such pages: 127 us from
//              one warp, 96 from four; pages of 64: 96 and 94)
// The keys of a sequence are split over CTAs and joined, o = sum 2^(m_c - M) o_c /
// sum 2^(m_c - M) l_c, in one of two ways:
//   * direct (few sequences, or short ones): a cluster of 1 to 8 CTAs shares a
//     sequence and KV head and joins through distributed shared memory.  One
//     launch, no workspace.
//   * planned: all sequences are cut into chunks of about one size, chosen from their true
//     lengths so that every SM gets several.  Up to 32 sequences: every CTA finds the chunks
//     for itself and takes each gridDim-th.  More: a one-CTA kernel lists them and zeroes a
//     counter that persistent CTAs take them from.  fp32 partials go to the workspace and a
//     last kernel joins them in chunk order.
// Every wait is bounded (llama_op_set_wait_budget).  A CTA that gives up records
// LLAMA_ERR_DEVICE_TIMEOUT and leaves once its copies and MMAs in flight are done: each
// loading warp arms the bytes that it is about to ask for itself, and at the end the
// warps arrive at the stages that only some of them came to (see settle_loads).
#include <float.h>

#include "paged_kernels.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int PD_KEYS = 128;    // keys of a tile
constexpr int PD_N = 16;        // head columns of a tile
constexpr int PD_LOADERS = 4;   // warps that load K and V
constexpr int PD_THREADS = 192 + PD_LOADERS * 32;
constexpr float PD_RESCALE = 8.0f;
constexpr int PD_MAX_CLUSTER = 8;
// Key tiles of a CTA in the direct form, at most, when clusters share items and when CTAs
// take whole ones.  The planned form costs about 6 us more to start and join, and then
// spreads ragged lengths evenly (direct for planned: 4 sequences of 7500 keys on 8 KV heads
// 25 us for 30, of up to 7500 19 for 20; 32 of 2000 keys, 16 tiles, 46 for 50, of up to
// 2000 39 for 34).
constexpr int PD_CLUSTER_TILES = 15, PD_WHOLE_TILES = 12;
constexpr int PD_ROUNDS = 12;       // chunks per SM that the planner aims at
// Key tiles that a split sequence's chunks may have, at least (6 make 3 + 3): a chunk costs
// about as much as a tile besides (4 sequences of 6000 keys on 8 KV heads, planned: 1: 31 us, 4: 23, 5: 21, 6: 22).
constexpr int PD_MIN_CHUNK = 5;
// Sequences that every CTA cuts into chunks for itself, at most (one per lane): no kernel in
// front, but chunks are dealt out in turn instead of taken (one sequence of 20000 keys on 8
// KV heads 17.8 us for 19.5; with 64 sequences of up to 4096 the turns cost as much as the
// kernel).
constexpr int PD_SHARED_SEQS = 32;
constexpr int PD_PLAN_THREADS = 1024;

template <int D>
struct PdLayout {
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr int ATOMS = D / 64;
  static constexpr int ATOM = PD_KEYS * 128;  // 128 rows x 64 columns
  static constexpr int TILE = ATOMS * ATOM;
  static constexpr int Q_BYTES = ATOMS * PD_N * 128;
  static constexpr int P_BYTES = 2 * PD_N * 128;  // 16 rows x 128 keys
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + STAGES * TILE;
  // With D = 64 the V^T operand is given 128 rows: rows 64-127 read the 16 KB
  // behind a stage's V (the next stage, or what follows the last one), and their
  // results are never looked at.
  static constexpr int OFF_Q = OFF_V + STAGES * TILE;
  static constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_RED = OFF_P + 2 * P_BYTES;           // [4][4 warps][PD_N] floats
  static constexpr int OFF_ITEM = OFF_RED + 4 * 4 * PD_N * 4;   // 2 items
  static constexpr int OFF_BAR = OFF_ITEM + 2 * 32;
  static constexpr int NBAR = 2 * STAGES + 18 + 3;
  static constexpr int END = OFF_BAR + NBAR * 8 + 16;
  static constexpr int BYTES = 1024 + (END > OFF_Q + ATOM ? END : OFF_Q + ATOM);
  static constexpr uint32_t TMEM_COLS = 64;  // S^T x2, O^T x2, 16 columns each
};

// A work item: key tiles [j0, j1) of one sequence for one block of heads.
struct PdItem {
  int seq;  // -1: no more items
  int g, h0, nh;
  int j0, j1, len;
  int slot;  // partial slot (planned); -1: this item is the whole sequence
};
static_assert(sizeof(PdItem) == 32, "PdItem fills its slot");

struct PdPlan {
  int n_entries, next, n_split, pad;
};
struct __align__(16) PdEntry {
  int seq, j0, j1, slot;
  int len, pad[3];
};
struct PdSplit {
  int seq, slot, n, pad;
};

struct PdArgs {
  bf16 *o;
  PagedView pv;
  const int *kv_lens;
  int n_seqs, max_kv_len;
  int H, G, D, r, subs, box;  // D: the heads' width (the kernel's or less); subs: blocks of up to 16 heads per KV head
  float scale_log2;
  int cluster;     // direct: CTAs of a sequence and head block
  int shared_sms;  // at most 32 sequences, cut by every CTA for itself: SMs that share them (0: not so)
  PdPlan *plan;    // null: direct, or shared_sms
  PdEntry *entries;
  float *part;     // [slot][H][D + 2]
  int *status;
  long long wait_cycles;  // a wait's budget
};

// ------------------------------------------------------------------ plan ---
// Key tiles of a chunk, at most: PD_ROUNDS chunks per SM, so that the last ones to finish
// are short.  A sequence's chunks differ by no more than its last one is shorter.  Chunks
// of split sequences then number less than 2 * PD_ROUNDS * sms / units, which sizes the
// workspace.
__device__ __forceinline__ int chunk_of(unsigned long long tiles, int units, int sms) {
  const unsigned long long share = (tiles * units + (unsigned)(PD_ROUNDS * sms) - 1) / (unsigned)(PD_ROUNDS * sms);
  return share > 65535 ? 65535 : share > PD_MIN_CHUNK ? (int)share : PD_MIN_CHUNK;  // no sequence is longer
}

// The chunks of up to 32 sequences, found by a warp for itself: lane i has sequence i's
// length, key tiles, chunks and the number of its first one.
struct WarpPlan {
  int len = 0, tiles = 0, n = 0, first = 0, total = 0;
  __device__ __forceinline__ void find(const PagedView &pv, const int *kv_lens, int n_seqs, int max_kv_len, int units,
                                      int sms, int *status) {
    const int lane = threadIdx.x & 31;
    const int raw = lane < n_seqs ? ld_after_wait(kv_lens + lane) : 0;
    len = checked_len(raw, max_kv_len, pv);
    if (len != raw) report_status(status, LLAMA_ERR_RANGE);
    tiles = (len + PD_KEYS - 1) / PD_KEYS;
    const int chunk = chunk_of(__reduce_add_sync(0xffffffffu, (unsigned)tiles), units, sms);
    n = lane < n_seqs ? max(1, (tiles + chunk - 1) / chunk) : 0;
    int end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    first = end - n;
    total = __shfl_sync(0xffffffffu, end, 31);
  }
};

__global__ void __launch_bounds__(PD_PLAN_THREADS) decode_plan_kernel(PagedView pv, const int *kv_lens, int n_seqs,
                                                                      int max_kv_len, int units, int sms,
                                                                      int max_entries, PdPlan *plan, PdEntry *entries,
                                                                      PdSplit *splits, int *status) {
  __shared__ int first[LLAMA_PACKED_MAX_SEQS + 1];  // chunks before sequence i
  __shared__ int s_slot[LLAMA_PACKED_MAX_SEQS];     // first slot (-1: one chunk)
  __shared__ unsigned short s_tiles[LLAMA_PACKED_MAX_SEQS];
  static_assert(LLAMA_PACKED_MAX_KV / PD_KEYS <= 65535, "key tiles fit 16 bits");
  __shared__ int warp_sums[32];
  __shared__ unsigned long long total;
  __shared__ int n_split, n_slots;
  constexpr int PER = LLAMA_PACKED_MAX_SEQS / PD_PLAN_THREADS;
  const int tid = threadIdx.x;
  allow_dependents_launch();
  if (tid == 0) {
    total = 0;
    n_split = n_slots = 0;
    first[0] = 0;
  }
  __syncthreads();
  grid_dependency_wait();
  int tiles[PER];
  unsigned long long mine = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int i = k * PD_PLAN_THREADS + tid;
    tiles[k] = 0;
    if (i < n_seqs) {
      const int raw = ld_after_wait(kv_lens + i), len = checked_len(raw, max_kv_len, pv);
      if (len != raw) report_status(status, LLAMA_ERR_RANGE);
      tiles[k] = (len + PD_KEYS - 1) / PD_KEYS;
      mine += (unsigned)tiles[k];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if ((tid & 31) == 0 && mine != 0) atomicAdd(&total, mine);
  __syncthreads();
  // (a CTA that streams faster takes more of the chunks)
  const int chunk = chunk_of(total, units, sms);
  int base = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (k * PD_PLAN_THREADS >= n_seqs) break;
    const int i = k * PD_PLAN_THREADS + tid;
    const int n = i < n_seqs ? max(1, (tiles[k] + chunk - 1) / chunk) : 0;
    const int end = base + cta_scan(n, warp_sums);
    if (i < n_seqs) {
      first[i + 1] = end;
      int slot = -1;
      if (n > 1) {
        slot = atomicAdd(&n_slots, n);
        splits[atomicAdd(&n_split, 1)] = PdSplit{i, slot, n, 0};
      }
      s_slot[i] = slot;
      s_tiles[i] = (unsigned short)tiles[k];
    }
    if (tid == PD_PLAN_THREADS - 1) warp_sums[0] = end;
    __syncthreads();
    base = warp_sums[0];
    __syncthreads();
  }
  const int n_entries = min(base, max_entries);
  for (int e = tid; e < n_entries; e += PD_PLAN_THREADS) {
    int lo = 0, hi = n_seqs;  // the last sequence with first[i] <= e
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= e) lo = mid;
      else hi = mid;
    }
    const int n = first[lo + 1] - first[lo], each = (s_tiles[lo] + n - 1) / n;
    const int c = e - first[lo], j0 = c * each, slot = s_slot[lo];
    const int len = checked_len(ld_after_wait(kv_lens + lo), max_kv_len, pv);
    entries[e] = PdEntry{lo, j0, min((int)s_tiles[lo], j0 + each), slot < 0 ? -1 : slot + c, len, {0, 0, 0}};
  }
  if (tid == 0) {
    plan->n_entries = n_entries;
    plan->next = 0;
    plan->n_split = n_split;
  }
}

// ----------------------------------------------------------------- loads ---
// One warp's part of filling a stage with K and V of a key tile, in boxes of a page's
// rows (at most 128) and 64 columns; the loading warps' lanes share the 16 boxes of K and
// 16 of V at most.
template <int D>
struct TileLoads {
  using L = PdLayout<D>;
  static constexpr int ATOMS = L::ATOMS, MINE = 32 / PD_LOADERS;
  const PdArgs &a;
  const CUtensorMap *map;
  uint32_t dst;
  uint64_t once = ptx::policy_evict_first();  // each cached key is read once per call
  int box, at;    // this lane's box and 64-column atom
  int page = -1;  // of this lane's box in the coming tile

  __device__ __forceinline__ TileLoads(const PdArgs &args, const CUtensorMap *tmK, const CUtensorMap *tmV,
                                       uint32_t smem, int warp)
      : a(args) {
    const int lane = threadIdx.x & 31, slot = warp * MINE + lane;
    map = slot < 16 ? tmK : tmV;
    box = lane < MINE ? (slot & 15) / ATOMS : PD_KEYS;  // past the tile: no box
    at = (slot & 15) % ATOMS;
    dst = smem + (slot < 16 ? L::OFF_K : L::OFF_V) + at * L::ATOM + box * a.box * 128;
  }
  __device__ __forceinline__ int boxes_of(const PdItem &it, int j) const {
    return j < it.j1 ? min(PD_KEYS / a.box, (it.len - j * PD_KEYS + a.box - 1) / a.box) : 0;
  }
  // Page of this lane's box of key tile j: its id, n_pages (a page of zeros) when the id is
  // out of range, -1 when the tile has no such box.
  __device__ __forceinline__ void look_up(const PdItem &it, int j) {
    page = -1;
    if (box >= boxes_of(it, j)) return;
    page = a.pv.page(it.seq, (j * PD_KEYS + box * a.box) >> a.pv.page_log2);
    if (page < 0) {
      report_status(a.status, LLAMA_ERR_RANGE);
      page = a.pv.n_pages;
    }
  }
  // The page for tile j; looks the next tile's up.
  __device__ __forceinline__ int advance(const PdItem &it, int j) {
    const int now = page;
    look_up(it, j + 1);
    return now;
  }
  // Every loading warp arrives at the stage's barrier, with the bytes of its own boxes.
  __device__ __forceinline__ void issue(const PdItem &it, int j, int stage, int pg, uint32_t bar) const {
    const unsigned boxes = __ballot_sync(0xffffffffu, pg >= 0);
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive_expect_tx(bar, __popc(boxes) * a.box * 128u);
    __syncwarp();
    const int row = (j * PD_KEYS) & ((1 << a.pv.page_log2) - 1) & ~(a.box - 1);
    if (pg >= 0) ptx::tma_load_4d_hint(dst + stage * L::TILE, map, at * 64, row, it.g, pg, bar, once);
  }
};

// ------------------------------------------------------------- attention ---
// RN: head columns the softmax works on, the smallest of 2, 4, 8, 16 that holds
// the block's heads; P^T rows RN .. 15 stay zero.
template <int D, int RN>
__global__ void __launch_bounds__(PD_THREADS, 1)
    paged_decode_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PdArgs a) {
  using L = PdLayout<D>;
  constexpr int STAGES = L::STAGES, ATOMS = L::ATOMS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::NBAR);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *red = reinterpret_cast<float *>(smem + L::OFF_RED);
  PdItem *item_slot = reinterpret_cast<PdItem *>(smem + L::OFF_ITEM);

  __shared__ int s_loaded[PD_LOADERS];

  const uint32_t s0 = ptx::smem_u32(smem);
  const uint32_t b0 = ptx::smem_u32(bars);
  auto kv_full = [&](int s) { return b0 + 8u * s; };
  auto kv_empty = [&](int s) { return b0 + 8u * (STAGES + s); };
  auto q_full = [&](int i) { return b0 + 8u * (2 * STAGES + i); };
  auto q_empty = [&](int i) { return b0 + 8u * (2 * STAGES + 2 + i); };
  auto s_full = [&](int i) { return b0 + 8u * (2 * STAGES + 4 + i); };
  auto p_full = [&](int i) { return b0 + 8u * (2 * STAGES + 6 + i); };
  auto p_free = [&](int i) { return b0 + 8u * (2 * STAGES + 8 + i); };
  auto o_full = [&](int i) { return b0 + 8u * (2 * STAGES + 10 + i); };
  auto o_free = [&](int i) { return b0 + 8u * (2 * STAGES + 12 + i); };
  const uint32_t fin = b0 + 8u * (2 * STAGES + 14);
  auto red_full = [&](int i) { return b0 + 8u * (2 * STAGES + 15 + i); };
  const uint32_t lred_full = b0 + 8u * (2 * STAGES + 17);
  // an item has been handed over; the loads have come to its last tile
  auto i_full = [&](int i) { return b0 + 8u * (2 * STAGES + 18 + i); };
  const uint32_t near_end = b0 + 8u * (2 * STAGES + 20);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (ptx::mbar_wait_within(bar, parity, abort_flag, a.wait_cycles)) return true;
    report_status(a.status, LLAMA_ERR_DEVICE_TIMEOUT);
    return false;
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(kv_full(s), PD_LOADERS);
      ptx::mbar_init(kv_empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(q_full(i), 1);
      // the MMAs reading Q are done; each softmax and loading warp has read the item
      ptx::mbar_init(q_empty(i), 5 + PD_LOADERS);
      ptx::mbar_init(i_full(i), 1);
      ptx::mbar_init(s_full(i), 1);
      ptx::mbar_init(p_full(i), 128);
      ptx::mbar_init(p_free(i), 1);
      ptx::mbar_init(o_full(i), 1);
      ptx::mbar_init(o_free(i), 128);
      ptx::mbar_init(red_full(i), 4);
    }
    ptx::mbar_init(fin, 1);
    ptx::mbar_init(lred_full, 4);
    ptx::mbar_init(near_end, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (RN < PD_N && warp >= 2 && warp < 6) {  // P^T rows the softmax never writes
    uint4 *pz = reinterpret_cast<uint4 *>(smem + L::OFF_P);
    for (int i = threadIdx.x - 64; i < 2 * L::P_BYTES / 16; i += 128) pz[i] = make_uint4(0, 0, 0, 0);
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
  const int rank = a.cluster > 1 ? (int)(blockIdx.x % a.cluster) : 0;
  const int units = a.G * a.subs;

  if (warp == 0) {
    // ---------------------------------------------------------- producer ---
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tmQ);
      ptx::tma_prefetch_desc(&tmK);
      ptx::tma_prefetch_desc(&tmV);
    }
    const int n_items = a.plan != nullptr ? *reinterpret_cast<volatile int *>(&a.plan->n_entries) * units
                                          : a.n_seqs * units;
    const bool shared = a.shared_sms > 0;
    WarpPlan mine;
    if (shared)
      mine.find(a.pv, a.kv_lens, a.n_seqs, a.max_kv_len, units, a.shared_sms, blockIdx.x == 0 ? a.status : nullptr);
    auto fetch = [&](int k) {  // the CTA's k-th item (all lanes)
      PdItem it;
      it.seq = -1;
      int u = blockIdx.x;
      if (shared) {
        u += k * gridDim.x;
        if (u >= mine.total * units) return it;
        const int e = u / units, unit = u % units;
        const int src = 31 - __clz(__ballot_sync(0xffffffffu, mine.n > 0 && mine.first <= e));
        const int n = __shfl_sync(0xffffffffu, mine.n, src), c = e - __shfl_sync(0xffffffffu, mine.first, src);
        const int tiles = __shfl_sync(0xffffffffu, mine.tiles, src);
        it.seq = src;
        it.g = unit / a.subs;
        it.h0 = it.g * a.r + (unit % a.subs) * PD_N;
        it.nh = min(PD_N, (it.g + 1) * a.r - it.h0);
        const int each = (tiles + n - 1) / n;
        it.j0 = c * each;
        it.j1 = min(tiles, it.j0 + each);
        it.len = __shfl_sync(0xffffffffu, mine.len, src);
        it.slot = n > 1 ? e : -1;
        return it;
      }
      if (a.plan == nullptr) {
        u = blockIdx.x / a.cluster + k * (gridDim.x / a.cluster);
      } else if (k > 0) {
        if (lane == 0) u = gridDim.x + atomicAdd(&a.plan->next, 1);
        u = __shfl_sync(0xffffffffu, u, 0);
      }
      int4 x = make_int4(0, 0, 0, -1);
      int len = 0;
      if (a.plan != nullptr && (k == 0 || u < n_items)) {  // the first: there is room, if not an entry
        const PdEntry *e = a.entries + u / units;
        x = ld_after_wait(reinterpret_cast<const int4 *>(e));
        len = ld_after_wait(&e->len);
      }
      if (u >= n_items) return it;
      const int unit = u % units;
      it.g = unit / a.subs;
      it.h0 = it.g * a.r + (unit % a.subs) * PD_N;
      it.nh = min(PD_N, (it.g + 1) * a.r - it.h0);
      it.slot = x.w;
      if (a.plan != nullptr) {
        it.seq = x.x;
        it.j0 = x.y;
        it.j1 = x.z;
        it.len = len;
        return it;
      }
      it.seq = u / units;
      const int raw = ld_after_wait(a.kv_lens + it.seq);
      it.len = checked_len(raw, a.max_kv_len, a.pv);
      if (it.len != raw && lane == 0) report_status(a.status, LLAMA_ERR_RANGE);
      const int nt = (it.len + PD_KEYS - 1) / PD_KEYS, each = (nt + a.cluster - 1) / a.cluster;
      it.j0 = min(nt, rank * each);
      it.j1 = min(nt, it.j0 + each);
      return it;
    };
    int items = 0;
    bool ended = false;
    PdItem it = fetch(0);
    for (int nq = 0;; ++nq) {
      const int qi = nq & 1;
      if (!wait_warp(q_empty(qi), ((nq >> 1) & 1) ^ 1)) break;
      if (lane == 0) {
        item_slot[qi] = it;  // published by the arrivals
        ptx::mbar_arrive(i_full(qi));
        if (it.seq < 0) {
          ptx::mbar_arrive(q_full(qi));
        } else {
          ptx::mbar_arrive_expect_tx(q_full(qi), L::Q_BYTES);
          for (int at = 0; at < ATOMS; ++at)
            ptx::tma_load_3d(s0 + L::OFF_Q + qi * L::Q_BYTES + at * (PD_N * 128), &tmQ, at * 64, it.h0, it.seq,
                             q_full(qi));
        }
      }
      __syncwarp();
      ended = it.seq < 0;
      if (ended) break;
      ++items;
      // the next item's look-ups hide behind the last tile of this one
      if (!wait_warp(near_end, nq & 1)) break;
      it = fetch(nq + 1);
    }
    // Every issued copy lands before the CTA exits.  The last Q load's phase is the newest
    // of its barrier unless the end was handed over there; the MMA thread waited for the
    // one before it.
    if (lane == 0)
      for (int q = max(0, items - 2); q < items; ++q)
        if (!(ended && (items & 1) == (q & 1))) ptx::mbar_drain(q_full(q & 1), (q >> 1) & 1, nullptr, 0);
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA ---
    if (lane == 0) {
      constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(PD_KEYS, PD_N, false);
      // O^T = V^T P^T: A = V^T (MN-major), B = P^T (K-major)
      constexpr uint32_t idesc_o = ptx::idesc_bf16_f32(128, PD_N, false) | (1u << 15);
      int tile = 0;
      bool ok = true;
      for (int nq = 0; ok; ++nq) {
        const int qi = nq & 1, ob = nq & 1;
        if (!wait(q_full(qi), (nq >> 1) & 1)) break;
        const PdItem it = item_slot[qi];
        if (it.seq < 0) break;
        const int nt = it.j1 - it.j0;
        if (!wait(o_free(ob), ((nq >> 1) & 1) ^ 1)) break;
        const uint32_t qbase = s0 + L::OFF_Q + qi * L::Q_BYTES;
        auto issue_s = [&](int t) -> bool {
          const int st = t % STAGES;
          if (!wait(kv_full(st), (t / STAGES) & 1)) return false;
          ptx::tc_fence_after();
          const uint32_t kb = s0 + L::OFF_K + st * L::TILE;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ka = (kk / 4) * L::ATOM + (kk % 4) * 32;
            const uint32_t qa = (kk / 4) * (PD_N * 128) + (kk % 4) * 32;
            ptx::mma_bf16_ss(tmem + (t & 1) * PD_N, ptx::smem_desc_sw128(kb + ka), ptx::smem_desc_sw128(qbase + qa),
                             idesc_s, kk > 0 ? 1u : 0u);
          }
          ptx::mma_commit(s_full(t & 1));
          return true;
        };
        if (nt > 0) ok = issue_s(tile);
        for (int j = 0; j < nt && ok; ++j, ++tile) {
          // one tile ahead: the softmax of this tile overlaps the next S^T
          if (j + 1 < nt && !issue_s(tile + 1)) {
            ok = false;
            break;
          }
          const int st = tile % STAGES, sb = tile & 1;
          if (!wait(p_full(sb), (tile >> 1) & 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t vb = s0 + L::OFF_V + st * L::TILE;
          const uint32_t pb = s0 + L::OFF_P + sb * L::P_BYTES;
#pragma unroll
          for (int kk = 0; kk < PD_KEYS / 16; ++kk) {
            const uint64_t adesc = ptx::smem_desc_sw128_mn(vb + kk * 16 * 128, L::ATOM, 1024);
            const uint32_t pa = (kk / 4) * (PD_N * 128) + (kk % 4) * 32;
            ptx::mma_bf16_ss(tmem + 32 + ob * PD_N, adesc, ptx::smem_desc_sw128(pb + pa), idesc_o,
                             (j > 0 || kk > 0) ? 1u : 0u);
          }
          ptx::mma_commit(p_free(sb));
          ptx::mma_commit(kv_empty(st));
        }
        if (!ok) break;
        ptx::mma_commit(q_empty(qi));
        ptx::mma_commit(o_full(ob));
      }
      ptx::mma_commit(fin);
      ptx::mbar_drain(fin, 0, nullptr, 0);
    }
  } else if (warp >= 6) {
    // ------------------------------------------------------------- K and V ---
    TileLoads<D> loads(a, &tmK, &tmV, s0, warp - 6);
    int tile = 0;
    bool ok = true;
    for (int nq = 0; ok; ++nq) {
      const int qi = nq & 1;
      if (!wait_warp(i_full(qi), (nq >> 1) & 1)) break;
      const PdItem it = item_slot[qi];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_empty(qi));
      if (it.seq < 0) break;
      if (it.j0 >= it.j1 && warp == 6 && lane == 0) ptx::mbar_arrive(near_end);
      loads.look_up(it, it.j0);
      for (int j = it.j0; j < it.j1; ++j, ++tile) {
        const int st = tile % STAGES;
        const int page = loads.advance(it, j);
        if (j + 1 == it.j1 && warp == 6 && lane == 0) ptx::mbar_arrive(near_end);
        if (!wait_warp(kv_empty(st), ((tile / STAGES) & 1) ^ 1)) {
          ok = false;
          break;
        }
        loads.issue(it, j, st, page, kv_full(st));
      }
    }
    __syncwarp();
    ptx::settle_loads<PD_LOADERS, STAGES>(tile, warp - 6, s_loaded, kv_full);
  } else {
    // --------------------------------------------------- softmax, output ---
    const int w4 = warp - 2;
    const int qq = warp & 3;         // TMEM lane quarter
    const int row = qq * 32 + lane;  // key of a tile (S^T), column of the head (O^T)
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    // One value per head of each warp to all four: lane h of a warp stores its head's
    // and one arrival per warp completes the phase.
    auto exchange = [&](float *slots, const float(&v)[RN], uint32_t bar, uint32_t parity) -> bool {
      if (lane < RN) {
        float x = v[0];
#pragma unroll
        for (int h = 1; h < RN; ++h)
          if (lane == h) x = v[h];
        slots[w4 * PD_N + lane] = x;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
      return wait_warp(bar, parity);
    };
    int tile = 0;
    bool ok = true;
    for (int nq = 0; ok; ++nq) {
      const int qi = nq & 1, ob = nq & 1;
      if (!wait_warp(q_full(qi), (nq >> 1) & 1)) break;
      const PdItem it = item_slot[qi];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_empty(qi));
      if (it.seq < 0) break;
      const int nt = it.j1 - it.j0;
      float m_run[RN], l_run[RN];
#pragma unroll
      for (int h = 0; h < RN; ++h) {
        m_run[h] = -INFINITY;
        l_run[h] = 0.f;
      }
      for (int j = 0; j < nt; ++j, ++tile) {
        const int sb = tile & 1;
        if (!wait_warp(s_full(sb), (tile >> 1) & 1)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        float s[PD_N];
        ptx::tmem_ld16(lane_base + sb * PD_N, s);
        const int key0 = (it.j0 + j) * PD_KEYS;
        const bool valid = key0 + row < it.len;
        if (key0 + PD_KEYS > it.len) {  // the sequence's last tile: clear V behind its last key
          const int st = tile % STAGES;
          if (!wait_warp(kv_full(st), (tile / STAGES) & 1)) {
            ok = false;
            break;
          }
          if (!valid) {
            uint4 *vr = reinterpret_cast<uint4 *>(smem + L::OFF_V + st * L::TILE + row * 128);
#pragma unroll
            for (int at = 0; at < ATOMS; ++at)
#pragma unroll
              for (int c = 0; c < 8; ++c) vr[at * (L::ATOM / 16) + c] = make_uint4(0, 0, 0, 0);
          }
        }
        // per-head maximum over the tile: warp shuffles, then across the 4 warps
        float mx[RN];
#pragma unroll
        for (int h = 0; h < RN; ++h) mx[h] = ptx::warp_max_redux((valid && h < it.nh) ? s[h] : -INFINITY);
        float *rs = red + (tile & 1) * (4 * PD_N);
        if (!exchange(rs, mx, red_full(tile & 1), (tile >> 1) & 1)) {
          ok = false;
          break;
        }
        bool need_any = false;
        float alpha[RN];
#pragma unroll
        for (int h = 0; h < RN; ++h) {
          const float mt =
              fmaxf(fmaxf(rs[h], rs[PD_N + h]), fmaxf(rs[2 * PD_N + h], rs[3 * PD_N + h])) * a.scale_log2;
          alpha[h] = 1.f;
          if (h < it.nh && mt > m_run[h] + PD_RESCALE) {
            alpha[h] = ptx::ex2_approx(m_run[h] - mt);
            m_run[h] = mt;
            need_any = true;
          }
        }
        // P^T into shared memory: row h (query head), column = key, 128-byte swizzle
        if (!wait_warp(p_free(sb), ((tile >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        uint8_t *pbuf = smem + L::OFF_P + sb * L::P_BYTES + (row / 64) * (PD_N * 128);
        const int c = row % 64;
#pragma unroll
        for (int h = 0; h < RN; ++h) {
          const float p = (valid && h < it.nh) ? ptx::ex2_approx(fmaf(s[h], a.scale_log2, -m_run[h])) : 0.f;
          l_run[h] = l_run[h] * alpha[h] + p;
          // bf16 P: the tensor cores' operand; the sum keeps the unrounded values
          *reinterpret_cast<bf16 *>(pbuf + h * 128 + ((c >> 3) ^ (h & 7)) * 16 + (c & 7) * 2) = __float2bfloat16_rn(p);
        }
        if (need_any && j > 0) {  // rescale O^T (thread = column) before this tile's product
          if (!wait_warp(p_free(sb ^ 1), ((tile - 1) >> 1) & 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          float ov[PD_N];
          ptx::tmem_ld16(lane_base + 32 + ob * PD_N, ov);
          uint32_t wv[PD_N];
#pragma unroll
          for (int h = 0; h < PD_N; ++h) wv[h] = __float_as_uint(h < RN ? ov[h] * alpha[h < RN ? h : 0] : ov[h]);
          ptx::tmem_st16(lane_base + 32 + ob * PD_N, wv);
          ptx::tmem_st_wait();
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(p_full(sb));
      }
      if (!ok) break;
      // item end: sum l over the 128 keys, read O^T
      if (!wait_warp(o_full(ob), (nq >> 1) & 1)) break;
      ptx::tc_fence_after();
      float ov[PD_N];
      if (nt > 0) {
        ptx::tmem_ld16(lane_base + 32 + ob * PD_N, ov);
      } else {
#pragma unroll
        for (int h = 0; h < PD_N; ++h) ov[h] = 0.f;
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(o_free(ob));
#pragma unroll
      for (int h = 0; h < RN; ++h) l_run[h] = warp_sum(l_run[h]);
      float *ls = red + (2 + ob) * (4 * PD_N);
      if (!exchange(ls, l_run, lred_full, nq & 1)) break;
#pragma unroll
      for (int h = 0; h < RN; ++h) {
        if (h >= it.nh || row >= D) continue;
        const float l = ls[h] + ls[PD_N + h] + ls[2 * PD_N + h] + ls[3 * PD_N + h];
        if (a.cluster > 1) {  // for the join below: [PD_N][D + 2] over the first K stage, idle by now
          float *pp = reinterpret_cast<float *>(smem + L::OFF_K) + h * (D + 2);
          pp[row] = ov[h];
          if (row == 0) {
            pp[D] = m_run[h];
            pp[D + 1] = l;
          }
        } else if (it.slot < 0) {
          if (row < a.D)
            a.o[((size_t)it.seq * a.H + it.h0 + h) * a.D + row] = __float2bfloat16_rn(l == 0.f ? 0.f : ov[h] / l);
        } else {
          float *pp = a.part + ((size_t)it.slot * a.H + it.h0 + h) * (D + 2);
          pp[row] = ov[h];
          if (row == 0) {
            pp[D] = m_run[h];
            pp[D + 1] = l;
          }
        }
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (a.cluster > 1) {
    // one item per cluster: its CTAs' parts meet here, head h finished by CTA h % cluster
    ptx::cluster_sync();
    const int u = blockIdx.x / a.cluster, unit = u % units, seq = u / units;
    const int g = unit / a.subs, h0 = g * a.r + (unit % a.subs) * PD_N;
    const int nh = min(PD_N, (g + 1) * a.r - h0);
    if (*abort_flag == 0 && threadIdx.x < a.D) {
      const uint32_t part = s0 + L::OFF_K;
      for (int h = rank; h < nh; h += a.cluster) {
        float mc[PD_MAX_CLUSTER], lc[PD_MAX_CLUSTER], oc[PD_MAX_CLUSTER];
        float m = -INFINITY;
#pragma unroll
        for (int c = 0; c < PD_MAX_CLUSTER; ++c) {
          mc[c] = -INFINITY;
          lc[c] = oc[c] = 0.f;
          if (c < a.cluster) {
            const uint32_t p = ptx::mapa_shared(part, c) + (uint32_t)(h * (D + 2)) * 4;
            mc[c] = ptx::ld_cluster_f32(p + D * 4);
            lc[c] = ptx::ld_cluster_f32(p + (D + 1) * 4);
            oc[c] = ptx::ld_cluster_f32(p + threadIdx.x * 4);
          }
        }
#pragma unroll
        for (int c = 0; c < PD_MAX_CLUSTER; ++c) m = fmaxf(m, mc[c]);
        float l = 0.f, o = 0.f;
#pragma unroll
        for (int c = 0; c < PD_MAX_CLUSTER; ++c) {
          const float f = mc[c] == -INFINITY ? 0.f : ptx::ex2_approx(mc[c] - m);
          l = fmaf(f, lc[c], l);
          o = fmaf(f, oc[c], o);
        }
        a.o[((size_t)seq * a.H + h0 + h) * a.D + threadIdx.x] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
      }
    }
    ptx::cluster_sync();  // no CTA leaves while others read its shared memory
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Joins the chunks of one split sequence's head, o = sum 2^(m_c - M) o_c / sum
// 2^(m_c - M) l_c.  COLS columns per CTA of 256 threads, COLS / 4 threads per chunk:
// 32 columns when few rows would leave most SMs idle, else all.
template <int D, int COLS>
__global__ void __launch_bounds__(256) decode_join_kernel(const PdPlan *plan, const PdSplit *splits,
                                                          const float *part, bf16 *o, int H, int width,
                                                          const __grid_constant__ PdArgs a) {
  constexpr int LANES = COLS / 4, GROUPS = 256 / LANES, PER = D / COLS;
  __shared__ float sm[8], so[GROUPS][COLS], sl[GROUPS];
  grid_dependency_wait();
  const int c0 = (int)(blockIdx.x % PER) * COLS, h = blockIdx.x / PER % H, k = blockIdx.x / PER / H;
  PdSplit s;
  if (plan != nullptr) {
    if (k >= plan->n_split) return;
    s = splits[k];
  } else {  // the same chunks as the CTAs found
    WarpPlan x;
    x.find(a.pv, a.kv_lens, a.n_seqs, a.max_kv_len, a.G * a.subs, a.shared_sms, nullptr);
    s.seq = k;
    s.slot = __shfl_sync(0xffffffffu, x.first, k);
    s.n = __shfl_sync(0xffffffffu, x.n, k);
    if (s.n == 1) return;
  }
  const float *p = part + ((size_t)s.slot * H + h) * (D + 2);
  const size_t step = (size_t)H * (D + 2);
  float m = -INFINITY;
  for (int c = threadIdx.x; c < s.n; c += 256) m = fmaxf(m, p[c * step + D]);
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, sm[w]);
  const int grp = threadIdx.x / LANES, d = threadIdx.x % LANES * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int c = grp; c < s.n; c += GROUPS) {
    const float *pc = p + c * step;
    const float f = ptx::ex2_approx(pc[D] - m);
    const float2 x = *reinterpret_cast<const float2 *>(pc + c0 + d);
    const float2 y = *reinterpret_cast<const float2 *>(pc + c0 + d + 2);
    l = fmaf(f, pc[D + 1], l);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, y.x, acc.z);
    acc.w = fmaf(f, y.y, acc.w);
  }
  *reinterpret_cast<float4 *>(&so[grp][d]) = acc;
  if (d == 0) sl[grp] = l;
  __syncthreads();
  const int col = c0 + threadIdx.x;
  if (threadIdx.x < COLS && col < width) {
    float x = 0.f, z = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      x += so[g][threadIdx.x];
      z += sl[g];
    }
    o[((size_t)s.seq * H + h) * width + col] = __float2bfloat16_rn(x / z);
  }
}

// Clusters of a size that run at once: 152 SMs hold 15 of eight CTAs and 36 of four (16
// sequences of 1024 keys as clusters of eight take two turns: 18 us for 10.8).
int clusters_at_once(int cluster, int sms) {
  static ClusterRoom room;
  return room.at_once(paged_decode_tc_kernel<128, 4>, cluster, PD_THREADS, PdLayout<128>::BYTES, sms);
}

struct PdSizes {
  int units = 0, cluster = 0;  // cluster: CTAs of a direct item (0: planned)
  bool shared = false;         // planned by every CTA for itself
  long long max_entries = 0;
  int max_split = 0;
  size_t off_entries = 0, off_splits = 0, off_part = 0, bytes = 0;
};

PdSizes decode_sizes(int n_seqs, int max_kv_len, int H, int G, int D, int sms) {
  PdSizes z;
  z.units = G * ((H / G + PD_N - 1) / PD_N);
  const long long items = (long long)n_seqs * z.units;
  const int tiles = (max_kv_len + PD_KEYS - 1) / PD_KEYS;
  int cluster = 1;
  while (cluster < PD_MAX_CLUSTER && items <= clusters_at_once(cluster * 2, sms) && tiles > cluster) cluster *= 2;
  if ((tiles + cluster - 1) / cluster <= (cluster > 1 ? PD_CLUSTER_TILES : PD_WHOLE_TILES)) {
    z.cluster = cluster;
    return z;
  }
  const int most = 2 * ((PD_ROUNDS * sms + z.units - 1) / z.units) + 2;  // chunks of split sequences
  if (n_seqs <= PD_SHARED_SEQS) {
    z.shared = true;
    z.max_entries = (long long)n_seqs + most;
    z.max_split = n_seqs;
    z.bytes = (size_t)z.max_entries * H * (D + 2) * sizeof(float);
    return z;
  }
  z.max_entries = (long long)n_seqs + most;
  z.max_split = n_seqs < most / 2 ? n_seqs : most / 2;
  z.off_entries = sizeof(PdPlan);
  z.off_splits = z.off_entries + (size_t)z.max_entries * sizeof(PdEntry);
  z.off_part = z.off_splits + (size_t)z.max_split * sizeof(PdSplit);
  z.off_part = (z.off_part + 127) / 128 * 128;
  z.bytes = z.off_part + (size_t)most * H * (D + 2) * sizeof(float);
  return z;
}

template <int D, int RN>
cudaError_t launch_tc(const bf16 *q, const bf16 *k, const bf16 *v, bf16 *o, const PagedView &pv, const int *kv_lens,
                      int n_seqs, int max_kv_len, int H, int G, int width, void *workspace, int *status,
                      cudaStream_t st) {
  using L = PdLayout<D>;
  static PerContextOnce attr;
  cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(paged_decode_tc_kernel<D, RN>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  });
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  const PdSizes z = decode_sizes(n_seqs, max_kv_len, H, G, D, sms);
  PdArgs a;
  a.o = o;
  a.pv = pv;
  a.kv_lens = kv_lens;
  a.n_seqs = n_seqs;
  a.max_kv_len = max_kv_len;
  a.H = H;
  a.G = G;
  a.D = width;
  a.r = H / G;
  a.subs = z.units / G;
  a.box = 1 << (pv.page_log2 < 7 ? pv.page_log2 : 7);
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)width);
  a.cluster = 1;
  a.shared_sms = z.shared ? sms : 0;
  a.plan = nullptr;
  a.entries = nullptr;
  a.part = nullptr;
  a.status = status;
  a.wait_cycles = op_wait_cycles();
  CUtensorMap mq, mk, mv;
  if (!make_heads_map(&mq, q, n_seqs, H, width, PD_N, 1) || !make_paged_map(&mk, k, pv, G, width, a.box) ||
      !make_paged_map(&mv, v, pv, G, width, a.box))
    return cudaErrorInvalidValue;
  const long long items = (long long)n_seqs * z.units;
  if (z.cluster > 0) {
    a.cluster = z.cluster;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)z.cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    // clusters: one item each; single CTAs: one per SM, each looping over its items
    cfg.gridDim = dim3((unsigned)(z.cluster > 1 ? items * z.cluster : (items < sms ? items : sms)));
    cfg.blockDim = dim3(PD_THREADS);
    cfg.dynamicSmemBytes = L::BYTES;
    cfg.stream = st;
    cfg.attrs = attrs;
    cfg.numAttrs = z.cluster > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, paged_decode_tc_kernel<D, RN>, mq, mk, mv, a);
  }
  char *w = reinterpret_cast<char *>(workspace);
  PdSplit *splits = nullptr;
  a.part = reinterpret_cast<float *>(w);
  if (!z.shared) {
    a.plan = reinterpret_cast<PdPlan *>(w);
    a.entries = reinterpret_cast<PdEntry *>(w + z.off_entries);
    splits = reinterpret_cast<PdSplit *>(w + z.off_splits);
    a.part = reinterpret_cast<float *>(w + z.off_part);
    count_launch();
    e = launch_pdl(decode_plan_kernel, dim3(1), dim3(PD_PLAN_THREADS), 0, st, pv, kv_lens, n_seqs, max_kv_len,
                   z.units, sms, (int)z.max_entries, a.plan, a.entries, splits, status);
    if (e != cudaSuccess) return e;
  }
  count_launch();
  const long long most = z.max_entries * z.units;
  e = launch_pdl(paged_decode_tc_kernel<D, RN>, dim3((unsigned)(most < sms ? most : sms)), dim3(PD_THREADS), L::BYTES,
                 st, mq, mk, mv, a);
  if (e != cudaSuccess) return e;
  count_launch();
  const bool narrow = (long long)z.max_split * H < 2LL * sms;
  return launch_pdl(narrow ? decode_join_kernel<D, 32> : decode_join_kernel<D, D>,
                    dim3((unsigned)(z.max_split * H * (narrow ? D / 32 : 1))), dim3(256), 0, st,
                    (const PdPlan *)a.plan, (const PdSplit *)splits, (const float *)a.part, o, H, width, a);
}

template <int D>
cudaError_t launch_by_heads(const bf16 *q, const bf16 *k, const bf16 *v, bf16 *o, const PagedView &pv,
                            const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int width, void *workspace,
                            int *status, cudaStream_t st) {
  const int r = H / G;
  auto f = r <= 2 ? launch_tc<D, 2> : r <= 4 ? launch_tc<D, 4> : r <= 8 ? launch_tc<D, 8> : launch_tc<D, 16>;
  return f(q, k, v, o, pv, kv_lens, n_seqs, max_kv_len, H, G, width, workspace, status, st);
}

}  // namespace

size_t paged_decode_tc_workspace_bytes(int n_seqs, int max_kv_len, int H, int G, int D) {
  return decode_sizes(n_seqs, max_kv_len, H, G, D < 64 ? 64 : D, sm_count()).bytes;
}

cudaError_t launch_paged_decode_tc(const bf16 *q, const bf16 *k, const bf16 *v, bf16 *o, const PagedView &pv,
                                   const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int D,
                                   void *workspace, int *status, cudaStream_t st) {
  if (D == 128)
    return launch_by_heads<128>(q, k, v, o, pv, kv_lens, n_seqs, max_kv_len, H, G, D, workspace, status, st);
  return launch_by_heads<64>(q, k, v, o, pv, kv_lens, n_seqs, max_kv_len, H, G, D, workspace, status, st);
}

}  // namespace llama
