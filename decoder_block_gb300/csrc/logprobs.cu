// Log-probabilities of given tokens, entropy and the likeliest tokens of logits
// rows ("The Evolving Transformer 04 · LLaMA", §07 Assemble: the logits of a
// position are the unnormalised log-probabilities of its next token).
//   m = max_v x_v, Z = sum_v e^(x_v - m), U = sum_v e^(x_v - m) (x_v - m):
//   ln p(v) = (x_v - m) - ln Z,   entropy = ln Z - U / Z,
// and the top_k largest x in the order (x descending, id ascending).
//
// Every logit is read once, and that is what bounds it.  Each thread keeps a running
// (m, Z, U) -- a larger m' turns Z into f Z and U into f (U + Z (m - m')) with f =
// e^(m - m') -- and, for the top, only which three of its batches of 16 or 32 logits
// had the largest maxima and the fourth largest maximum: 14 instructions a batch.
// Then the k-th largest of 64 such maxima is a bound that at least k logits reach, so
// nothing below it is among the top; the few batches whose maximum reaches it are
// read again, and each of the k to about 2 k logits found takes the place given by
// how many of the others are ahead of it.  A row whose top is not found that way (a
// thread with four such batches, or a great many equal logits) is read a second time,
// its warps sorting candidates into lists of 32.  (Sorting candidates as they come
// took 202 us where this takes 171: votes and shuffles in every batch.)
// A row belongs to one warp, to a CTA, or to a cluster of CTAs whose parts meet
// through distributed shared memory (few rows: the row is what there is to split).
#include <float.h>
#include <limits.h>
#include <math.h>

#include "paged_kernels.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
// CTAs of an SM and 16-byte vectors of a lane's batch: 64 KB of an SM's loads in flight.
// 2048 x 128256, top 20, fp32: 171 to 175 us (1.05 GB at 0.89 to 0.91 of the measured copy
// rate); with 3 CTAs 181, with 5 252 us (64 registers spill 24 to 48 bytes of a thread, 48
// registers 52 to 136).  bf16, top 5: 104 us, 0.75 (the same number of logits in half the bytes).
// A row with fewer logits above -inf than top_k has no bound and is read twice: 419 us for 196
// in a loop with a cold L2.
constexpr int LP_CTAS = 4;
constexpr int LP_VECS = 4;
constexpr int LP_STEP = 32 * LP_VECS;  // vectors of a warp's batch
constexpr int LP_MAX_CLUSTER = 8;
constexpr float LP_LOG2E = 1.4426950408889634f;

struct LpArgs {
  const void *logits;
  long long stride;
  const int *targets;
  int rows, V;
  float *logprobs, *entropy;
  int top_k;
  int *top_ids;
  float *top_logprobs;
  int *status;
  int bad_target;
  int cluster;
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN when either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Order of the top: larger logit first, lower id among equals.
__device__ __forceinline__ bool ahead(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

// ------------------------------------------------------------ statistics ---
struct Stats {
  float m, z, u;
};
__device__ __forceinline__ Stats merge(const Stats &a, const Stats &b) {
  Stats r;
  r.m = fmaxf(a.m, b.m);
  // m is finite or +inf; the side that has the maximum (also +inf) stays as it is
  const float da = a.m == r.m ? 0.f : fmaxf(a.m - r.m, -200.f), db = b.m == r.m ? 0.f : fmaxf(b.m - r.m, -200.f);
  const float fa = ptx::ex2_approx(da * LP_LOG2E), fb = ptx::ex2_approx(db * LP_LOG2E);
  r.z = a.z * fa + b.z * fb;
  r.u = fa * fmaf(a.z, da, a.u) + fb * fmaf(b.z, db, b.u);
  return r;
}
// A row's statistics from one part in each of the first n lanes (a power of two).
__device__ __forceinline__ Stats lanes_merge(Stats s, int n) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= n) continue;
    Stats t;
    t.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    t.z = __shfl_xor_sync(0xffffffffu, s.z, o);
    t.u = __shfl_xor_sync(0xffffffffu, s.u, o);
    s = merge(s, t);
  }
  s.m = __shfl_sync(0xffffffffu, s.m, 0);
  s.z = __shfl_sync(0xffffffffu, s.z, 0);
  s.u = __shfl_sync(0xffffffffu, s.u, 0);
  return s;
}

// A batch: LP_VECS vectors per lane at v0 + 32 j + lane (index in the row's aligned
// part), -inf behind v_end.
template <typename T>
__device__ __forceinline__ void load_batch(Vec16<T> (&x)[LP_VECS], const Vec16<T> *vec, int v0, int v_end) {
#pragma unroll
  for (int j = 0; j < LP_VECS; ++j) {
    const int at = v0 + 32 * j + (int)(threadIdx.x & 31);
    if (at < v_end) {
      x[j].raw = ld_once_after_wait(vec + at);
    } else {
#pragma unroll
      for (int e = 0; e < Vec16<T>::N; ++e) x[j].set(e, -INFINITY);
    }
  }
}

// Largest logit of a lane's batch, NaN left out (-inf or NaN when there is nothing else).
// bf16 in pairs as they are: half the instructions.
__device__ __forceinline__ float batch_max(const Vec16<float> (&x)[LP_VECS]) {
  float bm = -INFINITY;
#pragma unroll
  for (int j = 0; j < LP_VECS; ++j)
#pragma unroll
    for (int e = 0; e < Vec16<float>::N; ++e) bm = fmaxf(bm, x[j].get(e));
  return bm;
}
__device__ __forceinline__ float batch_max(const Vec16<bf16> (&x)[LP_VECS]) {
  uint32_t m = 0xff80ff80u;  // -inf, -inf
#pragma unroll
  for (int j = 0; j < LP_VECS; ++j) {
    const uint32_t w[4] = {x[j].raw.x, x[j].raw.y, x[j].raw.z, x[j].raw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[e]));
  }
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// What a thread keeps of the part of a row that it reads.
template <typename T>
struct RowScan {
  static constexpr int V = Vec16<T>::N;
  float m = -FLT_MAX;  // finite, so that -inf alone gives weights of 0; a logit of -FLT_MAX itself counts
  uint64_t z[2], u[2];  // four independent sums each
  // m is the largest maximum of a batch, b2 to b4 the next ones; of batches i1 to i3
  float b2 = -INFINITY, b3 = -INFINITY, b4 = -INFINITY;
  int i1 = -1, i2 = -1, i3 = -1;

  __device__ __forceinline__ RowScan() { z[0] = z[1] = u[0] = u[1] = ptx::f2pack(0.f, 0.f); }
  __device__ __forceinline__ void raise(float nm) {
    const float d = fmaxf(m - nm, -200.f);  // the old sums are worth nothing beyond e^-200
    const float f = ptx::ex2_approx(d * LP_LOG2E);
    const uint64_t f2 = ptx::f2pack(f, f), d2 = ptx::f2pack(d, d);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u[i] = ptx::fmul2(ptx::ffma2(z[i], d2, u[i]), f2);
      z[i] = ptx::fmul2(z[i], f2);
    }
    m = nm;
  }
  __device__ __forceinline__ void add(float a, float b, int i) {
    float d0, d1;
    ptx::f2unpack(ptx::fadd2(ptx::f2pack(a, b), ptx::f2pack(-m, -m)), d0, d1);
    d0 = max_nan(d0, -200.f);  // -inf: weight 0 and 0 in U instead of 0 * inf
    d1 = max_nan(d1, -200.f);
    const uint64_t d2 = ptx::f2pack(d0, d1);
    float y0, y1;
    ptx::f2unpack(ptx::fmul2(d2, ptx::f2pack(LP_LOG2E, LP_LOG2E)), y0, y1);
    const uint64_t e2 = ptx::f2pack(ptx::ex2_approx(y0), ptx::ex2_approx(y1));
    z[i & 1] = ptx::fadd2(z[i & 1], e2);
    u[i & 1] = ptx::ffma2(e2, d2, u[i & 1]);
  }
  __device__ __forceinline__ Stats stats() const {
    float a, b, c, d;
    Stats s;
    s.m = m;
    ptx::f2unpack(z[0], a, b);
    ptx::f2unpack(z[1], c, d);
    s.z = (a + b) + (c + d);
    ptx::f2unpack(u[0], a, b);
    ptx::f2unpack(u[1], c, d);
    s.u = (a + b) + (c + d);
    return s;
  }
  __device__ __forceinline__ void batch(const Vec16<T> (&x)[LP_VECS], int round) {
    const float bm = batch_max(x);
    b4 = fmaxf(b4, fminf(bm, b3));
    i3 = bm > b2 ? i2 : bm > b3 ? round : i3;
    b3 = fmaxf(b3, fminf(bm, b2));
    i2 = bm > m ? i1 : bm > b2 ? round : i2;
    b2 = fmaxf(b2, fminf(bm, m));
    i1 = bm > m ? round : i1;
    if (bm > m) raise(bm);
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j)
#pragma unroll
      for (int e = 0; e < V; e += 2) add(x[j].get(e), x[j].get(e + 1), j + e / 2);
  }
};

// ------------------------------------------------------------------- top ---
struct __align__(8) Cand {
  float v;
  int id;
};

// A float as an integer of the same order, its six low bits replaced by `slot`.
__device__ __forceinline__ int slot_key(float x, int slot) {
  const int b = __float_as_int(x);
  return ((b < 0 ? b ^ 0x7fffffff : b) & ~63) | slot;
}
__device__ __forceinline__ float key_value(int key) {  // at most the value the key was made of
  key &= ~63;
  const float x = __int_as_float(key < 0 ? key ^ 0x7fffffff : key);
  return x == x ? x : -INFINITY;
}
// Calls f(i, key) with the i-th largest of the lanes' two keys each for i < n, in every lane.
template <typename F>
__device__ __forceinline__ void top_keys(int a, int b, int n, F &&f) {
  for (int i = 0; i < n; ++i) {
    const int best = __reduce_max_sync(0xffffffffu, max(a, b));
    if (a == best) a = INT_MIN;
    if (b == best) b = INT_MIN;
    f(i, best);
  }
}

// The logits of one thread's batch, its vectors `first` + 32 j, that reach `bound`,
// appended to all[].
template <typename T>
__device__ __forceinline__ void pick(const Vec16<T> *vec, int first, int v_end, int id0, float bound, Cand *all, int *n,
                                     int cap) {
  constexpr int V = Vec16<T>::N;
  Vec16<T> x[LP_VECS];
#pragma unroll
  for (int j = 0; j < LP_VECS; ++j)
    if (first + 32 * j < v_end) x[j] = load16<T>(reinterpret_cast<const T *>(vec + first + 32 * j));
#pragma unroll
  for (int j = 0; j < LP_VECS; ++j) {
    if (first + 32 * j >= v_end) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float v = x[j].get(e);
      if (v >= bound) {
        const int at = atomicAdd(n, 1);
        if (at < cap) all[at] = Cand{v, id0 + (first + 32 * j) * V + e};
      }
    }
  }
}

// A warp's sorted list: lane j holds the j-th entry.
struct TopList {
  float v;
  int id;
  // Keeps, of this lane's entry and that of the lane s away, the one ahead or behind.
  __device__ __forceinline__ void exchange(int s, bool keep_ahead) {
    const float xv = __shfl_xor_sync(0xffffffffu, v, s);
    const int xi = __shfl_xor_sync(0xffffffffu, id, s);
    if (keep_ahead == ahead(xv, xi, v, id)) {
      v = xv;
      id = xi;
    }
  }
  __device__ __forceinline__ void sort() {  // bitonic, the one that is ahead in the lower lane
    const int lane = threadIdx.x & 31;
    for (int size = 2; size <= 32; size *= 2)
      for (int s = size / 2; s > 0; s /= 2) exchange(s, ((lane & s) == 0) == ((lane & size) == 0));
  }
  // The 32 first of this list and another sorted one: the larger of entry j here and
  // entry 31 - j there are those 32, in a bitonic order that five steps sort.
  __device__ __forceinline__ void merge(float ov, int oi) {
    const int lane = threadIdx.x & 31;
    ov = __shfl_xor_sync(0xffffffffu, ov, 31);
    oi = __shfl_xor_sync(0xffffffffu, oi, 31);
    if (ahead(ov, oi, v, id)) {
      v = ov;
      id = oi;
    }
    for (int s = 16; s > 0; s >>= 1) exchange(s, (lane & s) == 0);
  }
};

// Candidates of a warp: fewer than 32 wait, a vector's logits of each lane join them.
template <typename T>
constexpr int LP_WAIT = 32 + 32 * Vec16<T>::N;

// The second pass over a warp's part of a row: everything that reaches `bound` and is
// ahead of the k-th entry of the warp's list waits in `wait` and is sorted into the
// list 32 at a time.  Leaves list and rest together in `wait`; returns their number,
// less than 64.
template <typename T>
__device__ __noinline__ int second_pass(const Vec16<T> *vec, int v0, int step, int n_vec, int id0, int k, float bound,
                                        Cand *wait) {
  constexpr int V = Vec16<T>::N;
  const int lane = threadIdx.x & 31;
  TopList top{-INFINITY, INT_MAX};
  float kth = -INFINITY;
  int kth_id = INT_MAX, waiting = 0;
  Vec16<T> x[LP_VECS], next[LP_VECS];
  load_batch<T>(next, vec, v0, n_vec);
  for (; v0 < n_vec; v0 += step) {
    float bm = -INFINITY;
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) {
      x[j] = next[j];
#pragma unroll
      for (int e = 0; e < V; ++e) bm = fmaxf(bm, x[j].get(e));
    }
    load_batch<T>(next, vec, v0 + step, n_vec);  // a batch ahead: nothing where the row ends
    if (!__any_sync(0xffffffffu, bm >= bound && bm >= kth)) continue;
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) {
      const int at = v0 + 32 * j + lane;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = x[j].get(e);
        const int id = id0 + at * V + e;
        const bool c = at < n_vec && v >= bound && ahead(v, id, kth, kth_id);
        const unsigned mask = __ballot_sync(0xffffffffu, c);
        if (c) wait[waiting + __popc(mask & ((1u << lane) - 1u))] = Cand{v, id};
        waiting += __popc(mask);
      }
      if (waiting < 32) continue;
      __syncwarp();
      while (waiting >= 32) {
        waiting -= 32;
        TopList c{wait[waiting + lane].v, wait[waiting + lane].id};
        c.sort();
        top.merge(c.v, c.id);
      }
      __syncwarp();
      kth = __shfl_sync(0xffffffffu, top.v, k - 1);
      kth_id = __shfl_sync(0xffffffffu, top.id, k - 1);
    }
  }
  const bool c = top.id != INT_MAX;
  const unsigned mask = __ballot_sync(0xffffffffu, c);
  if (c) wait[waiting + __popc(mask & ((1u << lane) - 1u))] = Cand{top.v, top.id};
  __syncwarp();
  return waiting + __popc(mask);
}

// Entry of this candidate in the order of all n of `all`: how many are ahead of it.
__device__ __forceinline__ int rank_of(const Cand &c, const Cand *all, int n) {
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const Cand o = all[i];
    rank += ahead(o.v, o.id, c.v, c.id) ? 1 : 0;
  }
  return rank;
}

// --------------------------------------------------------------- results ---
// The given token of a row, looked up while the row is read.
template <typename T>
struct Target {
  int id = -1;
  float logit = 0.f;
  __device__ __forceinline__ Target(const LpArgs &a, int row, const T *x, bool needed) {
    if (!needed || a.logprobs == nullptr) return;
    id = ld_after_wait(a.targets + row);
    if (id >= 0 && id < a.V) logit = to_f32<T>(x[id]);
  }
};

// A row's results from its statistics and its n candidates, by one warp (THREADS =
// 32) or by a whole CTA.
template <typename T, int THREADS>
__device__ __forceinline__ void finish_row(const LpArgs &a, int row, const Target<T> &y, const Stats &s,
                                           const Cand *all, int n) {
  const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
  const bool empty = s.m == -FLT_MAX && s.z == 0.f;  // nothing but -inf
  const float log_z = logf(s.z);
  auto logprob = [&](float v) { return empty ? -INFINITY : (v - s.m) - log_z; };
  if (tid == 0) {
    if (a.logprobs != nullptr) {
      float lp = y.id == -1 ? 0.f : NAN;
      if (y.id >= 0 && y.id < a.V) lp = logprob(y.logit);
      else if (y.id != -1) report_status(a.status, a.bad_target);
      a.logprobs[row] = lp;
    }
    if (a.entropy != nullptr) a.entropy[row] = empty ? 0.f : log_z - s.u / s.z;
  }
  if (a.top_k == 0) return;
  int *ids = a.top_ids + (size_t)row * a.top_k;
  float *lps = a.top_logprobs + (size_t)row * a.top_k;
  for (int i = tid; i < n; i += THREADS) {
    const Cand c = all[i];
    const int at = rank_of(c, all, n);
    if (at < a.top_k) {
      ids[at] = c.id;
      lps[at] = logprob(c.v);
    }
  }
  for (int at = n + tid; at < a.top_k; at += THREADS) {  // fewer logits than top_k that are not NaN
    ids[at] = -1;
    lps[at] = NAN;
  }
}

// WPR: warps of a row in this CTA (1: eight rows per CTA; 8: one row, or a
// cluster's part of one).
template <typename T, int WPR>
__global__ void __launch_bounds__(LP_THREADS, LP_CTAS) token_logprobs_kernel(const __grid_constant__ LpArgs a) {
  constexpr int V = Vec16<T>::N, GROUPS = LP_WARPS / WPR;  // rows of this CTA
  constexpr int CAP = WPR * 64, ENDS = 2 * (V - 1);        // candidates kept; logits outside whole vectors
  __shared__ Cand s_wait[LP_WARPS][LP_WAIT<T>];
  __shared__ Cand s_all[GROUPS][CAP + ENDS];
  __shared__ Cand s_first[32];  // a CTA's top, for the cluster's first CTA
  __shared__ Stats s_stats[LP_WARPS];
  __shared__ int s_max[GROUPS][64];
  __shared__ int s_batch[GROUPS][CAP];  // batches to read again
  __shared__ int s_n[GROUPS], s_batches[GROUPS];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, k = a.top_k, group = WPR == 1 ? warp : 0;
  const int parts = WPR == 1 ? 1 : WPR * a.cluster;  // warps that share a row
  const int rank = WPR == 1 ? 0 : (int)(blockIdx.x % a.cluster);
  const int row = WPR == 1 ? (int)blockIdx.x * LP_WARPS + warp : (int)(blockIdx.x / a.cluster);
  const int part = WPR == 1 ? 0 : rank * WPR + warp;
  grid_dependency_wait();
  if (WPR == 1 && row >= a.rows) return;
  auto sync = [] {
    if (WPR == 1) __syncwarp();
    else __syncthreads();
  };
  const T *x = reinterpret_cast<const T *>(a.logits) + (long long)row * a.stride;
  const Target<T> y(a, row, x, part == 0);
  // logits before the first 16-byte boundary, then whole vectors, then the rest
  const int head = min(a.V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T));
  const int n_vec = (a.V - head) / V;
  const Vec16<T> *vec = reinterpret_cast<const Vec16<T> *>(x + head);
  if (WPR == 1 || warp == 0) {
    s_max[group][lane] = s_max[group][lane + 32] = slot_key(-INFINITY, 0);
    if (lane == 0) s_n[group] = s_batches[group] = 0;
  }
  if (k > 0) sync();
  RowScan<T> r;
  int round = 0;
  for (int v0 = part * LP_STEP; v0 < n_vec; v0 += parts * LP_STEP, ++round) {
    Vec16<T> b[LP_VECS];
    load_batch<T>(b, vec, v0, n_vec);
    r.batch(b, round);
  }
  // in front of the first 16-byte boundary and behind the last one
  const bool has_ends = part == parts - 1;
  const int n_ends = has_ends ? a.V - n_vec * V : 0;  // at most ENDS
  const int end_id = lane < head ? lane : lane + n_vec * V;
  const float end = lane < n_ends ? to_f32<T>(x[end_id]) : -INFINITY;
  if (has_ends) {
    if (end > r.m) r.raise(end);
    r.add(end, -INFINITY, 0);
  }
  Stats s = lanes_merge(r.stats(), 32);
  if (WPR > 1 && lane == 0) s_stats[warp] = s;
  int n = 0;
  Cand *all = s_all[group];
  if (k > 0) {
    // 64 of the threads' two largest maxima: the largest of every warp that read a batch
    const int active = WPR == 1 ? 1 : max(1, min(WPR, (n_vec - rank * WPR * LP_STEP + LP_STEP - 1) / LP_STEP));
    const int share = (64 + active - 1) / active;
    // (a first batch above -FLT_MAX leaves the start value of m as b2, behind which no batch
    // stands and which no logit need reach: i2 < 0)
    const int k1 = slot_key(r.m == -FLT_MAX ? -INFINITY : r.m, lane);
    const int k2 = slot_key(r.i2 < 0 ? -INFINITY : r.b2, 32 + lane);
    if (share == 64) {
      if (warp < active || WPR == 1) {
        s_max[group][lane] = k1;
        s_max[group][lane + 32] = k2;
      }
    } else if (warp < active) {
      top_keys(k1, k2, share, [&](int i, int best) {
        if (lane == 0 && warp * share + i < 64) s_max[0][warp * share + i] = best;
      });
    }
    sync();
    float bound = -INFINITY;
    top_keys((s_max[group][lane] & ~63) | lane, (s_max[group][lane + 32] & ~63) | (32 + lane), k,
             [&](int i, int best) { bound = key_value(best); });
    // No bound, or a thread with a fourth batch that reaches it: read the row again.
    const bool again = bound == -INFINITY || r.b4 >= bound;
    bool redo = WPR == 1 ? __any_sync(0xffffffffu, again) != 0 : __syncthreads_or(again) != 0;
    if (!redo) {
      const int step = parts * LP_STEP, first = part * LP_STEP + lane;
      auto need = [&](float max, int i) {
        if (!(max >= bound) || i < 0) return;
        const int at = atomicAdd(&s_batches[group], 1);
        if (at < CAP) s_batch[group][at] = first + i * step;
      };
      need(r.m, r.i1);
      need(r.b2, r.i2);
      need(r.b3, r.i3);
      sync();
      const int n_batch = min(s_batches[group], CAP);
      for (int i = WPR == 1 ? lane : threadIdx.x; i < n_batch; i += 32 * WPR)
        pick<T>(vec, s_batch[group][i], n_vec, head, bound, all, &s_n[group], CAP);
      sync();
      n = s_n[group];
      redo = n > CAP || s_batches[group] > CAP;
      sync();
    }
    if (redo) {
      if (WPR == 1 ? lane == 0 : threadIdx.x == 0) s_n[group] = 0;
      sync();
      const int mine =
          second_pass<T>(vec, part * LP_STEP, parts * LP_STEP, n_vec, head, k, bound, s_wait[warp]);
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_n[group], mine);
      at = __shfl_sync(0xffffffffu, at, 0);
      for (int i = lane; i < mine; i += 32) all[at + i] = s_wait[warp][i];
      sync();
      n = s_n[group];
    }
    if (has_ends && lane < n_ends && end >= bound) all[atomicAdd(&s_n[group], 1)] = Cand{end, end_id};  // never a NaN
    sync();
    n = s_n[group];
  } else if (WPR > 1) {
    __syncthreads();
  }
  if (WPR == 1) {
    finish_row<T, 32>(a, row, y, s, all, n);
    return;
  }
  s = lanes_merge(s_stats[lane & (LP_WARPS - 1)], LP_WARPS);
  if (a.cluster == 1) {
    finish_row<T, LP_THREADS>(a, row, y, s, all, n);
    return;
  }
  // The CTAs' tops and statistics meet in the cluster's first CTA.
  if (k > 0) {
    if (threadIdx.x < 32) s_first[threadIdx.x] = Cand{-INFINITY, INT_MAX};
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += LP_THREADS) {
      const Cand c = all[i];
      const int at = rank_of(c, all, n);
      if (at < k) s_first[at] = c;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) s_stats[0] = s;
  if (threadIdx.x == 0) s_n[0] = 0;
  __syncthreads();
  ptx::cluster_sync();
  if (rank == 0) {
    if (k > 0 && warp < a.cluster) {
      const uint32_t from = ptx::mapa_shared(ptx::smem_u32(&s_first[lane]), warp);
      Cand c;
      c.v = ptx::ld_cluster_f32(from);
      c.id = __float_as_int(ptx::ld_cluster_f32(from + 4));
      const unsigned mask = __ballot_sync(0xffffffffu, c.id != INT_MAX);
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_n[0], __popc(mask));
      at = __shfl_sync(0xffffffffu, at, 0);
      if (c.id != INT_MAX) all[at + __popc(mask & ((1u << lane) - 1u))] = c;
    }
    const uint32_t st = ptx::mapa_shared(ptx::smem_u32(&s_stats[0]), lane & (a.cluster - 1));
    s.m = ptx::ld_cluster_f32(st);
    s.z = ptx::ld_cluster_f32(st + 4);
    s.u = ptx::ld_cluster_f32(st + 8);
    s = lanes_merge(s, a.cluster);
    __syncthreads();
  }
  ptx::cluster_sync();  // no CTA leaves while its parts are read
  if (rank == 0) finish_row<T, LP_THREADS>(a, row, y, s, all, k > 0 ? s_n[0] : 0);
}

}  // namespace

template <typename T>
cudaError_t launch_token_logprobs(const T *logits, long long row_stride, const int *targets, int rows, int V,
                                  float *logprobs, float *entropy, int top_k, int *top_ids, float *top_logprobs,
                                  int *status, int bad_target, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const int sms = sm_count();
  LpArgs a;
  a.logits = logits;
  a.stride = row_stride;
  a.targets = targets;
  a.rows = rows;
  a.V = V;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_k = top_k;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.status = status;
  a.bad_target = bad_target;
  a.cluster = 1;
  constexpr int CTA_LOGITS = LP_THREADS * LP_VECS * Vec16<T>::N;  // one batch of a CTA
  count_launch();
  // A warp per row has no barriers and no idle warps, but it needs four times as many rows as
  // CTAs run at once, or as many times more as a row has batches of a CTA; and with a larger
  // top one of its lanes more often has four batches that reach the bound, and the row is
  // read again (warp / CTA per row: 8000 rows of 32000 bf16, top 1 96 / 135 us, top 20 207 /
  // 162; 3000 rows of 8000 fp32, top 20 34 / 41 us, 1300 rows 27 / 20).
  if (V <= 8 * CTA_LOGITS && (long long)rows * CTA_LOGITS >=
                                 (long long)sms * (V > CTA_LOGITS ? V : CTA_LOGITS) * (top_k > 4 ? top_k : 4)) {
    return launch_pdl(token_logprobs_kernel<T, 1>, dim3((unsigned)((rows + LP_WARPS - 1) / LP_WARPS)),
                      dim3(LP_THREADS), 0, st, a);
  }
  // Too few rows to fill the SMs: split each over a cluster, down to one batch per CTA, while
  // three CTAs per SM do not have work (four when parts are long; 64 rows of 128255 bf16: 10.1
  // us as 4 x 64 CTAs, 12.0 as 8 x 64; 304 rows of 128256 fp32: 33.7 us whole, 28.0 in two
  // parts) and all clusters run at once (76 rows of 128255 bf16: 15.7 us as clusters of
  // eight, two of which wait, 12.3 of four).
  static ClusterRoom room;
  for (int c = 2; c <= LP_MAX_CLUSTER && V / c >= CTA_LOGITS; c *= 2) {
    if ((long long)rows * c > (V / c >= 8 * CTA_LOGITS ? 4LL : 3LL) * sms ||
        rows > room.at_once(token_logprobs_kernel<T, LP_WARPS>, c, LP_THREADS, 0, 4 * sms))
      break;
    a.cluster = c;
  }
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = (unsigned)a.cluster;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  if ((long long)rows * a.cluster > 0x7fffffffLL) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)(rows * a.cluster));
  cfg.blockDim = dim3(LP_THREADS);
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, LP_WARPS>, a);
}

template cudaError_t launch_token_logprobs<float>(const float *, long long, const int *, int, int, float *, float *,
                                                  int, int *, float *, int *, int, cudaStream_t);
template cudaError_t launch_token_logprobs<bf16>(const bf16 *, long long, const int *, int, int, float *, float *, int,
                                                 int *, float *, int *, int, cudaStream_t);

}  // namespace llama
