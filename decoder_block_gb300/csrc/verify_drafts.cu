// Keeps or replaces drafted tokens by the target's probabilities ("The Evolving
// Transformer 04 · LLaMA", §07 Assemble: the logits of a position are the unnormalised
// log-probabilities of its next token).  With p and q the target's and the draft's
// softmax, a draft x is kept with probability min(1, p[x] / q[x]) and otherwise replaced
// by one drawn from max(p - q, 0): what comes out is distributed as p.  Drawing is a race
// of exponential variates E: the id with the smallest E_v / w_v, the largest w_v / E_v,
// is v with probability w_v / sum w.  No running sum is needed for it, so nothing depends
// on the order in which a row's parts are added up, and its parts can be searched apart.
//
// How near p / q is: an exponent (x - m) log2(e) / T has four roundings, 2^-22 of its size, which
// is log2 V at most on average over a row's weights; p / q is off by ln 2 log2(V) 2^-22 (2.8e-6 for
// 128256 ids), 2^-22 for each exponential and 2^-24 for each of a thread's additions.  Measured over
// 4099 to 200003 ids: 6.5e-7 at most.
//
// Every logit has to be read once, and that bounds it.  Two kernels:
//   rows   a CTA takes a part of a row, target's or draft's, and leaves its maximum m,
//          sum of e^((x - m) / T) and, for greedy sequences, the id of m;
//   draw   a cluster takes a sequence: every CTA of it adds up the parts of its rows,
//          takes the decisions, and searches a part of the one row (with its draft's and
//          the noise) that the next token is drawn from.  The CTAs meet through
//          distributed shared memory.
// 64 sequences of four drafts over 128256 ids (fp32, with a draft's logits): 69.5 to 72 us, 43 of
// them the rows kernel at 6.2 TB/s (0.91 of the copy rate); in the draw kernel the decisions take
// 3 us, the search the rest.
// Rows behind the first refused draft are summed in vain: knowing it first would take a
// chain of kernels as long as the drafts, each too small to fill the GPU.
#include <float.h>
#include <limits.h>
#include <math.h>
#include <string.h>

#include "paged_kernels.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int VD_THREADS = 256;
constexpr int VD_WARPS = VD_THREADS / 32;
constexpr int VD_MOST_THREADS = 768;  // of a CTA that draws
constexpr int VD_VECS = 4;          // 16-byte vectors of a thread in flight
// CTAs of an SM, and CTAs for an SM that the parts aim at: 265 MB in 42.9 us by itself, 0.91 of the
// measured rate (4 and 32: 45.2, 6 and 16: 43.5, 4 and 16: 43.5; rows left in L2 for the drawing, by
// loads that do not say that they are the last: 74 to 77 us in all for 71).  With bf16 logits 40
// registers spill 28 bytes: 64 x 4 drafts 62 us.
constexpr int VD_CTAS = 6, VD_AIM = 32;
constexpr int VD_RACE = 2;          // of each of a race's rows
constexpr int VD_MAX_PARTS = 32;    // of a row: a lane each when they are added up
constexpr int VD_MIN_PART = 4096;   // logits of a part, at least
// Ids of a CTA of a cluster, at least: while SMs are idle, and above that.  (6 and 3 sequences of
// 22085 and 12828 ids: 15.8 and 13.9 us at 1024, 15.8 and 14.5 at 2048, 16.9 and 16.1 at 4096, 20.9 and
// 17.5 at 8192; 197 sequences of 2833: 19.0 at 1024, 17.6 at 2048.)
constexpr int VD_MIN_RACE = 1024, VD_MIN_RACE_BUSY = 4096;
constexpr int VD_MAX_CLUSTER = 8;
constexpr float VD_LOG2E = 1.4426950408889634f;

struct VdPart {
  float m, z;  // largest logit that is not NaN (-FLT_MAX at least); z: NaN where the row holds NaN or +inf
  int id;      // of m (greedy alone)
  int pad;
};

struct VdArgs {
  const void *target, *draft;
  long long target_stride, seq_stride, step_stride;
  int V;
  const int *q_offsets, *tokens;
  const float *temperatures, *uniforms, *noise;
  long long noise_stride;
  int n_seqs, n_rows, max_drafts;
  int parts;    // of a row
  VdPart *part; // [n_rows][2: target, draft][parts]
  int *out_tokens, *n_accepted;
  float *logprobs;
  int *status;
  int cluster;
};

__device__ __forceinline__ float ld_float_after_wait(const float *p) {
  return __int_as_float(ld_after_wait(reinterpret_cast<const int *>(p)));
}
template <typename T> __device__ __forceinline__ float ld_logit(const T *p);
template <> __device__ __forceinline__ float ld_logit<float>(const float *p) { return ld_float_after_wait(p); }
template <> __device__ __forceinline__ float ld_logit<bf16>(const bf16 *p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return __uint_as_float((uint32_t)v << 16);
}

// Temperature of sequence i; 0: greedy.  (Denormals divide to infinities.)
__device__ __forceinline__ float temperature_of(const VdArgs &a, int i) {
  if (a.noise == nullptr) return 0.f;
  if (a.temperatures == nullptr) return 1.f;
  const float t = ld_float_after_wait(a.temperatures + i);
  return fabsf(t) < FLT_MIN ? 0.f : t;
}
__device__ __forceinline__ bool temperature_ok(float t) { return t >= 0.f && t <= FLT_MAX; }

// Rows of sequence i: n < 0 when they are out of range.
__device__ __forceinline__ void rows_of(const VdArgs &a, int i, int &first, int &n) {
  first = ld_after_wait(a.q_offsets + i);
  const int end = ld_after_wait(a.q_offsets + i + 1);
  n = first >= 0 && end >= first && end <= a.n_rows && end - first <= a.max_drafts + 1 ? end - first : -1;
}

// (maximum, sum) of two parts; c: log2(e) / T.
__device__ __forceinline__ void merge(float &m, float &z, float om, float oz, float c) {
  const float up = fmaxf(m, om);
  z = z * ptx::ex2_approx((m - up) * c) + oz * ptx::ex2_approx((om - up) * c);
  m = up;
}

// ------------------------------------------------------------------ rows ---
template <typename T, bool GREEDY>
struct VdScan {
  float m = -FLT_MAX, z = 0.f;  // finite: -inf alone leaves weights of 0
  int at = -1;                  // greedy: first batch that has the maximum
  // N logits, a batch or some that are in no whole vector.
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float c, int batch) {
    float bm = x[0];
#pragma unroll
    for (int e = 1; e < N; ++e) bm = fmaxf(bm, x[e]);
    if (GREEDY && bm >= m && (bm > m || at < 0)) at = batch;
    if (bm > m) {
      z *= ptx::ex2_approx((m - bm) * c);
      m = bm;
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < N; ++e) s[e & 3] += ptx::ex2_approx((x[e] - m) * c);
    z += (s[0] + s[1]) + (s[2] + s[3]);
  }
};

// Part `part` of a row: this thread's (m, z, id of m).
template <typename T, bool GREEDY>
__device__ __forceinline__ void scan_part(const T *x, int V, int part, int parts, float c, float &m, float &z, int &id) {
  constexpr int N = Vec16<T>::N;
  const int head0 = (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T);
  const int head = head0 < V ? head0 : V;  // logits in front of the first whole vector
  const int n_vec = (V - head) / N, rest = V - head - n_vec * N;
  const T *body = x + head;
  const int v0 = (int)((long long)n_vec * part / parts), v1 = (int)((long long)n_vec * (part + 1) / parts);
  VdScan<T, GREEDY> s;
  for (int v = v0; v < v1; v += VD_VECS * VD_THREADS) {
    Vec16<T> w[VD_VECS];
#pragma unroll
    for (int k = 0; k < VD_VECS; ++k) {
      const int at = v + k * VD_THREADS + (int)threadIdx.x;
      if (at < v1) {
        w[k].raw = ld_once_after_wait(body + (size_t)at * N);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) w[k].set(e, -INFINITY);
      }
    }
    float f[VD_VECS * N];
#pragma unroll
    for (int k = 0; k < VD_VECS; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e) f[k * N + e] = w[k].get(e);
    s.add(f, c, v);
  }
  id = INT_MAX;
  if (GREEDY && s.at >= 0) {  // the batch again, for the place of its maximum
#pragma unroll 1
    for (int k = VD_VECS - 1; k >= 0; --k) {
      const int at = s.at + k * VD_THREADS + (int)threadIdx.x;
      if (at >= v1) continue;
      const Vec16<T> w = load16<T>(body + (size_t)at * N);
#pragma unroll
      for (int e = N - 1; e >= 0; --e)
        if (w.get(e) == s.m) id = head + at * N + e;
    }
  }
  m = s.m;
  z = s.z;
  // the ends: one logit of each of the first part's first threads
  if (part == 0 && (int)threadIdx.x < head + rest) {
    const int at = (int)threadIdx.x < head ? threadIdx.x : V - rest + (int)threadIdx.x - head;
    const float f = ld_logit<T>(x + at);
    if (GREEDY && (f > m || (f == m && at < id))) id = at;
    if (f > m) {
      z *= ptx::ex2_approx((m - f) * c);
      m = f;
    }
    z += ptx::ex2_approx((f - m) * c);
  }
}

template <typename T>
__global__ void __launch_bounds__(VD_THREADS, VD_CTAS) verify_rows_kernel(const __grid_constant__ VdArgs a) {
  __shared__ float s_m[VD_WARPS], s_z[VD_WARPS];
  __shared__ int s_id[VD_WARPS];
  allow_dependents_launch();
  grid_dependency_wait();
  const int part = blockIdx.x % a.parts, side = blockIdx.x / a.parts % 2, row = blockIdx.x / a.parts / 2;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  PackedView b;
  b.q_offsets = a.q_offsets;
  b.n_seqs = a.n_seqs;
  b.n_tokens = a.n_rows;
  const int seq = find_seq(b, row);  // (every warp for itself)
  if (seq < 0) return;
  int first, n;
  rows_of(a, seq, first, n);
  const float t = temperature_of(a, seq);
  if (n < 0 || !temperature_ok(t)) return;
  const T *x;
  if (side == 0) {
    x = reinterpret_cast<const T *>(a.target) + (size_t)row * a.target_stride;
  } else {
    if (a.draft == nullptr || t == 0.f || row - first >= n - 1) return;
    x = reinterpret_cast<const T *>(a.draft) + (size_t)seq * a.seq_stride + (size_t)(row - first) * a.step_stride;
  }
  const float c = t == 0.f ? VD_LOG2E : VD_LOG2E / t;
  float m, z;
  int id = INT_MAX;
  if (t == 0.f) scan_part<T, true>(x, a.V, part, a.parts, c, m, z, id);
  else scan_part<T, false>(x, a.V, part, a.parts, c, m, z, id);
  auto join = [&](float om, float oz, int oid) {
    if (om > m) id = oid;
    else if (om == m) id = min(id, oid);
    merge(m, z, om, oz, c);
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_down_sync(0xffffffffu, m, o), oz = __shfl_down_sync(0xffffffffu, z, o);
    const int oid = __shfl_down_sync(0xffffffffu, id, o);
    join(om, oz, oid);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_z[warp] = z;
    s_id[warp] = id;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < VD_WARPS; ++w) join(s_m[w], s_z[w], s_id[w]);
  a.part[((size_t)row * 2 + side) * a.parts + part] = VdPart{m, z, id, 0};
}

// ------------------------------------------------------------------ draw ---
// This lane's part of a row.
__device__ __forceinline__ VdPart load_part(const VdArgs &a, int row, int side, bool there = true) {
  const int lane = threadIdx.x & 31;
  VdPart p{-FLT_MAX, 0.f, INT_MAX, 0};
  if (there && lane < a.parts) {
    const int4 v = ld_after_wait(reinterpret_cast<const int4 *>(a.part + ((size_t)row * 2 + side) * a.parts + lane));
    p = VdPart{__int_as_float(v.x), __int_as_float(v.y), v.z, 0};
  }
  return p;
}
// The row's (m, z, id), from the lanes' parts, in every lane.
__device__ __forceinline__ VdPart sum_parts(VdPart p, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, p.m, o), oz = __shfl_xor_sync(0xffffffffu, p.z, o);
    const int oid = __shfl_xor_sync(0xffffffffu, p.id, o);
    if (om > p.m) p.id = oid;
    else if (om == p.m) p.id = min(p.id, oid);
    merge(p.m, p.z, om, oz, c);
  }
  // (the lanes add in different orders)
  p.z = __shfl_sync(0xffffffffu, p.z, 0);
  return p;
}
__device__ __forceinline__ bool row_ok(float z) { return z > 0.f && z <= FLT_MAX; }

// N elements side by side, whatever their alignment (bytes, 16 at most): rows of an odd
// vocabulary begin anywhere, and differently in each array.
template <typename E, int N>
__device__ __forceinline__ void load_group(const E *p, int align, E (&x)[N]) {
  static_assert(N * sizeof(E) % 16 == 0, "whole vectors");
  constexpr int WORDS = N * (int)sizeof(E) / 4;
  uint32_t w[WORDS];
  if (align >= 16) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const uint4 v = ld_once_after_wait(reinterpret_cast<const char *>(p) + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if (align == 8) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 2)
      asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];"
                   : "=r"(w[i]), "=r"(w[i + 1])
                   : "l"(reinterpret_cast<const char *>(p) + 4 * i));
  } else if (align == 4) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = (uint32_t)ld_after_wait(reinterpret_cast<const int *>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      uint16_t a, b;
      asm volatile("ld.global.u16 %0, [%1];" : "=h"(a) : "l"(reinterpret_cast<const char *>(p) + 4 * i));
      asm volatile("ld.global.u16 %0, [%1];" : "=h"(b) : "l"(reinterpret_cast<const char *>(p) + 4 * i + 2));
      w[i] = (uint32_t)a | (uint32_t)b << 16;
    }
  }
  memcpy(x, w, sizeof(w));
}
__device__ __forceinline__ int align_of(const void *p) {
  const uint32_t low = (uint32_t)reinterpret_cast<uintptr_t>(p) | 16u;
  return (int)(low & (0u - low));
}

// The best so far of a race; of equals the lowest id.
struct VdBest {
  float score;
  int id;
  __device__ __forceinline__ void join(float s, int i) {
    if (s > score || (s == score && i < id)) {
      score = s;
      id = i;
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(VD_MOST_THREADS) verify_draw_kernel(const __grid_constant__ VdArgs a) {
  constexpr int MOST = LLAMA_MAX_DRAFTS + 1;
  __shared__ float s_m[2][MOST], s_z[2][MOST];
  __shared__ int s_id[MOST];
  __shared__ bool s_keep[MOST];
  __shared__ VdBest s_best[VD_MOST_THREADS / 32];
  __shared__ VdBest s_cta[3][VD_MAX_CLUSTER];  // every CTA's, of each search
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, threads = blockDim.x, warps = threads / 32;
  const int seq = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  if (a.cluster > 1) ptx::cluster_sync();  // every CTA runs: the first one's shared memory may be written
  grid_dependency_wait();
  int first, n;
  rows_of(a, seq, first, n);
  const float t = temperature_of(a, seq);
  const bool fine = n >= 0 && temperature_ok(t);
  if (!fine && rank == 0 && threadIdx.x == 0) report_status(a.status, LLAMA_ERR_RANGE);
  const int width = a.max_drafts + 1;
  int kept = 0, token = -1;
  if (fine && n > 0) {  // the same in every CTA of the cluster
    const bool greedy = t == 0.f;
    const float c = greedy ? VD_LOG2E : VD_LOG2E / t;
    // This CTA's share of the noise, which does not wait for the decisions, into L2, a piece for each
    // lane; behind the loads that the decisions wait for.
    auto ask_for_noise = [&] {
      const long long ids = ((long long)a.V + 32 * a.cluster - 1) / (32 * a.cluster);
      const long long from = (rank * 32 + lane) * ids, to = min((long long)a.V, from + ids);
      const uintptr_t p = reinterpret_cast<uintptr_t>(a.noise + (size_t)seq * a.noise_stride);
      const uintptr_t b0 = (p + 4 * (uintptr_t)from + 15) & ~uintptr_t(15);
      const uintptr_t b1 = (p + 4 * (uintptr_t)max(from, to)) & ~uintptr_t(15);
      if (b1 > b0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(b0), "r"((uint32_t)(b1 - b0)) : "memory");
    };
    // (loads first, as far as they are known: each takes about as long as all else here)
    for (int k = warp; k < n; k += warps) {
      const bool has_draft = a.draft != nullptr && !greedy && k + 1 < n, random = k + 1 < n && !greedy;
      const int x = k + 1 < n ? ld_after_wait(a.tokens + first + k + 1) : 0;
      const float u = random ? ld_float_after_wait(a.uniforms + (size_t)seq * a.max_drafts + k) : 0.f;
      VdPart p = load_part(a, first + k, 0), q = load_part(a, first + k, 1, has_draft);
      const bool in = x >= 0 && x < a.V;
      float fx = 0.f, fy = 0.f;
      if (random && in) {
        fx = ld_logit<T>(reinterpret_cast<const T *>(a.target) + (size_t)(first + k) * a.target_stride + x);
        if (has_draft)
          fy = ld_logit<T>(reinterpret_cast<const T *>(a.draft) + (size_t)seq * a.seq_stride + (size_t)k * a.step_stride + x);
      }
      if (!greedy && k == 0) ask_for_noise();
      p = sum_parts(p, c);
      if (has_draft) q = sum_parts(q, c);
      if (lane == 0) {
        s_m[0][k] = p.m;
        s_z[0][k] = p.z;
        s_m[1][k] = q.m;
        const float zq = has_draft && row_ok(q.z) ? q.z : 0.f;  // 0: the draft was certain
        s_z[1][k] = zq;
        s_id[k] = p.id;
        if (k + 1 < n) {
          bool keep = false;
          if (!in) {
            if (rank == 0) report_status(a.status, LLAMA_ERR_RANGE);
          } else if (row_ok(p.z)) {
            if (greedy) {
              keep = x == p.id;
            } else {
              // p / q = e^((x - m) / T - (y - m_q) / T) z_q / z, the exponent in fp64 and what its
              // fp32 part leaves of it as a factor
              double d = (double)fx - (double)p.m, z = p.z;
              if (zq > 0.f) {
                d -= (double)fy - (double)q.m;
                z /= zq;
              }
              d /= (double)t;
              const float hi = (float)d, lo = (float)(d - (double)hi);
              const double ratio = (double)expf(hi) * (fabsf(hi) <= FLT_MAX ? 1.0 + (double)lo : 1.0);
              keep = (double)u * z < ratio;
            }
          }
          s_keep[k] = keep;
        }
      }
    }
    __syncthreads();
    while (kept + 1 < n && s_keep[kept]) ++kept;
    const bool refused = kept + 1 < n;
    const float z = s_z[0][kept];
    if (greedy) {
      // (offsets that descend may leave rows that no CTA has summed: any id may stand there)
      token = row_ok(z) && (unsigned)s_id[kept] < (unsigned)a.V ? s_id[kept] : -1;
    } else if (row_ok(z)) {
      const T *x = reinterpret_cast<const T *>(a.target) + (size_t)(first + kept) * a.target_stride;
      const float *noise = a.noise + (size_t)seq * a.noise_stride;
      const bool both = refused && s_z[1][kept] > 0.f;
      const T *y = both ? reinterpret_cast<const T *>(a.draft) + (size_t)seq * a.seq_stride + (size_t)kept * a.step_stride
                        : nullptr;
      const int banned = refused && !both ? ld_after_wait(a.tokens + first + kept + 1) : -1;
      const float m = s_m[0][kept], mq = s_m[1][kept], inv = 1.f / z, inv_q = both ? 1.f / s_z[1][kept] : 0.f;
      VdBest best{0.f, INT_MAX};  // in the end the CTA's, in its first warp
      // What cannot beat the best so far is found without a division: `bar` is a little below it.
      float bar = 0.f;
      auto race = [&](float fx, float fy, float e, int id, bool residual) {
        const float p = ptx::ex2_approx((fx - m) * c) * inv;
        float w = p;
        if (residual && both) w = p - ptx::ex2_approx((fy - mq) * c) * inv_q;
        if (residual && id == banned) w = 0.f;
        if (w > bar * e && e > 0.f) {  // (0 does not win: ids start behind every other)
          const float s = w / e;
          if (s > best.score) {
            best.score = s;
            best.id = id;
            bar = s * (1.f - 0x1p-21f);
          }
        }
      };
      constexpr int N = Vec16<T>::N;
      const int ax = align_of(x), ay = both ? align_of(y) : 16, ae = align_of(noise);
      const int stride = a.cluster * threads, me = rank * threads + (int)threadIdx.x;
      auto search = [&](bool residual) {
        const int groups = a.V / N;
        for (int v = me; v < groups; v += VD_RACE * stride) {
          T fx[VD_RACE][N], fy[VD_RACE][N];
          float e[VD_RACE][N];
#pragma unroll
          for (int k = 0; k < VD_RACE; ++k) {
            const int at = v + k * stride;
            if (at >= groups) continue;
            load_group(x + (size_t)at * N, ax, fx[k]);
            if (both) load_group(y + (size_t)at * N, ay, fy[k]);
            load_group(noise + (size_t)at * N, ae, e[k]);
          }
#pragma unroll
          for (int k = 0; k < VD_RACE; ++k) {
            const int at = v + k * stride;
            if (at >= groups) continue;
#pragma unroll
            for (int i = 0; i < N; ++i)
              race(to_f32<T>(fx[k][i]), both ? to_f32<T>(fy[k][i]) : 0.f, e[k][i], at * N + i, residual);
          }
        }
        const int at = groups * N + me;  // what is left of the row
        if (at < a.V)
          race(ld_logit<T>(x + at), both ? ld_logit<T>(y + at) : 0.f, ld_float_after_wait(noise + at), at, residual);
      };
      // the CTA's best into every CTA's array, through distributed shared memory
      auto publish = [&](int which) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float s = __shfl_xor_sync(0xffffffffu, best.score, o);
          const int i = __shfl_xor_sync(0xffffffffu, best.id, o);
          best.join(s, i);
        }
        if (lane == 0) s_best[warp] = best;
        __syncthreads();
        if (warp == 0) {
          best = s_best[lane < warps ? lane : 0];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float s = __shfl_xor_sync(0xffffffffu, best.score, o);
            const int i = __shfl_xor_sync(0xffffffffu, best.id, o);
            best.join(s, i);
          }
        }
        __syncthreads();  // (the next search writes there again)
        if (threadIdx.x < a.cluster) {
          uint32_t dst = ptx::smem_u32(&s_cta[which][rank]);
          if (a.cluster > 1) dst = ptx::mapa_shared(dst, threadIdx.x);
          ptx::st_cluster_u32(dst, __float_as_uint(best.score));
          ptx::st_cluster_u32(dst + 4, (uint32_t)best.id);
        }
        if (a.cluster > 1) ptx::cluster_sync();
        else __syncthreads();
      };
      search(true);
      publish(0);
      int last = 0;
      if (refused) {  // (in every CTA of the cluster alike)
        auto nobody_won = [&](int which) {
          float top = 0.f;
          for (int k = 0; k < a.cluster; ++k) top = fmaxf(top, s_cta[which][k].score);
          return top == 0.f;
        };
        // Either p - q is 0 everywhere, and the token is drawn from p, or no id that it leaves may be
        // drawn, and there is no token: a race without the noise tells.  (Rare: an id at a time, in
        // few registers.)
#pragma unroll 1
        for (int which = 1; which <= 2 && nobody_won(which - 1); ++which) {
#pragma unroll 1
          for (int at = me; at < a.V; at += stride)
            race(ld_logit<T>(x + at), both ? ld_logit<T>(y + at) : 0.f,
                 which == 1 ? 1.f : ld_float_after_wait(noise + at), at, which == 1);
          publish(which);
          last = which == 2 ? 2 : 0;
        }
      }
      if (rank == 0) {
        VdBest all = s_cta[last][0];
        for (int k = 1; k < a.cluster; ++k) all.join(s_cta[last][k].score, s_cta[last][k].id);
        token = all.score > 0.f ? all.id : -1;
      }
    }
  }
  if (rank != 0) return;
  for (int k = threadIdx.x; k < width; k += threads) {
    int x = -1;
    float lp = 0.f;
    if (k < kept) x = ld_after_wait(a.tokens + first + k + 1);
    else if (k == kept) x = token;
    if (x >= 0 && a.logprobs != nullptr) {
      const T *row = reinterpret_cast<const T *>(a.target) + (size_t)(first + k) * a.target_stride;
      lp = (ld_logit<T>(row + x) - s_m[0][k]) / (t == 0.f ? 1.f : t) - logf(s_z[0][k]);
    }
    a.out_tokens[(size_t)seq * width + k] = x;
    if (a.logprobs != nullptr) a.logprobs[(size_t)seq * width + k] = lp;
  }
  if (threadIdx.x == 0) a.n_accepted[seq] = kept;
}

// Parts of a row: enough CTAs to fill the GPU several times over, none with less than
// VD_MIN_PART logits.
int parts_of(int n_rows, int V) {
  const long long aim = (long long)VD_AIM * sm_count(), want = (aim + 2LL * n_rows - 1) / (2LL * n_rows);
  const int most = V / VD_MIN_PART < VD_MAX_PARTS ? V / VD_MIN_PART : VD_MAX_PARTS;
  return want < most ? (int)want : most > 1 ? most : 1;
}

}  // namespace

size_t verify_drafts_workspace_bytes(int n_rows, int V) {
  return n_rows == 0 ? 0 : (size_t)n_rows * 2 * parts_of(n_rows, V) * sizeof(VdPart);
}

template <typename T>
cudaError_t launch_verify_drafts(const T *target, long long target_stride, const T *draft, long long seq_stride,
                                 long long step_stride, int V, const llama_draft_batch &b, int *out_tokens,
                                 int *n_accepted, float *logprobs, void *workspace, int *status, cudaStream_t st) {
  VdArgs a;
  a.target = target;
  a.draft = draft;
  a.target_stride = target_stride;
  a.seq_stride = seq_stride;
  a.step_stride = step_stride;
  a.V = V;
  a.q_offsets = b.q_offsets;
  a.tokens = b.tokens;
  a.temperatures = b.temperatures;
  a.uniforms = b.uniforms;
  a.noise = b.noise;
  a.noise_stride = b.noise_stride;
  a.n_seqs = b.n_seqs;
  a.n_rows = b.n_rows;
  a.max_drafts = b.max_drafts;
  a.part = reinterpret_cast<VdPart *>(workspace);
  a.out_tokens = out_tokens;
  a.n_accepted = n_accepted;
  a.logprobs = logprobs;
  a.status = status;
  a.parts = 1;
  if (b.n_rows > 0) {
    a.parts = parts_of(b.n_rows, V);
    count_launch();
    const cudaError_t e = launch_pdl(verify_rows_kernel<T>, dim3((unsigned)(b.n_rows * 2LL * a.parts)),
                                     dim3(VD_THREADS), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  a.cluster = 1;
  for (int c = 2; c <= VD_MAX_CLUSTER; c *= 2) {
    const long long ctas = (long long)c * b.n_seqs;
    if (ctas > 4 * sm_count() || V / c < (ctas <= sm_count() ? VD_MIN_RACE : VD_MIN_RACE_BUSY)) break;
    a.cluster = c;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(b.n_seqs * a.cluster));
  // few sequences: a thread for each vector (8 sequences of 35468 ids 17.0 -> 15.4 us, 3 of 12828
  // 13.2 -> 12.4; 1024 threads, where a row has as many: two sequences of 49152 12.0 for 11.5)
  const int vectors = V / (a.cluster * (16 / (int)sizeof(T)));
  int threads = VD_THREADS;
  if (b.noise != nullptr && b.n_seqs * a.cluster <= sm_count()) {
    while (threads < vectors && threads < VD_MOST_THREADS) threads += VD_THREADS;
  }
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, verify_draw_kernel<T>, a);
}

template cudaError_t launch_verify_drafts<float>(const float *, long long, const float *, long long, long long, int,
                                                 const llama_draft_batch &, int *, int *, float *, void *, int *,
                                                 cudaStream_t);
template cudaError_t launch_verify_drafts<bf16>(const bf16 *, long long, const bf16 *, long long, long long, int,
                                                const llama_draft_batch &, int *, int *, float *, void *, int *,
                                                cudaStream_t);

}  // namespace llama
