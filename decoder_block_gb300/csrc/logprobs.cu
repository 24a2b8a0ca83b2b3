// Log-probabilities of given tokens, entropy and the likeliest tokens of logits
// rows ("The Evolving Transformer 04 · LLaMA", §07 Assemble: the logits of a
// position are the unnormalised log-probabilities of its next token).
//   m = max_v x_v, Z = sum_v e^(x_v - m):  ln p(v) = x_v - m - ln Z,
//   entropy = ln Z - sum_v e^(x_v - m) (x_v - m) / Z.
#include <limits.h>
#include <math.h>

#include "paged_kernels.h"

namespace llama {
namespace {

constexpr int LP_THREADS = 512;

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float *buf, F &&op) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < LP_THREADS / 32; ++w) v = op(v, buf[w]);
  __syncthreads();
  return v;
}

template <typename T>
__global__ void __launch_bounds__(LP_THREADS) token_logprobs_kernel(const T *__restrict__ logits, long long stride,
                                                                    const int *__restrict__ targets, int V,
                                                                    float *__restrict__ logprobs,
                                                                    float *__restrict__ entropy, int top_k,
                                                                    int *__restrict__ top_ids,
                                                                    float *__restrict__ top_logprobs, int *status, int bad_target) {
  __shared__ float buf[LP_THREADS / 32];
  __shared__ int ibuf[LP_THREADS / 32];
  const int row = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const T *x = logits + (size_t)row * stride;
  float m = -INFINITY;
  for (int v = threadIdx.x; v < V; v += LP_THREADS) m = fmaxf(m, to_f32<T>(x[v]));
  m = block_reduce(m, buf, [](float a, float b) { return fmaxf(a, b); });
  float z = 0.f, u = 0.f;
  if (m > -INFINITY)
    for (int v = threadIdx.x; v < V; v += LP_THREADS) {
      const float d = to_f32<T>(x[v]) - m, e = expf(d);
      z += e;
      u += d == -INFINITY ? 0.f : e * d;
    }
  else  // no logit above -inf; NaN still has to show
    for (int v = threadIdx.x; v < V; v += LP_THREADS)
      if (isnan(to_f32<T>(x[v]))) z = NAN;
  auto add = [](float a, float b) { return a + b; };
  z = block_reduce(z, buf, add);
  u = block_reduce(u, buf, add);
  const float log_z = logf(z);  // -inf for a row of nothing but -inf
  auto logprob = [&](float v) { return (m == -INFINITY && z == 0.f) ? -INFINITY : (v - m) - log_z; };
  if (threadIdx.x == 0) {
    if (logprobs != nullptr) {
      const int y = targets[row];
      if (y >= 0 && y < V) {
        logprobs[row] = logprob(to_f32<T>(x[y]));
      } else {
        logprobs[row] = y == -1 ? 0.f : NAN;
        if (y != -1) report_status(status, bad_target);
      }
    }
    if (entropy != nullptr) entropy[row] = (m == -INFINITY && z == 0.f) ? 0.f : log_z - u / z;
  }
  // top_k times the best logit behind the last one taken
  float last = INFINITY;
  int last_id = -1;
  for (int j = 0; j < top_k; ++j) {
    float best = -INFINITY;
    int id = INT_MAX;
    for (int v = threadIdx.x; v < V; v += LP_THREADS) {
      const float a = to_f32<T>(x[v]);
      if (!(a < last || (a == last && v > last_id))) continue;
      if (a > best || (a == best && v < id)) {
        best = a;
        id = v;
      }
    }
    auto merge = [&](float ob, int oi) {
      if (ob > best || (ob == best && oi < id)) {
        best = ob;
        id = oi;
      }
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      merge(__shfl_xor_sync(0xffffffffu, best, o), __shfl_xor_sync(0xffffffffu, id, o));
    if (lane == 0) {
      buf[warp] = best;
      ibuf[warp] = id;
    }
    __syncthreads();
    best = buf[0];
    id = ibuf[0];
    for (int w = 1; w < LP_THREADS / 32; ++w) merge(buf[w], ibuf[w]);
    __syncthreads();
    if (threadIdx.x == 0) {
      top_ids[(size_t)row * top_k + j] = id == INT_MAX ? -1 : id;
      top_logprobs[(size_t)row * top_k + j] = id == INT_MAX ? NAN : logprob(best);
    }
    last = id == INT_MAX ? -INFINITY : best;
    last_id = id;
  }
}

}  // namespace

template <typename T>
cudaError_t launch_token_logprobs(const T *logits, long long row_stride, const int *targets, int rows, int V,
                                  float *logprobs, float *entropy, int top_k, int *top_ids, float *top_logprobs,
                                  int *status, int bad_target, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  count_launch();
  token_logprobs_kernel<T><<<(unsigned)rows, LP_THREADS, 0, st>>>(logits, row_stride, targets, V, logprobs, entropy,
                                                                  top_k, top_ids, top_logprobs, status, bad_target);
  return cudaGetLastError();
}

template cudaError_t launch_token_logprobs<float>(const float *, long long, const int *, int, int, float *, float *,
                                                  int, int *, float *, int *, int, cudaStream_t);
template cudaError_t launch_token_logprobs<bf16>(const bf16 *, long long, const int *, int, int, float *, float *, int,
                                                 int *, float *, int *, int, cudaStream_t);

}  // namespace llama
