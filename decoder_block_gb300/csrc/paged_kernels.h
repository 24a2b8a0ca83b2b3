// Internal launch wrappers of the packed / paged operators (not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include <mutex>

#include "common.cuh"
#include "paged.cuh"

namespace llama {

// How many clusters of a kernel run at once on the current device, asked once per device
// and size.  A cluster's SMs are neighbours (one processing cluster of the GPU), so there
// are fewer than the number of SMs says: those left over in each hold smaller ones only.
class ClusterRoom {
 public:
  // slots: CTAs that run at once without clusters, for when the device cannot be asked
  template <typename K>
  int at_once(K kernel, int cluster, int threads, int smem, int slots) {
    int dev = 0;
    if (cluster <= 1 || cluster > MOST || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= DEVICES)
      return slots / cluster;
    std::lock_guard<std::mutex> lock(mutex_);
    int &n = known_[dev][cluster];
    if (n > 0) return n;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int found = 0;
    if ((smem > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) ||
        cudaOccupancyMaxActiveClusters(&found, kernel, &cfg) != cudaSuccess || found <= 0) {
      cudaGetLastError();
      return slots / cluster;
    }
    return n = found;
  }

 private:
  static constexpr int DEVICES = 64, MOST = 8;
  std::mutex mutex_;
  int known_[DEVICES][MOST + 1] = {};
};

// SMs of the current device, by which work is split and workspaces sized; 1 without a GPU.
inline int sm_count() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

// Budget of a wait in the packed and paged-decode attention kernels, in SM clock cycles
// (llama_op_set_wait_budget).
long long op_wait_cycles();

// RoPE on the q and k of packed rows and the write of k and v into their pages
// (paged_write.cu); halves as for launch_rope_kv.
template <typename T>
cudaError_t launch_rope_kv_paged(const T *qkv, T *q_out, T *k, T *v, const PagedView &pv, const PackedView &b,
                                 const float2 *table, int table_max_seq, int H, int G, int D, int halves, int *status,
                                 cudaStream_t st);

// Tensor maps (packed_tc.cu), 64 columns wide in the 128-byte swizzle: `box` rows of
// one page and KV head, coordinates (column, row in page, head, page); box_heads x
// box_rows of packed query rows [rows][H][D], coordinates (column, head, row).
bool make_paged_map(CUtensorMap *map, const bf16 *pool, const PagedView &pv, int G, int D, int box);
bool make_heads_map(CUtensorMap *map, const bf16 *q, int rows, int H, int D, int box_heads, int box_rows);

// Tensor-core attention of packed rows (packed_tc.cu).
size_t packed_tc_workspace_bytes(const PackedView &b, int H, int G, int D);
cudaError_t launch_packed_tc(const bf16 *q, const bf16 *k, const bf16 *v, bf16 *o, const PagedView &pv,
                             const PackedView &b, int H, int G, int D, void *workspace, int *status, cudaStream_t st);

// Tensor-core decode attention (paged_decode_tc.cu).
size_t paged_decode_tc_workspace_bytes(int n_seqs, int max_kv_len, int H, int G, int D);
cudaError_t launch_paged_decode_tc(const bf16 *q, const bf16 *k, const bf16 *v, bf16 *o, const PagedView &pv,
                                   const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int D,
                                   void *workspace, int *status, cudaStream_t st);

// fp32 attention over pages on CUDA cores (paged_simt.cu).
size_t packed_simt_workspace_bytes(const PackedView &b, int H, int G, int D);
cudaError_t launch_packed_simt(const float *q, const float *k, const float *v, float *o, const PagedView &pv,
                               const PackedView &b, int H, int G, int D, float *part, int *status, cudaStream_t st);
size_t paged_decode_simt_workspace_bytes(int n_seqs, int max_kv_len, int H, int G, int D);
cudaError_t launch_paged_decode_simt(const float *q, const float *k, const float *v, float *o, const PagedView &pv,
                                     const int *kv_lens, int n_seqs, int max_kv_len, int H, int G, int D, float *part,
                                     int *status, cudaStream_t st);

// Log-probabilities, entropy and top_k of logits rows (logprobs.cu); targets
// and logprobs may both be null, entropy too.  A target outside [0, V) other than
// -1 records the code bad_target.
template <typename T>
cudaError_t launch_token_logprobs(const T *logits, long long row_stride, const int *targets, int rows, int V,
                                  float *logprobs, float *entropy, int top_k, int *top_ids, float *top_logprobs,
                                  int *status, int bad_target, cudaStream_t st);

}  // namespace llama
