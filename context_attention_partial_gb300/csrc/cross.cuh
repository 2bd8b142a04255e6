// cross.cuh -- parameters of the cross-attention kernels and what they share
// (not part of the public ABI).
#pragma once
#include <atomic>
#include <cmath>

#include "internal.h"

namespace cpattn {

// A [B, H, S, D] (or, for lse, [B, H, S]) tensor: strides (b, h, s) in elements.
struct CrossTensor {
  void* data;
  int64_t s[3];
  Span span;   // (CPATTN_CHECK builds)
};

struct CrossParams {
  CrossTensor q, k, v, out, lse;
  CrossTensor dout, dq, dk, dv;      // backward
  const int32_t* lengths;            // [B] valid keys, or nullptr: s_kv everywhere
  Span lengths_span;
  float* ws;                         // workspace (see the launches)
  Span ws_span;
  int batch, heads, kv_heads, s_q, s_kv;
  float scale, scale_log2;           // softmax scale, and times log2(e)
  int splits;                        // forward: parts of the key axis (1: no join)
                                     // backward: parts of the query axis for dk, dv
  unsigned long long timeout_ns;
  int fault_skip_kv;                 // testing: the producer issues no copies
  unsigned int* err;                 // device error word
};

// A value that is the same in every lane, passed through a shuffle so that the
// compiler knows it: loops and addresses that depend on it then stay in
// uniform registers (whole warps only).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Valid keys of batch b: the given length, brought into [0, s_kv].
__device__ __forceinline__ int cross_length(const CrossParams& p, int b) {
  if (p.lengths == nullptr) return p.s_kv;
  const int32_t* at = p.lengths + b;
  const int n = CPATTN_IN(p.lengths_span, at, 4, p.err) ? *at : 0;
  return max(0, min(n, p.s_kv));
}

// A row's lse in base 2, as the gradients subtract it.  A row whose scores are all
// -inf has lse -inf and no weights: against +inf its exponentials are 0.
__device__ __forceinline__ float cross_lse2(float lse) {
  return lse == -INFINITY ? INFINITY : lse * 1.442695040888963407f;
}

// Raises a kernel's dynamic shared-memory limit once per device (bit d of
// `ready`: device d is set up; the call costs about 5 us of host time).  A kernel
// that splits its registers between its warps needs exactly `regs` at launch and
// is refused otherwise.
template <typename K>
cudaError_t cross_set_up(K kernel, size_t smem, std::atomic<unsigned long long>& ready, int regs = 0) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit != 0 && (ready.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  if (regs > 0) {
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
    if (attr.numRegs != regs) return cudaErrorInvalidConfiguration;
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Launches `kernel` on blocks x splits blocks (one instantiation, so one set-up
// record, per kernel).
template <auto kernel, typename... Args>
cudaError_t cross_run(int64_t blocks, int splits, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
  static std::atomic<unsigned long long> ready{0};
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const cudaError_t e = cross_set_up(kernel, smem, ready);
  if (e != cudaSuccess) return e;
  return launch_behind(kernel, dim3(static_cast<unsigned>(blocks), splits), threads, smem, stream, args...);
}

// Clusters of `size` blocks of a kernel that the idle current device holds at
// once; -1 if that cannot be asked (no device).
template <typename... Params>
int cross_clusters(void (*kernel)(Params...), dim3 cluster, int threads, size_t smem) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  cudaLaunchConfig_t config = {};
  config.gridDim = cluster;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster.x;
  attr.val.clusterDim.y = cluster.y;
  attr.val.clusterDim.z = cluster.z;
  config.attrs = &attr;
  config.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &config) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return n;
}
// The same for the two bf16 forward kernels at D = 128 (one block an SM, and two).
int cross_fwd_clusters(int size);
int cross_few_clusters(int size);

// Blocks of a cluster, at most.  bf16 forward calls have p.splits up to it, or a
// multiple of it: a cluster joins its parts itself, and the workspace gets
// p.splits / kCrossCluster parts to join.
constexpr int kCrossCluster = 8;
// bf16 inputs, D 64 or 128, on the tensor cores (s_kv >= 1; the maps' boxes
// have 128 rows, the output's 32).
cudaError_t launch_cross_fwd(int head_dim, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, const CUtensorMap& tm_o, const CrossParams& p,
                             cudaStream_t stream);
// the same for at most 64 query rows a key head (s_q * H / H_kv)
cudaError_t launch_cross_few(int head_dim, const CrossParams& p, cudaStream_t stream);
// its gradient (s_q, s_kv >= 1; the kernels write delta to the workspace's start
// and, when p.splits > 1, partial sums of dk and dv `partials` floats into it;
// the outputs' maps have boxes of 32 rows, dq's of 32 columns, dense, at D = 64)
struct CrossBwdMaps {
  CUtensorMap q, k, v, out, dout, dq, dk, dv;
};
cudaError_t launch_cross_bwd(int head_dim, const CrossBwdMaps& maps, const CrossParams& p, int64_t partials,
                             cudaStream_t stream);
// parts of the query axis for key_units 128-key tiles that walk `steps`
// 128-row query tiles each
int cross_backward_parts(int64_t key_units, int64_t steps);
// fp32 inputs (D 64 or 128; s_q, s_kv >= 1); the gradient keeps delta, [B, H, S_q],
// at the workspace's start, and, when p.splits > 1, partial sums of dk and dv
// `partials` floats into it.
cudaError_t launch_cross_simt(int head_dim, const CrossParams& p, cudaStream_t stream);
cudaError_t launch_cross_simt_backward(int head_dim, const CrossParams& p, int64_t partials, cudaStream_t stream);
// whether fp32 calls with that many 64-row query blocks, which walk `values`
// elements of a key head (S_kv D), or 64 x 64 tiles of dk and dv, take 64-row blocks
bool cross_f32_rows(int64_t blocks, int64_t values);
bool cross_f32_keys(int64_t tiles);
// parts of the query axis for key_units 64-key tiles that walk `steps` 64-row
// query tiles each
int cross_f32_parts(int64_t key_units, int64_t steps);
// the same in 64-row blocks, for calls with many rows (dq takes no splits)
cudaError_t launch_cross_f32(int head_dim, const CrossParams& p, cudaStream_t stream);
cudaError_t launch_cross_f32_dq(int head_dim, const CrossParams& p, cudaStream_t stream);
cudaError_t launch_cross_f32_dkv(int head_dim, const CrossParams& p, int64_t partials, cudaStream_t stream);
// adds up p.splits partial sums of dk and dv
cudaError_t launch_cross_dkv_join(InDtype dt, int head_dim, const CrossParams& p, int64_t partials, cudaStream_t stream);
// dq, dk, dv = 0 (no queries, or no keys).
cudaError_t launch_cross_zeros(InDtype dt, int head_dim, const CrossParams& p, cudaStream_t stream);
// joins p.splits partial outputs of the workspace into out and lse
cudaError_t launch_cross_join(InDtype dt, int head_dim, const CrossParams& p, cudaStream_t stream);

}  // namespace cpattn
