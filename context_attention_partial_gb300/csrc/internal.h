// internal.h -- declarations shared by the translation units of libcpattn.so
// (not part of the public ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/cpattn.h"
#include "check.cuh"

namespace cpattn {

// Parameters of one attention launch (ring or single partial).
struct AttnParams {
  void* out;             // [B, H, S_q, D], f32 or the input dtype
  int64_t out_sb, out_sh, out_ss;
  float* lse;            // [B, H, S_q] f32
  int64_t lse_sb, lse_sh, lse_ss;
  // running merged partial (ring_degree > 1), per 128-row query tile t of
  // the B*H*ceil(S_q/128) tiles: ws_o f32 [t][D/4][128 rows][4] (a warp's
  // float4 accesses at one column group are 512 contiguous bytes), ws_lse
  // f32 [t][128 rows]
  float* ws_o;
  float* ws_lse;
  int batch, heads, s_q, s_kv;
  float scale_log2;      // softmax scale times log2(e)
  int ring_degree;
  int out_f32;           // 1: out is f32, 0: out has the input dtype (bf16)
  unsigned long long timeout_ns;
  int fault_skip_kv;     // testing: the producer issues no K/V loads
  int causal;            // 1: query i attends keys j <= i (is_causal)
  // Ulysses Anything: 0, or G when the batch axis is (group, batch) and the
  // head axis holds ceil(H/G) slots of which group g fills its first h_g
  // (tensor_split sizes of group_heads = H); padding slots are skipped
  int group_count;
  int group_heads;
  int n_tiles_all;       // key tiles over all chunks (the count without causal masking)
  int resident_ctas;     // CTAs in flight at once (one per SM; set at launch)
  int chunk_start[CPATTN_MAX_RING_DEGREE + 1];
  // extents of out, lse and the workspace (checked in CPATTN_CHECK builds)
  Span out_span, lse_span, ws_span;
};

enum class InDtype { F32, BF16 };

// Keys per K/V tile of the attention kernel for this input type and head
// size (the row count of the K and V tensor maps' boxes; query boxes have
// 128 rows).
int attn_kv_tile_rows(InDtype dt, int head_dim);

// Launches the attention kernel; tensor maps already encoded.
cudaError_t launch_attention(InDtype dt, int head_dim, const CUtensorMap& tm_q,
                             const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             const AttnParams& p, cudaStream_t stream);

struct MergeParams {
  float* o_a;
  float* l_a;
  const float* o_b;
  const float* l_b;
  int64_t rows;          // B * H * S
  int head_dim;
  int heads, seq;        // for the strided index map
  int64_t oa_s[3], ob_s[3], la_s[3], lb_s[3];   // strides (b, h, s) in elements
  int dense;             // 1: all four tensors are dense row-major
  Span oa_span, ob_span, la_span, lb_span;   // (CPATTN_CHECK builds)
  unsigned int* err;     // device error word
};
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);

// Up to kMaxPermuteBatch tensors of one shape and dtype regrouped by one
// launch (tensor i: x[i] -> y[i]).
constexpr int kMaxPermuteBatch = CPATTN_MAX_PERMUTE_BATCH;
struct PermuteParams {
  int n;
  const void* x[kMaxPermuteBatch];
  void* y[kMaxPermuteBatch];
  int64_t batch, seq, heads, head_dim, degree;
  int dir;               // +1 forward, -1 inverse
  int elem_bytes;
  uint64_t x_bytes, y_bytes;   // extent of every x[i] / y[i] (CPATTN_CHECK builds)
  unsigned int* err;           // device error word
};
cudaError_t launch_permute(const PermuteParams& p, cudaStream_t stream);
// Ulysses Anything regroup between [B, S, H, D] and [G, B, S, ceil(H/G), D]
// (heads = H; H need not divide by G).
cudaError_t launch_permute_anything(const PermuteParams& p, cudaStream_t stream);

// Rotary positions on up to kMaxPermuteBatch tensors x[i] -> y[i] of one
// dtype, batch, sequence and head size (head counts may differ).
struct RotaryParams {
  int n;
  const void* x[kMaxPermuteBatch];
  void* y[kMaxPermuteBatch];
  int64_t x_sb[kMaxPermuteBatch], x_sh[kMaxPermuteBatch], x_ss[kMaxPermuteBatch];   // elements
  int64_t y_sb[kMaxPermuteBatch], y_sh[kMaxPermuteBatch], y_ss[kMaxPermuteBatch];
  int head_start[kMaxPermuteBatch + 1];   // first head of tensor i in the count over all tensors
  int batch, seq, head_dim;
  const float* pos;
  int64_t pos_sb, pos_ss, pos_sa;
  int axes;
  int axis_dim[CPATTN_MAX_ROTARY_AXES];
  int pair_start[CPATTN_MAX_ROTARY_AXES];
  int rotary_pairs;        // pairs that turn (the rest of the features is copied)
  int interleaved, inverse;
  float2 freq[CPATTN_MAX_ROTARY_DIM / 2];   // turns per position, hi + lo
  Span x_span[kMaxPermuteBatch], y_span[kMaxPermuteBatch], pos_span;   // (CPATTN_CHECK builds)
  unsigned int* err;
};
cudaError_t launch_rotary(InDtype dt, const RotaryParams& p, cudaStream_t stream);

// Launches a kernel that may start while the one before it in the stream still
// runs, whoever launched that.  Every block of it calls launch_wait() before it
// touches memory that an earlier kernel writes or reads -- so it never
// completes before that kernel -- and launch_next() after that, so a kernel
// behind it only starts once everything before it has completed.  (Hides the
// launch and the start of the blocks, 2 to 4 us a kernel.)
template <typename... Params, typename... Args>
cudaError_t launch_behind_clustered(void (*kernel)(Params...), dim3 grid, dim3 cluster, unsigned threads,
                                    size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster.x;
  attr[1].val.clusterDim.y = cluster.y;
  attr[1].val.clusterDim.z = cluster.z;
  config.attrs = attr;
  config.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                          const Args&... args) {
  return launch_behind_clustered(kernel, grid, dim3(1), threads, smem, stream, args...);
}
#ifdef __CUDACC__
// Waits until the kernel before this one has completed (nothing to wait for
// when it was launched the ordinary way).
__device__ __forceinline__ void launch_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Asks for a line in L2, also before launch_wait(): no value is read, and what an
// earlier kernel still writes there it writes in L2.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// Lets the kernel behind this one start (once every block has called it).
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// Error word helpers (defined with the device symbol).
cudaError_t read_and_clear_device_error(unsigned int* value, cudaStream_t stream);
// Device address of the error word on the current device (nullptr on
// failure); looked up once per device.
unsigned int* device_error_word();

// SM count of the current device (152, GB300's, if it cannot be read).
int sm_count();

}  // namespace cpattn
