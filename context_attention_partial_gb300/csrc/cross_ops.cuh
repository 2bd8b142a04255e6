// cross_ops.cuh -- device helpers shared by the tensor-core cross-attention
// kernels: tile loads, and the way of a warp's output rows to memory.
#pragma once
#include "cross.cuh"
#include "ptx.cuh"
#include "tile_ops.cuh"
#include "tmem_ops.cuh"

namespace cpattn {

// A 128-row tile of D bf16 features (128-byte column blocks, swizzled).
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int row, int h, int b,
                                          uint64_t pol) {
#pragma unroll
  for (int kb = 0; kb < D / 64; ++kb) tma_load_4d_hint(dst + kb * 128 * 128, tm, bar, kb * 64, row, h, b, pol);
}

// The same tile into L2 only.
template <int D>
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* tm, int row, int h, int b) {
#pragma unroll
  for (int kb = 0; kb < D / 64; ++kb) tma_prefetch_l2_4d(tm, kb * 64, row, h, b);
}

// Rows valid.. of a 128-row tile become zeros (whole warp; before the MMAs
// that read the tile are issued): keys past a length get no weight, but
// 0 * NaN would still be NaN.
template <int D>
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int valid) {
  const int per = (128 - valid) * 8;   // 16-byte chunks of a column block
  for (int i = threadIdx.x % 32; i < per * (D / 64); i += 32) {
    const int kb = i / per;
    *reinterpret_cast<uint4*>(tile + kb * 128 * 128 + (valid * 8 + i - kb * per) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// The kernels place their tiles from the start of dynamic shared memory, which
// a 128-byte swizzle needs at a multiple of 1024 bytes: asked for by the
// declaration, and checked (there is no room for a runtime alignment).
__device__ __forceinline__ bool tiles_aligned(const CrossParams& p, const void* smem) {
  if ((smem_addr(smem) & 1023u) == 0) return true;
  if (threadIdx.x == 0) atomicOr(p.err, 0x10u);
  return false;
}

// A warp's 32 rows x N columns (fp32 in registers, one row per lane), times f,
// as bf16 to rows row0.. and columns c0.. of a tensor: through `stage` (32 N
// bf16, 1024-byte aligned) and one tensor store that leaves out rows past the
// tensor's end.  N = 64: the staged rows are 128 bytes in the 128-byte
// swizzle; N = 32: 64 bytes, dense.  The caller waits (bulk_wait_read by lane
// 0) before the stage is written again or given up.
// Check builds store with plain, checked stores instead.
template <int N>
__device__ __forceinline__ void store_rows(const CrossParams& p, const CrossTensor& t, const CUtensorMap* tm,
                                           uint8_t* stage, const uint32_t (&o)[N], float f, int b, int h, int row0,
                                           int rows, int c0) {
  constexpr int CH = N / 8;   // 16-byte chunks of a row
  constexpr int MASK = N == 64 ? 7 : 0;
  const int lane = threadIdx.x % 32;
  uint4* srow = reinterpret_cast<uint4*>(stage) + lane * CH;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    uint32_t x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b2;
      fmul2(a, b2, u2f(o[8 * i + 2 * e]), u2f(o[8 * i + 2 * e + 1]), f, f);
      x[e] = pack_bf16x2(a, b2);
    }
    srow[i ^ (lane & MASK)] = make_uint4(x[0], x[1], x[2], x[3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
#ifdef CPATTN_CHECK
  uint8_t* out = static_cast<uint8_t*>(t.data) + (b * t.s[0] + h * t.s[1]) * 2;
  for (int it = 0; it < CH; ++it) {
    const int idx = it * 32 + lane, r = idx / CH, c = idx % CH;
    if (row0 + r < rows) {
      const uint4 val = reinterpret_cast<const uint4*>(stage)[r * CH + (c ^ (r & MASK))];
      uint8_t* dst = out + (static_cast<int64_t>(row0 + r) * t.s[2] + c0) * 2 + c * 16;
      if (CPATTN_IN(t.span, dst, 16, p.err)) *reinterpret_cast<uint4*>(dst) = val;
    }
  }
  __syncwarp();
#else
  if (lane == 0 && row0 < rows) {
    tma_store_4d(tm, smem_addr(stage), c0, row0, h, b);
    bulk_commit();
  }
#endif
}

}  // namespace cpattn
