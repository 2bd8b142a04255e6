// tile_ops.cuh -- per-thread helpers of the tensor-core attention kernels:
// bit casts, bf16 packing, the 128-byte-swizzled tile layout, and the row
// operations of a softmax over a TMEM tile.
#pragma once
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"
#include "tmem_ops.cuh"

namespace cpattn {

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Byte offset of (row r, byte b of the row) in a tile stored as 128-byte
// column blocks of `rows` rows each, with the 128-byte swizzle (16-byte
// chunk index XOR row % 8), the layout TMA writes and tcgen05 reads.
__device__ __forceinline__ uint32_t sw128_offset(int r, int b, int rows) {
  return (b >> 7) * rows * 128 + r * 128 + ((((b >> 4) & 7) ^ (r & 7)) << 4) + (b & 15);
}

// Largest of the first `valid` scores of this thread's row; the others are
// set to -inf in place (keys past a chunk's end or, causal, after the row).
template <int N>
__device__ __forceinline__ float masked_row_max(uint32_t (&s)[N], int valid) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i >= valid) s[i] = f2u(-INFINITY);
  float mx[4] = {u2f(s[0]), u2f(s[1]), u2f(s[2]), u2f(s[3])};
#pragma unroll
  for (int i = 4; i < N; i += 8) {
    mx[0] = fmax3(mx[0], u2f(s[i + 0]), u2f(s[i + 1]));
    mx[1] = fmax3(mx[1], u2f(s[i + 2]), u2f(s[i + 3]));
    if (i + 4 < N) {
      mx[2] = fmax3(mx[2], u2f(s[i + 4]), u2f(s[i + 5]));
      mx[3] = fmax3(mx[3], u2f(s[i + 6]), u2f(s[i + 7]));
    }
  }
  return fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
}

// Multiplies this thread's O row (TMEM) by `factor`.
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t tO, float factor) {
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += 32) {
    uint32_t o[32];
    tmem_ld_x32(tO + c0, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * factor);
    tmem_st_x32(tO + c0, o);
  }
  tmem_wait_st();
}

}  // namespace cpattn
