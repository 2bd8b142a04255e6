// args.h -- what the C entry points share: checks of tensor descriptors, the
// driver's tensor-map encoder, and the library's process-wide settings (host code;
// not part of the public ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/cpattn.h"

namespace cpattn {

// (defined in cpattn_api.cu: one of each per build of the library, also where two are loaded)
extern std::atomic<unsigned long long> g_timeout_ns;
extern std::atomic<int> g_fault_skip_kv;
extern std::atomic<long long> g_check_shrink;   // testing: output extents shrunk by this many bytes

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (nullptr without a driver).
EncodeTiledFn encode_fn();

// 4-D map over a [B, H, S, D] tensor: dims (D, S, H, B), box (128 bytes of D,
// box_rows rows, 1, 1), 128-byte swizzle, zero fill out of bounds; with
// half_rows, 64 bytes of D and no swizzle.
cpattn_status make_tmap(CUtensorMap* m, const cpattn_tensor* t, int box_rows, bool half_rows = false);

inline int elem_bytes(int32_t dtype) { return dtype == CPATTN_BF16 ? 2 : 4; }

inline bool dtype_known(int32_t dtype) { return dtype == CPATTN_F32 || dtype == CPATTN_BF16; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Inner stride 1; other strides of extent>1 dims are multiples of 16 bytes
// and non-negative; data 16-byte aligned.
inline bool layout_ok(const cpattn_tensor* t) {
  if (t->ndim < 1) return false;
  if (t->shape[t->ndim - 1] > 1 && t->stride[t->ndim - 1] != 1) return false;
  if (!aligned16(t->data)) return false;
  const int eb = elem_bytes(t->dtype);
  for (int i = 0; i < t->ndim - 1; ++i) {
    if (t->stride[i] < 0) return false;
    if (t->shape[i] > 1 && (t->stride[i] * eb) % 16 != 0) return false;
  }
  return true;
}

inline bool shape_ok(const cpattn_tensor* t, int ndim) {
  if (t->ndim != ndim) return false;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] < 0) return false;
  return true;
}

// Bytes from a tensor's data pointer to the end of its last element (0 if
// it has none), less `shrink` (the bounds-check testing hook).
inline uint64_t extent_bytes(const cpattn_tensor* t, long long shrink = 0) {
  int64_t last = 0;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] == 0) return 0;
    last += (t->shape[i] - 1) * t->stride[i];
  }
  const int64_t bytes = (last + 1) * elem_bytes(t->dtype) - shrink;
  return bytes > 0 ? static_cast<uint64_t>(bytes) : 0;
}

inline bool contiguous(const cpattn_tensor* t) {
  int64_t expect = 1;
  for (int i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] > 1 && t->stride[i] != expect) return false;
    expect *= t->shape[i];
  }
  return true;
}

// Stride of a dimension as the TMA map sees it: dims of extent 1 get the
// dense stride so that every stride stays a positive multiple of 16 bytes.
inline int64_t tma_stride(const cpattn_tensor* t, int dim, int64_t dense) {
  return t->shape[dim] > 1 ? t->stride[dim] : dense;
}

// layout_ok, and no extent above 1 walks on the spot (broadcast views).
inline bool layout_distinct(const cpattn_tensor* t) {
  if (!layout_ok(t)) return false;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] <= 0) return false;
  return true;
}

inline bool lse_layout_ok(const cpattn_tensor* t) {
  if (reinterpret_cast<uintptr_t>(t->data) & 3u) return false;
  for (int i = 0; i < 3; ++i)
    if (t->shape[i] > 1 && t->stride[i] <= 0) return false;
  return t->shape[2] <= 1 || t->stride[2] == 1;
}

inline bool same_shape(const cpattn_tensor* a, const cpattn_tensor* b, int ndim) {
  for (int i = 0; i < ndim; ++i)
    if (a->shape[i] != b->shape[i]) return false;
  return true;
}

// Axes and frequencies of a rotary call's parameters (checked axis_dims).
template <typename P>
void fill_turns(P& p, int axes, const int32_t* axis_dims, double theta) {
  p.axes = axes;
  if (!(theta > 0.0) || !std::isfinite(theta)) theta = 10000.0;
  int j = 0;
  for (int a = 0; a < axes; ++a) {
    p.axis_dim[a] = axis_dims[a];
    p.pair_start[a] = j;
    // theta^(-2i/d) / 2 pi: every sixteenth of its own, those behind it by repeated
    // products (an exponential costs some 15 ns of host time): relative error
    // below 2^-47 and 2^-51 of |log| of the power; hi + lo leave out 2^-48
    const double rate = -2.0 / axis_dims[a] * std::log(theta), step = std::exp(rate);
    double f = 0.15915494309189535;
    for (int i = 0; i < axis_dims[a] / 2; ++i, f *= step) {
      if (i > 0 && i % 16 == 0) f = 0.15915494309189535 * std::exp(i * rate);
      const float hi = static_cast<float>(f);
      p.freq[j++] = make_float2(hi, static_cast<float>(f - hi));
    }
  }
  p.rotary_pairs = j;
}

}  // namespace cpattn
