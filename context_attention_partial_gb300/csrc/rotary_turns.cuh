// rotary_turns.cuh -- what turns features to positions: the size of a row's vectors and a
// pair's cosine and sine (the angles' arithmetic and its error: rotary.cu), which rotary.cu
// and norm_rotary.cu use; vectors in fp32 and a thread's turns in registers, which rotary.cu
// does (norm_rotary.cu has packed pairs, and a block's turns in shared memory).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace cpattn {

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8], __nv_bfloat16) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4], float) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
// (bf16: the only rounding to fewer bits, to nearest, of the fp32 result)
__device__ __forceinline__ uint4 repack(const float (&f)[8], __nv_bfloat16) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return v;
}
__device__ __forceinline__ uint4 repack(const float (&f)[4], float) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}

// Cosine and sine of a pair with frequency w (turns per position, hi + lo) at `pos`.
__device__ __forceinline__ float2 rotary_turn(float pos, float2 w) {
  const float hi = __fmul_rn(pos, w.x);
  const float lo = fmaf(pos, w.y, fmaf(pos, w.x, -hi));
  float2 cs;
  sincospif(2.f * ((hi - rintf(hi)) + lo), &cs.y, &cs.x);
  return cs;
}

// Cosines and sines of vector v's features at (b, token), and the features that
// are turned (bit e).  PAIRING 0: interleaved, a turn per pair.  Halves (1, 2): a
// turn per feature, s with the sign that its partner, feature partner[e], is
// multiplied with.  P: parameters with a rotary call's positions and axes.
template <int PAIRING, int N, int NC, typename P>
__device__ __forceinline__ unsigned load_turns(const P& p, int v, int b, int token, bool active, bool inverse,
                                               float (&c)[NC], float (&s)[NC], int (&partner)[N]) {
  unsigned turned = 0;
#pragma unroll
  for (int e = 0; e < NC; ++e) {
    const int f = PAIRING == 0 ? v * N + 2 * e : v * N + e;
    c[e] = 1.f;
    s[e] = 0.f;
    if (PAIRING != 0) partner[e] = f;
    if (f < 2 * p.rotary_pairs) {
      turned |= 1u << e;
      int axis = 0;
#pragma unroll
      for (int a = 0; a < CPATTN_MAX_ROTARY_AXES - 1; ++a)
        if (a + 1 < p.axes && f >= 2 * p.pair_start[a + 1]) axis = a + 1;
      int pair = f / 2;
      bool upper = false;
      if constexpr (PAIRING != 0) {
        const int half = p.axis_dim[axis] / 2, i = f - 2 * p.pair_start[axis];
        upper = i >= half;
        pair = p.pair_start[axis] + (upper ? i - half : i);
        partner[e] = upper ? f - half : f + half;
      }
      if (active) {
        const float* src = p.pos + b * p.pos_sb + token * p.pos_ss + axis * p.pos_sa;
        const float2 cs = rotary_turn(CPATTN_IN(p.pos_span, src, 4, p.err) ? *src : 0.f, p.freq[pair]);
        c[e] = cs.x;
        s[e] = cs.y;
        // (sign: what this feature's partner is multiplied with)
        if (inverse != (PAIRING != 0 && !upper)) s[e] = -s[e];
      }
    }
  }
  return turned;
}

}  // namespace cpattn
