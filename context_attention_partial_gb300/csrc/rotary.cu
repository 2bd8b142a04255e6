// rotary.cu -- rotary positions with several axes (time, height, width, ...)
// for queries and keys, and their gradient.
//
// Mathematics.  The D features of a head hold one block of d_a features per
// position axis a (blocks in axis order; features past the last block are
// copied).  Pair i of block a turns by the angle pos_a * theta^(-2 i / d_a):
//     y_u = x_u cos - x_w sin,   y_w = x_u sin + x_w cos
// with (u, w) = (2i, 2i + 1) or (i, i + d_a / 2) inside the block.  The turn
// is orthogonal, so the gradient is the turn by the negative angle.
//
// Angles.  An fp32 product pos * frequency is off by pos * 2^-24 radians: 6e-3
// at position 100,000.  Frequencies therefore come from the host as two
// floats, in turns per position (theta^(-2i/d) / 2 pi in fp64, split hi + lo);
// pos * hi is taken exactly as a product and its fused remainder, whole turns
// are dropped from the product (exact), and sincospif sees the rest: the
// angle's error is below 2^-24 turns at any position fp32 can hold exactly.
// (fp64 sines would cost 29 us at 4608 tokens on this GPU's FP64 units.)
//
// What bounds it: HBM, each tensor read and written once.  A block turns one
// tile of tokens for a group of heads of all tensors: the (cos, sin) of a
// token are computed once in shared memory and shared by the heads, and a
// thread keeps one 16-byte column of the rows it walks, four rows in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
constexpr int kTileTokens = 16;
constexpr int kRowsInFlight = 4;

struct RotaryKernelParams {
  RotaryParams p;
  int head_group;     // heads (over all tensors) a block takes
  int heads_total;
  int token_tiles;    // per sequence
};

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

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryKernelParams kp) {
  constexpr int N = Vec<T>::N;
  const RotaryParams& p = kp.p;
  extern __shared__ __align__(16) unsigned char smem[];
  const int pairs = p.head_dim / 2;
  float2* cs = reinterpret_cast<float2*>(smem);                    // [token][pair]
  T* stage = reinterpret_cast<T*>(cs + kTileTokens * pairs);       // halves: [row][D] in flight

  const int tile = blockIdx.x % kp.token_tiles;
  const int b = blockIdx.x / kp.token_tiles;
  const int s0 = tile * kTileTokens;
  const int tokens = min(kTileTokens, p.seq - s0);
  const int head0 = blockIdx.y * kp.head_group;
  const int heads = min(kp.head_group, kp.heads_total - head0);

  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    float c = 1.f, s = 0.f;
    if (j < p.rotary_pairs) {
      int axis = 0;
#pragma unroll
      for (int a = 0; a < CPATTN_MAX_ROTARY_AXES - 1; ++a)
        if (a + 1 < p.axes && j >= p.pair_start[a + 1]) axis = a + 1;
      const float* src = p.pos + b * p.pos_sb + (s0 + t) * p.pos_ss + axis * p.pos_sa;
      const float pos = CPATTN_IN(p.pos_span, src, 4, p.err) ? *src : 0.f;
      const float2 f = p.freq[j];   // turns per position, hi + lo
      const float hi = __fmul_rn(pos, f.x);
      const float lo = fmaf(pos, f.y, fmaf(pos, f.x, -hi));
      sincospif(2.f * ((hi - rintf(hi)) + lo), &s, &c);
      if (p.inverse) s = -s;
    }
    cs[i] = make_float2(c, s);
  }
  __syncthreads();

  const int vpr = p.head_dim / N;             // 16-byte vectors per row
  const int rows_par = kThreads / vpr;        // rows the block walks at once
  const int rows = tokens * heads;
  const bool active = threadIdx.x < rows_par * vpr;
  const int row0 = threadIdx.x / vpr, v = threadIdx.x - row0 * vpr;

  // halves: partner feature and pair of each of this thread's N features
  int partner[N], pair[N];
  unsigned second = 0, turned = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int f = v * N + e;
    partner[e] = f;
    pair[e] = f / 2;
    if (f < 2 * p.rotary_pairs) turned |= 1u << e;
    if (!INTERLEAVED && f < 2 * p.rotary_pairs) {
      int axis = 0;
#pragma unroll
      for (int a = 0; a < CPATTN_MAX_ROTARY_AXES - 1; ++a)
        if (a + 1 < p.axes && f >= 2 * p.pair_start[a + 1]) axis = a + 1;
      const int base = 2 * p.pair_start[axis];
      const int half = p.axis_dim[axis] / 2, i = f - base;
      const bool upper = i >= half;
      partner[e] = upper ? f - half : f + half;
      pair[e] = p.pair_start[axis] + (upper ? i - half : i);
      if (upper) second |= 1u << e;
    }
  }

  for (int base = 0; base < rows; base += rows_par * kRowsInFlight) {
    uint4 val[kRowsInFlight];
    const char* src[kRowsInFlight];
    char* dst[kRowsInFlight];
    int tok[kRowsInFlight], tensor[kRowsInFlight];
    bool live[kRowsInFlight];
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      const int row = base + u * rows_par + row0;
      live[u] = active && row < rows;
      int h, t;
      if (p.token_inner) {
        h = row / tokens;
        t = row - h * tokens;
      } else {
        t = row / heads;
        h = row - t * heads;
      }
      h += head0;
      int n = 0;
#pragma unroll
      for (int i = 1; i < CPATTN_MAX_PERMUTE_BATCH; ++i)
        if (i < p.n && h >= p.head_start[i]) n = i;
      tok[u] = t;
      tensor[u] = n;
      if (live[u]) {
        const int64_t hh = h - p.head_start[n], ss = s0 + t;
        src[u] = static_cast<const char*>(p.x[n]) +
                 (b * p.x_sb[n] + hh * p.x_sh[n] + ss * p.x_ss[n]) * static_cast<int64_t>(sizeof(T)) + v * 16;
        dst[u] = static_cast<char*>(p.y[n]) +
                 (b * p.y_sb[n] + hh * p.y_sh[n] + ss * p.y_ss[n]) * static_cast<int64_t>(sizeof(T)) + v * 16;
        live[u] = CPATTN_IN(p.x_span[n], src[u], 16, p.err);
      }
      if (live[u]) val[u] = __ldcs(reinterpret_cast<const uint4*>(src[u]));
    }
    if constexpr (!INTERLEAVED) {
      // a pair's members sit in different threads' vectors: rows pass through
      // shared memory (so an output may also be its own input)
      __syncthreads();   // the previous rows have been read
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u)
        if (live[u])
          *reinterpret_cast<uint4*>(stage + ((u * rows_par + row0) * vpr + v) * N) = val[u];
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      if (!live[u]) continue;
      float x[N], y[N];
      unpack(val[u], x, T());
      const float2* turn = cs + tok[u] * pairs;
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 c = turn[(v * N + e) / 2];
          const bool on = (turned >> e) & 1u;
          y[e] = on ? fmaf(x[e], c.x, -x[e + 1] * c.y) : x[e];
          y[e + 1] = on ? fmaf(x[e], c.y, x[e + 1] * c.x) : x[e + 1];
        }
      } else {
        const T* row = stage + (u * rows_par + row0) * p.head_dim;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 c = turn[pair[e]];
          const float o = static_cast<float>(row[partner[e]]);
          const float r = fmaf(x[e], c.x, ((second >> e) & 1u) ? o * c.y : -o * c.y);
          y[e] = ((turned >> e) & 1u) ? r : x[e];
        }
      }
      if (CPATTN_IN(p.y_span[tensor[u]], dst[u], 16, p.err))
        __stcs(reinterpret_cast<uint4*>(dst[u]), repack(y, T()));
    }
  }
}

template <typename T>
cudaError_t launch_typed(const RotaryParams& p, cudaStream_t stream) {
  RotaryKernelParams kp;
  kp.p = p;
  kp.heads_total = p.head_start[p.n];
  kp.token_tiles = (p.seq + kTileTokens - 1) / kTileTokens;
  const int64_t tiles = static_cast<int64_t>(kp.token_tiles) * p.batch;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  // heads split over blocks until there are about 8 blocks per SM; each block
  // recomputes its tile's angles, so no finer than that
  int64_t groups = (static_cast<int64_t>(sm_count()) * 8 + tiles - 1) / tiles;
  if (groups > kp.heads_total) groups = kp.heads_total;
  kp.head_group = static_cast<int>((kp.heads_total + groups - 1) / groups);
  groups = (kp.heads_total + kp.head_group - 1) / kp.head_group;
  if (groups > 65535) return cudaErrorInvalidValue;
  const int rows_par = kThreads / (p.head_dim / Vec<T>::N);
  const size_t turns = static_cast<size_t>(kTileTokens) * (p.head_dim / 2) * sizeof(float2);
  const size_t stage = p.interleaved ? 0
                                     : static_cast<size_t>(kRowsInFlight) * rows_par * p.head_dim * sizeof(T);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(groups));
  if (p.interleaved)
    rotary_kernel<T, true><<<grid, kThreads, turns + stage, stream>>>(kp);
  else
    rotary_kernel<T, false><<<grid, kThreads, turns + stage, stream>>>(kp);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(InDtype dt, const RotaryParams& p, cudaStream_t stream) {
  return dt == InDtype::BF16 ? launch_typed<__nv_bfloat16>(p, stream) : launch_typed<float>(p, stream);
}

}  // namespace cpattn
