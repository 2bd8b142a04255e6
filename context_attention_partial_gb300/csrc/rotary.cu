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
// are dropped from the product (exact), and sincospif sees the rest.  With theta
// >= 1 and |pos| <= 2^24 that is at most 2^21.4 turns, and off by
//     2^-25.0   the frequency, 1.5 * 2^-47 of the turns
//   + 2^-26     the sum of remainder and pos * lo, below half a turn
//   + 2^-25     the sum of both with the product, below one turn
// or 2^-23.6 turns in all (2^-24.6 is the largest found).  Past 2^24 the first two
// grow with the position: 2^-23.4 found at 2^27, 2^-20.4 at 2^30.
// (fp64 sines would cost 29 us at 4608 tokens on this GPU's FP64 units.)
//
// A thread keeps one 16-byte column of one token for a group of heads of all
// tensors, so its cosines and sines are formed once and stay in registers, and
// walks the heads with four rows in flight.  Back to back, q and k of 24 heads,
// bf16, D = 128: 32768 tokens (806 MB) 123 us, 6.5 TB/s, bound by HBM; 4608 tokens
// (113 MB, [B, S, H, D]) 22.9 us, 4.9 TB/s, where HBM would take 16.7.  The short
// call is not bound by HBM: its 576 blocks start and end together, and a thread has
// no load in flight between one group of four rows and the next.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "rotary_turns.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsInFlight = 4;

struct RotaryKernelParams {
  RotaryParams p;
  int head_group;     // heads (over all tensors) a block takes
  int tile_tokens;    // tokens a block takes: kThreads / vectors of a row
  int token_tiles;    // per sequence
};

// PAIRING 0: interleaved.  Halves: a pair's members sit in different threads'
// vectors, and rows pass through shared memory (so an output may also be its
// own input); 1: every half is whole vectors, the partner is one vector,
// 2: element by element.
template <typename T, int PAIRING>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryKernelParams kp) {
  constexpr int N = Vec<T>::N;
  constexpr int NC = PAIRING == 0 ? N / 2 : N;   // turns a thread keeps
  const RotaryParams& p = kp.p;
  extern __shared__ __align__(16) unsigned char smem[];
  const int vpr = p.head_dim / N;   // 16-byte vectors of a row
  const int t = threadIdx.x / vpr, v = threadIdx.x - t * vpr;
  const int b = blockIdx.x / kp.token_tiles;
  const int token = (blockIdx.x - b * kp.token_tiles) * kp.tile_tokens + t;
  const bool active = t < kp.tile_tokens && token < p.seq;
  launch_wait();
  launch_next();

  float c[NC], s[NC];
  int partner[N];
  const unsigned turned = load_turns<PAIRING>(p, v, b, token, active, p.inverse != 0, c, s, partner);

  T* row = reinterpret_cast<T*>(smem) + t * p.head_dim;   // halves: rows in flight, [u][token][D]
  const int head0 = blockIdx.y * kp.head_group, head1 = min(head0 + kp.head_group, p.head_start[p.n]);
  for (int n = 0; n < p.n; ++n) {
    const int h0 = max(head0, p.head_start[n]) - p.head_start[n];
    const int h1 = min(head1, p.head_start[n + 1]) - p.head_start[n];
    if (h0 >= h1) continue;
    constexpr int64_t es = sizeof(T);
    const char* src = static_cast<const char*>(p.x[n]) + (b * p.x_sb[n] + h0 * p.x_sh[n] + token * p.x_ss[n]) * es + v * 16;
    char* dst = static_cast<char*>(p.y[n]) + (b * p.y_sb[n] + h0 * p.y_sh[n] + token * p.y_ss[n]) * es + v * 16;
    const int64_t src_step = p.x_sh[n] * es, dst_step = p.y_sh[n] * es;
    for (int h = h0; h < h1; h += kRowsInFlight) {
      uint4 val[kRowsInFlight];
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u)
        if (active && h + u < h1 && CPATTN_IN(p.x_span[n], src + u * src_step, 16, p.err))
          val[u] = __ldcs(reinterpret_cast<const uint4*>(src + u * src_step));
      if constexpr (PAIRING != 0) {
        __syncthreads();   // the previous rows have been read
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u)
          if (active && h + u < h1)
            reinterpret_cast<uint4*>(row + u * kp.tile_tokens * p.head_dim)[v] = val[u];
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u) {
        if (!active || h + u >= h1) continue;
        float x[N], y[N];
        unpack(val[u], x, T());
        if constexpr (PAIRING == 0) {
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            const bool on = (turned >> (e / 2)) & 1u;
            y[e] = on ? fmaf(x[e], c[e / 2], -x[e + 1] * s[e / 2]) : x[e];
            y[e + 1] = on ? fmaf(x[e], s[e / 2], x[e + 1] * c[e / 2]) : x[e + 1];
          }
        } else {
          const T* r = row + u * kp.tile_tokens * p.head_dim;
          float o[N];
          if constexpr (PAIRING == 1) {
            unpack(reinterpret_cast<const uint4*>(r)[partner[0] / N], o, T());
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = static_cast<float>(r[partner[e]]);
          }
#pragma unroll
          for (int e = 0; e < N; ++e) y[e] = ((turned >> e) & 1u) ? fmaf(x[e], c[e], o[e] * s[e]) : x[e];
        }
        if (CPATTN_IN(p.y_span[n], dst + u * dst_step, 16, p.err))
          __stcs(reinterpret_cast<uint4*>(dst + u * dst_step), repack(y, T()));
      }
      src += kRowsInFlight * src_step;
      dst += kRowsInFlight * dst_step;
    }
  }
}

template <typename T>
cudaError_t launch_typed(const RotaryParams& p, cudaStream_t stream) {
  RotaryKernelParams kp;
  kp.p = p;
  const int heads = p.head_start[p.n];
  kp.tile_tokens = kThreads / (p.head_dim / Vec<T>::N);
  kp.token_tiles = (p.seq + kp.tile_tokens - 1) / kp.tile_tokens;
  const int64_t tiles = static_cast<int64_t>(kp.token_tiles) * p.batch;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  // heads split over blocks until there are about 3 blocks per SM (4608 tokens
  // x 24 heads: 22.4 us with 3, 23.8 with 8, 27 with 24, 24 with 1): each
  // block forms its own turns, and a second round of blocks is a short one
  int64_t groups = (static_cast<int64_t>(sm_count()) * 3 + tiles - 1) / tiles;
  if (groups > heads) groups = heads;
  kp.head_group = static_cast<int>((heads + groups - 1) / groups);
  groups = (heads + kp.head_group - 1) / kp.head_group;
  if (groups > 65535) return cudaErrorInvalidValue;
  bool whole = true;   // every half whole vectors
  for (int a = 0; a < p.axes; ++a) whole = whole && p.axis_dim[a] % (2 * Vec<T>::N) == 0;
  const size_t stage = p.interleaved ? 0 : static_cast<size_t>(kRowsInFlight) * kp.tile_tokens * p.head_dim * sizeof(T);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(groups));
  return launch_behind(p.interleaved ? rotary_kernel<T, 0> : whole ? rotary_kernel<T, 1> : rotary_kernel<T, 2>, grid,
                       kThreads, stage, stream, kp);
}

}  // namespace

cudaError_t launch_rotary(InDtype dt, const RotaryParams& p, cudaStream_t stream) {
  return dt == InDtype::BF16 ? launch_typed<__nv_bfloat16>(p, stream) : launch_typed<float>(p, stream);
}

}  // namespace cpattn
