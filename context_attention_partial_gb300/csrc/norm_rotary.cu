// norm_rotary.cu -- norms of each head with rotary positions in the same pass, for
// queries and keys; their gradient; and new tokens' keys and values on their way to
// a paged cache.
//
// Mathematics.  A row x of D features (one token's, of one head), weights w:
//     r = 1 / sqrt(sum_d x_d^2 / D + eps),   y = Turn(x r w)
// with Turn the rotation of rotary.cu.  Given dy, with dz = Turn^-1(dy):
//     dx = r (dz w - x r^2 sum_d(dz_d w_d x_d) / D),   dw = sum over rows of dz x r.
// Everything is fp32 from the load to the one rounding of each result; dw is summed
// in fp32: a thread's rows, a block's threads, then the blocks, each in a fixed order.
//
// A row's D features are L lanes of a warp (16 bytes each; twice that for fp32 rows
// past 128 features), so both sums are butterflies within the warp, and a pair's
// members that sit in different lanes meet in the warp's own part of shared memory.
// A thread keeps its column of one token for a group of heads of all tensors: the
// cosines and sines are formed once, and four rows are in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache.cuh"
#include "rotary_turns.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsInFlight = 4;

// Weight of feature f (1 where there are none).
__device__ __forceinline__ float weight(const NormParams& p, const NormTensor& t, int f) {
  if (t.w == nullptr || f >= p.head_dim) return 1.f;
  if (p.w_f32) {
    const float* at = static_cast<const float*>(t.w) + f;
    return CPATTN_IN(t.w_span, at, 4, p.err) ? *at : 0.f;
  }
  const __nv_bfloat16* at = static_cast<const __nv_bfloat16*>(t.w) + f;
  return CPATTN_IN(t.w_span, at, 2, p.err) ? __bfloat162float(*at) : 0.f;
}

// Sums over the L lanes of a row, in every lane.
template <int L, int U>
__device__ __forceinline__ void row_sums(float (&x)[U]) {
#pragma unroll
  for (int m = L / 2; m > 0; m /= 2) {
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] += __shfl_xor_sync(0xffffffffu, x[u], m);
  }
}

// A thread's place: vectors l, l + L, ... of the row of token `row`, counted over
// the batch.
template <int L>
struct Place {
  int l, t, b, token;
  bool active;
  __device__ Place(const NormParams& p, int64_t tile) {
    l = threadIdx.x % L;
    t = threadIdx.x / L;
    const int64_t row = tile * (kThreads / L) + t;
    active = row < static_cast<int64_t>(p.batch) * p.seq;
    b = active ? static_cast<int>(row / p.seq) : 0;
    token = active ? static_cast<int>(row - static_cast<int64_t>(b) * p.seq) : 0;
  }
};

// The partner values of the vector at `v` from a staged row.
template <typename T, int PAIRING, int N>
__device__ __forceinline__ void partners(const T* row, const int (&partner)[N], float (&o)[N]) {
  if constexpr (PAIRING == 1) {
    unpack(reinterpret_cast<const uint4*>(row)[partner[0] / N], o, T());
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = static_cast<float>(row[partner[e]]);
  }
}

// PAIRING: 0 interleaved; halves: 1 where every half is whole vectors, 2 element by
// element (and vectors past the turned features are their own partners).
template <typename T, int PAIRING, int L, int V>
__global__ void __launch_bounds__(kThreads) norm_rotary_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = Vec<T>::N, U = kRowsInFlight;
  constexpr int NC = PAIRING == 0 ? N / 2 : N;
  extern __shared__ __align__(16) unsigned char smem[];
  const Place<L> at(p, blockIdx.x);
  const int vpr = p.head_dim / N;
  launch_wait();
  launch_next();

  float c[V][NC], s[V][NC];
  int partner[V][N];
  unsigned turned[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    turned[i] = load_turns<PAIRING>(p, at.l + i * L, at.b, at.token, at.active, false, c[i], s[i], partner[i]);
  CachePlace place = {0, 0, false};
  if (p.cache.lengths != nullptr && at.active) place = cache_place(p.cache, at.b, at.token, p.seq, p.err);

  // halves: rows in flight, [warp][u][token of the warp][D]
  T* stage = reinterpret_cast<T*>(smem) + (threadIdx.x / 32 * U * (32 / L) + threadIdx.x % 32 / L) * p.head_dim;
  const int stage_step = 32 / L * p.head_dim;
  const float inv_d = 1.f / p.head_dim;
  const int head0 = blockIdx.y * p.head_group, head1 = min(head0 + p.head_group, p.head_start[p.n]);
  for (int n = 0; n < p.n; ++n) {
    const NormTensor& t = p.t[n];
    const int h0 = max(head0, p.head_start[n]) - p.head_start[n];
    const int h1 = min(head1, p.head_start[n + 1]) - p.head_start[n];
    if (h0 >= h1) continue;
    float w[V][N], wp[V][N];   // this feature's weight, halves: its partner's
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        w[i][e] = weight(p, t, (at.l + i * L) * N + e);
        if (PAIRING != 0) wp[i][e] = weight(p, t, partner[i][e]);
      }
    constexpr int64_t es = sizeof(T);
    const char* src = static_cast<const char*>(t.x) +
                      (at.b * t.x_s[0] + h0 * t.x_s[1] + at.token * t.x_s[2]) * es + at.l * 16;
    char* dst = static_cast<char*>(t.y) + (h0 * t.y_s[1]) * es + at.l * 16;
    dst += (t.paged ? place.page * t.y_s[0] + place.row * t.y_s[2] : at.b * t.y_s[0] + at.token * t.y_s[2]) * es;
    const bool store = t.paged ? place.valid : at.active;
    const int64_t src_step = t.x_s[1] * es, dst_step = t.y_s[1] * es;
    for (int h = h0; h < h1; h += U, src += U * src_step, dst += U * dst_step) {
      uint4 val[U][V];
      float sum[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const char* from = src + u * src_step + i * (L * 16);
          val[u][i] = make_uint4(0, 0, 0, 0);
          if (at.active && h + u < h1 && at.l + i * L < vpr && CPATTN_IN(t.x_span, from, 16, p.err))
            val[u][i] = __ldcs(reinterpret_cast<const uint4*>(from));
        }
      if (t.norm) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          sum[u] = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float x[N];
            unpack(val[u][i], x, T());
#pragma unroll
            for (int e = 0; e < N; ++e) sum[u] = fmaf(x[e], x[e], sum[u]);
          }
        }
        row_sums<L>(sum);
#pragma unroll
        for (int u = 0; u < U; ++u) sum[u] = rsqrtf(fmaf(sum[u], inv_d, p.eps));
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) sum[u] = 1.f;
      }
      if constexpr (PAIRING != 0) {
        if (t.turn) {
          __syncwarp();   // the previous rows have been read
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (at.l + i * L < vpr) reinterpret_cast<uint4*>(stage + u * stage_step)[at.l + i * L] = val[u][i];
          __syncwarp();
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!store || h + u >= h1) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (at.l + i * L >= vpr) continue;
          if (t.norm || t.turn) {
            float x[N], y[N];
            unpack(val[u][i], x, T());
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] *= sum[u] * w[i][e];
            if (!t.turn) {
#pragma unroll
              for (int e = 0; e < N; ++e) y[e] = x[e];
            } else if constexpr (PAIRING == 0) {
#pragma unroll
              for (int e = 0; e < N; e += 2) {
                const bool on = (turned[i] >> (e / 2)) & 1u;
                y[e] = on ? fmaf(x[e], c[i][e / 2], -x[e + 1] * s[i][e / 2]) : x[e];
                y[e + 1] = on ? fmaf(x[e], s[i][e / 2], x[e + 1] * c[i][e / 2]) : x[e + 1];
              }
            } else {
              float o[N];
              partners<T, PAIRING>(stage + u * stage_step, partner[i], o);
#pragma unroll
              for (int e = 0; e < N; ++e)
                y[e] = ((turned[i] >> e) & 1u) ? fmaf(x[e], c[i][e], o[e] * (sum[u] * wp[i][e]) * s[i][e]) : x[e];
            }
            val[u][i] = repack(y, T());
          }
          char* to = dst + u * dst_step + i * (L * 16);
          if (CPATTN_IN(t.y_span, to, 16, p.err)) *reinterpret_cast<uint4*>(to) = val[u][i];
        }
      }
    }
  }
}

// dx, and this block's sums of dw to the workspace.
template <typename T, int PAIRING, int L, int V>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = Vec<T>::N, U = kRowsInFlight;
  constexpr int NC = PAIRING == 0 ? N / 2 : N, ROWS = kThreads / L;
  extern __shared__ __align__(16) unsigned char smem[];
  const int vpr = p.head_dim / N;
  const bool sums = p.ws != nullptr;
  // a thread's sums of dw over its rows, [n][e of a thread][thread]; then, where
  // halves meet, the rows in flight
  float* acc = reinterpret_cast<float*>(smem);
  T* stage = reinterpret_cast<T*>(acc + (sums ? p.n * V * N * kThreads : 0)) +
             (threadIdx.x / 32 * U * (32 / L) + threadIdx.x % 32 / L) * p.head_dim;
  const int stage_step = 32 / L * p.head_dim;
  const float inv_d = 1.f / p.head_dim;
  const int64_t tiles = (static_cast<int64_t>(p.batch) * p.seq + ROWS - 1) / ROWS;
  if (sums)
    for (int i = 0; i < p.n * V * N; ++i) acc[i * kThreads + threadIdx.x] = 0.f;
  launch_wait();
  launch_next();
  const int head0 = blockIdx.y * p.head_group, head1 = min(head0 + p.head_group, p.head_start[p.n]);
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Place<L> at(p, tile);
    float c[V][NC], s[V][NC];
    int partner[V][N];
    unsigned turned[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      turned[i] = load_turns<PAIRING>(p, at.l + i * L, at.b, at.token, at.active, true, c[i], s[i], partner[i]);
    for (int n = 0; n < p.n; ++n) {
      const NormTensor& t = p.t[n];
      const int h0 = max(head0, p.head_start[n]) - p.head_start[n];
      const int h1 = min(head1, p.head_start[n + 1]) - p.head_start[n];
      if (h0 >= h1) continue;
      float w[V][N], dw[V][N];
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          w[i][e] = weight(p, t, (at.l + i * L) * N + e);
          dw[i][e] = 0.f;
        }
      constexpr int64_t es = sizeof(T);
      const char* src = static_cast<const char*>(t.x) +
                        (at.b * t.x_s[0] + h0 * t.x_s[1] + at.token * t.x_s[2]) * es + at.l * 16;
      const char* grad = static_cast<const char*>(t.dy) +
                         (at.b * t.dy_s[0] + h0 * t.dy_s[1] + at.token * t.dy_s[2]) * es + at.l * 16;
      char* dst = static_cast<char*>(t.y) + (at.b * t.y_s[0] + h0 * t.y_s[1] + at.token * t.y_s[2]) * es + at.l * 16;
      const int64_t src_step = t.x_s[1] * es, grad_step = t.dy_s[1] * es, dst_step = t.y_s[1] * es;
      for (int h = h0; h < h1; h += U, src += U * src_step, grad += U * grad_step, dst += U * dst_step) {
        uint4 val[U][V], dval[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            val[u][i] = dval[u][i] = make_uint4(0, 0, 0, 0);
            if (!at.active || h + u >= h1 || at.l + i * L >= vpr) continue;
            const char* from = src + u * src_step + i * (L * 16);
            const char* gfrom = grad + u * grad_step + i * (L * 16);
            if (CPATTN_IN(t.x_span, from, 16, p.err)) val[u][i] = __ldcs(reinterpret_cast<const uint4*>(from));
            if (CPATTN_IN(t.dy_span, gfrom, 16, p.err)) dval[u][i] = __ldcs(reinterpret_cast<const uint4*>(gfrom));
          }
        if constexpr (PAIRING != 0) {
          __syncwarp();
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (at.l + i * L < vpr) reinterpret_cast<uint4*>(stage + u * stage_step)[at.l + i * L] = dval[u][i];
          __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[V][N], dz[V][N], sum[2] = {0.f, 0.f};
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float dy[N];
            unpack(val[u][i], x[i], T());
            unpack(dval[u][i], dy, T());
            if constexpr (PAIRING == 0) {
#pragma unroll
              for (int e = 0; e < N; e += 2) {
                const bool on = (turned[i] >> (e / 2)) & 1u;
                dz[i][e] = on ? fmaf(dy[e], c[i][e / 2], -dy[e + 1] * s[i][e / 2]) : dy[e];
                dz[i][e + 1] = on ? fmaf(dy[e], s[i][e / 2], dy[e + 1] * c[i][e / 2]) : dy[e + 1];
              }
            } else {
              float o[N];
#pragma unroll
              for (int e = 0; e < N; ++e) o[e] = 0.f;
              if (at.l + i * L < vpr) partners<T, PAIRING>(stage + u * stage_step, partner[i], o);
#pragma unroll
              for (int e = 0; e < N; ++e)
                dz[i][e] = ((turned[i] >> e) & 1u) ? fmaf(dy[e], c[i][e], o[e] * s[i][e]) : dy[e];
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
              sum[0] = fmaf(x[i][e], x[i][e], sum[0]);
              sum[1] = fmaf(dz[i][e] * w[i][e], x[i][e], sum[1]);
            }
          }
          row_sums<L>(sum);
          const float r = rsqrtf(fmaf(sum[0], inv_d, p.eps));
          const float f = -(r * sum[1] * inv_d) * r;   // (r first: r^2 alone may leave fp32's range)
          if (!at.active || h + u >= h1) continue;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (at.l + i * L >= vpr) continue;
            float dx[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
              dx[e] = r * fmaf(x[i][e], f, dz[i][e] * w[i][e]);
              dw[i][e] = fmaf(dz[i][e], x[i][e] * r, dw[i][e]);
            }
            char* to = dst + u * dst_step + i * (L * 16);
            if (CPATTN_IN(t.y_span, to, 16, p.err)) __stcs(reinterpret_cast<uint4*>(to), repack(dx, T()));
          }
        }
      }
      if (sums) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) acc[((n * V + i) * N + e) * kThreads + threadIdx.x] += dw[i][e];
      }
    }
  }
  if (!sums) return;
  __syncthreads();
  const int part = blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = threadIdx.x; i < p.n * p.head_dim; i += kThreads) {
    const int n = i / p.head_dim, f = i - n * p.head_dim;
    const int v = f / N, e = f % N;
    const float* from = acc + ((n * V + v / L) * N + e) * kThreads + v % L;
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < ROWS; ++t) sum += from[t * L];
    float* to = p.ws + static_cast<int64_t>(part) * p.n * p.head_dim + i;
    if (CPATTN_IN(p.ws_span, to, 4, p.err)) *to = sum;
  }
}

// dw: the parts' sums, in their order (32 columns a block, 8 threads a column).
__global__ void __launch_bounds__(256) norm_weight_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[8][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
  const int all = p.n * p.head_dim;
  launch_wait();
  launch_next();
  float sum = 0.f;
  if (col < all)
    for (int i = y; i < p.parts; i += 8) {
      const float* from = p.ws + static_cast<int64_t>(i) * all + col;
      sum += CPATTN_IN(p.ws_span, from, 4, p.err) ? *from : 0.f;
    }
  sums[y][threadIdx.x % 32] = sum;
  __syncthreads();
  if (y != 0 || col >= all) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) sum += sums[i][threadIdx.x];
  const int n = col / p.head_dim, f = col - n * p.head_dim;
  const NormTensor& t = p.t[n];
  if (p.w_f32) {
    float* to = static_cast<float*>(t.dw) + f;
    if (CPATTN_IN(t.dw_span, to, 4, p.err)) *to = sum;
  } else {   // (the weights' type: one rounding)
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(t.dw) + f;
    if (CPATTN_IN(t.dw_span, to, 2, p.err)) *to = __float2bfloat16_rn(sum);
  }
}

// Lanes of a row.
int lanes(InDtype dt, int head_dim) {
  const int vpr = head_dim * (dt == InDtype::BF16 ? 2 : 4) / 16;
  return vpr <= 8 ? 8 : vpr <= 16 ? 16 : 32;
}

// Head groups for `tiles` blocks of tokens: about 3 blocks per SM.
int head_groups(int64_t tiles, int64_t heads) {
  const int64_t groups = (static_cast<int64_t>(sm_count()) * 3 + tiles - 1) / tiles;
  return static_cast<int>(groups < heads ? groups : heads);
}

struct Grid {
  int64_t x;   // blocks along the tokens
  int y;       // along the heads
  int head_group;
};
Grid backward_grid(InDtype dt, int head_dim, int64_t tokens, int64_t heads) {
  const int rows = kThreads / lanes(dt, head_dim);
  Grid g;
  g.x = (tokens + rows - 1) / rows;
  const int64_t groups = head_groups(g.x, heads);
  g.head_group = static_cast<int>((heads + groups - 1) / groups);
  g.y = static_cast<int>((heads + g.head_group - 1) / g.head_group);
  const int64_t most = static_cast<int64_t>(sm_count()) * 4;
  if (g.x > most) g.x = most;
  return g;
}

// (four fp32 tensors of 256 features, halves, backward: 32 KB of sums, 32 KB of rows)
constexpr size_t kMostShared = 64 * 1024;
template <auto kernel>
cudaError_t norm_run(dim3 grid, size_t smem, cudaStream_t stream, const NormParams& p) {
  static std::atomic<unsigned long long> ready{0};
  const cudaError_t e = cross_set_up(kernel, kMostShared, ready);
  return e == cudaSuccess ? launch_behind(kernel, grid, kThreads, smem, stream, p) : e;
}

template <bool BACKWARD, typename T, int PAIRING, int L, int V>
cudaError_t launch_typed(const NormParams& p, dim3 grid, size_t sums, cudaStream_t stream) {
  const size_t stage = PAIRING == 0 ? 0 : static_cast<size_t>(kRowsInFlight) * p.head_dim * sizeof(T) * (kThreads / L);
  if constexpr (BACKWARD) return norm_run<norm_backward_kernel<T, PAIRING, L, V>>(grid, sums + stage, stream, p);
  else return norm_run<norm_rotary_kernel<T, PAIRING, L, V>>(grid, sums + stage, stream, p);
}

template <bool BACKWARD, typename T, int PAIRING>
cudaError_t launch_lanes(InDtype dt, const NormParams& p, dim3 grid, size_t sums, cudaStream_t stream) {
  if constexpr (sizeof(T) == 4)
    if (p.head_dim > 128) return launch_typed<BACKWARD, T, PAIRING, 32, 2>(p, grid, sums, stream);
  const int l = lanes(dt, p.head_dim);
  return l == 8 ? launch_typed<BACKWARD, T, PAIRING, 8, 1>(p, grid, sums, stream)
                : l == 16 ? launch_typed<BACKWARD, T, PAIRING, 16, 1>(p, grid, sums, stream)
                          : launch_typed<BACKWARD, T, PAIRING, 32, 1>(p, grid, sums, stream);
}

template <bool BACKWARD, typename T>
cudaError_t launch_pairs(InDtype dt, const NormParams& p, dim3 grid, size_t sums, cudaStream_t stream) {
  bool whole = true;   // every half whole vectors
  for (int a = 0; a < p.axes; ++a) whole = whole && p.axis_dim[a] % (2 * Vec<T>::N) == 0;
  if (p.interleaved || p.rotary_pairs == 0) return launch_lanes<BACKWARD, T, 0>(dt, p, grid, sums, stream);
  return whole ? launch_lanes<BACKWARD, T, 1>(dt, p, grid, sums, stream)
               : launch_lanes<BACKWARD, T, 2>(dt, p, grid, sums, stream);
}

}  // namespace

int norm_backward_parts(InDtype dt, int head_dim, int64_t tokens, int64_t heads) {
  if (tokens == 0 || heads == 0) return 0;
  const Grid g = backward_grid(dt, head_dim, tokens, heads);
  return static_cast<int>(g.x) * g.y;
}

cudaError_t launch_norm_rotary(InDtype dt, const NormParams& params, cudaStream_t stream) {
  NormParams p = params;
  const int64_t heads = p.head_start[p.n], rows = kThreads / lanes(dt, p.head_dim);
  const int64_t tiles = (static_cast<int64_t>(p.batch) * p.seq + rows - 1) / rows;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const int64_t groups = head_groups(tiles, heads);
  p.head_group = static_cast<int>((heads + groups - 1) / groups);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((heads + p.head_group - 1) / p.head_group));
  if (grid.y > 65535) return cudaErrorInvalidValue;
  return dt == InDtype::BF16 ? launch_pairs<false, __nv_bfloat16>(dt, p, grid, 0, stream)
                             : launch_pairs<false, float>(dt, p, grid, 0, stream);
}

cudaError_t launch_norm_backward(InDtype dt, const NormParams& params, cudaStream_t stream) {
  NormParams p = params;
  const int64_t tokens = static_cast<int64_t>(p.batch) * p.seq;
  const bool sums = p.ws != nullptr;
  if (tokens > 0 && p.head_start[p.n] > 0) {
    const Grid g = backward_grid(dt, p.head_dim, tokens, p.head_start[p.n]);
    p.head_group = g.head_group;
    p.parts = static_cast<int>(g.x) * g.y;
    if (g.y > 65535) return cudaErrorInvalidValue;
    const int vectors = dt == InDtype::F32 && p.head_dim > 128 ? 2 : 1;
    const size_t bytes = sums ? static_cast<size_t>(p.n) * vectors * (dt == InDtype::BF16 ? 8 : 4) * kThreads * 4 : 0;
    const dim3 grid(static_cast<unsigned>(g.x), g.y);
    const cudaError_t e = dt == InDtype::BF16 ? launch_pairs<true, __nv_bfloat16>(dt, p, grid, bytes, stream)
                                              : launch_pairs<true, float>(dt, p, grid, bytes, stream);
    if (e != cudaSuccess) return e;
  } else {
    p.parts = 0;   // (no rows: dw is 0)
  }
  if (p.t[0].dw == nullptr) return cudaSuccess;
  return launch_behind(norm_weight_kernel, dim3((p.n * p.head_dim + 31) / 32), 256, 0, stream, p);
}

}  // namespace cpattn
