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
// past 128 features), so both sums are butterflies within the warp.  A thread keeps its
// column of one token and walks a group of heads of all tensors; the next rows are on
// their way by asynchronous copies to shared memory, where a pair's members that sit
// in different lanes meet, too.  A long call is bound by HBM and nearly by the issue of
// its instructions: rows go four at a time (backward two), features in packed pairs.  A
// short one waits for its first instructions, which also come from HBM, so the code is
// kept short, and a block's sines and cosines are formed in one loop, to shared memory.
//
// Measured: q and k of 24 heads, bf16, D = 128, 4608 tokens (113 MB) 21.4 us, 5.3 TB/s, in runs
// of 60 calls, 23.8 in shorter ones; the gradient at 32768 tokens (1.21 GB) 187 us, 6.5 TB/s,
// in fp32 (2.42 GB) 357 us, 6.8 TB/s; four prompts of up to 4001 tokens, 48 heads, to a cache
// (336 MB) 58 to 59 us, 5.7 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache.cuh"
#include "ptx.cuh"
#include "rotary_turns.cuh"
#include "tile_ops.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 128;

// Two fp32 values in a register pair: one instruction for both.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 halves_of(f2 a) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
  return d;
}
__device__ __forceinline__ f2 mul(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 swapped(f2 a) {
  const float2 t = halves_of(a);
  return pack2(t.y, t.x);
}

// A 16-byte vector's pairs, and back (bf16: the only rounding to fewer bits, to
// nearest, of the fp32 result).
__device__ __forceinline__ void to_pairs(const uint4& v, f2 (&x)[4], __nv_bfloat16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void to_pairs(const uint4& v, f2 (&x)[2], float) {
  x[0] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
  x[1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ uint4 from_pairs(const f2 (&x)[4], __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = halves_of(x[i]);
    w[i] = pack_bf16x2(t.x, t.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 from_pairs(const f2 (&x)[2], float) {
  const float2 a = halves_of(x[0]), b = halves_of(x[1]);
  return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}

// How a kernel lays a block out: rows of L lanes, V vectors a lane, U rows at a time, and a
// ring of P such steps of each input, of which P - 1 are on their way.
template <typename T, int L, int V, int INPUTS>
struct Shape {
  static constexpr int N = Vec<T>::N;
  static constexpr int TOKENS = kThreads / L;
  static constexpr int U = INPUTS == 2 || V == 2 ? 2 : 4;
  static constexpr int P = INPUTS == 2 && V == 2 ? 2 : 3;
  static constexpr int SLOTS = INPUTS * P * U;   // rows of a token
  // bytes of shared memory: turns [token][pair], positions [token][4], weights [n][D], rows
  static constexpr size_t kPositions = static_cast<size_t>(TOKENS) * CPATTN_MAX_ROTARY_AXES * sizeof(float);
  static constexpr size_t turns(int pairs) { return static_cast<size_t>(TOKENS) * pairs * sizeof(float2); }
  static constexpr size_t weights(int n, int head_dim) { return static_cast<size_t>(n) * head_dim * sizeof(float); }
  static constexpr size_t rows(int head_dim) { return static_cast<size_t>(SLOTS) * TOKENS * head_dim * sizeof(T); }
};

// Value i of all tensors' weights, [n][D], as fp32 (1 where there are none).
__device__ __forceinline__ float weight(const NormParams& p, int i) {
  const int n = i / p.head_dim, f = i - n * p.head_dim;
  const NormTensor& t = p.t[n];
  if (t.w == nullptr) return 1.f;
  if (p.w_f32) {
    const float* from = static_cast<const float*>(t.w) + f;
    return CPATTN_IN(t.w_span, from, 4, p.err) ? *from : 0.f;
  }
  const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(t.w) + f;
  return CPATTN_IN(t.w_span, from, 2, p.err) ? __bfloat162float(*from) : 0.f;
}

// A tile's first token, counted over the batch, as sequence and token (one division of
// 64 bits a block), and the token `t` of the tile; b >= batch: none.
struct Tile {
  int b0, token0;
  __device__ Tile(const NormParams& p, int64_t first) {
    b0 = static_cast<int>(first / p.seq);
    token0 = static_cast<int>(first - static_cast<int64_t>(b0) * p.seq);
  }
  __device__ void at(const NormParams& p, int t, int& b, int& token) const {
    const unsigned local = static_cast<unsigned>(token0) + t, more = local / p.seq;
    b = b0 + static_cast<int>(more);
    token = static_cast<int>(local - more * p.seq);
  }
};

// A thread's place: vectors l, l + L, ... of the row of token t of the tile.
template <int L>
struct Place {
  int l, t, b, token;
  bool active;
  __device__ Place(const NormParams& p, const Tile& tile) {
    l = threadIdx.x % L;
    t = threadIdx.x / L;
    tile.at(p, t, b, token);
    active = b < p.batch;
    if (!active) b = token = 0;
  }
};

// Position i of a tile's, [token][axis].
__device__ __forceinline__ float position(const NormParams& p, const Tile& tile, int i) {
  const int t = i / p.axes;
  int b, token;
  tile.at(p, t, b, token);
  const float* from = p.pos + b * p.pos_sb + token * p.pos_ss + (i - t * p.axes) * p.pos_sa;
  return b < p.batch && CPATTN_IN(p.pos_span, from, 4, p.err) ? *from : 0.f;
}

// The cosines and sines of a tile's tokens, [token][pair], from their positions (all
// threads).
template <int L>
__device__ __forceinline__ void tile_turns(const NormParams& p, const float* positions, float2* turns) {
  const int pairs = p.rotary_pairs, lanes = kThreads / pairs, t0 = threadIdx.x / pairs, pair = threadIdx.x - t0 * pairs;
  if (t0 >= lanes) return;
  int axis = 0;
#pragma unroll
  for (int a = 1; a < CPATTN_MAX_ROTARY_AXES; ++a)
    if (a < p.axes && pair >= p.pair_start[a]) axis = a;
  const float2 w = p.freq[pair];
#pragma unroll 1
  for (int t = t0; t < kThreads / L; t += lanes) turns[t * pairs + pair] = rotary_turn(positions[t * p.axes + axis], w);
}

// How a vector turns: y = c x + s o, with o the pairs' members swapped (interleaved: in
// x's own pairs) or their partners (halves).  Features that do not turn have (1, 0), and
// `all` is false: they stay as they are, also beside an infinite one.
template <int N>
struct Turns {
  f2 c[N / 2], s[N / 2];
  int partner[N];
  unsigned turned;   // bit e: feature e turns
  bool all;
};
// PAIRING: 0 interleaved; halves: 1 where every half is whole vectors, 2 element by
// element.
template <int PAIRING, int N>
__device__ __forceinline__ void vector_turns(const NormParams& p, const float2* turns, int v, bool active, bool inverse,
                                             Turns<N>& r) {
  r.turned = 0;
  int start = 0, half = 0;   // of the axis of the vector's first feature (PAIRING 1: of all)
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    float c[2], s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int f = v * N + e + k;
      c[k] = 1.f;
      s[k] = 0.f;
      r.partner[e + k] = f;
      if (!active || f >= 2 * p.rotary_pairs) continue;
      r.turned |= 1u << (e + k);
      bool plus;   // the sign of the sine
      int pair;
      if constexpr (PAIRING == 0) {
        pair = f / 2;
        plus = k == 1;
        r.partner[e + k] = f ^ 1;
      } else {
        if (PAIRING == 2 || (e == 0 && k == 0)) {
          int axis = 0;
#pragma unroll
          for (int a = 1; a < CPATTN_MAX_ROTARY_AXES; ++a)
            if (a < p.axes && f >= 2 * p.pair_start[a]) axis = a;
          start = 2 * p.pair_start[axis];
          half = p.axis_dim[axis] / 2;
        }
        const int i = f - start;
        plus = i >= half;
        pair = start / 2 + (plus ? i - half : i);
        r.partner[e + k] = plus ? f - half : f + half;
      }
      const float2 cs = turns[pair];
      c[k] = cs.x;
      s[k] = inverse != plus ? cs.y : -cs.y;
    }
    r.c[e / 2] = pack2(c[0], c[1]);
    r.s[e / 2] = pack2(s[0], s[1]);
  }
  r.all = r.turned == (1u << N) - 1;
}

// The partner values of a vector from its row in shared memory.
template <typename T, int PAIRING, int N>
__device__ __forceinline__ void partners(const T* row, const Turns<N>& r, f2 (&o)[N / 2]) {
  if constexpr (PAIRING == 1) {
    to_pairs(reinterpret_cast<const uint4*>(row)[r.partner[0] / N], o, T());
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2)
      o[e / 2] = pack2(static_cast<float>(row[r.partner[e]]), static_cast<float>(row[r.partner[e + 1]]));
  }
}
// Where not all of a vector's features turn: 0 in o beside those that do not.
template <int N>
__device__ __forceinline__ void mask_partners(const Turns<N>& r, f2 (&o)[N / 2]) {
  if (r.all) return;
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float2 t = halves_of(o[e / 2]);
    o[e / 2] = pack2((r.turned >> e) & 1u ? t.x : 0.f, (r.turned >> (e + 1)) & 1u ? t.y : 0.f);
  }
}

// The rows that a thread asks for, in their order: heads head0 .. head1 - 1 of all
// tensors, counted together.
struct Cursor {
  int n, left;     // tensor, its rows left
  int64_t at;      // elements from the tensor's start: this token's row of the head
};
__device__ __forceinline__ bool next_tensor(const NormParams& p, int head0, int head1, int& n, int& h0, int& rows) {
  for (++n; n < p.n; ++n) {
    h0 = max(head0, p.head_start[n]) - p.head_start[n];
    rows = min(head1, p.head_start[n + 1]) - p.head_start[n] - h0;
    if (rows > 0) return true;
  }
  return false;
}

template <typename T, int PAIRING, int L, int V>
__global__ void __launch_bounds__(kThreads, V == 1 && PAIRING != 0 ? 5 : 4)
    norm_rotary_kernel(const __grid_constant__ NormParams p) {
  using S = Shape<T, L, V, 1>;
  constexpr int N = S::N, P = S::P, U = S::U;
  constexpr int64_t es = sizeof(T);
  extern __shared__ __align__(16) unsigned char smem[];
  float2* turns = reinterpret_cast<float2*>(smem);
  float* positions = reinterpret_cast<float*>(smem + S::turns(p.rotary_pairs));
  float* weights = positions + S::TOKENS * CPATTN_MAX_ROTARY_AXES;
  const Tile tile(p, static_cast<int64_t>(blockIdx.x) * S::TOKENS);
  const Place<L> at(p, tile);
  const int vpr = p.head_dim / N;
  // this token's rows on their way: step i's at ring + i U step
  T* ring = reinterpret_cast<T*>(weights + p.n * p.head_dim) + at.t * p.head_dim;
  const int step = S::TOKENS * p.head_dim;
  const int head0 = blockIdx.y * p.head_group, head1 = min(head0 + p.head_group, p.head_start[p.n]);
  bool lane[V];   // whether the lane has this vector of a row
#pragma unroll
  for (int i = 0; i < V; ++i) lane[i] = at.l + i * L < vpr;
  launch_wait();
  launch_next();

  // (asked for before the rows, which fill the way to memory)
  static_assert(S::TOKENS * CPATTN_MAX_ROTARY_AXES <= kThreads, "a position a thread");
  const int n_weights = p.n * p.head_dim;
  const float w0 = threadIdx.x < n_weights ? weight(p, threadIdx.x) : 0.f;
  const float pos0 = threadIdx.x < S::TOKENS * p.axes ? position(p, tile, threadIdx.x) : 0.f;
  CachePlace place = {0, 0, false};
  bool placed = false;   // where the token goes, found when a paged tensor comes up
  Cursor ask = {-1, 0, 0};
  int64_t ask_step = 0;  // bytes from head to head
  const char* ask_from = nullptr;
  bool ask_read = false;
  uint32_t ask_to = smem_addr(ring) + at.l * 16;
  const uint32_t row_bytes = step * es, ask_end = ask_to + P * U * row_bytes;
  auto request = [&]() {
    if (ask.left <= 0) {
      int h0;
      ask.left = 0;
      if (ask.n < p.n && next_tensor(p, head0, head1, ask.n, h0, ask.left)) {
        const NormTensor& t = p.t[ask.n];
        ask_step = t.x_s[1] * es;
        ask_from = static_cast<const char*>(t.x) + (at.b * t.x_s[0] + at.token * t.x_s[2]) * es + h0 * ask_step + at.l * 16;
        if (t.paged && !placed) {
          placed = true;
          if (at.active) place = cache_place(p.cache, at.b, at.token, p.seq, p.err);
        }
        ask_read = t.paged ? place.valid : at.active;
      }
    }
    if (ask.left > 0 && ask_read) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const char* from = ask_from + u * ask_step;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (u < ask.left && lane[i] && CPATTN_IN(p.t[ask.n].x_span, from + i * (L * 16), 16, p.err))
            copy16(ask_to + u * row_bytes + i * (L * 16), from + i * (L * 16), true);
      }
    }
    ask_from += U * ask_step;
    ask.left -= U;
    ask_to += U * row_bytes;
    if (ask_to == ask_end) ask_to -= P * U * row_bytes;
    copies_commit();
  };
#pragma unroll 1
  for (int i = 0; i < P - 1; ++i) request();

  if (threadIdx.x < n_weights) weights[threadIdx.x] = w0;
#pragma unroll 1
  for (int i = threadIdx.x + kThreads; i < n_weights; i += kThreads) weights[i] = weight(p, i);
  if (threadIdx.x < S::TOKENS * CPATTN_MAX_ROTARY_AXES) positions[threadIdx.x] = pos0;
  __syncthreads();
  if (p.rotary_pairs > 0) {
    tile_turns<L>(p, positions, turns);
    __syncthreads();
  }

  const float inv_d = 1.f / p.head_dim;
  int n = -1, h0 = 0, rows = 0, slot = 0;
  while (next_tensor(p, head0, head1, n, h0, rows)) {
    const NormTensor& t = p.t[n];
    const bool norm = t.norm, turn = t.turn;
    // y = inv (x wc + o ws), o the partners: this feature's weight times its cosine, and
    // its partner's times the sine
    f2 wc[V][N / 2], ws[V][N / 2];
    Turns<N> vec[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float* w = weights + n * p.head_dim;
      vector_turns<PAIRING>(p, turns + at.t * p.rotary_pairs, at.l + i * L, turn && at.active && lane[i], false, vec[i]);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const int f = lane[i] ? (at.l + i * L) * N + e : 0;
        wc[i][e / 2] = mul(pack2(w[f], w[f + 1]), vec[i].c[e / 2]);
        ws[i][e / 2] = 0;
        if (lane[i])   // (0 for a feature that does not turn, whatever its weight is)
          ws[i][e / 2] = mul(pack2((vec[i].turned >> e) & 1u ? w[vec[i].partner[e]] : 0.f,
                                   (vec[i].turned >> (e + 1)) & 1u ? w[vec[i].partner[e + 1]] : 0.f),
                             vec[i].s[e / 2]);
      }
    }
    if (t.paged && !placed) {
      placed = true;
      if (at.active) place = cache_place(p.cache, at.b, at.token, p.seq, p.err);
    }
    char* dst = static_cast<char*>(t.y) + h0 * t.y_s[1] * es + at.l * 16;
    dst += (t.paged ? place.page * t.y_s[0] + place.row * t.y_s[2] : at.b * t.y_s[0] + at.token * t.y_s[2]) * es;
    const bool store = t.paged ? place.valid : at.active;
    const int64_t dst_step = t.y_s[1] * es;
#pragma unroll 1
    for (int left = rows; left > 0; left -= U, dst += U * dst_step) {
      copies_wait<P - 2>();
      __syncwarp();   // (the rows before have been read, too)
      request();
      const T* row = ring + slot * step;
      slot = slot + U == P * U ? 0 : slot + U;
      if (!norm && !turn) {   // values: as they are
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            char* to = dst + u * dst_step + i * (L * 16);
            if (store && u < left && lane[i] && CPATTN_IN(t.y_span, to, 16, p.err))
              *reinterpret_cast<uint4*>(to) = reinterpret_cast<const uint4*>(row + u * step)[at.l + i * L];
          }
        continue;
      }
      f2 x[U][V][N / 2], inv[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i)
          // (slots of rows that are not there hold anything: nothing of them is kept)
          to_pairs(lane[i] ? reinterpret_cast<const uint4*>(row + u * step)[at.l + i * L] : make_uint4(0, 0, 0, 0), x[u][i], T());
      if (norm) {
        float sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          f2 two = 0;
#pragma unroll
          for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < N / 2; ++e) two = fma(x[u][i][e], x[u][i][e], two);
          const float2 h = halves_of(two);
          sum[u] = h.x + h.y;
        }
#pragma unroll
        for (int m = L / 2; m > 0; m /= 2)
#pragma unroll
          for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], m);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float f = rsqrtf(fmaf(sum[u], inv_d, p.eps));
          inv[u] = pack2(f, f);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          f2 y[N / 2], o[N / 2];
          if constexpr (PAIRING == 0) {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) o[e] = swapped(x[u][i][e]);
          } else if (lane[i]) {
            partners<T, PAIRING>(row + u * step, vec[i], o);
          }
          mask_partners(vec[i], o);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) y[e] = fma(o[e], ws[i][e], mul(x[u][i][e], wc[i][e]));
          if (norm) {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) y[e] = mul(y[e], inv[u]);
          }
          char* to = dst + u * dst_step + i * (L * 16);
          if (store && u < left && lane[i] && CPATTN_IN(t.y_span, to, 16, p.err))
            *reinterpret_cast<uint4*>(to) = from_pairs(y, T());
        }
    }
  }
}

// dx, and this block's sums of dw to the workspace.
template <typename T, int PAIRING, int L, int V>
__global__ void __launch_bounds__(kThreads, 4) norm_backward_kernel(const __grid_constant__ NormParams p) {
  using S = Shape<T, L, V, 2>;
  constexpr int N = S::N, P = S::P;
  constexpr int64_t es = sizeof(T);
  extern __shared__ __align__(16) unsigned char smem[];
  const int vpr = p.head_dim / N;
  const bool sums = p.ws != nullptr;
  float2* turns = reinterpret_cast<float2*>(smem);
  float* positions = reinterpret_cast<float*>(smem + S::turns(p.rotary_pairs));
  float* weights = positions + S::TOKENS * CPATTN_MAX_ROTARY_AXES;
  T* const rings = reinterpret_cast<T*>(weights + p.n * p.head_dim);
  // a thread's sums of dw over its rows, [n][pair of a thread][thread]
  f2* acc = reinterpret_cast<f2*>(reinterpret_cast<unsigned char*>(rings) + S::rows(p.head_dim));
  const int step = S::TOKENS * p.head_dim;
  const float inv_d = 1.f / p.head_dim;
  const int64_t tiles = (static_cast<int64_t>(p.batch) * p.seq + S::TOKENS - 1) / S::TOKENS;
  if (sums)
    for (int i = 0; i < p.n * V * N / 2; ++i) acc[i * kThreads + threadIdx.x] = 0;
  const int head0 = blockIdx.y * p.head_group, head1 = min(head0 + p.head_group, p.head_start[p.n]);
  launch_wait();
  launch_next();
#pragma unroll 1
  for (int i = threadIdx.x; i < p.n * p.head_dim; i += kThreads) weights[i] = weight(p, i);
#pragma unroll 1
  for (int64_t x = blockIdx.x; x < tiles; x += gridDim.x) {
    const Tile tile(p, x * S::TOKENS);
    const Place<L> at(p, tile);
    T* ring = rings + at.t * p.head_dim;   // step u's: x's two rows at 4 u step, dy's behind them
    Cursor ask = {-1, 0, 0};
    int64_t ask_dy = 0;
    int ask_slot = 0;
    auto request = [&]() {
      if (ask.left <= 0) {
        int h0;
        ask.left = 0;
        if (ask.n < p.n && next_tensor(p, head0, head1, ask.n, h0, ask.left)) {
          const NormTensor& t = p.t[ask.n];
          ask.at = at.b * t.x_s[0] + h0 * t.x_s[1] + at.token * t.x_s[2];
          ask_dy = at.b * t.dy_s[0] + h0 * t.dy_s[1] + at.token * t.dy_s[2];
        }
      }
      if (ask.left > 0) {
        const NormTensor& t = p.t[ask.n];
        const char* src = static_cast<const char*>(t.x) + ask.at * es + at.l * 16;
        const char* grad = static_cast<const char*>(t.dy) + ask_dy * es + at.l * 16;
        const uint32_t dst = smem_addr(ring + ask_slot * 4 * step) + at.l * 16;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (u >= ask.left || !at.active || at.l + i * L >= vpr) continue;
            const char* from = src + u * t.x_s[1] * es + i * (L * 16);
            const char* gfrom = grad + u * t.dy_s[1] * es + i * (L * 16);
            if (CPATTN_IN(t.x_span, from, 16, p.err)) copy16(dst + u * step * es + i * (L * 16), from, true);
            if (CPATTN_IN(t.dy_span, gfrom, 16, p.err)) copy16(dst + (2 + u) * step * es + i * (L * 16), gfrom, true);
          }
        ask.at += 2 * t.x_s[1];
        ask_dy += 2 * t.dy_s[1];
        ask.left -= 2;
      }
      ask_slot = ask_slot + 1 == P ? 0 : ask_slot + 1;
      copies_commit();
    };
    const float pos0 = threadIdx.x < S::TOKENS * p.axes ? position(p, tile, threadIdx.x) : 0.f;
    __syncthreads();   // (the tile before has read its rows and turns)
#pragma unroll 1
    for (int u = 0; u < P - 1; ++u) request();
    if (threadIdx.x < S::TOKENS * CPATTN_MAX_ROTARY_AXES) positions[threadIdx.x] = pos0;
    __syncthreads();
    tile_turns<L>(p, positions, turns);
    __syncthreads();
    Turns<N> turn[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      vector_turns<PAIRING>(p, turns + at.t * p.rotary_pairs, at.l + i * L, at.active, true, turn[i]);
    int n = -1, h0 = 0, rows = 0, slot = 0;
    while (next_tensor(p, head0, head1, n, h0, rows)) {
      const NormTensor& t = p.t[n];
      f2 w[V][N / 2], dw[V][N / 2];
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const int f = n * p.head_dim + (at.l + i * L < vpr ? (at.l + i * L) * N + e : 0);
          w[i][e / 2] = pack2(weights[f], weights[f + 1]);
          dw[i][e / 2] = 0;
        }
      char* dst = static_cast<char*>(t.y) + (at.b * t.y_s[0] + h0 * t.y_s[1] + at.token * t.y_s[2]) * es + at.l * 16;
      const int64_t dst_step = t.y_s[1] * es;
#pragma unroll 1
      for (int r = 0; r < rows; r += 2, dst += 2 * dst_step) {
        copies_wait<P - 2>();
        __syncwarp();   // (the rows before have been read, too)
        request();
        const T* row = ring + slot * 4 * step;
        slot = slot + 1 == P ? 0 : slot + 1;
        f2 x[2][V][N / 2], dz[2][V][N / 2];
        float sum[2], dot[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f2 two = 0, dots = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            uint4 val = make_uint4(0, 0, 0, 0), dval = val;
            const bool in = at.active && r + u < rows && at.l + i * L < vpr;
            if (in) {
              val = reinterpret_cast<const uint4*>(row + u * step)[at.l + i * L];
              dval = reinterpret_cast<const uint4*>(row + (2 + u) * step)[at.l + i * L];
            }
            f2 dy[N / 2], o[N / 2];
            to_pairs(val, x[u][i], T());
            to_pairs(dval, dy, T());
            if constexpr (PAIRING == 0) {
#pragma unroll
              for (int e = 0; e < N / 2; ++e) o[e] = swapped(dy[e]);
            } else {
#pragma unroll
              for (int e = 0; e < N / 2; ++e) o[e] = 0;
              if (in) partners<T, PAIRING>(row + (2 + u) * step, turn[i], o);
            }
            mask_partners(turn[i], o);
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
              dz[u][i][e] = fma(o[e], turn[i].s[e], mul(dy[e], turn[i].c[e]));
              two = fma(x[u][i][e], x[u][i][e], two);
              dots = fma(mul(dz[u][i][e], w[i][e]), x[u][i][e], dots);
            }
          }
          const float2 a = halves_of(two), b = halves_of(dots);
          sum[u] = a.x + a.y;
          dot[u] = b.x + b.y;
        }
#pragma unroll
        for (int m = L / 2; m > 0; m /= 2)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], m);
            dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], m);
          }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // dx = inv (dz w + n f), dw += dz n, with n = x inv
          const float r1 = rsqrtf(fmaf(sum[u], inv_d, p.eps)), r2 = -(r1 * dot[u]) * inv_d;
          const f2 inv = pack2(r1, r1), f = pack2(r2, r2);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (!at.active || r + u >= rows || at.l + i * L >= vpr) continue;
            f2 dx[N / 2];
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
              const f2 normed = mul(x[u][i][e], inv);
              dx[e] = mul(fma(normed, f, mul(dz[u][i][e], w[i][e])), inv);
              dw[i][e] = fma(dz[u][i][e], normed, dw[i][e]);
            }
            char* to = dst + u * dst_step + i * (L * 16);
            if (CPATTN_IN(t.y_span, to, 16, p.err)) __stcs(reinterpret_cast<uint4*>(to), from_pairs(dx, T()));
          }
        }
      }
      if (sums) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            f2& a = acc[((n * V + i) * (N / 2) + e) * kThreads + threadIdx.x];
            const float2 old = halves_of(a), more = halves_of(dw[i][e]);
            a = pack2(old.x + more.x, old.y + more.y);
          }
      }
    }
  }
  if (!sums) return;
  __syncthreads();
  const int part = blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = threadIdx.x; i < p.n * p.head_dim / 2; i += kThreads) {   // a pair of features
    // (neighbouring threads read neighbouring lanes' sums)
    const int n = i / (p.head_dim / 2), k = i - n * (p.head_dim / 2), v = k % vpr, e = k / vpr;
    const f2* from = acc + ((n * V + v / L) * (N / 2) + e) * kThreads + v % L;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int t = 0; t < S::TOKENS; ++t) {
      const float2 more = halves_of(from[t * L]);
      sum = make_float2(sum.x + more.x, sum.y + more.y);
    }
    float2* to = reinterpret_cast<float2*>(p.ws + (static_cast<int64_t>(part) * p.n + n) * p.head_dim + v * N + 2 * e);
    if (CPATTN_IN(p.ws_span, to, 8, p.err)) *to = sum;
  }
}

// dw: the parts' sums, in a fixed order (8 columns a block, 32 threads a column).
__global__ void __launch_bounds__(256) norm_weight_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[32][9];
  const int col = blockIdx.x * 8 + threadIdx.x % 8, y = threadIdx.x / 8;
  const int all = p.n * p.head_dim;
  launch_wait();
  launch_next();
  float sum = 0.f;
  if (col < all)
#pragma unroll 8
    for (int i = y; i < p.parts; i += 32) {
      const float* from = p.ws + static_cast<int64_t>(i) * all + col;
      sum += CPATTN_IN(p.ws_span, from, 4, p.err) ? *from : 0.f;
    }
  sums[y][threadIdx.x % 8] = sum;
  __syncthreads();
  if (y != 0 || col >= all) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += sums[i][threadIdx.x];
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

// Blocks of an SM, forward (registers: see the kernels' launch bounds; interleaved pairs
// with 4 blocks and 5, in turn three times, runs of 60 calls: 4608 tokens x 48 heads 21.3 and
// 23.5 us; halves, 16004 tokens x 48 heads to a cache: 67.0 and 59.1; no run 0.3 off).
int blocks_of_sm(InDtype dt, const NormParams& p) {
  return p.interleaved || p.rotary_pairs == 0 || (dt == InDtype::F32 && p.head_dim > 128) ? 4 : 5;
}
constexpr int64_t kBackwardBlocks = 4;   // of an SM (registers)

// Head groups for `tiles` blocks of tokens: rounds of blocks times a block's heads, and
// its start (turns, weights, first instructions), which costs about as much as 4 heads.
int head_groups(int64_t tiles, int64_t heads, int64_t slots) {
  int64_t best = 1, least = INT64_MAX;
  for (int64_t g = 1; g <= (heads + 3) / 4; ++g) {
    const int64_t cost = (tiles * g + slots - 1) / slots * ((heads + g - 1) / g + 4);
    if (cost < least) {
      least = cost;
      best = g;
    }
    if (tiles * g > 8 * slots) break;   // (a last round is a small part)
  }
  return static_cast<int>(best);
}

struct Grid {
  int64_t x;   // blocks along the tokens
  int y;       // along the heads
  int head_group;
};
// rows: tokens of a block; slots: blocks that run at once.
Grid norm_grid(int rows, int64_t slots, int64_t tokens, int64_t heads, bool backward) {
  Grid g;
  g.x = (tokens + rows - 1) / rows;
  const int64_t groups = head_groups(g.x, heads, slots);
  g.head_group = static_cast<int>((heads + groups - 1) / groups);
  g.y = static_cast<int>((heads + g.head_group - 1) / g.head_group);
  // (backward: a block walks tiles, and leaves one sum of dw)
  if (backward && g.x > slots / g.y) g.x = slots / g.y > 1 ? slots / g.y : 1;
  return g;
}

// Turns and positions (5 KB), weights (4 KB), rows (24 KB, fp32 past 128 features 32) and,
// backward, sums (4 KB a tensor, fp32 past 128 features too).
constexpr size_t kMostShared = 64 * 1024;
template <auto kernel>
cudaError_t norm_run(dim3 grid, size_t smem, cudaStream_t stream, const NormParams& p) {
  static std::atomic<unsigned long long> ready{0};
  const cudaError_t e = cross_set_up(kernel, kMostShared, ready);
  return e == cudaSuccess ? launch_behind(kernel, grid, kThreads, smem, stream, p) : e;
}

template <bool BACKWARD, typename T, int PAIRING, int L, int V>
cudaError_t launch_typed(const NormParams& p, dim3 grid, size_t sums, cudaStream_t stream) {
  using S = Shape<T, L, V, BACKWARD ? 2 : 1>;
  const size_t smem = S::turns(p.rotary_pairs) + S::kPositions + S::weights(p.n, p.head_dim) + S::rows(p.head_dim) + sums;
  if constexpr (BACKWARD) return norm_run<norm_backward_kernel<T, PAIRING, L, V>>(grid, smem, stream, p);
  else return norm_run<norm_rotary_kernel<T, PAIRING, L, V>>(grid, smem, stream, p);
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
  const Grid g = norm_grid(kThreads / lanes(dt, head_dim), kBackwardBlocks * sm_count(), tokens, heads, true);
  return static_cast<int>(g.x) * g.y;
}

cudaError_t launch_norm_rotary(InDtype dt, const NormParams& params, cudaStream_t stream) {
  NormParams p = params;
  const Grid g = norm_grid(kThreads / lanes(dt, p.head_dim), static_cast<int64_t>(sm_count()) * blocks_of_sm(dt, p),
                           static_cast<int64_t>(p.batch) * p.seq, p.head_start[p.n], false);
  p.head_group = g.head_group;
  if (g.x > 0x7fffffff || g.y > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(g.x), g.y);
  return dt == InDtype::BF16 ? launch_pairs<false, __nv_bfloat16>(dt, p, grid, 0, stream)
                             : launch_pairs<false, float>(dt, p, grid, 0, stream);
}

cudaError_t launch_norm_backward(InDtype dt, const NormParams& params, cudaStream_t stream) {
  NormParams p = params;
  const int64_t tokens = static_cast<int64_t>(p.batch) * p.seq;
  const bool sums = p.ws != nullptr;
  if (tokens > 0 && p.head_start[p.n] > 0) {
    const Grid g = norm_grid(kThreads / lanes(dt, p.head_dim), kBackwardBlocks * sm_count(), tokens, p.head_start[p.n], true);
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
  return launch_behind(norm_weight_kernel, dim3((p.n * p.head_dim + 7) / 8), 256, 0, stream, p);
}

}  // namespace cpattn
