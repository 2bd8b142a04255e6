// cross_simt.cu -- cross attention of fp32 inputs and its gradient on the FP32
// pipes (no tf32 rounding), and the join of key-split partials of both types.
//
// Forward, per query row i over the first n = length[b] keys:
//     s_j = scale q_i . k_j,  o = sum_j e^(s_j - m) v_j / l,  lse = m + ln l
// in one pass with the running maximum m and sum l (fp32, base 2).
// Gradient, with p_ij = e^(s_ij - lse_i) and delta_i = sum_d do_id o_id:
//     ds_ij = p_ij (do_i . v_j - delta_i)
//     dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// dk and dv of a shared key head sum over its query heads.  Two kernels, one
// owning query rows (dq), one owning keys (dk, dv): every sum has one owner
// and a fixed order, at the price of forming s and do . v twice.
//
// Layout, for calls of fewer rows than cross_f32.cu takes: a warp owns R rows
// (query rows, or keys in the dk/dv kernel), its lanes own C rows each of a 32
// C-row tile of the other side for the dot products over D, and D / 32 features
// each for the products over the tile.
// A tile row is padded by 16 bytes, so both walks are free of bank conflicts.
// R = 2, C = 1: the blocks are small, so few rows make many of them; what
// bounds them is shared memory and the latency of a short walk (one query x 500
// keys x 16 heads 10.7 us, its gradient 52; 256 queries x 77 keys x 4 heads at
// D = 64 6.9, host-bound).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "cross.cuh"
#include "ptx.cuh"

namespace cpattn {
namespace {

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.442695040888963407f;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&f)[N]) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (N == 4)
      *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      *reinterpret_cast<__nv_bfloat162*>(p + i) = __floats2bfloat162_rn(f[i], f[i + 1]);
  }
}

template <int N>
__device__ __forceinline__ void load_lane(const float* p, float (&f)[N]) {
  if constexpr (N == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    f[0] = t.x; f[1] = t.y; f[2] = t.z; f[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(p);
    f[0] = t.x; f[1] = t.y;
  }
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Requests rows [row0, row0 + rows) of one head into a tile of padded rows;
// rows at or past `end` become zero and are not read (they may hold anything).
template <int D>
__device__ __forceinline__ void fill_tile(const CrossParams& p, const CrossTensor& t, int b, int h,
                                          int row0, int rows, int end, float* tile, int stride) {
  const float* head = static_cast<const float*>(t.data) + b * t.s[0] + h * t.s[1];
  for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    const float* src = head + static_cast<int64_t>(row0 + r) * t.s[2] + c;
    const bool read = row0 + r < end && CPATTN_IN(t.span, src, 16, p.err);
    copy16(smem_addr(tile + r * stride + c), read ? src : head, read);
  }
}

// dot products of R broadcast rows (dense, stride D) with this lane's tile
// rows, lane, lane + 32, ...
template <int D, int R, int C>
__device__ __forceinline__ void dots(const float* rows, const float* tile, float (&s)[R][C]) {
  const float* mine = tile + (threadIdx.x % 32) * (D + 4);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) s[r][c] = 0.f;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 k[C];
#pragma unroll
    for (int c = 0; c < C; ++c) k[c] = *reinterpret_cast<const float4*>(mine + c * 32 * (D + 4) + d);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 q = *reinterpret_cast<const float4*>(rows + r * D + d);
#pragma unroll
      for (int c = 0; c < C; ++c)
        s[r][c] = fmaf(q.x, k[c].x, fmaf(q.y, k[c].y, fmaf(q.z, k[c].z, fmaf(q.w, k[c].w, s[r][c]))));
    }
  }
}

// acc[r][f] += sum over the tile's 32 C rows j of w[r][j] tile[j][lane's features]
template <int D, int R, int C>
__device__ __forceinline__ void spread(const float* w, const float* tile, float (&acc)[R][D / 32]) {
  constexpr int F = D / 32;
  const int lane = threadIdx.x % 32;
#pragma unroll 2
  for (int j = 0; j < 32 * C; j += 4) {
    float t[4][F];
#pragma unroll
    for (int u = 0; u < 4; ++u) load_lane<F>(tile + (j + u) * (D + 4) + lane * F, t[u]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(w + r * 32 * C + j);
#pragma unroll
      for (int f = 0; f < F; ++f)
        acc[r][f] = fmaf(x.x, t[0][f], fmaf(x.y, t[1][f], fmaf(x.z, t[2][f], fmaf(x.w, t[3][f], acc[r][f]))));
    }
  }
}

// ------------------------------------------------------------------ forward
// W warps as W / KS groups of R query rows; the KS warps of a group take every
// KS-th 32 C-key tile and are joined at the end.
template <int D, int W, int R, int C, int KS>
__global__ void __launch_bounds__(W * 32) cross_simt_kernel(const __grid_constant__ CrossParams p) {
  constexpr int F = D / 32, ROWS = (W / KS) * R, PAD = D + 4, T1 = 32 * C, TK = T1 * KS;
  extern __shared__ __align__(16) float sm[];
  launch_wait();
  launch_next();
  float* sQ = sm;                          // [ROWS][D]
  float* sKV = sQ + ROWS * D;              // two stages of K and V, [TK][PAD] each
  float* sP = sKV + 4 * TK * PAD;          // [W][R][T1]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int group = warp / KS, part = warp % KS;
  const int tiles = (p.s_q + ROWS - 1) / ROWS, bh = blockIdx.x / tiles;
  const int row0 = (blockIdx.x - bh * tiles) * ROWS;
  const int h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.kv_heads);
  const int len = cross_length(p, b);
  // this split's keys: whole tiles, dealt out evenly
  const int all_tiles = (len + TK - 1) / TK;
  const int per = (all_tiles + p.splits - 1) / p.splits;
  const int t_begin = min(static_cast<int>(blockIdx.y) * per, all_tiles), t_end = min(t_begin + per, all_tiles);

  fill_tile<D>(p, p.q, b, h, row0, ROWS, p.s_q, sQ, D);
  float o[R][F], m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int f = 0; f < F; ++f) o[r][f] = 0.f;
  }
  float* myP = sP + warp * R * T1;
  auto request = [&](int t) {
    if (t < t_end) {
      float* stage = sKV + ((t - t_begin) & 1) * 2 * TK * PAD;
      fill_tile<D>(p, p.k, b, hk, t * TK, TK, len, stage, PAD);
      fill_tile<D>(p, p.v, b, hk, t * TK, TK, len, stage + TK * PAD, PAD);
    }
    copies_commit();
  };
  request(t_begin);   // (with the query rows)
  for (int t = t_begin; t < t_end; ++t) {
    request(t + 1);
    copies_wait<1>();
    __syncthreads();
    const float* sK = sKV + ((t - t_begin) & 1) * 2 * TK * PAD;
    const float* sV = sK + TK * PAD;
    const int valid = len - (t * KS + part) * T1 - lane;   // row lane + 32 c is a key where 32 c < valid
    float s[R][C];
    dots<D, R, C>(sQ + group * R * D, sK + part * T1 * PAD, s);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x = -INFINITY;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        s[r][c] = 32 * c < valid ? s[r][c] * p.scale_log2 : -INFINITY;
        x = fmaxf(x, s[r][c]);
      }
      const float top = fmaxf(m[r], warp_max(x));
      const float base = top == -INFINITY ? 0.f : top;
      const float f = exp2f(m[r] - base);
      m[r] = top;
      l[r] *= f;   // (this lane's share of the sum)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float e = exp2f(s[r][c] - base);
        l[r] += e;
        myP[r * T1 + c * 32 + lane] = e;
      }
#pragma unroll
      for (int i = 0; i < F; ++i) o[r][i] *= f;
    }
    __syncwarp();
    spread<D, R, C>(myP, sV + part * T1 * PAD, o);
    __syncthreads();   // (this stage may be filled again)
  }
  copies_wait<0>();
#pragma unroll
  for (int r = 0; r < R; ++r) l[r] = warp_sum(l[r]);
  if constexpr (KS > 1) {
    // join the group's KS parts through shared memory (K and V are done with)
    __syncthreads();
    float* so = sKV;                       // [W][R][D]
    float* sml = sP;                       // [W][R][2]
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int f = 0; f < F; ++f) so[(warp * R + r) * D + lane * F + f] = o[r][f];
      if (lane == 0) {
        sml[(warp * R + r) * 2] = m[r];
        sml[(warp * R + r) * 2 + 1] = l[r];
      }
    }
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = m[r];
      for (int x = 1; x < KS; ++x) top = fmaxf(top, sml[((warp + x) * R + r) * 2]);
      const float base = top == -INFINITY ? 0.f : top;
      const float f0 = exp2f(m[r] - base);
      l[r] *= f0;
#pragma unroll
      for (int f = 0; f < F; ++f) o[r][f] *= f0;
      for (int x = 1; x < KS; ++x) {
        const float fx = exp2f(sml[((warp + x) * R + r) * 2] - base);
        l[r] = fmaf(sml[((warp + x) * R + r) * 2 + 1], fx, l[r]);
#pragma unroll
        for (int f = 0; f < F; ++f)
          o[r][f] = fmaf(so[((warp + x) * R + r) * D + lane * F + f], fx, o[r][f]);
      }
      m[r] = top;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + group * R + r;
    if (row >= p.s_q) continue;
    const bool empty = !(l[r] > 0.f);   // (NaN sums stay NaN below)
    const bool none = empty && !(l[r] != l[r]);
    const float inv = none ? 0.f : 1.f / l[r];
    float res[F];
#pragma unroll
    for (int f = 0; f < F; ++f) res[f] = o[r][f] * inv;
    const float lse = none ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
    if (p.splits > 1) {
      const int64_t n = static_cast<int64_t>(p.batch) * p.heads * p.s_q;
      const int64_t at = blockIdx.y * n + static_cast<int64_t>(bh) * p.s_q + row;
      float* dst = p.ws + at * D + lane * F;
      float* dl = p.ws + p.splits * n * D + at;
      if (CPATTN_IN(p.ws_span, dst, 4 * F, p.err)) store_n<float, F>(dst, res);
      if (lane == 0 && CPATTN_IN(p.ws_span, dl, 4, p.err)) *dl = lse;
    } else {
      float* dst = static_cast<float*>(p.out.data) + b * p.out.s[0] + h * p.out.s[1] + row * p.out.s[2] + lane * F;
      if (CPATTN_IN(p.out.span, dst, 4 * F, p.err)) store_n<float, F>(dst, res);
      float* dl = static_cast<float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + row * p.lse.s[2];
      if (lane == 0 && CPATTN_IN(p.lse.span, dl, 4, p.err)) *dl = lse;
    }
  }
}

// ------------------------------------------------------------------ join
// One warp per query row: weights e^(lse_x - lse) of the row's parts.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ CrossParams p) {
  constexpr int F = D / 32;
  const int lane = threadIdx.x % 32;
  const int64_t n = static_cast<int64_t>(p.batch) * p.heads * p.s_q;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  launch_wait();   // (the parts are written)
  launch_next();
  if (at >= n) return;
  const float* pl = p.ws + p.splits * n * D + at;
  float top = -INFINITY;
  for (int x = lane; x < p.splits; x += 32)
    if (CPATTN_IN(p.ws_span, pl + x * n, 4, p.err)) top = fmaxf(top, pl[x * n]);
  top = warp_max(top);
  float o[F] = {}, total = 0.f;
  const float base = top == -INFINITY ? 0.f : top;
  for (int x0 = 0; x0 < p.splits; x0 += 32) {
    // a lane's own part's weight, 0 for a part without keys (which is not read)
    float mine = 0.f;
    if (x0 + lane < p.splits && CPATTN_IN(p.ws_span, pl + (x0 + lane) * n, 4, p.err))
      mine = exp2f((pl[(x0 + lane) * n] - base) * kLog2e);
    const int count = min(32, p.splits - x0);
#pragma unroll 8
    for (int x = 0; x < count; ++x) {
      const float w = __shfl_sync(0xffffffffu, mine, x);
      const float* src = p.ws + ((x0 + x) * n + at) * D + lane * F;
      float t[F] = {};
      if (w != 0.f && CPATTN_IN(p.ws_span, src, 4 * F, p.err)) load_lane<F>(src, t);
      total += w;
#pragma unroll
      for (int f = 0; f < F; ++f) o[f] = fmaf(w, t[f], o[f]);
    }
  }
  const bool none = total == 0.f;
  const float inv = none ? 0.f : 1.f / total;
#pragma unroll
  for (int f = 0; f < F; ++f) o[f] *= inv;
  const int64_t row = at % p.s_q, bh = at / p.s_q, h = bh % p.heads, b = bh / p.heads;
  T* dst = static_cast<T*>(p.out.data) + b * p.out.s[0] + h * p.out.s[1] + row * p.out.s[2] + lane * F;
  if (CPATTN_IN(p.out.span, dst, F * sizeof(T), p.err)) store_n<T, F>(dst, o);
  float* dl = static_cast<float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + row * p.lse.s[2];
  if (lane == 0 && CPATTN_IN(p.lse.span, dl, 4, p.err))
    *dl = none ? -INFINITY : base + log2f(total) * kLn2;
}

// ------------------------------------------------------------------ gradient
// delta_i = sum_d do_id o_id, one warp per query row, dense [B, H, S_q] fp32
// at the workspace's start.
template <int D>
__global__ void __launch_bounds__(256) cross_delta_kernel(const __grid_constant__ CrossParams p) {
  constexpr int PER = D / 4;   // lanes of a row
  const int64_t n = static_cast<int64_t>(p.batch) * p.heads * p.s_q;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t at = i / PER;
  const int c = static_cast<int>(i % PER) * 4;
  float d = 0.f;
  launch_wait();
  launch_next();
  if (at < n) {
    const int64_t row = at % p.s_q, bh = at / p.s_q, h = bh % p.heads, b = bh / p.heads;
    const float* o = static_cast<const float*>(p.out.data) + b * p.out.s[0] + h * p.out.s[1] + row * p.out.s[2] + c;
    const float* g = static_cast<const float*>(p.dout.data) + b * p.dout.s[0] + h * p.dout.s[1] + row * p.dout.s[2] + c;
    if (CPATTN_IN(p.out.span, o, 16, p.err) && CPATTN_IN(p.dout.span, g, 16, p.err)) {
      const float4 x = load4(o), y = load4(g);
      d = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
    }
  }
#pragma unroll
  for (int o = PER / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (at < n && c == 0 && CPATTN_IN(p.ws_span, p.ws + at, 4, p.err)) p.ws[at] = d;
}

// dq: a warp owns R query rows and walks the keys.
template <int D, int W, int R, int C>
__global__ void __launch_bounds__(W * 32) cross_simt_dq_kernel(const __grid_constant__ CrossParams p) {
  constexpr int F = D / 32, ROWS = W * R, PAD = D + 4, T1 = 32 * C;
  extern __shared__ __align__(16) float sm[];
  launch_wait();
  launch_next();
  float* sQ = sm;                          // [ROWS][D]
  float* sG = sQ + ROWS * D;               // [ROWS][D] dout
  float* sKV = sG + ROWS * D;              // two stages of K and V, [T1][PAD] each
  float* sS = sKV + 4 * T1 * PAD;          // [W][R][T1]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tiles = (p.s_q + ROWS - 1) / ROWS, bh = blockIdx.x / tiles;
  const int row0 = (blockIdx.x - bh * tiles) * ROWS;
  const int h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.kv_heads);
  const int len = cross_length(p, b);
  fill_tile<D>(p, p.q, b, h, row0, ROWS, p.s_q, sQ, D);
  fill_tile<D>(p, p.dout, b, h, row0, ROWS, p.s_q, sG, D);
  float dq[R][F], lse2[R], delta[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + warp * R + r;
    lse2[r] = INFINITY;   // (rows past the end: p = 0)
    delta[r] = 0.f;
    if (row < p.s_q) {
      const float* l = static_cast<const float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + row * p.lse.s[2];
      const float* d = p.ws + static_cast<int64_t>(bh) * p.s_q + row;
      if (CPATTN_IN(p.lse.span, l, 4, p.err)) lse2[r] = cross_lse2(*l);
      if (CPATTN_IN(p.ws_span, d, 4, p.err)) delta[r] = *d;
    }
#pragma unroll
    for (int f = 0; f < F; ++f) dq[r][f] = 0.f;
  }
  float* myS = sS + warp * R * T1;
  auto request = [&](int k0) {
    if (k0 < len) {
      float* stage = sKV + ((k0 / T1) & 1) * 2 * T1 * PAD;
      fill_tile<D>(p, p.k, b, hk, k0, T1, len, stage, PAD);
      fill_tile<D>(p, p.v, b, hk, k0, T1, len, stage + T1 * PAD, PAD);
    }
    copies_commit();
  };
  request(0);   // (with the query rows)
  for (int k0 = 0; k0 < len; k0 += T1) {
    request(k0 + T1);
    copies_wait<1>();
    __syncthreads();
    const float* sK = sKV + ((k0 / T1) & 1) * 2 * T1 * PAD;
    const float* sV = sK + T1 * PAD;
    float s[R][C], g[R][C];
    dots<D, R, C>(sQ + warp * R * D, sK, s);
    dots<D, R, C>(sG + warp * R * D, sV, g);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float e = k0 + 32 * c + lane < len ? exp2f(fmaf(s[r][c], p.scale_log2, -lse2[r])) : 0.f;
        // (one key has all the weight whatever q is)
        myS[r * T1 + c * 32 + lane] = len > 1 ? e * (g[r][c] - delta[r]) : 0.f;
      }
    __syncwarp();
    spread<D, R, C>(myS, sK, dq);
    __syncthreads();   // (this stage may be filled again)
  }
  copies_wait<0>();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + warp * R + r;
    if (row >= p.s_q) continue;
    float res[F];
#pragma unroll
    for (int f = 0; f < F; ++f) res[f] = dq[r][f] * p.scale;
    float* dst = static_cast<float*>(p.dq.data) + b * p.dq.s[0] + h * p.dq.s[1] + row * p.dq.s[2] + lane * F;
    if (CPATTN_IN(p.dq.span, dst, 4 * F, p.err)) store_n<float, F>(dst, res);
  }
}

// dk, dv: a warp owns R keys and walks the query rows of every query head
// that shares the key head.
template <int D, int W, int R, int C>
__global__ void __launch_bounds__(W * 32) cross_simt_dkv_kernel(const __grid_constant__ CrossParams p) {
  constexpr int F = D / 32, KEYS = W * R, PAD = D + 4, T1 = 32 * C;
  extern __shared__ __align__(16) float sm[];
  launch_wait();
  launch_next();
  float* sK = sm;                          // [KEYS][D]
  float* sV = sK + KEYS * D;
  float* sQG = sV + KEYS * D;              // two stages of Q and dO, [T1][PAD] each
  float* sS = sQG + 4 * T1 * PAD;          // [W][R][T1] ds
  float* sP = sS + W * R * T1;             // [W][R][T1] p
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tiles = (p.s_kv + KEYS - 1) / KEYS, bk = blockIdx.x / tiles;
  const int key0 = (blockIdx.x - bk * tiles) * KEYS;
  const int hk = bk % p.kv_heads, b = bk / p.kv_heads;
  const int share = p.heads / p.kv_heads;
  const int len = cross_length(p, b);
  float dk[R][F], dv[R][F];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int f = 0; f < F; ++f) dk[r][f] = dv[r][f] = 0.f;
  float* myS = sS + warp * R * T1;
  float* myP = sP + warp * R * T1;
  if (key0 < len) {
    fill_tile<D>(p, p.k, b, hk, key0, KEYS, len, sK, D);
    fill_tile<D>(p, p.v, b, hk, key0, KEYS, len, sV, D);
    // steps: the query tiles of one head after the other
    const int tiles_q = (p.s_q + T1 - 1) / T1, steps = share * tiles_q;
    auto request = [&](int x) {
      if (x < steps) {
        float* stage = sQG + (x & 1) * 2 * T1 * PAD;
        const int g = x / tiles_q, i0 = (x - g * tiles_q) * T1, h = hk * share + g;
        fill_tile<D>(p, p.q, b, h, i0, T1, p.s_q, stage, PAD);
        fill_tile<D>(p, p.dout, b, h, i0, T1, p.s_q, stage + T1 * PAD, PAD);
      }
      copies_commit();
    };
    request(0);   // (with the keys and values)
    for (int x = 0; x < steps; ++x) {
      request(x + 1);
      const int g = x / tiles_q, i0 = (x - g * tiles_q) * T1, h = hk * share + g;
      float lse2[C], delta[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int row = i0 + 32 * c + lane;
        lse2[c] = INFINITY;
        delta[c] = 0.f;
        if (row < p.s_q) {
          const float* l = static_cast<const float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + row * p.lse.s[2];
          const float* d = p.ws + (static_cast<int64_t>(b) * p.heads + h) * p.s_q + row;
          if (CPATTN_IN(p.lse.span, l, 4, p.err)) lse2[c] = cross_lse2(*l);
          if (CPATTN_IN(p.ws_span, d, 4, p.err)) delta[c] = *d;
        }
      }
      copies_wait<1>();
      __syncthreads();
      const float* sQ = sQG + (x & 1) * 2 * T1 * PAD;
      const float* sG = sQ + T1 * PAD;
      float s[R][C], e[R][C];
      dots<D, R, C>(sK + warp * R * D, sQ, s);
      dots<D, R, C>(sV + warp * R * D, sG, e);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          // (rows past the end: 0 k_j need not be 0)
          const bool on = key0 + warp * R + r < len && i0 + 32 * c + lane < p.s_q;
          const float pr = on ? exp2f(fmaf(s[r][c], p.scale_log2, -lse2[c])) : 0.f;
          myP[r * T1 + c * 32 + lane] = pr;
          myS[r * T1 + c * 32 + lane] = on && len > 1 ? pr * (e[r][c] - delta[c]) : 0.f;   // (as in the dq kernel)
        }
      __syncwarp();
      spread<D, R, C>(myP, sG, dv);
      spread<D, R, C>(myS, sQ, dk);
      __syncthreads();   // (this stage may be filled again)
    }
    copies_wait<0>();
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int key = key0 + warp * R + r;
    if (key >= p.s_kv) continue;
    float res[F];
#pragma unroll
    for (int f = 0; f < F; ++f) res[f] = dk[r][f] * p.scale;
    float* d1 = static_cast<float*>(p.dk.data) + b * p.dk.s[0] + hk * p.dk.s[1] + key * p.dk.s[2] + lane * F;
    float* d2 = static_cast<float*>(p.dv.data) + b * p.dv.s[0] + hk * p.dv.s[1] + key * p.dv.s[2] + lane * F;
    if (CPATTN_IN(p.dk.span, d1, 4 * F, p.err)) store_n<float, F>(d1, res);
#pragma unroll
    for (int f = 0; f < F; ++f) res[f] = dv[r][f];
    if (CPATTN_IN(p.dv.span, d2, 4 * F, p.err)) store_n<float, F>(d2, res);
  }
}


// Sums the parts of dk and dv in their order: one thread per four values.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_dkv_join_kernel(const __grid_constant__ CrossParams p, const int64_t partials) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.kv_heads * p.s_kv, n = rows * (D / 4);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  launch_wait();   // (the parts are written)
  launch_next();
  if (i >= 2 * n) return;
  const int which = i >= n;   // 0: dk, 1: dv
  const int64_t at = i - which * n;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* src = reinterpret_cast<const float4*>(p.ws + partials) + which * n + at;
#pragma unroll 4
  for (int x = 0; x < p.splits; ++x) {
    const float4* s = src + 2 * x * n;
    if (!CPATTN_IN(p.ws_span, s, 16, p.err)) continue;
    const float4 v = *s;
    sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
  }
  const float f = which ? 1.f : p.scale;
  const CrossTensor& t = which ? p.dv : p.dk;
  const int64_t row = at / (D / 4), key = row % p.s_kv, bh = row / p.s_kv, h = bh % p.kv_heads, b = bh / p.kv_heads;
  T* dst = static_cast<T*>(t.data) + b * t.s[0] + h * t.s[1] + key * t.s[2] + (at % (D / 4)) * 4;
  const float res[4] = {sum.x * f, sum.y * f, sum.z * f, sum.w * f};
  if (CPATTN_IN(t.span, dst, 4 * sizeof(T), p.err)) store_n<T, 4>(dst, res);
}

// A gradient without terms (no queries, or no keys): zeros.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_zero_kernel(const CrossTensor t, int batch, int heads, int rows, unsigned int* err) {
  constexpr int PER = D * sizeof(T) / 16;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t at = i / PER;
  const int64_t row = at % rows, h = at / rows % heads, b = at / rows / heads;
  launch_wait();
  launch_next();
  if (b >= batch) return;
  T* dst = static_cast<T*>(t.data) + b * t.s[0] + h * t.s[1] + row * t.s[2] + (i % PER) * (16 / sizeof(T));
  if (CPATTN_IN(t.span, dst, 16, err)) *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
}

int64_t tiles_of(int rows, int per) { return (rows + per - 1) / per; }

// Shared memory of the kernels in floats: the rows a block owns, two stages of
// two tiles, the warps' weights.
constexpr size_t simt_smem(int D, int rows, int tile, int weights) {
  return sizeof(float) * (static_cast<size_t>(rows) * D + 4 * tile * (D + 4) + weights);
}


template <int D>
cudaError_t forward_typed(const CrossParams& p, cudaStream_t stream) {
  const int64_t bh = static_cast<int64_t>(p.batch) * p.heads;
  if (cross_f32_rows(tiles_of(p.s_q, 64) * bh, static_cast<int64_t>(p.s_kv) * D)) return launch_cross_f32(D, p, stream);
  // 8 or 16 rows a block, and for one or two queries 2, the KS warps of each
  // row taking every KS-th tile
  constexpr int KS = D == 64 ? 4 : 2;
  if (p.s_q > 2)
    return cross_run<cross_simt_kernel<D, 16, 2, 1, KS>>(tiles_of(p.s_q, 32 / KS) * bh, p.splits, 512,
                                                         simt_smem(D, 32 / KS, 32 * KS, 16 * 2 * 32), stream, p);
  return cross_run<cross_simt_kernel<D, KS, 2, 1, KS>>(tiles_of(p.s_q, 2) * bh, p.splits, 32 * KS,
                                                       simt_smem(D, 2, 32 * KS, KS * 2 * 32), stream, p);
}

template <int D>
cudaError_t backward_typed(const CrossParams& p, int64_t partials, cudaStream_t stream) {
  const int64_t bh = static_cast<int64_t>(p.batch) * p.heads;
  const int64_t bk = static_cast<int64_t>(p.batch) * p.kv_heads;
  const int64_t n = bh * p.s_q * (D / 4);
  if ((n + 255) / 256 > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = launch_behind(cross_delta_kernel<D>, dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, stream, p);
  if (e != cudaSuccess) return e;
  // (dq takes no splits: 64-row blocks from a quarter of the SMs; 32 blocks x
  // 100 keys at D = 64: 26 us without, 30 with)
  if (tiles_of(p.s_q, 64) * bh * 4 >= sm_count())
    e = launch_cross_f32_dq(D, p, stream);
  else
    e = cross_run<cross_simt_dq_kernel<D, 4, 2, 1>>(tiles_of(p.s_q, 8) * bh, 1, 128, simt_smem(D, 16, 32, 4 * 2 * 32),
                                                    stream, p);
  if (e != cudaSuccess) return e;
  if (cross_f32_keys(tiles_of(p.s_kv, 64) * bk * tiles_of(p.s_q, 64) * (p.heads / p.kv_heads))) {
    e = launch_cross_f32_dkv(D, p, partials, stream);
    return e == cudaSuccess && p.splits > 1 ? launch_cross_dkv_join(InDtype::F32, D, p, partials, stream) : e;
  }
  return cross_run<cross_simt_dkv_kernel<D, 4, 2, 1>>(tiles_of(p.s_kv, 8) * bk, 1, 128,
                                                      simt_smem(D, 16, 32, 2 * 4 * 2 * 32), stream, p);
}

template <typename T, int D>
cudaError_t zero_typed(const CrossParams& p, const CrossTensor& t, int heads, int rows, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(p.batch) * heads * rows * (D * sizeof(T) / 16);
  if (n == 0) return cudaSuccess;
  if ((n + 255) / 256 > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_behind(cross_zero_kernel<T, D>, dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, stream, t, p.batch,
                       heads, rows, p.err);
}

template <typename T, int D>
cudaError_t zeros_typed(const CrossParams& p, cudaStream_t stream) {
  cudaError_t e = zero_typed<T, D>(p, p.dq, p.heads, p.s_q, stream);
  if (e == cudaSuccess) e = zero_typed<T, D>(p, p.dk, p.kv_heads, p.s_kv, stream);
  return e == cudaSuccess ? zero_typed<T, D>(p, p.dv, p.kv_heads, p.s_kv, stream) : e;
}

}  // namespace

cudaError_t launch_cross_simt(int head_dim, const CrossParams& p, cudaStream_t stream) {
  return head_dim == 64 ? forward_typed<64>(p, stream) : forward_typed<128>(p, stream);
}

cudaError_t launch_cross_simt_backward(int head_dim, const CrossParams& p, int64_t partials, cudaStream_t stream) {
  return head_dim == 64 ? backward_typed<64>(p, partials, stream) : backward_typed<128>(p, partials, stream);
}

// Against the kernels of this file, us, this / 64-row blocks.  Forward, 8 heads at
// D = 128: 64 queries (8 blocks) x 512 keys 23.7 / 20.7, 128 queries (16 blocks) x
// 512 keys 38.6 / 21.0, x 1500 keys 109.6 / 36.3, x 100 keys 11.9 / 16.3; at D = 64
// x 512 keys 14.2 / 15.2, x 1500 keys 36.2 / 23.7; 512 queries x 512 keys at D = 128
// 77 / 36.  Gradient (dk, dv), 128 queries x 100 keys x 16 heads at D = 64 (64 tiles)
// 26 / 41, 256 x 512 x 2 heads (64 tiles) 75 / 61, 128 x 512 x 8 heads (128 tiles)
// 99 / 92, 300 x 256 x 16 heads at D = 64 (320 tiles) 84 / 76.
bool cross_f32_rows(int64_t blocks, int64_t values) {
  return blocks * 8 >= sm_count() || (blocks * 16 >= sm_count() && values >= 512 * 128);
}
bool cross_f32_keys(int64_t tiles) { return tiles * 2 >= sm_count(); }

int cross_f32_parts(int64_t key_units, int64_t steps) {
  if (!cross_f32_keys(key_units * steps)) return 1;
  // as cross_backward_parts: a block's start and end count as one step, the
  // join as one
  const int64_t sms = sm_count();
  int best = 1;
  int64_t least = 0;
  for (int parts = 1; parts <= 32 && parts <= steps; ++parts) {
    const int64_t waves = (key_units * parts + sms - 1) / sms;
    const int64_t cost = waves * ((steps + parts - 1) / parts + 1) + (parts > 1 ? 1 : 0);
    if (parts == 1 || cost < least) {
      best = parts;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_cross_dkv_join(InDtype dt, int head_dim, const CrossParams& p, int64_t partials,
                                  cudaStream_t stream) {
  const int64_t blocks = (2 * static_cast<int64_t>(p.batch) * p.kv_heads * p.s_kv * (head_dim / 4) + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (dt == InDtype::BF16)
    return launch_behind(head_dim == 64 ? cross_dkv_join_kernel<__nv_bfloat16, 64> : cross_dkv_join_kernel<__nv_bfloat16, 128>,
                         grid, 256, 0, stream, p, partials);
  return launch_behind(head_dim == 64 ? cross_dkv_join_kernel<float, 64> : cross_dkv_join_kernel<float, 128>, grid, 256, 0,
                       stream, p, partials);
}

cudaError_t launch_cross_zeros(InDtype dt, int head_dim, const CrossParams& p, cudaStream_t stream) {
  if (dt == InDtype::BF16)
    return head_dim == 64 ? zeros_typed<__nv_bfloat16, 64>(p, stream) : zeros_typed<__nv_bfloat16, 128>(p, stream);
  return head_dim == 64 ? zeros_typed<float, 64>(p, stream) : zeros_typed<float, 128>(p, stream);
}

cudaError_t launch_cross_join(InDtype dt, int head_dim, const CrossParams& p, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(p.batch) * p.heads * p.s_q;
  if ((n + 7) / 8 > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 blocks(static_cast<unsigned>((n + 7) / 8));
  if (dt == InDtype::BF16)
    return launch_behind(head_dim == 64 ? cross_join_kernel<__nv_bfloat16, 64> : cross_join_kernel<__nv_bfloat16, 128>,
                         blocks, 256, 0, stream, p);
  return launch_behind(head_dim == 64 ? cross_join_kernel<float, 64> : cross_join_kernel<float, 128>, blocks, 256, 0,
                       stream, p);
}

}  // namespace cpattn
