// cross_f32.cu -- cross attention of fp32 inputs and its gradient on the FP32
// pipes, for calls with rows enough to fill the GPU with 64-row blocks (the
// others: cross_simt.cu, which has the formulas).
//
// What bounds it: the FP32 pipes, 128 multiply-adds a cycle and SM, as long as
// shared memory keeps up.  A 16-byte load costs a warp two cycles there as long
// as its address depends on at most one of lane bits 0 and 1 (up to 16 distinct
// addresses), four otherwise, even where one broadcast address serves all.  So a
// thread takes 8 x 4 elements of a product, (8 + 4) loads = 24 cycles for 128
// multiply-adds of a warp = 32 cycles, and the lanes lie 4 x 8 over a warp's
// 32 x 32 elements with row bits {0, 2} and column bits {1, 3, 4}.  Dot products
// add two features at once (fma.f32x2), which halves their issue slots.
//
// 8 warps own 64 rows and walk the other side in tiles.  In the gradient warps
// 0-3 form a tile's q.k, warps 4-7 its do.v, so a thread holds one of the two;
// they meet in shared memory.  dk and dv take the query axis in parts where
// that fills the GPU's last round, joined by cross_dkv_join.
// Measured at 1024 queries x 512 keys x 24 heads, D = 128: forward 173 us (37
// TFLOP/s; 203 with a warp's rows read as broadcasts), gradient 615 us (37
// TFLOP/s of its seven products; 848); 48 heads at D = 64: 187 and 778 us.  The
// pipes reach 75 TFLOP/s alone; a tile's exponentials, their exchange and the
// barriers, and a third round of blocks that is half full, take the rest.
#include <cuda_runtime.h>

#include <cmath>

#include "cross.cuh"
#include "ptx.cuh"

namespace cpattn {
namespace {

constexpr int kOwn = 64;         // rows a block owns
constexpr int kThreads = 256;
constexpr float kLn2 = 0.693147180559945309f;

// This lane's row of 4 and column of 8 in a warp's tile (see above).
__device__ __forceinline__ int lane_row() { return (threadIdx.x & 1) | ((threadIdx.x >> 1) & 2); }
__device__ __forceinline__ int lane_col() { return ((threadIdx.x >> 1) & 1) | ((threadIdx.x >> 2) & 6); }
// A sum, a maximum over the 8 lanes of a row.
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

__device__ __forceinline__ void fma_pair(unsigned long long& acc, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// s[i][j] = row i of a . row j of b: a at this lane's first row of 8 in steps
// of 4, b at its first of 4 in steps of 8; rows are D + 4 floats apart.
template <int D>
__device__ __forceinline__ void dots(const float* a, const float* b, float (&s)[8][4]) {
  constexpr int PAD = D + 4;
  if constexpr (D == 64) {   // (two blocks an SM: no registers for pairs)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
    for (int d = 0; d < D; d += 4) {
      float4 y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + j * 8 * PAD + d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(a + i * 4 * PAD + d);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(x.x, y[j].x, fmaf(x.y, y[j].y, fmaf(x.z, y[j].z, fmaf(x.w, y[j].w, s[i][j]))));
      }
    }
    return;
  }
  unsigned long long acc[8][4];   // sums over even and over odd features
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    ulonglong2 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(b + j * 8 * PAD + d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(a + i * 4 * PAD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        fma_pair(acc[i][j], x.x, y[j].x);
        fma_pair(acc[i][j], x.y, y[j].y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s[i][j] = __uint_as_float(static_cast<unsigned>(acc[i][j])) + __uint_as_float(static_cast<unsigned>(acc[i][j] >> 32));
}

// N consecutive floats.
template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&f)[N]) {
  if constexpr (N == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    f[0] = t.x; f[1] = t.y; f[2] = t.z; f[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(p);
    f[0] = t.x; f[1] = t.y;
  }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&f)[N], float scale) {
  if constexpr (N == 4)
    *reinterpret_cast<float4*>(p) = make_float4(f[0] * scale, f[1] * scale, f[2] * scale, f[3] * scale);
  else
    *reinterpret_cast<float2*>(p) = make_float2(f[0] * scale, f[1] * scale);
}

// acc[i][f] += sum over tile rows j < n of w[row i][j] tile[j][feature f]: w at
// this lane's first row of 8 in steps of 4 (rows W floats apart), tile at its
// first feature; n a multiple of 4.
template <int D, int W>
__device__ __forceinline__ void spread(const float* w, const float* tile, int n, float (&acc)[8][D / 32]) {
  constexpr int F = D / 32;
#pragma unroll 4
  for (int j = 0; j < n; j += 4) {
    float t[4][F];
#pragma unroll
    for (int u = 0; u < 4; ++u) load_n<F>(tile + (j + u) * (D + 4), t[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(w + i * 4 * W + j);
#pragma unroll
      for (int f = 0; f < F; ++f)
        acc[i][f] = fmaf(x.x, t[0][f], fmaf(x.y, t[1][f], fmaf(x.z, t[2][f], fmaf(x.w, t[3][f], acc[i][f]))));
    }
  }
}

// Requests rows [row0, row0 + ROWS) of one head into a tile of padded rows;
// rows at or past `end` become zero and are not read (they may hold anything).
template <int D, int ROWS>
__device__ __forceinline__ void fill_tile(const CrossParams& p, const CrossTensor& t, int b, int h, int row0, int end,
                                          float* tile) {
  constexpr int CH = D / 4, STEP = kThreads / CH;
  const float* head = static_cast<const float*>(t.data) + b * t.s[0] + h * t.s[1];
  const int r0 = threadIdx.x / CH, c = threadIdx.x % CH * 4;
  const float* src = head + static_cast<int64_t>(row0 + r0) * t.s[2] + c;
  float* dst = tile + r0 * (D + 4) + c;
#pragma unroll 4
  for (int r = 0; r < ROWS; r += STEP) {
    const bool read = row0 + r0 + r < end && CPATTN_IN(t.span, src, 16, p.err);
    copy16(smem_addr(dst), read ? src : head, read);
    src += STEP * t.s[2];
    dst += STEP * (D + 4);
  }
}

// A row's place in a [B, H, S] tensor.
__device__ __forceinline__ float* lse_at(const CrossTensor& t, int b, int h, int row) {
  return static_cast<float*>(t.data) + b * t.s[0] + h * t.s[1] + row * t.s[2];
}

// ------------------------------------------------------------------ forward
// Key tiles of 128: warps as 2 row groups x 4 key groups for the scores, and
// 2 x 4 feature groups for P V.  K and V have one buffer each: the next K
// arrives under P V, the next V under the scores.  blockIdx.y: a split of the
// key axis.
constexpr int kTileF = 128, kWF = kTileF + 4;

template <int D>
constexpr size_t fwd_smem() {
  return sizeof(float) * (kOwn * (D + 4) + 2 * kTileF * (D + 4) + (D == 64 ? 0 : kOwn * kWF) + 4 * kOwn);
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1) cross_f32_kernel(const __grid_constant__ CrossParams p) {
  constexpr int F = D / 32, PAD = D + 4;
  constexpr bool OVER = D == 64;       // P over K: two blocks an SM take turns instead
  static_assert(!OVER || kOwn * kWF <= kTileF * PAD, "P fits K's buffer");
  extern __shared__ __align__(16) float sm[];
  launch_wait();
  launch_next();
  float* sQ = sm;                      // [64][PAD]
  float* sK = sQ + kOwn * PAD;         // [128][PAD]
  float* sV = sK + kTileF * PAD;       // [128][PAD]
  float* sP = OVER ? sK : sV + kTileF * PAD;                   // [64][kWF]
  float* sX = sV + kTileF * PAD + (OVER ? 0 : kOwn * kWF);     // [4][64] row maxima, then sums, of a key group
  const int warp = threadIdx.x / 32, group = warp & 1, part = warp >> 1, lr = lane_row(), lc = lane_col();
  const int tiles = (p.s_q + kOwn - 1) / kOwn, bh = blockIdx.x / tiles;
  const int row0 = (blockIdx.x - bh * tiles) * kOwn, mine = group * 32 + lr;   // this lane's rows: mine + 4 i
  const int h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.kv_heads);
  // this split's keys: whole tiles, dealt out evenly
  const int all = cross_length(p, b), all_tiles = (all + kTileF - 1) / kTileF;
  const int per = (all_tiles + p.splits - 1) / p.splits;
  const int begin = min(static_cast<int>(blockIdx.y) * per, all_tiles) * kTileF;
  const int end = min(all, begin + per * kTileF);

  fill_tile<D, kOwn>(p, p.q, b, h, row0, p.s_q, sQ);
  fill_tile<D, kTileF>(p, p.k, b, hk, begin, end, sK);
  copies_commit();
  fill_tile<D, kTileF>(p, p.v, b, hk, begin, end, sV);
  copies_commit();
  float o[8][F], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int f = 0; f < F; ++f) o[i][f] = 0.f;
  }
  copies_wait<1>();
  __syncthreads();
  for (int k0 = begin; k0 < end; k0 += kTileF) {
    const int valid = min(end - k0, kTileF), col = part * 32 + lc;   // this lane's keys: col + 8 j
    float s[8][4] = {};
    if (part * 32 < valid) dots<D>(sQ + mine * PAD, sK + col * PAD, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = col + 8 * j < valid ? s[i][j] * p.scale_log2 : -INFINITY;
        x = fmaxf(x, s[i][j]);
      }
      x = row_max(x);
      if (lc == 0) sX[part * kOwn + mine + 4 * i] = x;
    }
    __syncthreads();   // (K is done with)
    if (!OVER && k0 + kTileF < end) fill_tile<D, kTileF>(p, p.k, b, hk, k0 + kTileF, end, sK);
    copies_commit();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float top = m[i];
#pragma unroll
      for (int x = 0; x < 4; ++x) top = fmaxf(top, sX[x * kOwn + mine + 4 * i]);
      const float base = top == -INFINITY ? 0.f : top;
      const float f = exp2f(m[i] - base);
      m[i] = top;
      l[i] *= f;   // (this lane's share of the sum)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - base);
        l[i] += e;
        sP[(mine + 4 * i) * kWF + col + 8 * j] = e;
      }
#pragma unroll
      for (int x = 0; x < F; ++x) o[i][x] *= f;
    }
    copies_wait<1>();
    __syncthreads();   // (P and V are there)
    spread<D, kWF>(sP + mine * kWF, sV + (part * 8 + lc) * F, (valid + 3) & ~3, o);
    copies_wait<0>();
    __syncthreads();   // (the next K is there, P and V are done with)
    if (k0 + kTileF < end) {
      if (OVER) fill_tile<D, kTileF>(p, p.k, b, hk, k0 + kTileF, end, sK);
      if (OVER) copies_commit();
      fill_tile<D, kTileF>(p, p.v, b, hk, k0 + kTileF, end, sV);
      copies_commit();
      if (OVER) {
        copies_wait<1>();
        __syncthreads();
      }
    }
  }
  copies_wait<0>();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    l[i] = row_sum(l[i]);
    if (lc == 0) sX[part * kOwn + mine + 4 * i] = l[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + mine + 4 * i;
    if (row >= p.s_q) continue;
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) sum += sX[x * kOwn + mine + 4 * i];
    const bool none = sum == 0.f;   // (NaN sums stay NaN below)
    const float inv = none ? 0.f : 1.f / sum;
    // (several splits: their outputs and lse, for the join)
    const bool split = p.splits > 1;
    const int64_t n = static_cast<int64_t>(p.batch) * p.heads * p.s_q;
    const int64_t at = blockIdx.y * n + static_cast<int64_t>(bh) * p.s_q + row;
    float* dst = (split ? p.ws + at * D
                        : static_cast<float*>(p.out.data) + b * p.out.s[0] + h * p.out.s[1] + row * p.out.s[2]) +
                 (part * 8 + lc) * F;
    if (CPATTN_IN(split ? p.ws_span : p.out.span, dst, 4 * F, p.err)) store_n<F>(dst, o[i], inv);
    float* dl = split ? p.ws + p.splits * n * D + at : lse_at(p.lse, b, h, row);
    if (part == 0 && lc == 0 && CPATTN_IN(split ? p.ws_span : p.lse.span, dl, 4, p.err))
      *dl = none ? -INFINITY : (m[i] + log2f(sum)) * kLn2;
  }
}

// ------------------------------------------------------------------ gradient
constexpr int kTile = 64, kW = kTile + 4;

template <int D>
constexpr size_t grad_smem() {
  return sizeof(float) * (2 * kOwn * (D + 4) + 4 * kTile * (D + 4) + kOwn * kW);
}

// dq of 64 query rows (delta from the workspace's start, as cross_simt.cu).
template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1) cross_f32_dq_kernel(const __grid_constant__ CrossParams p) {
  constexpr int F = D / 32, PAD = D + 4;
  extern __shared__ __align__(16) float sm[];
  launch_wait();
  launch_next();
  float* sQ = sm;                      // [64][PAD]
  float* sG = sQ + kOwn * PAD;         // [64][PAD] dout
  float* sKV = sG + kOwn * PAD;        // two stages of K and V, [64][PAD] each
  float* sS = sKV + 4 * kTile * PAD;   // [64][kW] p, then ds
  const int warp = threadIdx.x / 32, group = warp & 1, half = (warp >> 1) & 1, lr = lane_row(), lc = lane_col();
  const bool scores = warp < 4;        // else do.v
  const int tiles = (p.s_q + kOwn - 1) / kOwn, bh = blockIdx.x / tiles;
  const int row0 = (blockIdx.x - bh * tiles) * kOwn, mine = group * 32 + lr;
  const int h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.kv_heads);
  const int len = cross_length(p, b);
  fill_tile<D, kOwn>(p, p.q, b, h, row0, p.s_q, sQ);
  fill_tile<D, kOwn>(p, p.dout, b, h, row0, p.s_q, sG);
  auto request = [&](int k0) {
    if (k0 < len) {
      float* stage = sKV + ((k0 / kTile) & 1) * 2 * kTile * PAD;
      fill_tile<D, kTile>(p, p.k, b, hk, k0, len, stage);
      fill_tile<D, kTile>(p, p.v, b, hk, k0, len, stage + kTile * PAD);
    }
    copies_commit();
  };
  request(0);   // (with the query rows)
  float dq[8][F], stat[8];   // stat: lse log2e, or delta
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + mine + 4 * i;
    stat[i] = scores ? INFINITY : 0.f;   // (rows past the end: p = 0)
    if (row < p.s_q) {
      const float* at = scores ? lse_at(p.lse, b, h, row) : p.ws + static_cast<int64_t>(bh) * p.s_q + row;
      if (CPATTN_IN(scores ? p.lse.span : p.ws_span, at, 4, p.err)) stat[i] = scores ? cross_lse2(*at) : *at;
    }
#pragma unroll
    for (int f = 0; f < F; ++f) dq[i][f] = 0.f;
  }
  for (int k0 = 0; k0 < len; k0 += kTile) {
    request(k0 + kTile);
    copies_wait<1>();
    __syncthreads();
    const float* sK = sKV + ((k0 / kTile) & 1) * 2 * kTile * PAD;
    const int valid = min(len - k0, kTile), col = half * 32 + lc;
    float s[8][4] = {};
    if (half * 32 < valid)
      dots<D>((scores ? sQ : sG) + mine * PAD, (scores ? sK : sK + kTile * PAD) + col * PAD, s);
    float* at = sS + mine * kW + col;
    if (scores) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          at[i * 4 * kW + 8 * j] = col + 8 * j < valid ? exp2f(fmaf(s[i][j], p.scale_log2, -stat[i])) : 0.f;
    }
    __syncthreads();
    if (!scores) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (one key has all the weight whatever q is)
          const bool on = col + 8 * j < valid && len > 1;
          at[i * 4 * kW + 8 * j] = on ? at[i * 4 * kW + 8 * j] * (s[i][j] - stat[i]) : 0.f;
        }
    }
    __syncthreads();
    spread<D, kW>(sS + mine * kW, sK + ((warp >> 1) * 8 + lc) * F, (valid + 3) & ~3, dq);
    __syncthreads();   // (this stage may be filled again)
  }
  copies_wait<0>();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + mine + 4 * i;
    float* dst = static_cast<float*>(p.dq.data) + b * p.dq.s[0] + h * p.dq.s[1] + row * p.dq.s[2] +
                 ((warp >> 1) * 8 + lc) * F;
    if (row < p.s_q && CPATTN_IN(p.dq.span, dst, 4 * F, p.err)) store_n<F>(dst, dq[i], p.scale);
  }
}

// dk, dv of 64 keys over part blockIdx.y of the query tiles of every query
// head that shares the key head; sums of several parts go to the workspace,
// `partials` floats into it.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
    cross_f32_dkv_kernel(const __grid_constant__ CrossParams p, const int64_t partials) {
  constexpr int F = D / 32, PAD = D + 4;
  extern __shared__ __align__(16) float sm[];
  launch_wait();
  launch_next();
  float* sK = sm;                      // [64][PAD]
  float* sV = sK + kOwn * PAD;
  float* sQG = sV + kOwn * PAD;        // two stages of Q and dO, [64][PAD] each
  float* sS = sQG + 4 * kTile * PAD;   // [64][kW] p, then ds
  const int warp = threadIdx.x / 32, group = warp & 1, half = (warp >> 1) & 1, lr = lane_row(), lc = lane_col();
  const bool scores = warp < 4;
  const int tiles = (p.s_kv + kOwn - 1) / kOwn, bk = blockIdx.x / tiles;
  const int key0 = (blockIdx.x - bk * tiles) * kOwn, mine = group * 32 + lr;
  const int hk = bk % p.kv_heads, b = bk / p.kv_heads;
  const int share = p.heads / p.kv_heads;
  const int len = cross_length(p, b);
  float dk[8][F], dv[8][F];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int f = 0; f < F; ++f) dk[i][f] = dv[i][f] = 0.f;
  if (key0 < len) {
    fill_tile<D, kOwn>(p, p.k, b, hk, key0, len, sK);
    fill_tile<D, kOwn>(p, p.v, b, hk, key0, len, sV);
    // steps: the query tiles of one head after the other, dealt out evenly
    const int tiles_q = (p.s_q + kTile - 1) / kTile, steps = share * tiles_q;
    const int per = (steps + p.splits - 1) / p.splits;
    const int x0 = min(static_cast<int>(blockIdx.y) * per, steps), x1 = min(x0 + per, steps);
    auto request = [&](int x) {
      if (x < x1) {
        float* stage = sQG + ((x - x0) & 1) * 2 * kTile * PAD;
        const int g = x / tiles_q, i0 = (x - g * tiles_q) * kTile, h = hk * share + g;
        fill_tile<D, kTile>(p, p.q, b, h, i0, p.s_q, stage);
        fill_tile<D, kTile>(p, p.dout, b, h, i0, p.s_q, stage + kTile * PAD);
      }
      copies_commit();
    };
    request(x0);   // (with the keys and values)
    for (int x = x0; x < x1; ++x) {
      request(x + 1);
      const int g = x / tiles_q, i0 = (x - g * tiles_q) * kTile, h = hk * share + g;
      const int valid = min(p.s_q - i0, kTile), col = half * 32 + lc;
      float stat[4];   // lse log2e, or delta
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = i0 + col + 8 * j;
        stat[j] = scores ? INFINITY : 0.f;
        if (row < p.s_q) {
          const float* at =
              scores ? lse_at(p.lse, b, h, row) : p.ws + (static_cast<int64_t>(b) * p.heads + h) * p.s_q + row;
          if (CPATTN_IN(scores ? p.lse.span : p.ws_span, at, 4, p.err)) stat[j] = scores ? cross_lse2(*at) : *at;
        }
      }
      copies_wait<1>();
      __syncthreads();
      const float* sQ = sQG + ((x - x0) & 1) * 2 * kTile * PAD;
      const float* sG = sQ + kTile * PAD;
      float s[8][4] = {};
      if (half * 32 < valid) dots<D>((scores ? sK : sV) + mine * PAD, (scores ? sQ : sG) + col * PAD, s);
      float* at = sS + mine * kW + col;
      if (scores) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            at[i * 4 * kW + 8 * j] = key0 + mine + 4 * i < len && col + 8 * j < valid
                                         ? exp2f(fmaf(s[i][j], p.scale_log2, -stat[j])) : 0.f;
      }
      __syncthreads();
      const int n = (valid + 3) & ~3;
      if (!scores) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool on = key0 + mine + 4 * i < len && col + 8 * j < valid && len > 1;   // (as in the dq kernel)
            s[i][j] = on ? at[i * 4 * kW + 8 * j] * (s[i][j] - stat[j]) : 0.f;
          }
      }
      spread<D, kW>(sS + mine * kW, sG + ((warp >> 1) * 8 + lc) * F, n, dv);
      __syncthreads();
      if (!scores) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) at[i * 4 * kW + 8 * j] = s[i][j];
      }
      __syncthreads();
      spread<D, kW>(sS + mine * kW, sQ + ((warp >> 1) * 8 + lc) * F, n, dk);
      __syncthreads();   // (this stage may be filled again)
    }
    copies_wait<0>();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int key = key0 + mine + 4 * i, c = ((warp >> 1) * 8 + lc) * F;
    if (key >= p.s_kv) continue;
    if (p.splits > 1) {
      const int64_t rows = static_cast<int64_t>(p.batch) * p.kv_heads * p.s_kv;
      float* d1 = p.ws + partials + ((2 * blockIdx.y * rows) + static_cast<int64_t>(bk) * p.s_kv + key) * D + c;
      float* d2 = d1 + rows * D;
      if (CPATTN_IN(p.ws_span, d1, 4 * F, p.err)) store_n<F>(d1, dk[i], 1.f);
      if (CPATTN_IN(p.ws_span, d2, 4 * F, p.err)) store_n<F>(d2, dv[i], 1.f);
    } else {
      float* d1 = static_cast<float*>(p.dk.data) + b * p.dk.s[0] + hk * p.dk.s[1] + key * p.dk.s[2] + c;
      float* d2 = static_cast<float*>(p.dv.data) + b * p.dv.s[0] + hk * p.dv.s[1] + key * p.dv.s[2] + c;
      if (CPATTN_IN(p.dk.span, d1, 4 * F, p.err)) store_n<F>(d1, dk[i], p.scale);
      if (CPATTN_IN(p.dv.span, d2, 4 * F, p.err)) store_n<F>(d2, dv[i], 1.f);
    }
  }
}

int64_t tiles_of(int rows, int per) { return (rows + per - 1) / per; }

}  // namespace

cudaError_t launch_cross_f32(int head_dim, const CrossParams& p, cudaStream_t stream) {
  const int64_t blocks = tiles_of(p.s_q, kOwn) * p.batch * p.heads;
  return head_dim == 64 ? cross_run<cross_f32_kernel<64>>(blocks, p.splits, kThreads, fwd_smem<64>(), stream, p)
                        : cross_run<cross_f32_kernel<128>>(blocks, p.splits, kThreads, fwd_smem<128>(), stream, p);
}

cudaError_t launch_cross_f32_dq(int head_dim, const CrossParams& p, cudaStream_t stream) {
  const int64_t blocks = tiles_of(p.s_q, kOwn) * p.batch * p.heads;
  return head_dim == 64 ? cross_run<cross_f32_dq_kernel<64>>(blocks, 1, kThreads, grad_smem<64>(), stream, p)
                        : cross_run<cross_f32_dq_kernel<128>>(blocks, 1, kThreads, grad_smem<128>(), stream, p);
}

cudaError_t launch_cross_f32_dkv(int head_dim, const CrossParams& p, int64_t partials, cudaStream_t stream) {
  const int64_t blocks = tiles_of(p.s_kv, kOwn) * p.batch * p.kv_heads;
  return head_dim == 64
             ? cross_run<cross_f32_dkv_kernel<64>>(blocks, p.splits, kThreads, grad_smem<64>(), stream, p, partials)
             : cross_run<cross_f32_dkv_kernel<128>>(blocks, p.splits, kThreads, grad_smem<128>(), stream, p, partials);
}

}  // namespace cpattn
