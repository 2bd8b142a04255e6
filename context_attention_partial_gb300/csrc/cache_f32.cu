// cache_f32.cu -- attention of new tokens to a paged cache of fp32 keys and values,
// computed in fp32 (no tf32 rounding).
//
// Mathematics as in cache_few.cu.  A block of 128 threads takes 16 RT rows (tokens of
// the query heads that share a key head) and walks its keys in tiles of 32, the next
// one in flight by asynchronous copies.  Scores: a thread has RT rows, 16 apart, and
// every eighth key; P V: the same rows, and every eighth group of four features; the
// eight threads of a row share its maximum and sum by shuffles, and its weights through
// shared memory.  Rows of shared memory are D + 4 floats, so that eight neighbouring
// rows use all banks.  What bounds it is shared memory's reads: RT + 4 a thread for 4 RT
// products of four features, so RT = 4 where there are more than 16 rows.
//
// Measured: 13 drafts of 3 sequences of up to 700 keys, 8 heads on 2, D = 64, 15.5 to 17
// us (14.0 in a replayed graph), which is two launches' starts, a few key tiles and the
// join in series; 32 tokens of 3 sequences of up to 4000 keys, 16 heads on 4, D = 64 64 us,
// 14 TFLOP/s; 512 tokens behind 4096, 8 heads on 2, D = 128 257 us, 36 TFLOP/s.
#include <cuda_runtime.h>

#include <cmath>

#include "cache.cuh"
#include "ptx.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 128;
constexpr int kKeys = kCacheF32Keys;

template <int D, int RT>
struct Cfg {
  static constexpr int R = 16 * RT;
  static constexpr int ROW = D + 4;                      // floats of a staged row
  static constexpr int CH = D / 4;                       // 16-byte chunks of a row
  static constexpr int STAGES = 2;
  static constexpr int STAGE = 2 * kKeys * ROW;          // K and V, floats
  static constexpr int Q = STAGES * STAGE, P = Q + R * ROW, PATHS = P + R * (kKeys + 4);
  static constexpr int SMEM = (PATHS + R * kTreeWords + CPATTN_MAX_TREE) * 4;
};

// Over the eight threads of a row.
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int m = 4; m > 0; m /= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = 4; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

template <int D, int RT>
__global__ void __launch_bounds__(kThreads) cache_f32_kernel(const __grid_constant__ CacheParams p) {
  using C = Cfg<D, RT>;
  constexpr int R = C::R;
  extern __shared__ __align__(16) float shared[];
  float* sQ = shared + C::Q;
  float* sP = shared + C::P;
  uint32_t* paths = reinterpret_cast<uint32_t*>(shared + C::PATHS);
  int* parents = reinterpret_cast<int*>(paths + R * kTreeWords);
  const int r = threadIdx.x / 8, g = threadIdx.x % 8;   // this thread's first row, and place in its rows
  const int share = p.heads / p.kv_heads, rows = p.s_q * share;
  cache_prefetch(p);
  launch_wait();
  launch_next();
  CacheWalk<R, kKeys> walk;
  walk.start(p);
  CachePiece w;
  while (walk.next(p, w)) {
    if (threadIdx.x == 0) cache_note_unit<R, D>(p, w);
    const int k_begin = w.t0 * kKeys, k_end = min(w.len + w.count, w.t1 * kKeys), tiles = w.t1 - w.t0;
    // page numbers of a tile, at most two, read while the tile before it is asked for
    auto pages = [&](int t, int (&pg)[2]) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = k_begin + t * kKeys + (j << p.cache.shift);
        pg[j] = t < tiles && (j << p.cache.shift) < kKeys && key < k_end ? cache_page(p.cache, w.b, key, p.err) : -1;
      }
    };
    int pg[2];
    pages(0, pg);
    auto load = [&](int t) {
      if (t < tiles) {
        float* dst = shared + (t % C::STAGES) * C::STAGE;
        const float* kbase = static_cast<const float*>(p.k.data) + w.hk * p.k.s[1];
        const float* vbase = static_cast<const float*>(p.v.data) + w.hk * p.v.s[1];
#pragma unroll 4
        for (int i = threadIdx.x; i < kKeys * C::CH; i += kThreads) {
          const int kr = i / C::CH, d = i % C::CH * 4, key = k_begin + t * kKeys + kr;
          const int64_t page = (kr >> p.cache.shift) == 0 ? pg[0] : pg[1];
          const int at_row = key & ((1 << p.cache.shift) - 1);
          const float* kp = kbase + page * p.k.s[0] + at_row * p.k.s[2] + d;
          const float* vp = vbase + page * p.v.s[0] + at_row * p.v.s[2] + d;
          const bool in = key < k_end && page >= 0;
          copy16<true>(smem_addr(dst + kr * C::ROW + d), in ? static_cast<const void*>(kp) : p.q.data,
                       in && CPATTN_IN(p.k.span, kp, 16, p.err));
          copy16<true>(smem_addr(dst + (kKeys + kr) * C::ROW + d), in ? static_cast<const void*>(vp) : p.q.data,
                       in && CPATTN_IN(p.v.span, vp, 16, p.err));
        }
      }
      copies_commit();
      pages(t + 1, pg);
    };
    __syncthreads();   // (the piece before has read its rows and paths)
    load(0);
    if (p.parents != nullptr) {
      for (int i = threadIdx.x; i < p.s_q; i += kThreads) {
        const int32_t* from = p.parents + w.b * p.parents_stride + i;
        parents[i] = CPATTN_IN(p.parents_span, from, 4, p.err) ? *from : -1;
      }
    }
    for (int i = threadIdx.x; i < R * C::CH; i += kThreads) {
      const int row = w.rt * R + i / C::CH, d = i % C::CH * 4, t = row / share, h = w.hk * share + row % share;
      const float* src = static_cast<const float*>(p.q.data) + w.b * p.q.s[0] + h * p.q.s[1] + t * p.q.s[2] + d;
      *reinterpret_cast<float4*>(sQ + i / C::CH * C::ROW + d) =
          row < rows && CPATTN_IN(p.q.span, src, 16, p.err) ? *reinterpret_cast<const float4*>(src)
                                                           : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    if (p.parents != nullptr) tree_paths<R>(p, parents, w.rt, threadIdx.x, kThreads, paths);
    int token[RT];
    float m[RT], l[RT];
    float4 o[RT][D / 32];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      token[i] = (w.rt * R + r + 16 * i) / share;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    bool unclean = false;

    for (int t = 0; t < tiles; ++t) {
      load(t + 1);
      copies_wait<1>();
      __syncthreads();                 // tile t has arrived
      const float* sK = shared + (t % C::STAGES) * C::STAGE;
      float* sV = shared + (t % C::STAGES) * C::STAGE + kKeys * C::ROW;
      const int start = k_begin + t * kKeys;
      const bool drafts = start + kKeys > w.open;
      if (drafts && w.count > 1) {     // (values that are not finite: as in cache_few.cu)
        bool found = false;
        for (int i = threadIdx.x; i < kKeys * C::CH; i += kThreads) {
          const int kr = i / C::CH;
          if (start + kr >= w.open && start + kr < k_end)
            found |= clear_unfinite(reinterpret_cast<float4*>(sV + kr * C::ROW + i % C::CH * 4));
        }
        unclean |= __syncthreads_or(found);
      }
      float s[RT][kKeys / 8];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 k[kKeys / 8];
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) k[j] = *reinterpret_cast<const float4*>(sK + (g + 8 * j) * C::ROW + d);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(sQ + (r + 16 * i) * C::ROW + d);
#pragma unroll
          for (int j = 0; j < kKeys / 8; ++j)
            s[i][j] = fmaf(q.x, k[j].x, fmaf(q.y, k[j].y, fmaf(q.z, k[j].z, fmaf(q.w, k[j].w, s[i][j]))));
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        unsigned long long seen = 0ull;
        if (token[i] < w.count)
          seen = !drafts ? ~0ull
                 : p.parents == nullptr ? chain_window(w.len, token[i], start)
                                        : tree_window(paths + (r + 16 * i) * kTreeWords, w.len, start);
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
          s[i][j] = (seen >> (g + 8 * j)) & 1 ? s[i][j] * p.scale_log2 : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
        top = fmaxf(m[i], row_max(top));
        const float base = top == -INFINITY ? 0.f : top, f = exp2f(m[i] - base);
        m[i] = top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
          s[i][j] = exp2f(s[i][j] - base);
          sum += s[i][j];
          sP[(r + 16 * i) * (kKeys + 4) + g + 8 * j] = s[i][j];
        }
        l[i] = fmaf(l[i], f, row_sum(sum));
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[i][c] = make_float4(o[i][c].x * f, o[i][c].y * f, o[i][c].z * f, o[i][c].w * f);
      }
      __syncwarp();                    // (a row's threads are of one warp)
#pragma unroll 2
      for (int k = 0; k < kKeys; k += 4) {
        float4 x[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) x[i] = *reinterpret_cast<const float4*>(sP + (r + 16 * i) * (kKeys + 4) + k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(sV + (k + e) * C::ROW + g * 4 + c * 32);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const float f = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
              o[i][c] = make_float4(fmaf(f, v.x, o[i][c].x), fmaf(f, v.y, o[i][c].y), fmaf(f, v.z, o[i][c].z),
                                    fmaf(f, v.w, o[i][c].w));
            }
          }
      }
      __syncthreads();                 // tile t is free
    }
    copies_wait<0>();
    const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = w.rt * R + r + 16 * i, h = w.hk * share + row - token[i] * share;
      if (row >= rows) continue;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const int d = g * 4 + c * 32;
        float4 sum = o[i][c];
        if (unclean && token[i] < w.count)
          add_unfinite<float>(p, w, token[i], p.parents != nullptr ? paths + (r + 16 * i) * kTreeWords : nullptr, k_begin,
                              k_end, d, sum);
        if (w.whole())
          cache_write_row<float>(p, w.b, h, token[i], d, sum, m[i], l[i]);
        else
          cache_write_part<R, D>(p, part, r + 16 * i, d, sum, m[i], l[i]);
      }
    }
  }
  cache_empty_units<float, R, kKeys, D>(p, threadIdx.x, kThreads);
}

template <int D, int RT>
cudaError_t launch_typed(const CacheParams& p, int blocks, cudaStream_t stream) {
  const cudaError_t e = cross_run<cache_f32_kernel<D, RT>>(blocks, 1, kThreads, Cfg<D, RT>::SMEM, stream, p);
  if (e != cudaSuccess || !p.split) return e;
  return cache_join<16 * RT, D, float>(p, blocks, stream);
}

}  // namespace

cudaError_t launch_cache_f32(int head_dim, int rows, const CacheParams& p, int blocks, cudaStream_t stream) {
  if (head_dim == 64) return rows == 16 ? launch_typed<64, 1>(p, blocks, stream) : launch_typed<64, 4>(p, blocks, stream);
  return rows == 16 ? launch_typed<128, 1>(p, blocks, stream) : launch_typed<128, 4>(p, blocks, stream);
}

}  // namespace cpattn
