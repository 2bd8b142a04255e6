// cache_f32.cu -- attention of new tokens to a paged cache of fp32 keys and values,
// computed in fp32 (no tf32 rounding).
//
// Mathematics as in cache_few.cu.  A block of 128 threads takes 16 rows (tokens of the
// query heads that share a key head) and walks its keys in tiles of 32, the next one in flight by asynchronous
// copies.  Scores: a thread has one row and every eighth key; P V: the
// same row, and every eighth group of four features; the eight threads of a row share
// its maximum and sum by shuffles, and its weights through shared memory.  Rows of
// shared memory are D + 4 floats, so that eight neighbouring rows use all banks.
#include <cuda_runtime.h>

#include <cmath>

#include "cache.cuh"
#include "ptx.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 128;
constexpr int R = kCacheF32Rows, kKeys = kCacheF32Keys;

template <int D>
struct Cfg {
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

template <int D>
__global__ void __launch_bounds__(kThreads) cache_f32_kernel(const __grid_constant__ CacheParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(16) float shared[];
  float* sQ = shared + C::Q;
  float* sP = shared + C::P;
  uint32_t* paths = reinterpret_cast<uint32_t*>(shared + C::PATHS);
  int* parents = reinterpret_cast<int*>(paths + R * kTreeWords);
  const int r = threadIdx.x / 8, g = threadIdx.x % 8;   // this thread's row, and place in it
  const int share = p.heads / p.kv_heads, rows = p.s_q * share;
  cache_prefetch(p);
  launch_wait();
  launch_next();
  CacheWalk<kKeys> walk;
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
    const int row = w.rt * R + r, token = row / share;
    float m = -INFINITY, l = 0.f;
    float4 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
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
      float s[kKeys / 8];
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j) s[j] = 0.f;
#pragma unroll 8
      for (int d = 0; d < D; d += 4) {
        const float4 q = *reinterpret_cast<const float4*>(sQ + r * C::ROW + d);
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
          const float4 k = *reinterpret_cast<const float4*>(sK + (g + 8 * j) * C::ROW + d);
          s[j] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[j]))));
        }
      }
      unsigned long long seen = 0ull;
      if (token < w.count)
        seen = !drafts ? ~0ull
               : p.parents == nullptr ? chain_window(w.len, token, start) : tree_window(paths + r * kTreeWords, w.len, start);
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j) {
        s[j] = (seen >> (g + 8 * j)) & 1 ? s[j] * p.scale_log2 : -INFINITY;
        top = fmaxf(top, s[j]);
      }
      top = fmaxf(m, row_max(top));
      const float base = top == -INFINITY ? 0.f : top;
      const float f = exp2f(m - base);
      m = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j) {
        s[j] = exp2f(s[j] - base);
        sum += s[j];
        sP[r * (kKeys + 4) + g + 8 * j] = s[j];
      }
      l = fmaf(l, f, row_sum(sum));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = make_float4(o[i].x * f, o[i].y * f, o[i].z * f, o[i].w * f);
      __syncwarp();                    // (a row's threads are of one warp)
#pragma unroll 4
      for (int k = 0; k < kKeys; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(sP + r * (kKeys + 4) + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f4 = e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(sV + (k + e) * C::ROW + g * 4 + i * 32);
            o[i] = make_float4(fmaf(f4, v.x, o[i].x), fmaf(f4, v.y, o[i].y), fmaf(f4, v.z, o[i].z), fmaf(f4, v.w, o[i].w));
          }
        }
      }
      __syncthreads();                 // tile t is free
    }
    copies_wait<0>();
    if (row < rows) {
      const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1);
      const int h = w.hk * share + row % share;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int d = g * 4 + i * 32;
        if (unclean && token < w.count)
          add_unfinite<float>(p, w, token, p.parents != nullptr ? paths + r * kTreeWords : nullptr, k_begin, k_end, d, o[i]);
        if (w.whole())
          cache_write_row<float>(p, w.b, h, token, d, o[i], m, l);
        else
          cache_write_part<R, D>(p, part, r, d, o[i], m, l);
      }
    }
  }
  cache_empty_units<float, R, kKeys, D>(p, threadIdx.x, kThreads);
}

template <int D>
cudaError_t launch_typed(const CacheParams& p, int blocks, cudaStream_t stream) {
  const cudaError_t e = cross_run<cache_f32_kernel<D>>(blocks, 1, kThreads, Cfg<D>::SMEM, stream, p);
    if (e != cudaSuccess || !p.split) return e;
  return cache_join<R, D, float>(p, blocks, stream);
}

}  // namespace

cudaError_t launch_cache_f32(int head_dim, const CacheParams& p, int blocks, cudaStream_t stream) {
  return head_dim == 64 ? launch_typed<64>(p, blocks, stream) : launch_typed<128>(p, blocks, stream);
}

}  // namespace cpattn
