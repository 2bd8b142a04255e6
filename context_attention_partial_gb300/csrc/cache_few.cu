// cache_few.cu -- attention of few rows (single tokens, small trees of drafts) to a
// paged cache, bf16.
//
// Mathematics: row (token i, head) sees the sequence's cached keys and, of the
// drafts behind them, those that are i or above it; over these
//     m = max_j scale log2e s_j,  P_j = 2^(scale log2e s_j - m),  l = sum_j P_j,
//     o = sum_j P_j v_j / l,  lse = (m + log2 l) ln2,
// one pass over the keys with the running m and l (fp32).  P is rounded to bf16 for
// its product with V (the tensor cores' operand type), and the output once.
//
// What bounds it is the read of the keys and values, 4 D bytes a key, once per key
// head: the rows of a tile are the tokens of every query head that shares it.  The
// key tiles of all sequences are dealt out evenly over the blocks (CacheWalk), two
// blocks an SM (D = 64: three).
//
// A block of 4 warps walks its keys in stages of 64, two of them (D = 64: three) on their
// way by 16-byte asynchronous copies while one is read, each row from its page; a warp
// holds 32 page numbers and has the next 32 on their way.  MT = 1 tile of 16 rows, whose 4 warps share a stage's keys
// and are joined at the end, or 4 (more than 128 query heads a key head, which the
// tensor cores' tiles do not hold), a warp each.
//
// Measured, both launches: single tokens of 8 sequences of up to 16384 keys, 32 heads on
// 8, D = 128 (302 MB) 53 us, 5.7 TB/s; of 4 sequences of 16384 keys, 24 heads, D = 64
// (403 MB) 66 us, 6.1 TB/s; of one sequence of 1000 keys 9.7 to 11 us, 8.6 in
// a replayed graph.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "cache.cuh"
#include "mma_ops.cuh"
#include "ptx.cuh"
#include "tile_ops.cuh"

namespace cpattn {
namespace {

constexpr int kKeys = 64;   // of a stage
constexpr int kThreads = 128;

template <int D, int MT>
struct Few {
  static constexpr int R = 16 * MT;
  static constexpr int ROW = D * 2;
  static constexpr int CH = ROW / 16;                     // 16-byte chunks of a row
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int STAGE = 2 * kKeys * ROW;           // K and V
  static constexpr int JOIN = 4 * 16 * (D + 4) * 4 + 2 * 4 * 16 * 8;
  static constexpr int TILES = STAGES * STAGE > JOIN ? STAGES * STAGE : JOIN;
  // behind them: a tree's paths and parents
  static constexpr int SMEM = TILES + R * kTreeWords * 4 + CPATTN_MAX_TREE * 4;
};

template <int D, int MT>
__global__ void __launch_bounds__(kThreads) cache_few_kernel(const __grid_constant__ CacheParams p) {
  using C = Few<D, MT>;
  constexpr int R = C::R, KG = 4 / MT, KW = kKeys / KG;   // key groups, keys of a warp and stage
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* paths = reinterpret_cast<uint32_t*>(smem + C::TILES);
  int* parents = reinterpret_cast<int*>(paths + R * kTreeWords);
  const uint32_t s0 = smem_addr(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int mt = warp % MT, kg = warp / MT;
  const int share = p.heads / p.kv_heads, rows = p.s_q * share;
  const int c = threadIdx.x % C::CH, r_first = threadIdx.x / C::CH;
  constexpr int RSTEP = kThreads / C::CH;
  cache_prefetch(p);
  launch_wait();
  launch_next();
  // (keys that one row tile reads leave L2 first: 8 sequences x 16384 keys 58.1 us, 61.0
  // when they are kept)
  const uint64_t policy = p.row_tiles > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
  CacheWalk<R, kKeys> walk;
  walk.start(p);
  CachePiece w;
  while (walk.next(p, w)) {
    if (threadIdx.x == 0) cache_note_unit<R, D>(p, w);
    const int k_begin = w.t0 * kKeys, k_end = min(w.len + w.count, w.t1 * kKeys), tiles = w.t1 - w.t0;
    // page numbers, 32 at a time, a lane each; the next 32 are read ahead, and checked
    // when their turn comes
    const int entry0 = k_begin >> p.cache.shift, in_page = k_begin & ((1 << p.cache.shift) - 1);
    auto key_of = [&](int window) { return (entry0 + window * 32 + lane) << p.cache.shift; };
    auto read_pages = [&](int window) {
      return key_of(window) < k_end ? cache_entry(p.cache, w.b, key_of(window), p.err) : -1;
    };
    auto checked = [&](int window, int entry) {
      return key_of(window) < k_end ? cache_checked(p.cache, entry, p.err) : -1;
    };
    const int first = read_pages(0);
    int window = 0, ahead = read_pages(1), here = checked(0, first);
    // this thread's copies of a stage: chunk c of rows r_first, r_first + RSTEP, ...
    const char* kbase = static_cast<const char*>(p.k.data) + w.hk * p.k.s[1] * 2 + c * 16;
    const char* vbase = static_cast<const char*>(p.v.data) + w.hk * p.v.s[1] * 2 + c * 16;
    auto load = [&](int t) {
      if (t < tiles) {
        // (a stage's pages are of one window: both begin at multiples of a stage's pages)
        if ((in_page + t * kKeys) >> p.cache.shift >> 5 != window) {
          ++window;
          here = checked(window, ahead);
          ahead = read_pages(window + 1);
        }
        const uint32_t dst = s0 + (t % C::STAGES) * C::STAGE;
#pragma unroll
        for (int i = 0; i < kKeys / RSTEP; ++i) {
          const int r = r_first + i * RSTEP, key = k_begin + t * kKeys + r;
          const int64_t page = __shfl_sync(0xffffffffu, here, (in_page + t * kKeys + r) >> p.cache.shift & 31);
          const int at_row = key & ((1 << p.cache.shift) - 1);
          const uint32_t at = r * C::ROW + ((c ^ (r & 7)) << 4);
          const char* kp = kbase + (page * p.k.s[0] + at_row * p.k.s[2]) * 2;
          const char* vp = vbase + (page * p.v.s[0] + at_row * p.v.s[2]) * 2;
          const bool in = key < k_end && page >= 0;
          copy16_hint(dst + at, in ? static_cast<const void*>(kp) : p.q.data, in && CPATTN_IN(p.k.span, kp, 16, p.err), policy);
          copy16_hint(dst + kKeys * C::ROW + at, in ? static_cast<const void*>(vp) : p.q.data, in && CPATTN_IN(p.v.span, vp, 16, p.err), policy);
        }
      }
      copies_commit();
    };
    __syncthreads();   // (the piece before has read its rows, paths and sums)
#pragma unroll
    for (int t = 0; t < C::STAGES - 1; ++t) load(t);

    if (p.parents != nullptr) {
      for (int i = threadIdx.x; i < p.s_q; i += kThreads) {
        const int32_t* from = p.parents + w.b * p.parents_stride + i;
        parents[i] = CPATTN_IN(p.parents_span, from, 4, p.err) ? *from : -1;
      }
      __syncthreads();
      tree_paths<R>(p, parents, w.rt, threadIdx.x, kThreads, paths);
      // (seen behind the first stage's barrier)
    }
    // this thread's rows of the tile: lane / 4 and lane / 4 + 8
    uint32_t q[D / 16][4];
    int token[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = w.rt * R + mt * 16 + lane / 4 + 8 * i, h = w.hk * share + r % share;
      token[i] = r / share;
      const char* src = static_cast<const char*>(p.q.data) +
                        (w.b * p.q.s[0] + h * p.q.s[1] + token[i] * p.q.s[2]) * 2 + (lane % 4) * 4;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const bool in = r < rows && CPATTN_IN(p.q.span, src + kk * 32 + 16, 4, p.err);
        q[kk][i] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 32) : 0u;
        q[kk][i + 2] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 32 + 16) : 0u;
      }
    }

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    bool unclean = false;   // some draft's value is not finite

    for (int t = 0; t < tiles; ++t) {
      copies_wait<C::STAGES - 2>();
      __syncthreads();                 // stage t has arrived, and stage t - 1 is free
      load(t + C::STAGES - 1);
      const uint32_t sK = s0 + (t % C::STAGES) * C::STAGE, sV = sK + kKeys * C::ROW;
      const int key0 = kg * KW, start = k_begin + t * kKeys;
      const bool drafts = start + kKeys > w.open;
      if (drafts && w.count > 1) {
        // a draft that a row does not see has weight 0, which does not keep an
        // infinite value out of the row's sum: such values are taken out here, and
        // added at the end to the rows that do see them
        bool found = false;
        for (int i = threadIdx.x; i < kKeys * C::CH; i += kThreads) {
          const int r = i / C::CH;
          if (start + r < w.open || start + r >= k_end) continue;
          uint4* at = reinterpret_cast<uint4*>(smem + (t % C::STAGES) * C::STAGE + kKeys * C::ROW + r * C::ROW +
                                               ((i % C::CH ^ (r & 7)) << 4));
          found |= clear_unfinite(at);
        }
        unclean |= __syncthreads_or(found);
      }
      float s[KW / 8][4];
#pragma unroll
      for (int n = 0; n < KW / 8; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
        const int row = key0 + n * 8 + lane % 8;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          uint32_t f[4];
          ldsm4(f, sK + row * C::ROW + (((kk * 4 + lane / 8) ^ (row & 7)) << 4));
          mma16816(s[n], q[2 * kk], f[0], f[1]);
          mma16816(s[n], q[2 * kk + 1], f[2], f[3]);
        }
      }
      unsigned long long seen[2] = {~0ull, ~0ull};   // of the keys of this warp
      if (drafts) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          seen[i] = token[i] >= w.count ? 0ull
                    : p.parents == nullptr
                        ? chain_window(w.len, token[i], start + key0)
                        : tree_window(paths + (mt * 16 + lane / 4 + 8 * i) * kTreeWords, w.len, start + key0);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (token[i] >= w.count) seen[i] = 0ull;
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 2; ++i) seen[i] >>= 2 * (lane % 4);
#pragma unroll
      for (int n = 0; n < KW / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = (seen[e / 2] >> (n * 8 + (e & 1))) & 1 ? s[n][e] * p.scale_log2 : -INFINITY;
          top[e / 2] = fmaxf(top[e / 2], s[n][e]);
        }
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mx = fmaxf(m[i], quad_max(top[i]));
        const float base = mx == -INFINITY ? 0.f : mx;
        f[i] = ex2_approx(m[i] - base);
        m[i] = mx;
        top[i] = base;
        l[i] *= f[i];
      }
      uint32_t pb[KW / 8][2];
#pragma unroll
      for (int n = 0; n < KW / 8; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = ex2_approx(s[n][e] - top[e / 2]);
        l[0] += s[n][0] + s[n][1];
        l[1] += s[n][2] + s[n][3];
        pb[n][0] = pack_bf16x2(s[n][0], s[n][1]);
        pb[n][1] = pack_bf16x2(s[n][2], s[n][3]);
      }
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= f[0];
          o[i][1] *= f[0];
          o[i][2] *= f[1];
          o[i][3] *= f[1];
        }
      }
#pragma unroll
      for (int k16 = 0; k16 < KW / 16; ++k16) {
        const uint32_t a[4] = {pb[2 * k16][0], pb[2 * k16][1], pb[2 * k16 + 1][0], pb[2 * k16 + 1][1]};
        const int row = key0 + k16 * 16 + ((lane / 8) & 1) * 8 + lane % 8;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t v[4];
          ldsm4t(v, sV + row * C::ROW + (((n * 2 + lane / 16) ^ (row & 7)) << 4));
          mma16816(o[2 * n], a, v[0], v[1]);
          mma16816(o[2 * n + 1], a, v[2], v[3]);
        }
      }
    }
    copies_wait<0>();
    __syncthreads();
    // every warp's rows to shared memory, then all threads join the key groups
    // and write: [warp][16 rows][D + 4] outputs, [warp][16 rows] (m, l)
    float* so = reinterpret_cast<float*>(smem);
    float2* sm = reinterpret_cast<float2*>(so + 4 * 16 * (D + 4));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] = quad_sum(l[i]);
      const int r = warp * 16 + lane / 4 + 8 * i;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(so + r * (D + 4) + n * 8 + 2 * (lane % 4)) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      if (lane % 4 == 0) sm[r] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1);   // (a piece's slot)
    const bool whole = w.whole();
    for (int i = threadIdx.x; i < R * (D / 4); i += kThreads) {
      // (rows of the result, or neighbouring places of a part, by neighbouring threads)
      const int r = whole ? i / (D / 4) : i % R, d = (whole ? i % (D / 4) : i / R) * 4;
      const int row = cache_row(p, w.rt, r);
      if (row < 0) continue;
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < KG; ++g) top = fmaxf(top, sm[g * R + r].x);
      const float base = top == -INFINITY ? 0.f : top;
      float total = 0.f;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        const int at = g * R + r;
        const float f = ex2_approx(sm[at].x - base);
        const float4 x = *reinterpret_cast<const float4*>(so + at * (D + 4) + d);
        total = fmaf(f, sm[at].y, total);
        sum = make_float4(fmaf(f, x.x, sum.x), fmaf(f, x.y, sum.y), fmaf(f, x.z, sum.z), fmaf(f, x.w, sum.w));
      }
      const int t = row / share, h = w.hk * share + row % share;
      if (unclean && t < w.count)
        add_unfinite<__nv_bfloat16>(p, w, t, p.parents != nullptr ? paths + r * kTreeWords : nullptr, k_begin, k_end, d, sum);
      if (whole)
        cache_write_row<__nv_bfloat16>(p, w.b, h, t, d, sum, top, total);
      else
        cache_write_part<R, D>(p, part, r, d, sum, top, total);
    }
  }
  cache_empty_units<__nv_bfloat16, R, kKeys, D>(p, threadIdx.x, kThreads);
}

template <int D, int MT>
cudaError_t launch_tiles(const CacheParams& p, int blocks, cudaStream_t stream) {
  using C = Few<D, MT>;
  const cudaError_t e = cross_run<cache_few_kernel<D, MT>>(blocks, 1, kThreads, C::SMEM, stream, p);
  if (e != cudaSuccess || !p.split) return e;
  return cache_join<C::R, D, __nv_bfloat16>(p, blocks, stream);
}

}  // namespace

cudaError_t launch_cache_few(int head_dim, int rows, const CacheParams& p, int blocks, cudaStream_t stream) {
  if (head_dim == 64)
    return rows == 16 ? launch_tiles<64, 1>(p, blocks, stream) : launch_tiles<64, 4>(p, blocks, stream);
  return rows == 16 ? launch_tiles<128, 1>(p, blocks, stream) : launch_tiles<128, 4>(p, blocks, stream);
}

}  // namespace cpattn
