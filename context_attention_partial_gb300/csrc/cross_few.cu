// cross_few.cu -- cross attention of few query rows (single new tokens) against
// long encoder states, bf16.
//
// Mathematics as in cross_fwd.cu; the rows are the S_q queries of every query
// head that shares a key head (at most 64), so each key and value is read once
// per key head.  What bounds it is that read: 4 D bytes a key.  The key axis
// is split over CTAs until the GPU is full.  8 parts (or fewer, where that is
// enough) are a cluster and join in its shared memory; the results of several
// clusters go to the workspace and are joined by their lse in a second kernel
// (cross_simt.cu).
//
// A CTA of 4 warps walks its keys in stages of 64, three or more stages in
// flight by 16-byte asynchronous copies (rows past the length are zero-filled
// by the copy and never read).  MT = 1, 2 or 4 tiles of 16 rows; the 4 / MT
// warps of a row tile share a stage's keys and are joined at the end.  With 16
// rows a warp-level m16n8k16 product is the right size: the 128-row tcgen05
// tile would be 7/8 padding, and its accumulators' way through TMEM is longer
// than the whole product.  P is rounded to bf16 for its product with V, sums
// and outputs of parts are fp32.
//
// Against the tensor-core kernel, which reads a key head once per query head
// (head size 128; us, this kernel / that one): 8 sequences x 8 key heads x 4096
// keys, 4 query heads each, 8 queries 28 / 81; 4 x 16 heads x 4096 keys, not
// shared, 48 queries 40 / 29; 24 heads x 4608 keys: 32 queries 18.7 / 17.6, 64
// queries 27 / 18; 4 key heads x 1024 keys, 4 query heads each: 8 queries 8.1 /
// 8.9, 16 queries 10.4 / 9.0; 8 heads x 2000 keys at D = 64, 32 queries 7.0 / 9.3;
// 2 x 2 key heads x 2500 keys, 8 query heads each, 7 queries 12.4 / 12.9.
// One query of 32 heads on 8, 8 sequences of up to 16384 keys: 302 MB in 56 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "cross.cuh"
#include "ptx.cuh"
#include "tile_ops.cuh"

namespace cpattn {
namespace {

constexpr int kKeys = 64;       // of a stage
constexpr float kLn2 = 0.693147180559945309f;

constexpr int kThreads = 128;

template <int D>
struct Few {
  static constexpr int ROW = D * 2;
  static constexpr int CH = ROW / 16;                     // 16-byte chunks of a row
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int STAGE = 2 * kKeys * ROW;           // K and V
  static constexpr int JOIN = 4 * 16 * (D + 4) * 4 + 2 * 4 * 16 * 8;
  static constexpr int SMEM = STAGES * STAGE > JOIN ? STAGES * STAGE : JOIN;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads) cross_few_kernel(const __grid_constant__ CrossParams p) {
  using C = Few<D>;
  constexpr int KG = 4 / MT, KW = kKeys / KG;    // key groups, keys of a warp and stage
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s0 = smem_addr(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int mt = warp % MT, kg = warp / MT;
  const int share = p.heads / p.kv_heads, rows = p.s_q * share;
  const int hk = blockIdx.x % p.kv_heads, b = blockIdx.x / p.kv_heads;
  {
    // the first stages, while the kernel before this one ends (where every key is
    // valid: lengths are not known yet); 36 key heads x 8192 keys, one query, 27.8
    // us without, 26.4 with
    const int first = min(static_cast<int>(blockIdx.y) * ceil_div(ceil_div(p.s_kv, kKeys), p.splits) * kKeys, p.s_kv);
    constexpr int LINES = C::ROW / 128;
    const int rows = p.lengths == nullptr ? min(p.s_kv - first, (C::STAGES - 1) * kKeys) : 0;
    for (int i = threadIdx.x; i < rows * LINES; i += kThreads) {
      const int64_t key = first + i / LINES;
      const int col = i % LINES * 64;
      prefetch_l2(static_cast<const __nv_bfloat16*>(p.k.data) + b * p.k.s[0] + hk * p.k.s[1] + key * p.k.s[2] + col);
      prefetch_l2(static_cast<const __nv_bfloat16*>(p.v.data) + b * p.v.s[0] + hk * p.v.s[1] + key * p.v.s[2] + col);
    }
  }
  launch_wait();
  launch_next();
  const int len = cross_length(p, b);
  const int all = ceil_div(len, kKeys), per = ceil_div(all, p.splits);
  const int t0 = min(static_cast<int>(blockIdx.y) * per, all), tiles = min(per, all - t0);
  const int k_begin = t0 * kKeys, k_end = min(len, (t0 + tiles) * kKeys);

  // this thread's copies of a stage: chunk c of rows r, r + kThreads / CH, ...
  const int c = threadIdx.x % C::CH, r_first = threadIdx.x / C::CH;
  constexpr int RSTEP = kThreads / C::CH;
  const char* kg_ptr = static_cast<const char*>(p.k.data) + (b * p.k.s[0] + hk * p.k.s[1]) * 2 + c * 16;
  const char* vg_ptr = static_cast<const char*>(p.v.data) + (b * p.v.s[0] + hk * p.v.s[1]) * 2 + c * 16;
  auto load = [&](int t) {
    if (t < tiles) {
      const uint32_t dst = s0 + (t % C::STAGES) * C::STAGE;
#pragma unroll
      for (int i = 0; i < kKeys / RSTEP; ++i) {
        const int r = r_first + i * RSTEP, key = k_begin + t * kKeys + r;
        const uint32_t at = r * C::ROW + ((c ^ (r & 7)) << 4);
        const char* kp = kg_ptr + static_cast<int64_t>(key) * p.k.s[2] * 2;
        const char* vp = vg_ptr + static_cast<int64_t>(key) * p.v.s[2] * 2;
        const bool in = key < k_end;
        copy16<true>(dst + at, in ? kp : kg_ptr, in && CPATTN_IN(p.k.span, kp, 16, p.err));
        copy16<true>(dst + kKeys * C::ROW + at, in ? vp : vg_ptr, in && CPATTN_IN(p.v.span, vp, 16, p.err));
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int t = 0; t < C::STAGES - 1; ++t) load(t);

  // this thread's rows of the query tile: lane / 4 and lane / 4 + 8
  uint32_t q[D / 16][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = mt * 16 + lane / 4 + 8 * i, qi = r / share, h = hk * share + r % share;
    const char* src = static_cast<const char*>(p.q.data) +
                      (b * p.q.s[0] + h * p.q.s[1] + static_cast<int64_t>(qi) * p.q.s[2]) * 2 + (lane % 4) * 4;
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

  for (int t = 0; t < tiles; ++t) {
    copies_wait<C::STAGES - 2>();
    __syncthreads();                 // stage t has arrived, and stage t - 1 is free
    load(t + C::STAGES - 1);
    const uint32_t sK = s0 + (t % C::STAGES) * C::STAGE, sV = sK + kKeys * C::ROW;
    const int key0 = kg * KW;        // within the stage
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
    const int valid = k_end - (k_begin + t * kKeys + key0) - 2 * (lane % 4);   // of this thread's columns n*8 + {0, 1}
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < KW / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = n * 8 + (e & 1) < valid ? s[n][e] * p.scale_log2 : -INFINITY;
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
  // the key groups of this block: their sums over group 0's, (m, l) to sj
  float2* sj = sm + 4 * 16;
  for (int i = threadIdx.x; i < MT * 16 * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < KG; ++g) top = fmaxf(top, sm[g * MT * 16 + r].x);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < KG; ++g) {
      const int at = g * MT * 16 + r;
      const float w = ex2_approx(sm[at].x - base);
      const float4 x = *reinterpret_cast<const float4*>(so + at * (D + 4) + d);
      total = fmaf(w, sm[at].y, total);
      sum = make_float4(fmaf(w, x.x, sum.x), fmaf(w, x.y, sum.y), fmaf(w, x.z, sum.z), fmaf(w, x.w, sum.w));
    }
    *reinterpret_cast<float4*>(so + r * (D + 4) + d) = sum;
    if (d == 0) sj[r] = make_float2(top, total);
  }
  // the blocks of a cluster share out the rows
  const int parts = min(p.splits, kCrossCluster), rank = blockIdx.y % parts, cluster = blockIdx.y / parts;
  const bool clustered = parts > 1;
  if (clustered) cluster_sync(); else __syncthreads();
  const int64_t n_rows = static_cast<int64_t>(p.batch) * p.heads * p.s_q;
  for (int i = rank * kThreads + threadIdx.x; i < MT * 16 * (D / 4); i += kThreads * parts) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    if (r >= rows) break;
    float top, total;
    float4 sum;
    if (!clustered) {
      top = sj[r].x;
      total = sj[r].y;
      sum = *reinterpret_cast<const float4*>(so + r * (D + 4) + d);
    } else {
      float2 ml[kCrossCluster];
      top = -INFINITY;
#pragma unroll
      for (int x = 0; x < kCrossCluster; ++x) {
        ml[x] = x < parts ? cluster_load2(cluster_addr(smem_addr(sj + r), x)) : make_float2(-INFINITY, 0.f);
        top = fmaxf(top, ml[x].x);
      }
      const float base = top == -INFINITY ? 0.f : top;
      total = 0.f;
      sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kCrossCluster; ++x) {
        if (x >= parts) continue;
        const float w = ex2_approx(ml[x].x - base);
        const float4 y = cluster_load4(cluster_addr(smem_addr(so + r * (D + 4) + d), x));
        total = fmaf(w, ml[x].y, total);
        sum = make_float4(fmaf(w, y.x, sum.x), fmaf(w, y.y, sum.y), fmaf(w, y.z, sum.z), fmaf(w, y.w, sum.w));
      }
    }
    const bool none = total == 0.f;   // (no keys in this cluster's parts, or scores of -inf only)
    const float inv = none ? 0.f : 1.f / total;
    sum = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
    const float lse = none ? -INFINITY : (top + log2f(total)) * kLn2;
    const int qi = r / share, h = hk * share + r % share;
    if (p.splits > parts) {
      const int64_t at = cluster * n_rows + (static_cast<int64_t>(b) * p.heads + h) * p.s_q + qi;
      float* dst = p.ws + at * D + d;
      float* dl = p.ws + p.splits / parts * n_rows * D + at;
      if (!none && CPATTN_IN(p.ws_span, dst, 16, p.err)) *reinterpret_cast<float4*>(dst) = sum;
      if (d == 0 && CPATTN_IN(p.ws_span, dl, 4, p.err)) *dl = lse;
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out.data) + b * p.out.s[0] + h * p.out.s[1] +
                           static_cast<int64_t>(qi) * p.out.s[2] + d;
      float* dl = static_cast<float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + qi * p.lse.s[2];
      if (CPATTN_IN(p.out.span, dst, 8, p.err))
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
      if (d == 0 && CPATTN_IN(p.lse.span, dl, 4, p.err)) *dl = lse;
    }
  }
  if (clustered) cluster_sync();   // (shared memory stays until every block has read it)
}

template <int D, int MT>
cudaError_t launch_tiles(const CrossParams& p, cudaStream_t stream) {
  using C = Few<D>;
  auto kernel = cross_few_kernel<D, MT>;
  static std::atomic<unsigned long long> ready{0};
  const cudaError_t e = cross_set_up(kernel, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(p.batch) * p.kv_heads;
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_behind_clustered(kernel, dim3(static_cast<unsigned>(units), p.splits),
                                 dim3(1, p.splits < kCrossCluster ? p.splits : kCrossCluster), kThreads, C::SMEM, stream, p);
}

template <int D>
cudaError_t launch_typed(const CrossParams& p, cudaStream_t stream) {
  const int rows = p.s_q * (p.heads / p.kv_heads);
  return rows <= 16 ? launch_tiles<D, 1>(p, stream)
                    : rows <= 32 ? launch_tiles<D, 2>(p, stream) : launch_tiles<D, 4>(p, stream);
}

}  // namespace

int cross_few_clusters(int size) {
  return cross_clusters(cross_few_kernel<128, 1>, dim3(1, size), kThreads, Few<128>::SMEM);
}

cudaError_t launch_cross_few(int head_dim, const CrossParams& p, cudaStream_t stream) {
  return head_dim == 64 ? launch_typed<64>(p, stream) : launch_typed<128>(p, stream);
}

}  // namespace cpattn
