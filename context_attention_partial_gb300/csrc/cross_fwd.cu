// cross_fwd.cu -- cross attention of bf16 inputs on the tensor cores.
//
// Mathematics: per query row, over the first n = length[b] keys,
//     m = max_j scale s_j,  P_j = 2^(scale log2e s_j - m),  l = sum_j P_j,
//     o = sum_j P_j v_j / l,  lse = m ln2 + ln l,
// one pass over the keys with the running m and l (fp32).  P is rounded to
// bf16 for its product with V (the tensor cores' operand type; l keeps the
// fp32 values), and the output once.
//
// What bounds it: an encoder's states are short (some 64 to 512 keys), so a
// unit of work -- 256 query rows of one head against its keys -- is only a
// few 128-key tiles, 1024 tensor-core cycles per query tile each, and the
// time to start and finish a unit weighs as much.  The kernel is therefore
// persistent, one CTA per SM walking units u, u + gridDim.x, ...: the next
// unit's queries and keys are fetched and its first Q K^T issued while this
// unit's last softmax, P V and output are under way.
//
// Roles (12 warps): warps 0-7 softmax and output, a warpgroup per 128-row
// query tile and one thread per row; warp 8 TMA producer; warp 9 MMA issuer;
// warps 10-11 only give up their registers.  TMEM: S_0 | S_1 | O_0 | O_1,
// P over S's first columns.  Shared memory: the two Q tiles, a ring of K / V
// tiles, and an output staging area per softmax warp.
//
// Measured: 4608 queries x 512 keys x 24 heads, D = 128: 24.4 us (1190 TFLOP/s);
// a step of two query tiles takes 2550 cycles, 2048 of them MMAs, near what
// shared memory gives (256 KB a step), a unit's boundary some 2000.  77 queries
// x 4481 keys x 32 heads, D = 64: 15.4 us.
//
// Keys past a length share their tile with valid ones: their scores are
// masked in registers, and their V rows are overwritten with zeros in shared
// memory before P V reads them (0 * NaN would not be 0).
// A unit may also be one part of the key axis (few queries): up to 8 parts are a
// cluster and join their fp32 rows in its shared memory (by way of the workspace
// and a second kernel this took 6 of 18 us at 77 queries x 4481 keys x 32 heads,
// 4 parts); the results of several clusters go to the workspace and are joined
// by that kernel.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "cross_ops.cuh"

namespace cpattn {
namespace {

constexpr int kBM = 128, kBN = 128;
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9;
constexpr int kLaunchRegs = 168;    // 65536 / 384, rounded down to 8
constexpr int kSoftmaxRegs = 208, kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays below 2^8
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.442695040888963407f;
constexpr unsigned kErrProducer = 1u, kErrMma = 2u, kErrSoftmax = 4u;

template <int D>
struct Cfg {
  static constexpr int ROW = D * 2;                       // bytes
  static constexpr int TILE = kBM * ROW;                  // bytes of a Q, K or V tile
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int STAGING = 8 * 32 * 128;            // 32 rows x 64 columns bf16 per warp
  static constexpr int BARS = 2 * STAGES + 11;
  static constexpr int SMEM = 1024 + 2 * TILE + STAGES * TILE + STAGING + BARS * 8 + 16;
  static constexpr int QK = ROW / 32, PV = kBN / 16;      // MMAs of a tile product
  static constexpr int O_COL = 2 * kBN;
  static constexpr uint32_t IDESC_QK = make_idesc(1, false, kBM, kBN);
  static constexpr uint32_t IDESC_PV = make_idesc(1, true, kBM, D);
  static_assert(O_COL + 2 * D <= 512, "TMEM");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct Unit {
  int b, h, q0, part;      // batch, head, first query row, part of the key axis
  int k0, k1;              // its keys
  int tiles, halves;       // key tiles, query tiles with rows
};

// Walks this CTA's units, blockIdx.x, blockIdx.x + gridDim.x, ..., part fastest
// (a cluster has one unit's), then query block, head and batch.  A step adds the grid's size digit by
// digit: divisions at every unit cost some 700 cycles between two units.
template <bool SPLIT>   // false: one part
struct UnitWalk {
  int q, part, h, b;       // digits of the unit
  int dq, dp, dh, db;      // digits of the grid's size
  int q_blocks;
  __device__ void split(const CrossParams& p, uint32_t u, int& q_, int& p_, int& h_, int& b_) const {
    const uint32_t splits = SPLIT ? p.splits : 1;
    uint32_t r = u / splits;
    p_ = static_cast<int>(u - r * splits);
    u = r / q_blocks;
    q_ = static_cast<int>(r - u * q_blocks);
    b_ = static_cast<int>(u / p.heads);
    h_ = static_cast<int>(u - b_ * p.heads);
  }
  __device__ explicit UnitWalk(const CrossParams& p) {
    q_blocks = ceil_div(p.s_q, 2 * kBM);
    split(p, blockIdx.x, q, part, h, b);
    split(p, gridDim.x, dq, dp, dh, db);
    for (int* x : {&q, &part, &h, &b, &dq, &dp, &dh, &db}) *x = uniform(*x);
  }
  __device__ bool more(const CrossParams& p) const { return b < p.batch; }
  __device__ void step(const CrossParams& p) {
    q += dq;
    if (SPLIT) part += dp;
    h += dh;
    b += db;
    if (SPLIT && part >= p.splits) {
      part -= p.splits;
      ++q;
    }
    if (q >= q_blocks) {
      q -= q_blocks;
      ++h;
    }
    if (h >= p.heads) {
      h -= p.heads;
      ++b;
    }
  }
  __device__ Unit unit(const CrossParams& p) const {
    Unit w;
    w.b = b;
    w.h = h;
    w.part = part;
    w.q0 = q * (2 * kBM);
    const int len = uniform(cross_length(p, b));
    const int all = ceil_div(len, kBN);
    int t0 = 0, t1 = all;
    if (SPLIT) {
      const int per = uniform(ceil_div(all, p.splits));
      t0 = min(part * per, all);
      t1 = min(t0 + per, all);
    }
    w.k0 = t0 * kBN;
    w.k1 = min(t1 * kBN, len);
    w.tiles = t1 - t0;
    w.halves = p.s_q - w.q0 > kBM ? 2 : 1;
    return w;
  }
  // Moves to the first unit with keys at or after this one.
  __device__ bool with_keys(const CrossParams& p, Unit& w) {
    for (; more(p); step(p)) {
      w = unit(p);
      if (w.tiles > 0) return true;
    }
    return false;
  }
};

// Joins the rows of a cluster's parts (256 threads of every block; the block's
// other threads meet the two cluster barriers): every block takes some of the
// rows, four 16-byte chunks a thread at a time.  Results of several clusters go
// to the workspace.  `weights`: [9][256] floats of this block's own.
template <int D>
__device__ __forceinline__ void join_cluster(const CrossParams& p, const float4* part_o, const float* part_lse,
                                             float* weights) {
  const int parts = min(p.splits, kCrossCluster);
  const Unit w = UnitWalk<true>(p).unit(p);
  const int rank = w.part % parts, cluster = w.part / parts, rows = min(p.s_q - w.q0, 2 * kBM);
  cluster_sync();
  // a row's weights, and the lse of its whole, where one of this block's threads
  // below takes the row
  const int t = threadIdx.x;
  if (t < rows && t * (D / 4) / 256 % parts == rank) {
    float lse[kCrossCluster], top = -INFINITY, total = 0.f;
#pragma unroll
    for (int x = 0; x < kCrossCluster; ++x) {
      lse[x] = x < parts ? cluster_load(cluster_addr(smem_addr(part_lse + t), x)) : -INFINITY;
      top = fmaxf(top, lse[x]);
    }
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int x = 0; x < kCrossCluster; ++x) {
      lse[x] = ex2_approx((lse[x] - base) * kLog2e);
      total += lse[x];
    }
    const bool none = total == 0.f;
    const float inv = none ? 0.f : 1.f / total;
#pragma unroll
    for (int x = 0; x < kCrossCluster; ++x)
      if (x < parts) weights[x * 256 + t] = lse[x] * inv;
    weights[8 * 256 + t] = none ? -INFINITY : base + log2f(total) * kLn2;
  }
  asm volatile("bar.sync 1, 256;" ::: "memory");
  const int64_t n = static_cast<int64_t>(p.batch) * p.heads * p.s_q;
  constexpr int U = 4;
  const int items = rows * (D / 4), step = parts * 256;
  for (int i0 = rank * 256 + t; i0 < items; i0 += U * step) {
    float4 sum[U];
    int at[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * step, items - 1);
      r[u] = i / (D / 4);
      at[u] = r[u] * (D / 4) + (i % (D / 4) ^ (r[u] & 7));
      sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 4
    for (int x = 0; x < parts; ++x) {
      float4 y[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * step < items) y[u] = cluster_load4(cluster_addr(smem_addr(part_o + at[u]), x));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = weights[x * 256 + r[u]];
        if (f != 0.f && i0 + u * step < items)   // (a part without keys has written no row)
          sum[u] = make_float4(fmaf(f, y[u].x, sum[u].x), fmaf(f, y[u].y, sum[u].y), fmaf(f, y[u].z, sum[u].z),
                               fmaf(f, y[u].w, sum[u].w));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * step >= items) break;
      const int c = (i0 + u * step) % (D / 4);
      const int64_t row = w.q0 + r[u];
      if (p.splits > parts) {
        const int64_t place = cluster * n + (static_cast<int64_t>(w.b) * p.heads + w.h) * p.s_q + row;
        float4* dst = reinterpret_cast<float4*>(p.ws + place * D) + c;
        float* dl = p.ws + p.splits / parts * n * D + place;
        if (CPATTN_IN(p.ws_span, dst, 16, p.err)) *dst = sum[u];
        if (c == 0 && CPATTN_IN(p.ws_span, dl, 4, p.err)) *dl = weights[8 * 256 + r[u]];
      } else {
        __nv_bfloat16* dst =
            static_cast<__nv_bfloat16*>(p.out.data) + w.b * p.out.s[0] + w.h * p.out.s[1] + row * p.out.s[2] + c * 4;
        float* dl = static_cast<float*>(p.lse.data) + w.b * p.lse.s[0] + w.h * p.lse.s[1] + row * p.lse.s[2];
        if (CPATTN_IN(p.out.span, dst, 8, p.err))
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(pack_bf16x2(sum[u].x, sum[u].y), pack_bf16x2(sum[u].z, sum[u].w));
        if (c == 0 && CPATTN_IN(p.lse.span, dl, 4, p.err)) *dl = weights[8 * 256 + r[u]];
      }
    }
  }
  cluster_sync();   // (shared memory stays until every block has read it)
}

// PAIR: the two query tiles are the same one (S_q <= 128), its key tiles
// alternate between them, each with sums of its own, and the warps of the first
// take the second's over at the end; a CTA has one unit.  A lone tile's products
// and exponentials wait for one another (some 2600 cycles a key tile); two
// chains fill each other's waits.
// SPLIT: parts of the key axis (one, with PAIR, where the units fill the GPU).
template <int D, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                     const __grid_constant__ CrossParams p) {
  using C = Cfg<D>;
  const bool split = SPLIT && p.splits > 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sQ = smem_addr(smem), sKV = sQ + 2 * C::TILE;
  uint8_t* staging = smem + (2 + C::STAGES) * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + C::STAGING);
  const uint32_t bar0 = smem_addr(bars);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto bar_q = [&](int i) { return bar0 + 8u * (2 * C::STAGES + i); };          // Q tile arrived
  auto bar_qfree = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 2 + i); };  // its last Q K^T is done
  auto bar_s = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 4 + i); };      // scores ready
  auto bar_p = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 6 + i); };      // P written
  auto bar_o = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 8 + i); };      // O of a unit ready
  const uint32_t bar_drain = bar0 + 8u * (2 * C::STAGES + 10);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q(i), 1);
      mbar_init(bar_qfree(i), 1);
      mbar_init(bar_s(i), 1);
      mbar_init(bar_p(i), 4);   // one arrival per softmax warp
      mbar_init(bar_o(i), 1);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_holder), 512);
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_o);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpProducer) {
    // the first unit's queries (and keys, unless their place depends on a
    // length), while the kernel before this one ends: 25.7 us without, 24.4 with,
    // at 4608 x 512 x 24 heads
    const UnitWalk<SPLIT> first(p);
    if (first.more(p) && lane == 0) {
      const int q0 = first.q * (2 * kBM);
      prefetch_tile<D>(&tm_q, q0, first.h, first.b);
      if (p.s_q - q0 > kBM) prefetch_tile<D>(&tm_q, q0 + kBM, first.h, first.b);
      if (!SPLIT) {
        prefetch_tile<D>(&tm_k, 0, first.h / (p.heads / p.kv_heads), first.b);
        prefetch_tile<D>(&tm_v, 0, first.h / (p.heads / p.kv_heads), first.b);
      }
    }
    __syncwarp();
  }
  launch_wait();
  launch_next();
  const uint32_t tmem = *tmem_holder;
  // every wait of a warp is voted on, so its lanes stay together
  auto wait_all = [&](uint32_t bar, uint32_t parity, unsigned code) {
    const bool r = mbar_wait(bar, parity, abort_flag, p.timeout_ns, p.err, code);
    return __all_sync(0xffffffffu, r) != 0;
  };

  if (warp >= 8) {
    regs_decrease<kControlRegs>();
    const bool leader = elect_one();
    if (warp == kWarpProducer) {
      // ---------------------------------------------------------- producer
      // K tiles on even stages, V tiles on odd ones: the first K alone, then
      // V_j and the K tile after it (of the next unit behind a unit's last V)
      // as one pair on the K stage's barrier, so the MMA warp waits once a
      // step; the very last V on its own.
      static_assert(C::STAGES % 2 == 0, "K / V pairs");
      const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
      int ld = 0, nq[2] = {0, 0};
      UnitWalk<SPLIT> walk(p);
      Unit w;
      const int share = p.heads / p.kv_heads;
      bool have = walk.with_keys(p, w);
      bool ok = p.fault_skip_kv == 0;
      auto load_q = [&](const Unit& x) {   // once the previous unit's last Q K^T is done
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= x.halves) break;
          ok = wait_all(bar_qfree(i), (nq[i] & 1) ^ 1, kErrProducer);
          if (!ok) return;
          if (leader) {
            mbar_arrive_expect_tx(bar_q(i), C::TILE);
            load_tile<D>(sQ + i * C::TILE, &tm_q, bar_q(i), x.q0 + i * kBM, x.h, x.b, pol_q);
          }
          __syncwarp();
          ++nq[i];
        }
      };
      if (have && ok) {
        if (leader) {
          mbar_arrive_expect_tx(bar_full(0), C::TILE);
          load_tile<D>(sKV, &tm_k, bar_full(0), w.k0, w.h / share, w.b, pol_kv);
        }
        __syncwarp();
        ld = 1;
        load_q(w);
      }
      while (have && ok) {
        Unit wn;
        walk.step(p);
        const bool more_units = walk.with_keys(p, wn);
        // (from HBM the next Q tiles arrived some 2000 cycles after they were wanted)
        if (more_units && leader)
          for (int i = 0; i < wn.halves; ++i) prefetch_tile<D>(&tm_q, wn.q0 + i * kBM, wn.h, wn.b);
        for (int j = 0; j < w.tiles && ok; ++j) {
          const bool in_unit = j + 1 < w.tiles, more = in_unit || more_units;
          const int sv = ld % C::STAGES, sk = (ld + 1) % C::STAGES;
          ok = wait_all(bar_empty(sv), ((ld / C::STAGES) & 1) ^ 1, kErrProducer);
          if (ok && more) ok = wait_all(bar_empty(sk), (((ld + 1) / C::STAGES) & 1) ^ 1, kErrProducer);
          if (!ok) break;
          if (leader) {
            const uint32_t bar = more ? bar_full(sk) : bar_full(sv);
            mbar_arrive_expect_tx(bar, (more ? 2 : 1) * C::TILE);
            load_tile<D>(sKV + sv * C::TILE, &tm_v, bar, w.k0 + j * kBN, w.h / share, w.b, pol_kv);
            if (in_unit)
              load_tile<D>(sKV + sk * C::TILE, &tm_k, bar, w.k0 + (j + 1) * kBN, w.h / share, w.b, pol_kv);
            else if (more)
              load_tile<D>(sKV + sk * C::TILE, &tm_k, bar, wn.k0, wn.h / share, wn.b, pol_kv);
          }
          __syncwarp();
          ld += more ? 2 : 1;
        }
        if (ok && more_units) load_q(wn);
        have = more_units;
        w = wn;
      }
      if (!ok && leader) {
        // leave no copy in flight into this CTA's shared memory
        for (int x = ld > C::STAGES ? ld - C::STAGES : 0; x < ld; ++x) {
          if (x % 2 == 0)
            mbar_drain(bar_full(x % C::STAGES), (x / C::STAGES) & 1, p.timeout_ns);
          else if (x + 1 >= ld)   // (a last V tile alone)
            mbar_drain(bar_full(x % C::STAGES), 0, p.timeout_ns);
        }
        for (int i = 0; i < 2; ++i)
          if (nq[i] > 0) mbar_drain(bar_q(i), (nq[i] - 1) & 1, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024), k_desc = smem_desc_sw128(sKV, 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(sKV, kBN * 128, 1024);
      const uint32_t hi = static_cast<uint32_t>(q_desc >> 32);   // (shared by all: low words hold the address)
      // Tests come before the descriptors are built, waits only where a test
      // failed: a wait costs this warp some 190 cycles beside the softmax
      // warps of its SM sub-partition, and the tensor pipe's queue is only a
      // few MMAs deep (four waits a step: 3310 cycles a step instead of 2400).
      uint32_t g = 0;                // key tiles so far, over all units
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
      bool ok = true;
      UnitWalk<SPLIT> walk(p);
      Unit w;
      bool have = walk.with_keys(p, w);
      // a unit's first scores, query tile by query tile (its K tile is here)
      auto first_qk = [&](const Unit& x, uint32_t at) {
        const uint32_t s = at % C::STAGES;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= x.halves) break;
          ok = wait_all(bar_q(i), nq[i] & 1, kErrMma);
          if (!ok) return;
          ++nq[i];
          uint32_t a[C::QK], b[C::QK];
#pragma unroll
          for (int kk = 0; kk < C::QK; ++kk) {
            const uint32_t off = ((kk / 4) * (kBM * 128) + (kk % 4) * 32) >> 4;
            a[kk] = static_cast<uint32_t>(q_desc) + ((i * C::TILE) >> 4) + off;
            b[kk] = static_cast<uint32_t>(k_desc) + ((s * C::TILE) >> 4) + off;
          }
          tc_fence_after();
          if (leader) {
            mma_group<C::QK, true>(tmem + i * kBN, a, b, hi, C::IDESC_QK, 0u);
            mma_commit(bar_s(i));
            if (x.tiles == 1) mma_commit(bar_qfree(i));
            if (i == x.halves - 1) mma_commit(bar_empty(s));
          }
          __syncwarp();
        }
      };
      if (have) {
        ok = wait_all(bar_full(0), 0, kErrMma);
        if (ok) first_qk(w, 0);
      }
      while (have && ok) {
        Unit wn;
        walk.step(p);
        const bool more_units = walk.with_keys(p, wn);
        for (int j = 0; j < w.tiles; ++j, ++g) {
          const bool more = j + 1 < w.tiles, two = w.halves == 2;
          const uint32_t sv = (2 * g + 1) % C::STAGES, lk = 2 * g + 2, sk = lk % C::STAGES;
          const bool pair = more || more_units;
          const uint32_t kv_bar = pair ? bar_full(sk) : bar_full(sv), kv_ph = pair ? (lk / C::STAGES) & 1 : 0u;
          const bool kv_now = mbar_test(kv_bar, kv_ph);
          const bool p0_now = !PAIR && mbar_test(bar_p(0), np[0] & 1);
          const uint32_t vb = static_cast<uint32_t>(v_desc) + ((sv * C::TILE) >> 4);
          const uint32_t kb = static_cast<uint32_t>(k_desc) + ((sk * C::TILE) >> 4);
          uint32_t vd[C::PV], kd[C::QK], qd[C::QK], pa[C::PV];
#pragma unroll
          for (int kk = 0; kk < C::PV; ++kk) {
            vd[kk] = vb + ((kk * 16 * 128) >> 4);
            pa[kk] = tmem + kk * 8;
          }
#pragma unroll
          for (int kk = 0; kk < C::QK; ++kk) {
            const uint32_t off = ((kk / 4) * (kBM * 128) + (kk % 4) * 32) >> 4;
            kd[kk] = kb + off;
            qd[kk] = static_cast<uint32_t>(q_desc) + off;
          }
          ok = __all_sync(0xffffffffu, kv_now) || wait_all(kv_bar, kv_ph, kErrMma);
          if (!ok) break;
          const int valid = w.k1 - (w.k0 + j * kBN);
          if (valid < kBN) zero_tile_rows<D>(smem + (2 + sv) * C::TILE, valid);
          if constexpr (PAIR) {
            const int i = j & 1;
            if (more && leader) {
              // (S_1-i's last P V was issued a step ago)
              tc_fence_after();
              mma_group<C::QK, true>(tmem + (i ^ 1) * kBN, qd, kd, hi, C::IDESC_QK, 0u);
              mma_commit(bar_s(i ^ 1));
              if (j + 2 == w.tiles) mma_commit(bar_qfree(0));
              mma_commit(bar_empty(sk));
            }
            __syncwarp();
            ok = wait_all(bar_p(i), np[i] & 1, kErrMma);
            if (!ok) break;
            ++np[i];
#pragma unroll
            for (int kk = 0; kk < C::PV; ++kk) pa[kk] += i * kBN;
            tc_fence_after();
            if (leader) {
              mma_group<C::PV, false>(tmem + C::O_COL + i * D, pa, vd, hi, C::IDESC_PV, j > 1);
              mma_commit(bar_empty(sv));
              if (j + 2 >= w.tiles) mma_commit(bar_o(i));
            }
            __syncwarp();
            continue;
          }
          ok = __all_sync(0xffffffffu, p0_now) || wait_all(bar_p(0), np[0] & 1, kErrMma);
          if (!ok) break;
          ++np[0];
          const bool p1_now = two && mbar_test(bar_p(1), np[1] & 1);
          tc_fence_after();
          if (leader) {
            mma_group<C::PV, false>(tmem + C::O_COL, pa, vd, hi, C::IDESC_PV, j > 0);
            if (!two) mma_commit(bar_empty(sv));
            if (more) {
              mma_group<C::QK, true>(tmem, qd, kd, hi, C::IDESC_QK, 0u);
              mma_commit(bar_s(0));
              if (j + 2 == w.tiles) mma_commit(bar_qfree(0));
              if (!two) mma_commit(bar_empty(sk));
            } else {
              mma_commit(bar_o(0));
            }
          }
          __syncwarp();
          if (!two) continue;
#pragma unroll
          for (int kk = 0; kk < C::PV; ++kk) pa[kk] += kBN;
#pragma unroll
          for (int kk = 0; kk < C::QK; ++kk) qd[kk] += C::TILE >> 4;
          ok = __all_sync(0xffffffffu, p1_now) || wait_all(bar_p(1), np[1] & 1, kErrMma);
          if (!ok) break;
          ++np[1];
          tc_fence_after();
          if (leader) {
            mma_group<C::PV, false>(tmem + C::O_COL + D, pa, vd, hi, C::IDESC_PV, j > 0);
            mma_commit(bar_empty(sv));
            if (more) {
              mma_group<C::QK, true>(tmem + kBN, qd, kd, hi, C::IDESC_QK, 0u);
              mma_commit(bar_s(1));
              if (j + 2 == w.tiles) mma_commit(bar_qfree(1));
              mma_commit(bar_empty(sk));
            } else {
              mma_commit(bar_o(1));
            }
          }
          __syncwarp();
        }
        if (ok && more_units) first_qk(wn, 2 * g);
        have = more_units;
        w = wn;
      }
      if (!ok && leader) {
        // let every MMA already issued finish before TMEM is released
        mma_commit(bar_drain);
        mbar_drain(bar_drain, 0, p.timeout_ns);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------- softmax, output
    regs_increase<kSoftmaxRegs>();
    const int wg = warp / 4, quarter = warp % 4;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + wg * kBN;
    const uint32_t tO = tmem + lane_base + C::O_COL + wg * D;
    const float sl2 = p.scale_log2;
    uint8_t* stage = staging + warp * 4096;
    // rows of a split, and before that PAIR's second O, over the K and V tiles;
    // their lse over the Q tiles
    float4* part_o = reinterpret_cast<float4*>(smem + 2 * C::TILE);   // [256][D / 4], chunks swizzled
    float* part_lse = reinterpret_cast<float*>(smem);                 // [256]
    float2* pair_ml = reinterpret_cast<float2*>(smem + C::TILE);      // [128]
    static_assert(2 * kBM * D * 4 <= C::STAGES * C::TILE && 4096 + 9 * 1024 <= 2 * C::TILE, "a split's rows");
    int ns = 0, no = 0;
    bool ok = true;
    for (UnitWalk<SPLIT> walk(p); ok && walk.more(p); walk.step(p)) {
      const Unit w = walk.unit(p);
      if (!PAIR && wg >= w.halves) continue;
      const int row0 = w.q0 + (PAIR ? 0 : wg * kBM) + quarter * 32, row = row0 + lane;
      float m = -INFINITY, l = 0.f;
      const int first = PAIR ? wg : 0;
      for (int j = first; j < w.tiles; j += PAIR ? 2 : 1) {
        ok = wait_all(bar_s(wg), ns & 1, kErrSoftmax);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        const int valid = w.k1 - (w.k0 + j * kBN);
        uint32_t s[kBN];
        float row_max;
        if (valid >= kBN) {
          tmem_ld_max_x128(tS, s, row_max);
        } else {
          tmem_ld_x128(tS, s);
          row_max = masked_row_max<kBN>(s, valid);
        }
        const float top = row_max * sl2;
        float factor = 1.f;
        bool raise = false;
        if (j == first) {
          m = top;
        } else if (top > m + kRescaleThreshold) {
          factor = ex2_approx(m - top);
          m = top;
          l *= factor;
          raise = true;
        }
        // (the previous P V completed before these scores: one issue order)
        if (__any_sync(0xffffffffu, raise)) rescale_o<D>(tO, factor);
        // (only scores of -inf so far: their exponentials are 0, not of -inf + inf)
        const float base = m == -INFINITY ? 0.f : -m;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kBN / 2; ++i) {
          float x0, x1;
          ffma2(x0, x1, u2f(s[2 * i]), u2f(s[2 * i + 1]), sl2, sl2, base, base);
          const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
          const int a = 2 * (i & 1);
          fadd2(acc[a], acc[a + 1], acc[a], acc[a + 1], e0, e1);
          s[i] = pack_bf16x2(e0, e1);
        }
        tmem_st_x64(tS, *reinterpret_cast<uint32_t(*)[64]>(&s[0]));
        l += (acc[0] + acc[1]) + (acc[2] + acc[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p(wg));
      }
      if (!PAIR && !ok) break;
      const bool none = w.tiles == 0;
      if constexpr (PAIR) {
        // the second tile's O (unnormalised), m and l to shared memory, whose K
        // and V tiles all products have read
        for (int i = 0; i <= wg && ok; ++i)
          if (w.tiles > i) ok = wait_all(bar_o(i), 0, kErrSoftmax);
        tc_fence_after();
        if (wg == 1 && ok && w.tiles > 1) {
          const int r = quarter * 32 + lane;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 64) {
            uint32_t o[64];
            tmem_ld_x64(tO + c0, o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              part_o[r * (D / 4) + c0 / 4 + (i ^ (r & 7))] =
                  make_float4(u2f(o[4 * i]), u2f(o[4 * i + 1]), u2f(o[4 * i + 2]), u2f(o[4 * i + 3]));
          }
          pair_ml[r] = make_float2(m, l);
        }
        // (all 8 warps come here, whether their waits ran out or not: a CTA has one unit)
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (!ok || wg == 1) break;
      }
      float own = 1.f, other = 0.f;   // weights of the two sums
      if (PAIR && w.tiles > 1) {
        const float2 ml = pair_ml[quarter * 32 + lane];
        const float top = fmaxf(m, ml.x), base = top == -INFINITY ? 0.f : top;
        own = ex2_approx(m - base);
        other = ex2_approx(ml.x - base);
        l = l * own + ml.y * other;
        m = top;
      }
      // (l is 0 where every score is -inf: no key has weight, as without keys)
      const float inv = none || l == 0.f ? 0.f : 1.f / l;
      const float lse = none ? -INFINITY : (m + log2f(l)) * kLn2;
      if (!PAIR && !none) {
        ok = wait_all(bar_o(wg), no & 1, kErrSoftmax);
        // (a split's rows go where the other tile's products read K and V)
        if (ok && split && w.halves == 2) ok = wait_all(bar_o(wg ^ 1), 0, kErrSoftmax);
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      if (split) {
        if (row < p.s_q) part_lse[(PAIR ? 0 : wg * kBM) + quarter * 32 + lane] = lse;
      } else if (row < p.s_q) {
        float* dst = static_cast<float*>(p.lse.data) + w.b * p.lse.s[0] + w.h * p.lse.s[1] + row * p.lse.s[2];
        if (CPATTN_IN(p.lse.span, dst, 4, p.err)) *dst = lse;
      }
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t o[64];
        __syncwarp();
        if (none) {
#pragma unroll
          for (int i = 0; i < 64; ++i) o[i] = 0u;
        } else {
          tmem_ld_x64(tO + c0, o);
          if (PAIR && w.tiles > 1) {
            const int r = quarter * 32 + lane;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 x = part_o[r * (D / 4) + c0 / 4 + (i ^ (r & 7))];
              o[4 * i] = f2u(u2f(o[4 * i]) * own + x.x * other);
              o[4 * i + 1] = f2u(u2f(o[4 * i + 1]) * own + x.y * other);
              o[4 * i + 2] = f2u(u2f(o[4 * i + 2]) * own + x.z * other);
              o[4 * i + 3] = f2u(u2f(o[4 * i + 3]) * own + x.w * other);
            }
          }
        }
        if (split) {
          const int r = (PAIR ? 0 : wg * kBM) + quarter * 32 + lane;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            part_o[r * (D / 4) + c0 / 4 + (i ^ (r & 7))] = make_float4(
                u2f(o[4 * i]) * inv, u2f(o[4 * i + 1]) * inv, u2f(o[4 * i + 2]) * inv, u2f(o[4 * i + 3]) * inv);
          continue;
        }
        // (the previous store has read the stage)
        if (lane == 0) bulk_wait_read();
        __syncwarp();
        store_rows<64>(p, p.out, &tm_o, stage, o, inv, w.b, w.h, row0, p.s_q, c0);
      }
    }
    if (split) join_cluster<D>(p, part_o, part_lse, reinterpret_cast<float*>(smem + 4096));
  }
  if (split && warp >= 8) {   // (as join_cluster)
    cluster_sync();
    cluster_sync();
  }
  if (lane == 0) bulk_wait_read();   // (no store reads this CTA's shared memory any more)
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool PAIR, bool SPLIT>
cudaError_t launch_typed(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                         const CUtensorMap& tm_o, const CrossParams& p, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kernel = cross_fwd_kernel<D, PAIR, SPLIT>;
  static std::atomic<unsigned long long> ready{0};
  const cudaError_t e = cross_set_up(kernel, C::SMEM, ready, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(p.batch) * p.heads * p.splits * ((p.s_q + 2 * kBM - 1) / (2 * kBM));
  const int64_t sms = sm_count();
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(PAIR || p.splits > 1 || units < sms ? units : sms));
  const unsigned cluster = p.splits < kCrossCluster ? p.splits : kCrossCluster;
  return launch_behind_clustered(kernel, grid, dim3(cluster), kThreads, C::SMEM, stream, tm_q, tm_k, tm_v, tm_o, p);
}

}  // namespace

int cross_fwd_clusters(int size) {
  return cross_clusters(cross_fwd_kernel<128, false, true>, dim3(size), kThreads, Cfg<128>::SMEM);
}

cudaError_t launch_cross_fwd(int head_dim, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             const CUtensorMap& tm_o, const CrossParams& p, cudaStream_t stream) {
  // one wave of a single query tile each: two sums a tile
  const int64_t units = static_cast<int64_t>(p.batch) * p.heads * p.splits;
  if (p.s_q <= kBM && units <= sm_count())
    return head_dim == 64 ? launch_typed<64, true, true>(tm_q, tm_k, tm_v, tm_o, p, stream)
                          : launch_typed<128, true, true>(tm_q, tm_k, tm_v, tm_o, p, stream);
  // (the code of splits costs calls without 3 %: 4608 x 512 x 24 heads 27.0 us, not 26.3)
  if (p.splits > 1)
    return head_dim == 64 ? launch_typed<64, false, true>(tm_q, tm_k, tm_v, tm_o, p, stream)
                          : launch_typed<128, false, true>(tm_q, tm_k, tm_v, tm_o, p, stream);
  return head_dim == 64 ? launch_typed<64, false, false>(tm_q, tm_k, tm_v, tm_o, p, stream)
                        : launch_typed<128, false, false>(tm_q, tm_k, tm_v, tm_o, p, stream);
}

}  // namespace cpattn
