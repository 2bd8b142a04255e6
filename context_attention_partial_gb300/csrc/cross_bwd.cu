// cross_bwd.cu -- the gradient of cross attention of bf16 inputs on the tensor
// cores.
//
// Mathematics (lse and delta_i = do_i . o_i given, per query row i, key j):
//     P_ij = 2^(scale log2e q_i.k_j - lse_i log2e),  dP_ij = do_i . v_j,
//     dS_ij = P_ij (dP_ij - delta_i),
//     dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij do_i.
// Two kernels.  One owns 128 query rows and walks the keys (dq: three tile
// products a step), one owns 128 keys and walks the query rows (dk, dv: four).
// The five products of a single kernel would need dq summed over key tiles by
// atomics, whose order changes the result, or written and read back once per
// key tile (226 MB at 4608 x 512 x 24 heads); forming S and dP twice costs
// two products more and keeps every sum in one place and order.
// P and dS are rounded to bf16 for their products (the tensor cores' operand
// type); sums, P and dS themselves are fp32, results are rounded once.
//
// Roles (12 warps): warps 0-7 elementwise, two warpgroups on the same 128 TMEM
// lanes taking 64 of the tile's 128 columns each; warp 8 TMA producer, warp 9
// MMA issuer, warp 10 row statistics (dk/dv kernel).
// TMEM columns, dq:     S 0 | dP 128 | dQ 256 | dS 384, 448 (two buffers)
//               dk, dv: S^T 0 | dP^T 128, then P^T and dS^T over it | dV, dK 256..
// The next step's S is issued as soon as this step's S is in registers, so the
// exponentials run under dQ (or dV and dK) and the products under the
// elementwise work.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "cross.cuh"
#include "ptx.cuh"
#include "tile_ops.cuh"
#include "tmem_ops.cuh"

namespace cpattn {
namespace {

constexpr int kBM = 128;            // rows of every tile
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpStats = 10;
constexpr int kLaunchRegs = 168;    // 65536 / 384, rounded down to 8
constexpr int kSoftmaxRegs = 208, kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr float kLog2e = 1.442695040888963407f;
constexpr unsigned kErrProducer = 1u, kErrMma = 2u, kErrSoftmax = 4u, kErrStats = 8u;

template <int D>
struct Cfg {
  static constexpr int ROW = D * 2;                    // bytes
  static constexpr int NKB = ROW / 128;                // 128-byte column blocks
  static constexpr int TILE = kBM * ROW;
  static constexpr int QK = ROW / 32, PV = kBM / 16;   // MMAs over D, over a tile's rows
  static constexpr uint32_t IDESC_S = make_idesc(1, false, kBM, kBM);
  static constexpr uint32_t IDESC_G = make_idesc(1, true, kBM, D);
  // dq kernel: K, V tiles in a ring, Q and dO of a unit
  static constexpr int RING = D == 128 ? 4 : 8;
  static constexpr int DQ_BARS = 2 * RING + 11;
  static constexpr int STAGING = 8 * 32 * (D / 2) * 2; // 32 rows x D / 2 columns per warp
  static constexpr int DQ_SMEM = 1024 + (2 + RING) * TILE + STAGING + DQ_BARS * 8 + 16;
  // dk, dv kernel: K, V tiles, stages of a Q and a dO tile with row statistics
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int STATS = 2 * kBM * 4;            // lse2, delta of a stage
  static constexpr int KV_BARS = 4 * STAGES + 7;
  static constexpr int KV_SMEM = 1024 + (2 + 2 * STAGES) * TILE + STAGES * STATS + KV_BARS * 8 + 16;
  static_assert(DQ_SMEM <= 227 * 1024 && KV_SMEM <= 227 * 1024, "shared memory");
};

// [rows x D] x [rows x D]^T: both tiles as TMA wrote them, row by row
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a_addr, uint32_t b_addr) {
  using C = Cfg<D>;
  const uint64_t base = smem_desc_sw128(0, 16, 1024);
  uint32_t a[C::QK], b[C::QK];
#pragma unroll
  for (int kk = 0; kk < C::QK; ++kk) {
    const uint32_t off = ((kk / 4) * (kBM * 128) + (kk % 4) * 32) >> 4;
    a[kk] = static_cast<uint32_t>(base) + (a_addr >> 4) + off;
    b[kk] = static_cast<uint32_t>(base) + (b_addr >> 4) + off;
  }
  mma_group<C::QK, true>(d, a, b, static_cast<uint32_t>(base >> 32), C::IDESC_S, 0u);
}

// (+)= A (TMEM, k-step kk at a_col(kk)) x the rows of a tile
template <int D, typename F>
__device__ __forceinline__ void mma_cols(uint32_t d, F a_col, uint32_t b_addr, uint32_t acc) {
  using C = Cfg<D>;
  const uint64_t base = smem_desc_sw128(0, kBM * 128, 1024);
  uint32_t a[C::PV], b[C::PV];
#pragma unroll
  for (int kk = 0; kk < C::PV; ++kk) {
    a[kk] = a_col(kk);
    b[kk] = static_cast<uint32_t>(base) + ((b_addr + kk * 16 * 128) >> 4);
  }
  mma_group<C::PV, false>(d, a, b, static_cast<uint32_t>(base >> 32), C::IDESC_G, acc);
}

template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int row, int h, int b,
                                          uint64_t pol) {
  for (int kb = 0; kb < Cfg<D>::NKB; ++kb)
    tma_load_4d_hint(dst + kb * kBM * 128, tm, bar, kb * 64, row, h, b, pol);
}

// A warp's 32 rows x N columns (fp32 in registers, one row per lane) as bf16
// through its staging area (16-byte chunks XOR-swizzled by row) to rows
// row0.. of a tensor, columns from c0; rows at or past `rows` are not written.
template <int N>
__device__ __forceinline__ void store_rows(const CrossParams& p, const CrossTensor& t, uint8_t* stage,
                                           const uint32_t (&o)[N], float f, int b, int h, int row0, int rows, int c0,
                                           uint64_t pol) {
  constexpr int CH = N / 8;   // chunks of a row
  const int lane = threadIdx.x % 32;
  __syncwarp();
  uint4* srow = reinterpret_cast<uint4*>(stage) + lane * CH;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    uint32_t x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack_bf16x2(u2f(o[8 * i + 2 * e]) * f, u2f(o[8 * i + 2 * e + 1]) * f);
    srow[i ^ (lane % CH)] = make_uint4(x[0], x[1], x[2], x[3]);
  }
  __syncwarp();
  uint8_t* out = static_cast<uint8_t*>(t.data) + (b * t.s[0] + h * t.s[1]) * 2;
#pragma unroll
  for (int it = 0; it < CH; ++it) {
    const int idx = it * 32 + lane, r = idx / CH, c = idx % CH;
    if (row0 + r < rows) {
      const uint4 val = reinterpret_cast<const uint4*>(stage)[r * CH + (c ^ (r % CH))];
      uint8_t* dst = out + (static_cast<int64_t>(row0 + r) * t.s[2] + c0) * 2 + c * 16;
      if (CPATTN_IN(t.span, dst, 16, p.err)) st_global_v4_hint(dst, val, pol);
    }
  }
}

// ------------------------------------------------------------------ dq
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_g,
                    const __grid_constant__ CrossParams p, const int64_t units) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sQ = smem_addr(smem), sG = sQ + C::TILE, sKV = sG + C::TILE;
  uint8_t* staging = smem + (2 + C::RING) * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + C::STAGING);
  const uint32_t bar0 = smem_addr(bars);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (C::RING + s); };
  const uint32_t B = bar0 + 8u * (2 * C::RING);
  const uint32_t BAR_Q = B, BAR_G = B + 8, BAR_QFREE = B + 16, BAR_GFREE = B + 24, BAR_S = B + 32, BAR_DP = B + 40,
                 BAR_SREAD = B + 48, BAR_DPREAD = B + 56, BAR_DS = B + 64, BAR_DQ = B + 72, BAR_DRAIN = B + 80;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::DQ_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::RING; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (uint32_t x : {BAR_Q, BAR_G, BAR_QFREE, BAR_GFREE, BAR_S, BAR_DP, BAR_DQ, BAR_DRAIN}) mbar_init(x, 1);
    for (uint32_t x : {BAR_SREAD, BAR_DPREAD, BAR_DS}) mbar_init(x, 8);   // one arrival per elementwise warp
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_holder), 512);
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_g);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait_all = [&](uint32_t bar, uint32_t parity, unsigned code) {
    const bool r = mbar_wait(bar, parity, abort_flag, p.timeout_ns, p.err, code);
    return __all_sync(0xffffffffu, r) != 0;
  };
  const int q_tiles = ceil_div(p.s_q, kBM);
  struct Unit {
    int b, h, q0, len, tiles;
  };
  auto unit_at = [&](int64_t u) {
    Unit w;
    w.q0 = static_cast<int>(u % q_tiles) * kBM;
    u /= q_tiles;
    w.h = static_cast<int>(u % p.heads);
    w.b = static_cast<int>(u / p.heads);
    w.len = cross_length(p, w.b);
    w.tiles = ceil_div(w.len, kBM);
    return w;
  };

  if (warp >= 8) {
    regs_decrease<kControlRegs>();
    const bool leader = elect_one();
    if (warp == kWarpProducer) {
      const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
      int ld = 0, nq = 0, ng = 0;
      bool ok = p.fault_skip_kv == 0;
      for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const Unit w = unit_at(u);
        const int hk = w.h / (p.heads / p.kv_heads);
        for (int x = 0; x < 2 * w.tiles && ok; ++x) {
          const int s = ld % C::RING;
          ok = wait_all(bar_empty(s), ((ld / C::RING) & 1) ^ 1, kErrProducer);
          if (!ok) break;
          if (leader) {
            mbar_arrive_expect_tx(bar_full(s), C::TILE);
            load_tile<D>(sKV + s * C::TILE, x % 2 ? &tm_v : &tm_k, bar_full(s), (x / 2) * kBM, hk, w.b, pol_kv);
          }
          __syncwarp();
          ++ld;
          if (x < 2) {   // Q after the first K tile, dO after the first V tile
            int& n = x ? ng : nq;
            ok = wait_all(x ? BAR_GFREE : BAR_QFREE, (n & 1) ^ 1, kErrProducer);
            if (!ok) break;
            if (leader) {
              mbar_arrive_expect_tx(x ? BAR_G : BAR_Q, C::TILE);
              load_tile<D>(x ? sG : sQ, x ? &tm_g : &tm_q, x ? BAR_G : BAR_Q, w.q0, w.h, w.b, pol_q);
            }
            __syncwarp();
            ++n;
          }
        }
      }
      if (!ok && leader) {
        // leave no copy in flight into this CTA's shared memory
        for (int x = ld > C::RING ? ld - C::RING : 0; x < ld; ++x)
          mbar_drain(bar_full(x % C::RING), (x / C::RING) & 1, p.timeout_ns);
        if (nq > 0) mbar_drain(BAR_Q, (nq - 1) & 1, p.timeout_ns);
        if (ng > 0) mbar_drain(BAR_G, (ng - 1) & 1, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      auto next_unit = [&](int64_t& u, Unit& w) {   // the next one with keys
        for (; u < units; u += gridDim.x) {
          w = unit_at(u);
          if (w.tiles > 0) return true;
        }
        return false;
      };
      int ld = 0, n = 0, it = 0;   // first load of the unit, units, steps over all units
      bool ok = true;
      int64_t u = blockIdx.x;
      Unit w;
      bool have = next_unit(u, w);
      // S and dP of key tile j (loads at and at + 1) of a unit; K's rows past
      // the last key become zeros first: dS is 0 there, and 0 * NaN is not
      auto issue_s = [&](const Unit& x, int j, int at) {
        const int s = at % C::RING;
        ok = wait_all(bar_full(s), (at / C::RING) & 1, kErrMma);
        if (ok && j == 0) ok = wait_all(BAR_Q, n & 1, kErrMma);
        if (!ok) return;
        const int valid = x.len - j * kBM;
        if (valid < kBM) {
          uint8_t* kt = smem + (2 + s) * C::TILE;
          const int per = (kBM - valid) * 8;
          for (int i = lane; i < per * C::NKB; i += 32) {
            const int kb = i / per;
            *reinterpret_cast<uint4*>(kt + kb * kBM * 128 + (valid * 8 + i - kb * per) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (leader) {
          mma_rows<D>(tmem, sQ, sKV + s * C::TILE);
          mma_commit(BAR_S);
          if (j + 1 == x.tiles) mma_commit(BAR_QFREE);
        }
        __syncwarp();
      };
      auto issue_dp = [&](const Unit& x, int j, int at) {
        const int s = (at + 1) % C::RING;
        ok = wait_all(bar_full(s), ((at + 1) / C::RING) & 1, kErrMma);
        if (ok && j == 0) ok = wait_all(BAR_G, n & 1, kErrMma);
        if (!ok) return;
        tc_fence_after();
        if (leader) {
          mma_rows<D>(tmem + 128, sG, sKV + s * C::TILE);
          mma_commit(BAR_DP);
          mma_commit(bar_empty(s));
          if (j + 1 == x.tiles) mma_commit(BAR_GFREE);
        }
        __syncwarp();
      };
      if (have) {
        issue_s(w, 0, 0);
        if (ok) issue_dp(w, 0, 0);
        ++n;
      }
      while (have && ok) {
        int64_t un = u + gridDim.x;
        Unit wn;
        const bool more_units = next_unit(un, wn);
        for (int j = 0; j < w.tiles && ok; ++j, ++it) {
          const bool more = j + 1 < w.tiles;
          if (more || more_units) {
            const Unit& x = more ? w : wn;
            const int jn = more ? j + 1 : 0, at = ld + 2 * j + 2;
            ok = wait_all(BAR_SREAD, it & 1, kErrMma);
            if (!ok) break;
            issue_s(x, jn, at);
            if (ok) ok = wait_all(BAR_DPREAD, it & 1, kErrMma);
            if (!ok) break;
            issue_dp(x, jn, at);
            if (!ok) break;
            if (!more) ++n;
          }
          ok = wait_all(BAR_DS, it & 1, kErrMma);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const int s = (ld + 2 * j) % C::RING;
            const uint32_t ds = tmem + 384 + (it & 1) * 64;
            mma_cols<D>(tmem + 256, [&](int kk) { return ds + kk * 8; }, sKV + s * C::TILE, j > 0);
            mma_commit(bar_empty(s));
            if (!more) mma_commit(BAR_DQ);
          }
          __syncwarp();
        }
        ld += 2 * w.tiles;
        have = more_units;
        u = un;
        w = wn;
      }
      if (!ok && leader) {
        // let every MMA already issued finish before TMEM is released
        mma_commit(BAR_DRAIN);
        mbar_drain(BAR_DRAIN, 0, p.timeout_ns);
      }
      __syncwarp();
    }
  } else {
    regs_increase<kSoftmaxRegs>();
    const int half = warp / 4, quarter = warp % 4;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint64_t pol = l2_policy_evict_first();
    uint8_t* stage = staging + warp * (C::STAGING / 8);
    const float sl2 = p.scale_log2;
    int it = 0, n = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Unit w = unit_at(u);
      const int row0 = w.q0 + quarter * 32, row = row0 + lane;
      float neg_lse = -INFINITY, delta = 0.f;   // (rows past the end: P = 0)
      if (row < p.s_q) {
        const float* l = static_cast<const float*>(p.lse.data) + w.b * p.lse.s[0] + w.h * p.lse.s[1] + row * p.lse.s[2];
        const float* d = p.ws + (static_cast<int64_t>(w.b) * p.heads + w.h) * p.s_q + row;
        if (CPATTN_IN(p.lse.span, l, 4, p.err)) neg_lse = -*l * kLog2e;
        if (CPATTN_IN(p.ws_span, d, 4, p.err)) delta = *d;
      }
      for (int j = 0; j < w.tiles; ++j, ++it) {
        ok = wait_all(BAR_S, it & 1, kErrSoftmax);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64], g[64];
        tmem_ld_x64(lanes + half * 64, s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR_SREAD);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x0, x1;
          ffma2(x0, x1, u2f(s[2 * i]), u2f(s[2 * i + 1]), sl2, sl2, neg_lse, neg_lse);
          s[2 * i] = f2u(ex2_approx(x0));
          s[2 * i + 1] = f2u(ex2_approx(x1));
        }
        ok = wait_all(BAR_DP, it & 1, kErrSoftmax);
        if (!ok) break;
        tc_fence_after();
        tmem_ld_x64(lanes + 128 + half * 64, g);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR_DPREAD);
        const int valid = w.len - j * kBM - half * 64;   // of this thread's 64 columns
        uint32_t ds[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x0, x1;
          fadd2(x0, x1, u2f(g[2 * i]), u2f(g[2 * i + 1]), -delta, -delta);
          x0 *= u2f(s[2 * i]);
          x1 *= u2f(s[2 * i + 1]);
          if (valid < 64) {   // (the same for the whole warpgroup)
            x0 = 2 * i < valid ? x0 : 0.f;
            x1 = 2 * i + 1 < valid ? x1 : 0.f;
          }
          ds[i] = pack_bf16x2(x0, x1);
        }
        tmem_st_x32(lanes + 384 + (it & 1) * 64 + half * 32, ds);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR_DS);
      }
      if (!ok) break;
      uint32_t o[D / 2];
      if (w.tiles > 0) {
        ok = wait_all(BAR_DQ, n & 1, kErrSoftmax);
        if (!ok) break;
        ++n;
        tc_fence_after();
        if constexpr (D == 128)
          tmem_ld_x64(lanes + 256 + half * 64, o);
        else
          tmem_ld_x32(lanes + 256 + half * 32, o);
      } else {
#pragma unroll
        for (int i = 0; i < D / 2; ++i) o[i] = 0u;
      }
      store_rows<D / 2>(p, p.dq, stage, o, p.scale, w.b, w.h, row0, p.s_q, half * (D / 2), pol);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dk, dv
// One CTA: 128 keys of one key head, and one of p.splits parts of the query
// tiles of all its query heads.  With several parts the fp32 sums go to the
// workspace (after delta): [part][dk, dv][B * H_kv * S_kv][D].
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_g,
                     const __grid_constant__ CrossParams p, const int64_t partials) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sK = smem_addr(smem), sV = sK + C::TILE, sQ = sV + C::TILE;   // stage s: Q, dO at sQ + 2 s TILE
  uint8_t* stats = smem + (2 + 2 * C::STAGES) * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stats + C::STAGES * C::STATS);
  const uint32_t bar0 = smem_addr(bars);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto bar_stats = [&](int s) { return bar0 + 8u * (2 * C::STAGES + s); };
  auto bar_stats_empty = [&](int s) { return bar0 + 8u * (3 * C::STAGES + s); };
  const uint32_t B = bar0 + 8u * (4 * C::STAGES);
  const uint32_t BAR_KV = B, BAR_S = B + 8, BAR_DP = B + 16, BAR_SREAD = B + 24, BAR_DS = B + 32, BAR_DONE = B + 40,
                 BAR_DRAIN = B + 48;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::KV_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x % 32;
  const int k_tiles = ceil_div(p.s_kv, kBM), q_tiles = ceil_div(p.s_q, kBM);
  const int share = p.heads / p.kv_heads;
  int64_t u = blockIdx.x;
  const int k0 = static_cast<int>(u % k_tiles) * kBM;
  u /= k_tiles;
  const int part = static_cast<int>(u % p.splits);
  u /= p.splits;
  const int hk = static_cast<int>(u % p.kv_heads), b = static_cast<int>(u / p.kv_heads);
  const int len = cross_length(p, b);
  const int all = share * q_tiles, per = ceil_div(all, p.splits);
  const int first = min(part * per, all), steps = k0 < len ? min(per, all - first) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
      mbar_init(bar_stats(s), 1);
      mbar_init(bar_stats_empty(s), 8);
    }
    for (uint32_t x : {BAR_KV, BAR_S, BAR_DP, BAR_DONE, BAR_DRAIN}) mbar_init(x, 1);
    for (uint32_t x : {BAR_SREAD, BAR_DS}) mbar_init(x, 8);   // one arrival per elementwise warp
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_holder), 512);
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_g);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait_all = [&](uint32_t bar, uint32_t parity, unsigned code) {
    const bool r = mbar_wait(bar, parity, abort_flag, p.timeout_ns, p.err, code);
    return __all_sync(0xffffffffu, r) != 0;
  };

  if (warp >= 8) {
    regs_decrease<kControlRegs>();
    const bool leader = elect_one();
    if (warp == kWarpProducer) {
      const uint64_t pol = l2_policy_evict_last();   // every tile is read again by another CTA
      bool ok = p.fault_skip_kv == 0;
      int t = 0;
      if (ok && steps > 0 && leader) {
        mbar_arrive_expect_tx(BAR_KV, 2 * C::TILE);
        load_tile<D>(sK, &tm_k, BAR_KV, k0, hk, b, pol);
        load_tile<D>(sV, &tm_v, BAR_KV, k0, hk, b, pol);
      }
      __syncwarp();
      for (; t < steps && ok; ++t) {
        const int s = t % C::STAGES, x = first + t;
        ok = wait_all(bar_empty(s), ((t / C::STAGES) & 1) ^ 1, kErrProducer);
        if (!ok) break;
        if (leader) {
          const int h = hk * share + x / q_tiles, q0 = (x % q_tiles) * kBM;
          mbar_arrive_expect_tx(bar_full(s), 2 * C::TILE);
          load_tile<D>(sQ + 2 * s * C::TILE, &tm_q, bar_full(s), q0, h, b, pol);
          load_tile<D>(sQ + (2 * s + 1) * C::TILE, &tm_g, bar_full(s), q0, h, b, pol);
        }
        __syncwarp();
      }
      if (!ok && leader && t > 0) {
        // leave no copy in flight into this CTA's shared memory
        mbar_drain(BAR_KV, 0, p.timeout_ns);
        for (int x = t > C::STAGES ? t - C::STAGES : 0; x < t; ++x)
          mbar_drain(bar_full(x % C::STAGES), (x / C::STAGES) & 1, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      bool ok = true;
      auto full = [&](int t) { return wait_all(bar_full(t % C::STAGES), (t / C::STAGES) & 1, kErrMma); };
      auto q_of = [&](int t) { return sQ + 2 * (t % C::STAGES) * C::TILE; };
      if (steps > 0) {
        ok = wait_all(BAR_KV, 0, kErrMma) && full(0);
        if (ok) {
          tc_fence_after();
          if (leader) {
            mma_rows<D>(tmem, sK, q_of(0));
            mma_commit(BAR_S);
            mma_rows<D>(tmem + 128, sV, q_of(0) + C::TILE);
            mma_commit(BAR_DP);
          }
          __syncwarp();
        }
      }
      for (int t = 0; t < steps && ok; ++t) {
        const bool more = t + 1 < steps;
        if (more) {
          ok = full(t + 1) && wait_all(BAR_SREAD, t & 1, kErrMma);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            mma_rows<D>(tmem, sK, q_of(t + 1));
            mma_commit(BAR_S);
          }
          __syncwarp();
        }
        ok = wait_all(BAR_DS, t & 1, kErrMma);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          // 64 of the 128 query columns per warpgroup: P^T in the first half
          // of its dP^T columns, dS^T in the second
          const uint32_t pt = tmem + 128;
          mma_cols<D>(tmem + 256, [&](int kk) { return pt + (kk / 4) * 64 + (kk % 4) * 8; }, q_of(t) + C::TILE, t > 0);
          mma_cols<D>(tmem + 256 + D, [&](int kk) { return pt + (kk / 4) * 64 + 32 + (kk % 4) * 8; }, q_of(t), t > 0);
          mma_commit(bar_empty(t % C::STAGES));
          if (more) {
            mma_rows<D>(tmem + 128, sV, q_of(t + 1) + C::TILE);
            mma_commit(BAR_DP);
          } else {
            mma_commit(BAR_DONE);
          }
        }
        __syncwarp();
      }
      if (!ok && leader) {
        // let every MMA already issued finish before TMEM is released
        mma_commit(BAR_DRAIN);
        mbar_drain(BAR_DRAIN, 0, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpStats) {
      bool ok = true;
      for (int t = 0; t < steps && ok; ++t) {
        const int s = t % C::STAGES, x = first + t;
        const int h = hk * share + x / q_tiles, q0 = (x % q_tiles) * kBM;
        float nl[4], dl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = q0 + i * 32 + lane;
          nl[i] = -INFINITY;   // (rows past the end: P = 0)
          dl[i] = 0.f;
          if (row < p.s_q) {
            const float* l = static_cast<const float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + row * p.lse.s[2];
            const float* d = p.ws + (static_cast<int64_t>(b) * p.heads + h) * p.s_q + row;
            if (CPATTN_IN(p.lse.span, l, 4, p.err)) nl[i] = -*l * kLog2e;
            if (CPATTN_IN(p.ws_span, d, 4, p.err)) dl[i] = -*d;
          }
        }
        ok = wait_all(bar_stats_empty(s), ((t / C::STAGES) & 1) ^ 1, kErrStats);
        if (!ok) break;
        float* st = reinterpret_cast<float*>(stats + s * C::STATS);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st[i * 32 + lane] = nl[i];
          st[kBM + i * 32 + lane] = dl[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_stats(s));
      }
      __syncwarp();
    }
  } else {
    regs_increase<kSoftmaxRegs>();
    const int half = warp / 4, quarter = warp % 4;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sl2 = p.scale_log2;
    const int key = k0 + quarter * 32 + lane;
    const bool ragged = k0 + kBM > len, live = key < len;
    bool ok = true;
    for (int t = 0; t < steps; ++t) {
      const int st = t % C::STAGES;
      const float4* nl = reinterpret_cast<const float4*>(stats + st * C::STATS) + half * 16;
      const float4* dl = nl + kBM / 4;
      ok = wait_all(BAR_S, t & 1, kErrSoftmax);
      if (ok) ok = wait_all(bar_stats(st), (t / C::STAGES) & 1, kErrSoftmax);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[64], g[64];
      tmem_ld_x64(lanes + half * 64, s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR_SREAD);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 m = nl[i];
        float x[4];
        ffma2(x[0], x[1], u2f(s[4 * i]), u2f(s[4 * i + 1]), sl2, sl2, m.x, m.y);
        ffma2(x[2], x[3], u2f(s[4 * i + 2]), u2f(s[4 * i + 3]), sl2, sl2, m.z, m.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * i + e] = f2u(ex2_approx(x[e]));
      }
      ok = wait_all(BAR_DP, t & 1, kErrSoftmax);
      if (!ok) break;
      tc_fence_after();
      tmem_ld_x64(lanes + 128 + half * 64, g);
      uint32_t pb[32], db[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 d = dl[i];
        float x[4];
        fadd2(x[0], x[1], u2f(g[4 * i]), u2f(g[4 * i + 1]), d.x, d.y);
        fadd2(x[2], x[3], u2f(g[4 * i + 2]), u2f(g[4 * i + 3]), d.z, d.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= u2f(s[4 * i + e]);
        pb[2 * i] = pack_bf16x2(u2f(s[4 * i]), u2f(s[4 * i + 1]));
        pb[2 * i + 1] = pack_bf16x2(u2f(s[4 * i + 2]), u2f(s[4 * i + 3]));
        db[2 * i] = pack_bf16x2(x[0], x[1]);
        db[2 * i + 1] = pack_bf16x2(x[2], x[3]);
      }
      if (ragged && !live) {
        // a key past the length (its k and v may hold anything): no weight
#pragma unroll
        for (int i = 0; i < 32; ++i) pb[i] = db[i] = 0u;
      }
      tmem_st_x32(lanes + 128 + half * 64, pb);
      tmem_st_x32(lanes + 128 + half * 64 + 32, db);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(BAR_DS);
        mbar_arrive(bar_stats_empty(st));
      }
    }
    if (ok && steps > 0) {
      ok = wait_all(BAR_DONE, 0, kErrSoftmax);
      if (ok) tc_fence_after();
    }
    if (ok) {
      // warpgroup 0 writes dv, warpgroup 1 dk; the Q and dO stages are idle
      const CrossTensor& t = half ? p.dk : p.dv;
      const float f = half ? p.scale : 1.f;
      const bool zero = steps == 0 || !live;
      const int64_t rows = static_cast<int64_t>(p.batch) * p.kv_heads * p.s_kv;
      float* ws = p.ws + partials + (2 * part + (half ? 0 : 1)) * rows * D +
                  ((static_cast<int64_t>(b) * p.kv_heads + hk) * p.s_kv + key) * D;
      const uint64_t pol = l2_policy_evict_first();
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t o[64];
        __syncwarp();
        if (steps > 0) tmem_ld_x64(lanes + 256 + half * D + c0, o);
#pragma unroll
        for (int i = 0; i < 64; ++i) o[i] = zero ? 0u : o[i];
        if (p.splits > 1) {
          if (key < p.s_kv) {
            float4* dst = reinterpret_cast<float4*>(ws + c0);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (CPATTN_IN(p.ws_span, dst + i, 16, p.err))
                dst[i] = make_float4(u2f(o[4 * i]), u2f(o[4 * i + 1]), u2f(o[4 * i + 2]), u2f(o[4 * i + 3]));
          }
        } else {
          store_rows<64>(p, t, smem + 2 * C::TILE + warp * 4096, o, f, b, hk, k0 + quarter * 32, p.s_kv, c0, pol);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sums the parts of dk and dv in their order: one thread per four values.
template <int D>
__global__ void __launch_bounds__(256) cross_dkv_join_kernel(const __grid_constant__ CrossParams p, const int64_t partials) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.kv_heads * p.s_kv, n = rows * (D / 4);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
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
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(t.data) + b * t.s[0] + h * t.s[1] + key * t.s[2] + (at % (D / 4)) * 4;
  if (CPATTN_IN(t.span, dst, 8, p.err))
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
}

// Once per device and kernel: the register split needs exactly kLaunchRegs at
// launch (refused otherwise), and the shared-memory limit is raised.
template <typename K>
cudaError_t set_up(K kernel, int smem, std::atomic<unsigned long long>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit != 0 && (ready.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
  if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  ready.fetch_or(bit, std::memory_order_acq_rel);
  return cudaSuccess;
}

template <int D>
cudaError_t launch_typed(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                         const CUtensorMap& tm_g, const CrossParams& p, int64_t partials, cudaStream_t stream) {
  using C = Cfg<D>;
  static std::atomic<unsigned long long> ready_q{0}, ready_kv{0};
  cudaError_t e = set_up(cross_dq_kernel<D>, C::DQ_SMEM, ready_q);
  if (e == cudaSuccess) e = set_up(cross_dkv_kernel<D>, C::KV_SMEM, ready_kv);
  if (e != cudaSuccess) return e;
  const int64_t sms = sm_count();
  const int64_t units = static_cast<int64_t>(p.batch) * p.heads * ((p.s_q + kBM - 1) / kBM);
  cross_dq_kernel<D><<<static_cast<unsigned>(units < sms ? units : sms), kThreads, C::DQ_SMEM, stream>>>(
      tm_q, tm_k, tm_v, tm_g, p, units);
  const int64_t ctas = static_cast<int64_t>(p.batch) * p.kv_heads * p.splits * ((p.s_kv + kBM - 1) / kBM);
  const int64_t rows = static_cast<int64_t>(p.batch) * p.kv_heads * p.s_kv, join = (2 * rows * (D / 4) + 255) / 256;
  if (ctas > 0x7fffffff || join > 0x7fffffff) return cudaErrorInvalidValue;
  cross_dkv_kernel<D><<<static_cast<unsigned>(ctas), kThreads, C::KV_SMEM, stream>>>(tm_q, tm_k, tm_v, tm_g, p,
                                                                                       partials);
  if (p.splits > 1) cross_dkv_join_kernel<D><<<static_cast<unsigned>(join), 256, 0, stream>>>(p, partials);
  return cudaGetLastError();
}

}  // namespace

int cross_backward_parts(int64_t key_units, int64_t steps) {
  // The parts share the GPU as whole CTAs, one per SM at a time: the fewest
  // query-tile steps over all waves, a CTA's start and end counting as three
  // steps and a part's share of the join as half a step.
  const int64_t sms = sm_count();
  int best = 1;
  double least = 0;
  for (int parts = 1; parts <= 32 && parts <= steps; ++parts) {
    const double waves = static_cast<double>((key_units * parts + sms - 1) / sms);
    const double cost = waves * ((steps + parts - 1) / parts + 3) + (parts > 1 ? 2 + 0.5 * parts : 0);
    if (parts == 1 || cost < least) {
      best = parts;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_cross_bwd(int head_dim, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             const CUtensorMap& tm_g, const CrossParams& p, int64_t partials, cudaStream_t stream) {
  return head_dim == 64 ? launch_typed<64>(tm_q, tm_k, tm_v, tm_g, p, partials, stream)
                        : launch_typed<128>(tm_q, tm_k, tm_v, tm_g, p, partials, stream);
}

}  // namespace cpattn
