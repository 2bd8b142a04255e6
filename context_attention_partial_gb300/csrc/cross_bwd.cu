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
// MMA issuer; warp 10 row statistics (dk, dv kernel).  The dq kernel forms
// delta, and writes it to the workspace for the other: each thread from its
// half row of dO in shared memory and of O, requested a unit ahead.  (By two
// warps of their own, 64 rows each, it took 17,500 cycles a unit: beside the
// elementwise warps they get few issue slots.)
// TMEM columns, dq:     S 0 | dP 128 | dQ 256 | dS 384, 448 (two buffers)
//               dk, dv: S^T 0 | dP^T 128, then P^T and dS^T over it | dV, dK 256..
// The next step's S is issued as soon as this step's S is in registers, so the
// exponentials run under dQ (or dV and dK) and the products under the
// elementwise work.
// Measured: 4608 queries x 512 keys x 24 heads, D = 128: dq 43 us, dk and dv 53 us;
// steps of 2000 and 2650 cycles against 1536 and 2048 of MMAs, near what shared
// memory gives (224 and 256 KB a step, and the statistics).
// Shared memory holds seven 32 KB tiles at D = 128.  dq: Q, dO, three K and two
// V tiles -- K_t is held until dQ_t, while S_{t+1} already needs K_{t+1}, so
// two K tiles would expose every load (3710 cycles a step); a unit's output
// leaves through its last K tile.  dk, dv: K, V, and five Q / dO tiles in turn
// (two whole pairs exposed 960 of 3400 cycles a step).
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "cross_ops.cuh"

namespace cpattn {
namespace {

constexpr int kBM = 128;            // rows of every tile
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpStats = 10;
constexpr int kLaunchRegs = 168;    // 65536 / 384, rounded down to 8
constexpr int kSoftmaxRegs = 208, kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr unsigned kErrProducer = 1u, kErrMma = 2u, kErrSoftmax = 4u, kErrStats = 8u;

template <int D>
struct Cfg {
  static constexpr int ROW = D * 2;                    // bytes
  static constexpr int TILE = kBM * ROW;
  static constexpr int QK = ROW / 32, PV = kBM / 16;   // MMAs over D, over a tile's rows
  static constexpr uint32_t IDESC_S = make_idesc(1, false, kBM, kBM);
  static constexpr uint32_t IDESC_G = make_idesc(1, true, kBM, D);
  static constexpr int STATS = 2 * kBM * 4;            // -lse log2e and delta of 128 rows
  // dq kernel: Q, dO of a unit, rings of K and of V tiles, halves of delta
  static constexpr int KR = D == 128 ? 3 : 5, VR = D == 128 ? 2 : 4;
  static constexpr int DQ_BARS = 2 * KR + 2 * VR + 13;
  static constexpr int DQ_SMEM = (2 + KR + VR) * TILE + STATS + DQ_BARS * 8 + 16;
  // dk, dv kernel: K, V tiles, a ring of Q and dO tiles, statistics of two steps
  static constexpr int RING = D == 128 ? 5 : 9;
  static constexpr int KV_BARS = 2 * RING + 12;
  static constexpr int KV_SMEM = (2 + RING) * TILE + 2 * STATS + KV_BARS * 8 + 16;
  static constexpr int PART_ROW = D * 4 + 16;          // staged fp32 row, padded against bank conflicts
  static_assert(DQ_SMEM <= 227 * 1024 && KV_SMEM <= 227 * 1024, "shared memory");
  static_assert(8 * 32 * PART_ROW <= RING * TILE && 8 * 4096 * (D / 64) <= RING * TILE, "staging");
};

// A place in a ring of N tiles and the parity of its use, stepped without
// divisions: the MMA warp gets an issue slot every eight cycles or so beside
// the elementwise warps, and its instructions between two groups of MMAs are
// time the tensor pipe waits.
template <int N>
struct Place {
  uint32_t i = 0, ph = 0;
  __device__ void next() {
    if (++i == N) {
      i = 0;
      ph ^= 1u;
    }
  }
};

// Sum of eight products of bf16 values, each added in fp32 with one rounding.
__device__ __forceinline__ float dot_bf16x8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float d = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
        "fma.rn.f32.bf16 %0, al, bl, %0;\n\tfma.rn.f32.bf16 %0, ah, bh, %0;\n\t}"
        : "+f"(d)
        : "r"(x[i]), "r"(y[i]));
  return d;
}

// Low descriptor words of a tile's k-steps: over its columns (the tile's rows
// times another's), and over its rows (a TMEM operand times the tile).  The
// high words are one constant; they are built before a group's waits.
constexpr uint64_t kRowsDesc = (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
constexpr uint64_t kColsDesc = (uint64_t((kBM * 128) >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
                               (uint64_t(2) << 61);
constexpr uint32_t kDescHi = static_cast<uint32_t>(kRowsDesc >> 32);
static_assert(kDescHi == static_cast<uint32_t>(kColsDesc >> 32), "one high word");

template <int N>
__device__ __forceinline__ void rows_desc(uint32_t (&d)[N], uint32_t addr) {
#pragma unroll
  for (int kk = 0; kk < N; ++kk)
    d[kk] = static_cast<uint32_t>(kRowsDesc) + (addr >> 4) + (((kk / 4) * (kBM * 128) + (kk % 4) * 32) >> 4);
}
template <int N>
__device__ __forceinline__ void cols_desc(uint32_t (&d)[N], uint32_t addr) {
#pragma unroll
  for (int kk = 0; kk < N; ++kk) d[kk] = static_cast<uint32_t>(kColsDesc) + ((addr + kk * 16 * 128) >> 4);
}

// ------------------------------------------------------------------ dq
struct DqUnit {
  int b, h, q0, len, tiles;
};

// Walks this CTA's units, blockIdx.x, blockIdx.x + gridDim.x, ..., query tile
// fastest, then head and batch; the grid's size is added digit by digit.
struct DqWalk {
  int q, h, b, dq, dh, db, q_tiles;
  __device__ explicit DqWalk(const CrossParams& p) {
    q_tiles = ceil_div(p.s_q, kBM);
    auto split = [&](uint32_t u, int& q_, int& h_, int& b_) {
      const uint32_t r = u / q_tiles;
      q_ = static_cast<int>(u - r * q_tiles);
      b_ = static_cast<int>(r / p.heads);
      h_ = static_cast<int>(r - b_ * p.heads);
    };
    split(blockIdx.x, q, h, b);
    split(gridDim.x, dq, dh, db);
    for (int* x : {&q, &h, &b, &dq, &dh, &db}) *x = uniform(*x);
  }
  __device__ bool more(const CrossParams& p) const { return b < p.batch; }
  __device__ void step(const CrossParams& p) {
    q += dq;
    h += dh;
    b += db;
    if (q >= q_tiles) {
      q -= q_tiles;
      ++h;
    }
    if (h >= p.heads) {
      h -= p.heads;
      ++b;
    }
  }
  __device__ DqUnit unit(const CrossParams& p) const {
    // (one key has all the weight whatever q is: dq is 0, as without keys)
    const int len = uniform(cross_length(p, b));
    return {b, h, q * kBM, len, len > 1 ? ceil_div(len, kBM) : 0};
  }
  // Moves to the first unit with keys at or after this one.
  __device__ bool with_keys(const CrossParams& p, DqUnit& w) {
    for (; more(p); step(p)) {
      w = unit(p);
      if (w.tiles > 0) return true;
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_g,
                    const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ CrossParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!tiles_aligned(p, smem)) return;
  const uint32_t sQ = smem_addr(smem), sG = sQ + C::TILE, sK = sG + C::TILE, sV = sK + C::KR * C::TILE;
  float* halves = reinterpret_cast<float*>(smem + (2 + C::KR + C::VR) * C::TILE);   // [2][128] of delta
  uint64_t* bars = reinterpret_cast<uint64_t*>(halves + C::STATS / 4);
  const uint32_t bar0 = smem_addr(bars);
  auto k_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto k_empty = [&](uint32_t s) { return bar0 + 8u * (C::KR + s); };
  auto v_full = [&](uint32_t s) { return bar0 + 8u * (2 * C::KR + s); };
  auto v_empty = [&](uint32_t s) { return bar0 + 8u * (2 * C::KR + C::VR + s); };
  const uint32_t B = bar0 + 8u * (2 * C::KR + 2 * C::VR);
  const uint32_t BAR_Q = B, BAR_G = B + 8, BAR_QFREE = B + 16, BAR_GFREE = B + 24, BAR_S = B + 32, BAR_DP = B + 40,
                 BAR_SREAD = B + 48, BAR_DPREAD = B + 56, BAR_DS = B + 64, BAR_DQ = B + 72, BAR_DRAIN = B + 80;
  const uint32_t BAR_OUT = B + 88, BAR_DELTA = B + 96;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::DQ_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::KR; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < C::VR; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    for (uint32_t x : {BAR_Q, BAR_G, BAR_QFREE, BAR_S, BAR_DP, BAR_DQ, BAR_DRAIN}) mbar_init(x, 1);
    mbar_init(BAR_GFREE, 2);   // the last product with dO, and delta formed
    for (uint32_t x : {BAR_SREAD, BAR_DPREAD, BAR_DS, BAR_OUT, BAR_DELTA}) mbar_init(x, 8);   // one arrival per elementwise warp
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_holder), 512);
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_g);
    tma_prefetch_desc(&tm_dq);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpProducer) {
    // the first unit's tiles, while the kernel before this one ends (the whole
    // gradient at 4608 x 512 x 24 heads 96.0 us without, 93.6 with)
    const DqWalk first(p);
    if (first.more(p) && lane == 0) {
      const int hk = first.h / (p.heads / p.kv_heads);
      prefetch_tile<D>(&tm_q, first.q * kBM, first.h, first.b);
      prefetch_tile<D>(&tm_k, 0, hk, first.b);
      prefetch_tile<D>(&tm_g, first.q * kBM, first.h, first.b);
      prefetch_tile<D>(&tm_v, 0, hk, first.b);
      prefetch_tile<D>(&tm_o, first.q * kBM, first.h, first.b);
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
      const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
      uint32_t ld = 0, nq = 0, ng = 0;   // K tiles (and V tiles) requested, Q and dO tiles
      uint32_t nv = 0;
      bool ok = p.fault_skip_kv == 0;
      DqWalk walk(p), ahead(p);
      DqUnit w, wa;
      // the next unit's Q, dO and O into L2
      auto prefetch = [&]() {
        if (ahead.with_keys(p, wa) && leader) {
          prefetch_tile<D>(&tm_g, wa.q0, wa.h, wa.b);
          prefetch_tile<D>(&tm_o, wa.q0, wa.h, wa.b);
          prefetch_tile<D>(&tm_q, wa.q0, wa.h, wa.b);
        }
        __syncwarp();
        ahead.step(p);
      };
      if (ok) prefetch();
      while (ok && walk.with_keys(p, w)) {
        const int hk = w.h / (p.heads / p.kv_heads);
        prefetch();
        for (int j = 0; j < w.tiles && ok; ++j) {
          ok = wait_all(k_empty(ld % C::KR), ((ld / C::KR) & 1) ^ 1, kErrProducer);
          if (!ok) break;
          if (leader) {
            mbar_arrive_expect_tx(k_full(ld % C::KR), C::TILE);
            load_tile<D>(sK + (ld % C::KR) * C::TILE, &tm_k, k_full(ld % C::KR), j * kBM, hk, w.b, pol_kv);
          }
          __syncwarp();
          ++ld;
          if (j == 0) {
            ok = wait_all(BAR_QFREE, (nq & 1) ^ 1, kErrProducer);
            if (!ok) break;
            if (leader) {
              mbar_arrive_expect_tx(BAR_Q, C::TILE);
              load_tile<D>(sQ, &tm_q, BAR_Q, w.q0, w.h, w.b, pol_q);
            }
            __syncwarp();
            ++nq;
          }
          ok = wait_all(v_empty(nv % C::VR), ((nv / C::VR) & 1) ^ 1, kErrProducer);
          if (!ok) break;
          if (leader) {
            mbar_arrive_expect_tx(v_full(nv % C::VR), C::TILE);
            load_tile<D>(sV + (nv % C::VR) * C::TILE, &tm_v, v_full(nv % C::VR), j * kBM, hk, w.b, pol_kv);
          }
          __syncwarp();
          ++nv;
          if (j == 0) {
            ok = wait_all(BAR_GFREE, (ng & 1) ^ 1, kErrProducer);
            if (!ok) break;
            if (leader) {
              mbar_arrive_expect_tx(BAR_G, C::TILE);
              load_tile<D>(sG, &tm_g, BAR_G, w.q0, w.h, w.b, pol_q);
            }
            __syncwarp();
            ++ng;
          }
        }
        walk.step(p);
      }
      if (!ok && leader) {
        // leave no copy in flight into this CTA's shared memory
        for (uint32_t x = ld > C::KR ? ld - C::KR : 0; x < ld; ++x)
          mbar_drain(k_full(x % C::KR), (x / C::KR) & 1, p.timeout_ns);
        for (uint32_t x = nv > C::VR ? nv - C::VR : 0; x < nv; ++x)
          mbar_drain(v_full(x % C::VR), (x / C::VR) & 1, p.timeout_ns);
        if (nq > 0) mbar_drain(BAR_Q, (nq - 1) & 1, p.timeout_ns);
        if (ng > 0) mbar_drain(BAR_G, (ng - 1) & 1, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      uint32_t n = 0, it = 0;              // units and steps so far
      Place<C::KR> kc, kn;                 // K tile of this step, and of the next S
      Place<C::VR> vn;                     // V tile of the next dP
      bool ok = true;
      DqWalk walk(p);
      DqUnit w;
      bool have = walk.with_keys(p, w);
      uint32_t qa[C::QK], ga[C::QK];
      rows_desc(qa, sQ);
      rows_desc(ga, sG);
      auto ready = [&](bool now, uint32_t bar, uint32_t parity) {   // after a test of the same phase
        return __all_sync(0xffffffffu, now) || wait_all(bar, parity, kErrMma);
      };
      // S and dP of a unit's key tile j; `read`: wait for the warps to have
      // read the ones before
      auto issue_s = [&](const DqUnit& x, int j, bool read) {
        const bool k_now = mbar_test(k_full(kn.i), kn.ph), r_now = read && mbar_test(BAR_SREAD, it & 1);
        uint32_t kb[C::QK];
        rows_desc(kb, sK + kn.i * C::TILE);
        ok = ready(k_now, k_full(kn.i), kn.ph);
        if (ok && j == 0) ok = wait_all(BAR_Q, n & 1, kErrMma);
        const int valid = x.len - j * kBM;
        if (ok && valid < kBM)
          zero_tile_rows<D>(smem + (2 + kn.i) * C::TILE, valid);   // (dS is 0 there, and 0 * NaN is not)
        if (ok && read) ok = ready(r_now, BAR_SREAD, it & 1);
        if (!ok) return;
        tc_fence_after();
        if (leader) {
          mma_group<C::QK, true>(tmem, qa, kb, kDescHi, C::IDESC_S, 0u);
          mma_commit(BAR_S);
          if (j + 1 == x.tiles) mma_commit(BAR_QFREE);
        }
        __syncwarp();
        kn.next();
      };
      auto issue_dp = [&](const DqUnit& x, int j, bool read) {
        const bool v_now = mbar_test(v_full(vn.i), vn.ph), r_now = read && mbar_test(BAR_DPREAD, it & 1);
        uint32_t vb[C::QK];
        rows_desc(vb, sV + vn.i * C::TILE);
        ok = ready(v_now, v_full(vn.i), vn.ph);
        if (ok && j == 0) ok = wait_all(BAR_G, n & 1, kErrMma);
        if (ok && read) ok = ready(r_now, BAR_DPREAD, it & 1);
        if (!ok) return;
        tc_fence_after();
        if (leader) {
          mma_group<C::QK, true>(tmem + 128, ga, vb, kDescHi, C::IDESC_S, 0u);
          mma_commit(BAR_DP);
          mma_commit(v_empty(vn.i));
          if (j + 1 == x.tiles) mma_commit(BAR_GFREE);
        }
        __syncwarp();
        vn.next();
      };
      auto issue_dq = [&](int j, bool last) {
        const bool now = mbar_test(BAR_DS, it & 1);
        uint32_t da[C::PV], kb[C::PV];
        cols_desc(kb, sK + kc.i * C::TILE);
#pragma unroll
        for (int kk = 0; kk < C::PV; ++kk) da[kk] = tmem + 384 + (it & 1) * 64 + kk * 8;
        ok = ready(now, BAR_DS, it & 1);
        if (!ok) return;
        tc_fence_after();
        if (leader) {
          mma_group<C::PV, false>(tmem + 256, da, kb, kDescHi, C::IDESC_G, j > 0);
          // (a unit's last K tile is given back once its output has left through it)
          mma_commit(last ? BAR_DQ : k_empty(kc.i));
        }
        __syncwarp();
        kc.next();
      };
      if (have) {
        issue_s(w, 0, false);
        if (ok) issue_dp(w, 0, false);
        ++n;
      }
      while (have && ok) {
        DqUnit wn;
        walk.step(p);
        const bool more_units = walk.with_keys(p, wn);
        for (int j = 0; j + 1 < w.tiles && ok; ++j, ++it) {
          issue_s(w, j + 1, true);
          if (ok) issue_dp(w, j + 1, true);
          if (ok) issue_dq(j, false);
        }
        if (!ok) break;
        // (the unit's last product before the next unit's first: its tiles may
        // still be on their way)
        issue_dq(w.tiles - 1, true);
        ++it;
        if (ok && more_units) {
          issue_s(wn, 0, false);
          if (ok) issue_dp(wn, 0, false);
          ++n;
        }
        have = more_units;
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
    const float sl2 = p.scale_log2;
    // delta's dot products: LPR lanes read a half row's 16-byte chunks, so a
    // load touches whole 128-byte lines
    constexpr int CH = D / 16, LPR = CH, RPI = 32 / LPR;   // CH loads cover the warp's 32 rows
    const int r = quarter * 32 + lane, r_in = quarter * 32 + lane / LPR, c_in = lane % LPR;
    const uint8_t* g_tile = smem + C::TILE + (D == 128 ? half * (kBM * 128) : 0);
    constexpr int kChunk0 = D == 128 ? 0 : CH;   // first chunk of the second half in its 128 bytes
    uint4 ox[CH];
    float lse = INFINITY;
    auto fetch = [&](const DqUnit& x) {
      if (x.tiles == 0) return;
      lse = INFINITY;   // (rows past the end: P = 0)
      const float* l = static_cast<const float*>(p.lse.data) + x.b * p.lse.s[0] + x.h * p.lse.s[1] + (x.q0 + r) * p.lse.s[2];
      if (x.q0 + r < p.s_q && CPATTN_IN(p.lse.span, l, 4, p.err)) lse = *l;   // (not used before the unit begins: no wait here)
      const uint4* o = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.out.data) + x.b * p.out.s[0] +
                                                      x.h * p.out.s[1] + half * (D / 2)) + c_in;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int64_t row = x.q0 + r_in + i * RPI;
        const uint4* at = o + row * (p.out.s[2] / 8);
        ox[i] = make_uint4(0, 0, 0, 0);
        if (row < p.s_q && CPATTN_IN(p.out.span, at, 16, p.err)) ox[i] = __ldcs(at);
      }
    };
    uint32_t it = 0, n = 0, slot = 0;
    // A unit's output leaves through its last K tile (n - 1: the unit before);
    // the tile is given back once all eight warps' rows have left it, looked
    // at when the next unit's first scores are done, not waited for.
    auto give_back = [&]() {
      if (lane == 0) {
        bulk_wait_read();
        mbar_arrive(BAR_OUT);
      }
      __syncwarp();
      bool done = true;
      if (warp == 0) {
        done = wait_all(BAR_OUT, (n - 1) & 1, kErrSoftmax);
        if (lane == 0) mbar_arrive(k_empty(slot));
      }
      return done;
    };
    bool ok = true;
    DqWalk walk(p);
    DqUnit wn = walk.unit(p);   // (the grid has no more CTAs than units)
    fetch(wn);
    while (ok && walk.more(p)) {
      const DqUnit w = wn;
      const float nl = -cross_lse2(lse);
      float neg_delta = 0.f;
      walk.step(p);
      const bool more = walk.more(p);
      if (more) wn = walk.unit(p);
      const int row0 = w.q0 + quarter * 32;
      if (w.tiles == 0) {
        // a sequence without keys, or with one: dq is 0
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.dq.data) + w.b * p.dq.s[0] + w.h * p.dq.s[1] +
                             static_cast<int64_t>(row0 + lane) * p.dq.s[2] + half * (D / 2);
        for (int i = 0; i < D / 16; ++i)
          if (row0 + lane < p.s_q && CPATTN_IN(p.dq.span, dst + 8 * i, 16, p.err))
            *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(0, 0, 0, 0);
        if (more) fetch(wn);
        continue;
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
          ffma2(x0, x1, u2f(s[2 * i]), u2f(s[2 * i + 1]), sl2, sl2, nl, nl);
          s[2 * i] = f2u(ex2_approx(x0));
          s[2 * i + 1] = f2u(ex2_approx(x1));
        }
        if (j == 0) {
          // delta of the unit's rows
          ok = (n == 0 || give_back()) && wait_all(BAR_G, n & 1, kErrSoftmax);
          if (!ok) break;
          float e[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int row = r_in + i * RPI;
            const uint4 gx = *reinterpret_cast<const uint4*>(g_tile + row * 128 + (((half * kChunk0 + c_in) ^ (row & 7)) << 4));
            e[i] = dot_bf16x8(ox[i], gx);
          }
          // LPR rows' sums over LPR lanes, each lane left with one row's
          // (LPR - 1 shuffles; one sum after the other took 1800 cycles)
#pragma unroll
          for (int x = LPR / 2; x > 0; x >>= 1) {
            const bool up = (c_in & x) != 0;
#pragma unroll
            for (int i = 0; i < x; ++i) {
              const float give = up ? e[i] : e[i + x];
              e[i] = (up ? e[i + x] : e[i]) + __shfl_xor_sync(0xffffffffu, give, x);
            }
          }
          halves[half * kBM + r_in + c_in * RPI] = e[0];
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR_DELTA);
          ok = wait_all(BAR_DELTA, n & 1, kErrSoftmax);
          if (!ok) break;
          const float d = halves[r] + halves[kBM + r];
          neg_delta = -d;
          if (threadIdx.x == 0) mbar_arrive(BAR_GFREE);
          float* dst = p.ws + (static_cast<int64_t>(w.b) * p.heads + w.h) * p.s_q + w.q0 + r;
          if (half == 0 && w.q0 + r < p.s_q && CPATTN_IN(p.ws_span, dst, 4, p.err)) *dst = d;
        }
        ok = wait_all(BAR_DP, it & 1, kErrSoftmax);
        if (!ok) break;
        tc_fence_after();
        tmem_ld_x64(lanes + 128 + half * 64, g);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR_DPREAD);
        uint32_t ds[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x0, x1;
          fadd2(x0, x1, u2f(g[2 * i]), u2f(g[2 * i + 1]), neg_delta, neg_delta);
          fmul2(x0, x1, x0, x1, u2f(s[2 * i]), u2f(s[2 * i + 1]));
          ds[i] = pack_bf16x2(x0, x1);
        }
        const int valid = w.len - j * kBM - half * 64;   // of this thread's 64 columns
        if (valid < 64) {   // (the same for the whole warpgroup; what was computed there may be NaN)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            ds[i] = 2 * i + 1 < valid ? ds[i] : 2 * i < valid ? ds[i] & 0xFFFFu : 0u;
        }
        tmem_st_x32(lanes + 384 + (it & 1) * 64 + half * 32, ds);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR_DS);
      }
      if (!ok) break;
      if (more) fetch(wn);
      ok = wait_all(BAR_DQ, n & 1, kErrSoftmax);
      if (!ok) break;
      tc_fence_after();
      uint32_t o[D / 2];
      if constexpr (D == 128)
        tmem_ld_x64(lanes + 256 + half * 64, o);
      else
        tmem_ld_x32(lanes + 256 + half * 32, o);
      // (every product has read the unit's last K tile)
      slot = (it - 1) % C::KR;
      store_rows<D / 2>(p, p.dq, &tm_dq, smem + (2 + slot) * C::TILE + warp * (C::TILE / 8), o, p.scale, w.b, w.h, row0,
                        p.s_q, half * (D / 2));
      ++n;
    }
    if (lane == 0) bulk_wait_read();   // (before this CTA's shared memory is given up)
    __syncwarp();
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
                     const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                     const __grid_constant__ CrossParams p, const int64_t partials) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!tiles_aligned(p, smem)) return;
  const uint32_t sK = smem_addr(smem), sV = sK + C::TILE, sR = sV + C::TILE;
  uint8_t* ring = smem + 2 * C::TILE;
  float* stats = reinterpret_cast<float*>(ring + C::RING * C::TILE);   // [2][-lse log2e, -delta][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(stats + 2 * C::STATS / 4);
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](uint32_t x) { return bar0 + 8u * (x % C::RING); };
  auto empty = [&](uint32_t x) { return bar0 + 8u * (C::RING + x % C::RING); };
  auto phase = [&](uint32_t x) { return (x / C::RING) & 1u; };
  auto tile = [&](uint32_t x) { return sR + (x % C::RING) * C::TILE; };
  const uint32_t B = bar0 + 8u * (2 * C::RING);
  const uint32_t BAR_KV = B, BAR_S = B + 8, BAR_DP = B + 16, BAR_SREAD = B + 24, BAR_DS = B + 32, BAR_DONE = B + 40,
                 BAR_DRAIN = B + 48, BAR_DS2 = B + 56;
  auto st_full = [&](uint32_t s) { return B + 64 + 8u * s; };
  auto st_empty = [&](uint32_t s) { return B + 80 + 8u * s; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::KV_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x % 32;
  const uint32_t k_tiles = (p.s_kv + kBM - 1) / kBM, q_tiles = (p.s_q + kBM - 1) / kBM;
  const uint32_t share = uniform(p.heads / p.kv_heads);
  const uint32_t r = uniform(blockIdx.x / k_tiles), u = uniform(r / p.splits);
  const int k0 = static_cast<int>(blockIdx.x - r * k_tiles) * kBM;
  const uint32_t part = r - u * p.splits;
  const int b = uniform(static_cast<int>(u / p.kv_heads)), hk = static_cast<int>(u - b * p.kv_heads);
  const int len = uniform(cross_length(p, b));
  const uint32_t all = share * q_tiles, per = uniform((all + p.splits - 1) / p.splits);
  const uint32_t first = min(part * per, all), steps = k0 < len ? min(per, all - first) : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::RING; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (uint32_t x : {BAR_KV, BAR_S, BAR_DP, BAR_DONE, BAR_DRAIN}) mbar_init(x, 1);
    for (uint32_t x : {BAR_SREAD, BAR_DS, BAR_DS2}) mbar_init(x, 8);   // one arrival per elementwise warp
    for (int s = 0; s < 2; ++s) {
      mbar_init(st_full(s), 1);
      mbar_init(st_empty(s), 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_holder), 512);
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_g);
    tma_prefetch_desc(&tm_dk);
    tma_prefetch_desc(&tm_dv);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // The copies and the first S and dP may run under the dq kernel.  What follows
  // them needs its delta, and the limit of a wait must not count the time that
  // kernel still takes: every warp waits for its end (launch_wait) before its
  // first wait for something behind the statistics.
  auto wait_all = [&](uint32_t bar, uint32_t parity, unsigned code) {
    const bool ok = mbar_wait(bar, parity, abort_flag, p.timeout_ns, p.err, code);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  if (warp >= 8) {
    regs_decrease<kControlRegs>();
    const bool leader = elect_one();
    if (warp == kWarpProducer) {
      const uint64_t pol = l2_policy_evict_last();   // every tile is read again by another CTA
      bool ok = p.fault_skip_kv == 0;
      uint32_t x = 0;   // Q tile of step t is load 2t, its dO tile load 2t + 1
      if (ok && steps > 0 && leader) {
        mbar_arrive_expect_tx(BAR_KV, 2 * C::TILE);
        load_tile<D>(sK, &tm_k, BAR_KV, k0, hk, b, pol);
        load_tile<D>(sV, &tm_v, BAR_KV, k0, hk, b, pol);
      }
      __syncwarp();
      uint32_t g = uniform(first / q_tiles), qt = first - g * q_tiles;
      for (; x < 2 * steps && ok; ++x) {
        if (x == C::RING) launch_wait();
        ok = wait_all(empty(x), phase(x) ^ 1, kErrProducer);
        if (!ok) break;
        if (leader) {
          mbar_arrive_expect_tx(full(x), C::TILE);
          load_tile<D>(tile(x), x % 2 ? &tm_g : &tm_q, full(x), qt * kBM, hk * share + g, b, pol);
        }
        __syncwarp();
        if (x % 2 == 1 && ++qt == q_tiles) {
          qt = 0;
          ++g;
        }
      }
      if (!ok && leader && x > 0) {
        // leave no copy in flight into this CTA's shared memory
        mbar_drain(BAR_KV, 0, p.timeout_ns);
        for (uint32_t y = x > C::RING ? x - C::RING : 0; y < x; ++y) mbar_drain(full(y), phase(y), p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      bool ok = true;
      auto ready = [&](bool now, uint32_t bar, uint32_t parity) {   // after a test of the same phase
        return __all_sync(0xffffffffu, now) || wait_all(bar, parity, kErrMma);
      };
      auto full_at = [&](uint32_t i) { return bar0 + 8u * i; };
      auto empty_at = [&](uint32_t i) { return bar0 + 8u * (C::RING + i); };
      Place<C::RING> qc, gc, qn, gn;   // this step's Q and dO tile, and the next step's
      gc.next();
      uint32_t ka[C::QK], va[C::QK];
      rows_desc(ka, sK);
      rows_desc(va, sV);
      if (steps > 0) {
        uint32_t qb[C::QK], gb[C::QK];
        rows_desc(qb, sR + qc.i * C::TILE);
        rows_desc(gb, sR + gc.i * C::TILE);
        ok = wait_all(BAR_KV, 0, kErrMma) && wait_all(full_at(qc.i), 0, kErrMma) && wait_all(full_at(gc.i), 0, kErrMma);
        if (ok) {
          tc_fence_after();
          if (leader) {
            mma_group<C::QK, true>(tmem, ka, qb, kDescHi, C::IDESC_S, 0u);
            mma_commit(BAR_S);
            mma_group<C::QK, true>(tmem + 128, va, gb, kDescHi, C::IDESC_S, 0u);
            mma_commit(BAR_DP);
          }
          __syncwarp();
        }
      }
      launch_wait();
      for (uint32_t t = 0; t < steps && ok; ++t) {
        const bool more = t + 1 < steps;
        qn = gc;
        qn.next();
        gn = qn;
        gn.next();
        if (more) {
          const bool q_now = mbar_test(full_at(qn.i), qn.ph), s_now = mbar_test(BAR_SREAD, t & 1);
          uint32_t qb[C::QK];
          rows_desc(qb, sR + qn.i * C::TILE);
          ok = ready(q_now, full_at(qn.i), qn.ph) && ready(s_now, BAR_SREAD, t & 1);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            mma_group<C::QK, true>(tmem, ka, qb, kDescHi, C::IDESC_S, 0u);
            mma_commit(BAR_S);
          }
          __syncwarp();
        }
        // P^T and dS^T arrive in two halves (32 of each warpgroup's 64 query
        // columns), so the products begin under the second half's arithmetic;
        // P^T lies in the first half of the warpgroup's dP^T columns, dS^T in
        // the second.  k-step kk covers query rows 16 kk..: steps 0, 1, 4, 5
        // belong to the first halves.
        const bool g_now = more && mbar_test(full_at(gn.i), gn.ph), d_now = mbar_test(BAR_DS, t & 1);
        uint32_t qb[C::PV], gb[C::PV], nb[C::QK];
        cols_desc(qb, sR + qc.i * C::TILE);
        cols_desc(gb, sR + gc.i * C::TILE);
        rows_desc(nb, sR + gn.i * C::TILE);
        const uint32_t pt = tmem + 128;
        auto products = [&](int part) {
          const int k0 = 2 * part;
          const uint32_t pa[4] = {pt + 8 * k0, pt + 8 * k0 + 8, pt + 64 + 8 * k0, pt + 64 + 8 * k0 + 8};
          const uint32_t da[4] = {pa[0] + 32, pa[1] + 32, pa[2] + 32, pa[3] + 32};
          const uint32_t q4[4] = {qb[k0], qb[k0 + 1], qb[k0 + 4], qb[k0 + 5]};
          const uint32_t g4[4] = {gb[k0], gb[k0 + 1], gb[k0 + 4], gb[k0 + 5]};
          mma_group<4, false>(tmem + 256 + D, da, q4, kDescHi, C::IDESC_G, t > 0 || part > 0);
          if (part == 1) mma_commit(empty_at(qc.i));
          mma_group<4, false>(tmem + 256, pa, g4, kDescHi, C::IDESC_G, t > 0 || part > 0);
          if (part == 1) mma_commit(more ? empty_at(gc.i) : BAR_DONE);
        };
        if (more) ok = ready(g_now, full_at(gn.i), gn.ph);
        if (ok) ok = ready(d_now, BAR_DS, t & 1);
        if (!ok) break;
        tc_fence_after();
        if (leader) products(0);
        __syncwarp();
        ok = ready(mbar_test(BAR_DS2, t & 1), BAR_DS2, t & 1);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          products(1);
          if (more) {
            mma_group<C::QK, true>(tmem + 128, va, nb, kDescHi, C::IDESC_S, 0u);
            mma_commit(BAR_DP);
          }
        }
        __syncwarp();
        qc = qn;
        gc = gn;
      }
      if (!ok && leader) {
        // let every MMA already issued finish before TMEM is released
        mma_commit(BAR_DRAIN);
        mbar_drain(BAR_DRAIN, 0, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpStats) {
      // (the next step's are requested before this step's are handed over)
      bool ok = true;
      uint32_t g = uniform(first / q_tiles), qt = first - g * q_tiles;
      float nl[4], dl[4], nn[4], dn[4];
      auto fetch = [&](float (&a)[4], float (&d)[4]) {
        const int h = hk * share + g, q0 = qt * kBM;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = q0 + i * 32 + lane;
          a[i] = INFINITY;   // (rows past the end: P = 0)
          d[i] = 0.f;
          if (row < p.s_q) {
            const float* l = static_cast<const float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + row * p.lse.s[2];
            const float* x = p.ws + (static_cast<int64_t>(b) * p.heads + h) * p.s_q + row;
            if (CPATTN_IN(p.lse.span, l, 4, p.err)) a[i] = *l;
            if (CPATTN_IN(p.ws_span, x, 4, p.err)) d[i] = *x;
          }
        }
        if (++qt == q_tiles) {
          qt = 0;
          ++g;
        }
      };
      launch_wait();   // (delta is written; everything older than the dq kernel was when this one started)
      launch_next();
      if (steps > 0) fetch(nl, dl);
      for (uint32_t t = 0; t < steps && ok; ++t) {
        if (t + 1 < steps) fetch(nn, dn);
        ok = wait_all(st_empty(t & 1), ((t >> 1) & 1) ^ 1, kErrStats);
        if (!ok) break;
        float* st = stats + (t & 1) * (C::STATS / 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st[i * 32 + lane] = -cross_lse2(nl[i]);
          st[kBM + i * 32 + lane] = -dl[i];
          nl[i] = nn[i];
          dl[i] = dn[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(st_full(t & 1));
      }
      __syncwarp();
    }
  } else {
    regs_increase<kSoftmaxRegs>();
    const int half = warp / 4, quarter = warp % 4;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sl2 = p.scale_log2;
    const int key = k0 + quarter * 32 + lane;
    const bool live = key < len;
    bool ok = true;
    uint32_t qt = first % q_tiles;
    launch_wait();
    for (uint32_t t = 0; t < steps; ++t) {
      const int rows = p.s_q - static_cast<int>(qt) * kBM - half * 64;   // of this thread's 64 query columns
      if (++qt == q_tiles) qt = 0;
      const float4* nl = reinterpret_cast<const float4*>(stats + (t & 1) * (C::STATS / 4)) + half * 16;
      const float4* dl = nl + kBM / 4;
      ok = wait_all(st_full(t & 1), (t >> 1) & 1, kErrSoftmax);
      if (ok) ok = wait_all(BAR_S, t & 1, kErrSoftmax);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[64], g[64], pb[32];
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
        pb[2 * i] = pack_bf16x2(u2f(s[4 * i]), u2f(s[4 * i + 1]));
        pb[2 * i + 1] = pack_bf16x2(u2f(s[4 * i + 2]), u2f(s[4 * i + 3]));
      }
      ok = wait_all(BAR_DP, t & 1, kErrSoftmax);
      if (!ok) break;
      tc_fence_after();
      tmem_ld_x64(lanes + 128 + half * 64, g);
      // two halves of the 64 query columns: P^T and dS^T of each over dP^T
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t px[16], dx[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = 32 * q + 4 * i;
          const float4 d = dl[8 * q + i];
          float x[4];
          fadd2(x[0], x[1], u2f(g[c]), u2f(g[c + 1]), d.x, d.y);
          fadd2(x[2], x[3], u2f(g[c + 2]), u2f(g[c + 3]), d.z, d.w);
          fmul2(x[0], x[1], x[0], x[1], u2f(s[c]), u2f(s[c + 1]));
          fmul2(x[2], x[3], x[2], x[3], u2f(s[c + 2]), u2f(s[c + 3]));
          px[2 * i] = pb[16 * q + 2 * i];
          px[2 * i + 1] = pb[16 * q + 2 * i + 1];
          dx[2 * i] = pack_bf16x2(x[0], x[1]);
          dx[2 * i + 1] = pack_bf16x2(x[2], x[3]);
        }
        if (!live) {
          // a key past the length (its k and v may hold anything): no weight
#pragma unroll
          for (int i = 0; i < 16; ++i) px[i] = dx[i] = 0u;
        }
        if (rows < 64) {
          // (the same for the whole warpgroup) rows past the end: their scores are
          // 0 k_j, and 0 * inf is not 0
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = 32 * q + 2 * i;
            const uint32_t keep = c + 1 < rows ? 0xFFFFFFFFu : c < rows ? 0xFFFFu : 0u;
            px[i] &= keep;
            dx[i] &= keep;
          }
        }
        __syncwarp();
        tmem_st_x16(lanes + 128 + half * 64 + q * 16, px);
        tmem_st_x16(lanes + 128 + half * 64 + 32 + q * 16, dx);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q == 0 ? BAR_DS : BAR_DS2);
      }
      if (lane == 0) mbar_arrive(st_empty(t & 1));
    }
    if (ok && steps > 0) {
      ok = wait_all(BAR_DONE, 0, kErrSoftmax);
      if (ok) tc_fence_after();
    }
    if (ok) {
      // warpgroup 0 writes dv, warpgroup 1 dk, through the idle ring
      const CrossTensor& t = half ? p.dk : p.dv;
      const CUtensorMap* tm = half ? &tm_dk : &tm_dv;
      const float f = half ? p.scale : 1.f;
      // (dk is 0 where one key has all the weight; delta was not formed there)
      const bool zero = steps == 0 || !live || (half == 1 && len == 1);
      const int64_t rows = static_cast<int64_t>(p.batch) * p.kv_heads * p.s_kv;
      float* ws = p.ws + partials + (2 * part + (half ? 0 : 1)) * rows * D +
                  ((static_cast<int64_t>(b) * p.kv_heads + hk) * p.s_kv + key) * D;
      uint8_t* row = ring + (warp * 32 + lane) * C::PART_ROW;   // (several parts: a row of fp32 each)
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t o[64];
        __syncwarp();
        if (steps > 0) tmem_ld_x64(lanes + 256 + half * D + c0, o);
#pragma unroll
        for (int i = 0; i < 64; ++i) o[i] = zero ? 0u : o[i];
        if (p.splits > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<uint4*>(row + c0 * 4 + i * 16) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
          store_rows<64>(p, t, tm, ring + (warp * (D / 64) + c0 / 64) * 4096, o, f, b, hk, k0 + quarter * 32, p.s_kv, c0);
        }
      }
      if (p.splits > 1 && key < p.s_kv) {
        // each lane's row leaves by one bulk copy
        if (CPATTN_IN(p.ws_span, ws, D * 4, p.err)) {
          fence_proxy_async_smem();
          bulk_store(ws, smem_addr(row), D * 4);
          bulk_commit();
        }
      }
      bulk_wait_read();   // (before this CTA's shared memory is given up)
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
template <int D>
cudaError_t launch_typed(const CrossBwdMaps& m, const CrossParams& p, int64_t partials, cudaStream_t stream) {
  using C = Cfg<D>;
  static std::atomic<unsigned long long> ready_q{0}, ready_kv{0};
  cudaError_t e = cross_set_up(cross_dq_kernel<D>, C::DQ_SMEM, ready_q, kLaunchRegs);
  if (e == cudaSuccess) e = cross_set_up(cross_dkv_kernel<D>, C::KV_SMEM, ready_kv, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const int64_t sms = sm_count();
  const int64_t units = static_cast<int64_t>(p.batch) * p.heads * ((p.s_q + kBM - 1) / kBM);
  const int64_t ctas = static_cast<int64_t>(p.batch) * p.kv_heads * p.splits * ((p.s_kv + kBM - 1) / kBM);
  if (units > 0x7fffffff || ctas > 0x7fffffff) return cudaErrorInvalidValue;
  e = launch_behind(cross_dq_kernel<D>, dim3(static_cast<unsigned>(units < sms ? units : sms)), kThreads, C::DQ_SMEM,
                    stream, m.q, m.k, m.v, m.dout, m.out, m.dq, p);
  if (e != cudaSuccess) return e;
  e = launch_behind(cross_dkv_kernel<D>, dim3(static_cast<unsigned>(ctas)), kThreads, C::KV_SMEM, stream, m.q, m.k, m.v,
                    m.dout, m.dk, m.dv, p, partials);
  return e == cudaSuccess && p.splits > 1 ? launch_cross_dkv_join(InDtype::BF16, D, p, partials, stream) : e;
}

}  // namespace

int cross_backward_parts(int64_t key_units, int64_t steps) {
  // The parts share the GPU as whole CTAs, one per SM at a time: the fewest
  // query-tile steps over all waves, a CTA's start and end (its sums leave at
  // some 28 bytes a cycle) counting as six steps and the join as eight.
  // (4608 x 512 x 24 heads: 1 part 105 us, 3 parts 108, 2 parts 119 in all.)
  const int64_t sms = sm_count();
  int best = 1;
  int64_t least = 0;
  for (int parts = 1; parts <= 32 && parts <= steps; ++parts) {
    const int64_t waves = (key_units * parts + sms - 1) / sms;
    const int64_t cost = waves * ((steps + parts - 1) / parts + 6) + (parts > 1 ? 8 : 0);
    if (parts == 1 || cost < least) {
      best = parts;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_cross_bwd(int head_dim, const CrossBwdMaps& maps, const CrossParams& p, int64_t partials,
                             cudaStream_t stream) {
  return head_dim == 64 ? launch_typed<64>(maps, p, partials, stream) : launch_typed<128>(maps, p, partials, stream);
}

}  // namespace cpattn
