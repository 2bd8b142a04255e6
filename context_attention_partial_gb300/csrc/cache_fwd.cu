// cache_fwd.cu -- attention of many rows (wide trees, pieces of prompts) to a paged
// cache, bf16, on the tensor cores.
//
// Mathematics as in cache_few.cu.  P is rounded to bf16 for its product with V (the
// tensor cores' operand type; l keeps the fp32 values), and the output once.
//
// What bounds it: with 256 rows a key head or more the products (4 D operations a row
// and key), below that the read of the keys and values.  Blocks are persistent, one an
// SM, and walk pieces of the line of all key tiles (CacheWalk): the next piece's
// queries and keys are fetched and its first Q K^T is issued while this piece's last
// softmax, P V and output are under way.
//
// Roles (12 warps): warps 0-7 softmax and output, one thread per row of a 128-row query
// tile and warpgroup; warp 8 TMA producer; warp 9 MMA issuer; warp 10 cleans the value
// tiles that hold drafts; warp 11 finds the block's pieces and announces them.  TMEM:
// S_0 | S_1 | O_0 | O_1, P over S's first columns.  Shared memory: the two Q tiles, a ring
// of K / V tiles, an output staging area and the paths of a tree's drafts per softmax warp.
//
// Rows.  A query tile is whole tokens, each with every query head that shares the key
// head: a TMA box [tokens][heads][64 features].  PAIR: a unit has one query tile, its
// key tiles alternate between the two sums, which are joined at the end of a piece:
// a lone tile's products and exponentials would wait for one another.  Otherwise a
// unit has two query tiles, which read the same keys.
//
// Keys.  A 128-key tile is up to eight pages' boxes; the producer's lanes hold 32 page
// numbers and have the next 32 on their way.  Scores of keys that a row does not see are
// masked in registers, by the bits of its path.  Value rows behind the last key are
// zeroed in shared memory, and so are a draft's values that are not finite (see
// cache_few.cu), by warp 10.
//
// Measured, with the join: trees of 27 drafts, 8 sequences of up to 8192 keys, 32 heads on
// 8, D = 128 (155 MB) 36.8 us, of which the join 6.3; trees of 64, 4 sequences of 16384
// keys, 24 heads, D = 64 (406 MB) 70 us, 5.8 TB/s; 1024 new tokens behind 16384, 32 heads
// on 8, D = 128 (283 GFLOP) 178 us, 1590 TFLOP/s, in longer runs 184 to 192 under the power cap.
#include <cmath>

#include "cache.cuh"
#include "cross_ops.cuh"

namespace cpattn {
namespace {

constexpr int kBM = 128, kBN = 128;
constexpr int kThreads = 384;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpClean = 10, kWarpWalk = 11;
constexpr int kPieces = 4;          // announced ahead
constexpr int kLaunchRegs = 168;    // 65536 / 384, rounded down to 8
constexpr int kSoftmaxRegs = 208, kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays below 2^8
constexpr unsigned kErrProducer = 1u, kErrMma = 2u, kErrSoftmax = 4u, kErrClean = 8u, kErrWalk = 0x10u;

template <int D>
struct Cfg {
  static constexpr int ROW = D * 2;                       // bytes
  static constexpr int TILE = kBM * ROW;                  // bytes of a Q, K or V tile
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int STAGING = 8 * 32 * 64;             // 32 rows x 64 bytes per warp
  static constexpr int PATHS = 8 * 32 * kTreeWords * 4;   // a path per row
  static constexpr int SUMS = 2 * kBM * 8;                // PAIR: m and l of both sums
  static constexpr int PIECES = (kPieces + 1) * 64;
  static constexpr int BARS = 2 * STAGES + 13 + 2 * kPieces;
  static constexpr int SMEM = 1024 + 2 * TILE + STAGES * TILE + STAGING + PATHS + SUMS + PIECES + BARS * 8 + 48;
  static constexpr int QK = ROW / 32, PV = kBN / 16;      // MMAs of a tile product
  static constexpr int KB = ROW / 128;                    // 128-byte column blocks
  static constexpr int O_COL = 2 * kBN;
  static constexpr uint32_t IDESC_QK = make_idesc(1, false, kBM, kBN);
  static constexpr uint32_t IDESC_PV = make_idesc(1, true, kBM, D);
  static_assert(O_COL + 2 * D <= 512, "TMEM");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// All 256 softmax threads meet and vote.
__device__ __forceinline__ bool vote_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.aligned.pred q, 1, 256, p;\n\tselp.u32 %0, 1, "
      "0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Sets the scores 32 C .. 32 C + 31 whose bits are not set to -inf.
template <int C>
__device__ __forceinline__ void mask_scores(uint32_t (&s)[128], uint32_t seen) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!((seen >> i) & 1u)) s[32 * C + i] = f2u(-INFINITY);
}

// A piece and what its roles derive from it.
struct Work : CachePiece {
  int k0, k1;     // its keys
  int n;          // its key tiles
  int drafts;     // the first of them with keys that not every row sees
  int halves;     // query tiles with rows
};

// The next piece of a block's walk (n = 0: no more).
template <bool PAIR>
__device__ __forceinline__ Work next_work(const CacheParams& p, CacheWalk<PAIR ? 128 : 256, kBN>& walk) {
  Work w;
  if (!walk.next(p, w)) {
    w.n = 0;
    return w;
  }
  w.k0 = w.t0 * kBN;
  w.k1 = min(w.len + w.count, w.t1 * kBN);
  w.n = w.t1 - w.t0;
  w.drafts = max(0, w.open - w.k0) / kBN;
  const int share = p.heads / p.kv_heads;
  w.halves = !PAIR && (w.rt * p.tile_rows + p.half_rows) / share < w.count ? 2 : 1;
  return w;
}

// Rows of a query tile as tokens and heads: row x is token x / share, head x % share of
// the tile's (x < 128, so 16 bits of the quotient's factor are exact).
struct Rows {
  int share, tokens, factor;   // heads, tokens of a tile
  __device__ explicit Rows(const CacheParams& p)
      : share(p.heads / p.kv_heads), tokens(p.half_rows / share), factor((65535 + share) / share) {}
  // Row x's token counted from the tile's, or -1: none.
  __device__ int token(int x) const {
    const int t = (x * factor) >> 16;
    return t < tokens ? t : -1;
  }
};

template <int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    cache_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CacheParams p) {
  using C = Cfg<D>;
  constexpr int R = PAIR ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sQ = smem_addr(smem), sKV = sQ + 2 * C::TILE;
  uint8_t* staging = smem + (2 + C::STAGES) * C::TILE;
  uint32_t* all_paths = reinterpret_cast<uint32_t*>(staging + C::STAGING);
  float2* sums = reinterpret_cast<float2*>(staging + C::STAGING + C::PATHS);   // [2][128]
  Work* pieces = reinterpret_cast<Work*>(staging + C::STAGING + C::PATHS + C::SUMS);
  static_assert(sizeof(Work) <= 64, "a piece");
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(pieces) + C::PIECES);
  const uint32_t bar0 = smem_addr(bars);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto bar_q = [&](int i) { return bar0 + 8u * (2 * C::STAGES + i); };          // Q tile arrived
  auto bar_qfree = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 2 + i); };  // its last Q K^T is done
  auto bar_s = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 4 + i); };      // scores ready
  auto bar_p = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 6 + i); };      // P written
  auto bar_o = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 8 + i); };      // O of a piece ready
  const uint32_t bar_drain = bar0 + 8u * (2 * C::STAGES + 10);
  const uint32_t bar_dirty = bar0 + 8u * (2 * C::STAGES + 11);                  // a value tile with drafts arrived
  const uint32_t bar_clean = bar0 + 8u * (2 * C::STAGES + 12);
  auto bar_piece = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 13 + i); };           // announced
  auto bar_done = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 13 + kPieces + i); };  // its output is written
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // pieces with values that are not finite, by the piece's number
  volatile int* unclean = reinterpret_cast<volatile int*>(tmem_holder + 2);     // [8]

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
    mbar_init(bar_dirty, 1);
    mbar_init(bar_clean, 1);
    for (int i = 0; i < kPieces; ++i) {
      pieces[i].n = 0;
      mbar_init(bar_piece(i), 1);
      mbar_init(bar_done(i), 9);   // softmax warps, cleaner
    }
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) unclean[i] = -1;
    fence_mbar_init();
    // the piece of nothing that the softmax warps begin with
    Work nothing = {};
    nothing.n = PAIR ? 2 : 1;   // (a tile for each group)
    nothing.drafts = nothing.halves = 2;
    pieces[kPieces] = nothing;
    mbar_arrive(bar_s(0));
    mbar_arrive(bar_s(1));
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_holder), 512);
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cache_prefetch(p);
  const uint32_t tmem = *tmem_holder;
  const Rows rows(p);
  const int share = rows.share;
  // every wait of a warp is voted on, so its lanes stay together
  auto wait_all = [&](uint32_t bar, uint32_t parity, unsigned code) {
    const bool r = mbar_wait(bar, parity, abort_flag, p.timeout_ns, p.err, code);
    return __all_sync(0xffffffffu, r) != 0;
  };

  // The same for a wait that is over only when some key tiles are: at 50 us a tile.
  auto wait_long = [&](uint32_t bar, uint32_t parity, long long tiles, unsigned code) {
    const bool r = mbar_wait(bar, parity, abort_flag, p.timeout_ns + tiles * 50000, p.err, code);
    return __all_sync(0xffffffffu, r) != 0;
  };
  // Key tiles of piece `number`'s place in the ring.  (The walk may be writing the next
  // piece there: then the one before has ended, and either number will do.)
  auto tiles_at = [&](int number) -> int { return *const_cast<const volatile int*>(&pieces[number % kPieces].n); };
  // Of all pieces announced and not known to have ended: a role with nothing to do in some
  // runs ahead of the others, and then waits for them.
  auto tiles_ahead = [&]() {
    long long tiles = 0;
    for (int i = 0; i < kPieces; ++i) tiles += tiles_at(i);
    return tiles;
  };
  // Piece `number` of this block, once announced, which is when piece number - kPieces has
  // ended; false: no more, or a wait ran out (ok).
  auto take = [&](int number, bool& ok, unsigned code) {
    ok = wait_long(bar_piece(number % kPieces), (number / kPieces) & 1, tiles_at(number), code);
    return ok && pieces[number % kPieces].n != 0;
  };

  if (warp >= 8) {
    launch_wait();
    launch_next();
    regs_decrease<kControlRegs>();
    const bool leader = elect_one();
    if (warp == kWarpProducer) {
      // ---------------------------------------------------------- producer
      // K tiles on even stages, V tiles on odd ones: the first K alone, then
      // V_j and the K tile after it (of the next piece behind a piece's last V)
      // as one pair on the K stage's barrier, so the MMA warp waits once a
      // step; the very last V on its own.  Keys that one row tile reads leave L2 first, so
      // that tables, parts and instructions stay (trees of 27 drafts x 8192 keys: 40.0
      // us, 43.6 when they are kept).
      static_assert(C::STAGES % 2 == 0, "K / V pairs");
      const uint64_t pol_q = l2_policy_evict_first(), pol_kv =
          p.row_tiles > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
      const int box = min(1 << p.cache.shift, kBN);
      const uint32_t q_bytes = static_cast<uint32_t>(p.half_rows) * C::ROW;
      int ld = 0, nq[2] = {0, 0};
      bool ok = true;
      bool have = take(0, ok, kErrProducer);
      ok = ok && p.fault_skip_kv == 0;
      // Pages of a piece's keys, 32 at a time, a lane each; a tile's are of one window, since
      // both begin at multiples of a tile's pages.  They are read a window ahead, and checked
      // when their turn comes (-1: no key, or not in the pool).
      auto key_of = [&](const Work& x, int window) {
        return ((x.k0 >> p.cache.shift) + window * 32 + lane) << p.cache.shift;
      };
      auto read_pages = [&](const Work& x, int window) {
        const int key = key_of(x, window);
        return key < x.k1 ? cache_entry(p.cache, x.b, key, p.err) : -1;
      };
      auto checked = [&](const Work& x, int window, int entry) {
        return key_of(x, window) < x.k1 ? cache_checked(p.cache, entry, p.err) : -1;
      };
      // where the first one of key tile j is among the piece's
      auto entry = [&](const Work& x, int j) { return ((x.k0 + j * kBN) >> p.cache.shift) - (x.k0 >> p.cache.shift); };
      // boxes of key tile j of piece x
      auto boxes = [&](const Work& x, int j) { return ceil_div(min(kBN, x.k1 - (x.k0 + j * kBN)), box); };
      // `n` boxes of key tile j of piece x, a lane each, their pages in lanes `from` on (us,
      // wide trees with pages of 128, 64, 16 rows: 70, 70, 95, by one lane in turn 73, 77,
      // 95).  A page that is not in the pool: zeros.
      const int part = lane / C::KB, kb = lane % C::KB;
      auto ask = [&](const CUtensorMap* tm, int stage, uint32_t bar, const Work& x, int j, int n, int pages, int from) {
        const int page = __shfl_sync(0xffffffffu, pages, from + part);
        if (part < n)
          tma_load_4d_hint(sKV + stage * C::TILE + kb * kBN * 128 + part * box * 128, tm, bar, kb * 64,
                           (x.k0 + j * kBN) & ((1 << p.cache.shift) - 1), x.hk, page, pol_kv);
        __syncwarp();
      };
      auto load_q = [&](const Work& x) {   // once the previous piece's last Q K^T is done
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= x.halves) break;
          ok = wait_all(bar_qfree(i), (nq[i] & 1) ^ 1, kErrProducer);
          if (!ok) return;
          if (leader) {
            mbar_arrive_expect_tx(bar_q(i), q_bytes);
            const int token = (x.rt * (PAIR ? 1 : 2) + i) * rows.tokens;
#pragma unroll
            for (int c = 0; c < C::KB; ++c)
              tma_load_4d_hint(sQ + i * C::TILE + c * kBM * 128, &tm_q, bar_q(i), c * 64, x.hk * share, token, x.b, pol_q);
          }
          __syncwarp();
          ++nq[i];
        }
      };
      // the key tile that is asked for next, j of a piece: its window, and the one behind it
      int here = -1, ahead = -1, window = 0;
      if (have && ok) {
        const Work& w = pieces[0];
        here = checked(w, 0, read_pages(w, 0));
        const int n = boxes(w, 0);
        if (leader) mbar_arrive_expect_tx(bar_full(0), n * box * C::ROW);
        __syncwarp();
        ask(&tm_k, 0, bar_full(0), w, 0, n, here, 0);
        ahead = read_pages(w, 1);
        ld = 1;
        load_q(w);
      }
      for (int number = 0; have && ok; ++number) {
        const bool more_units = take(number + 1, ok, kErrProducer);
        if (!ok) break;
        const Work w = pieces[number % kPieces], wn = pieces[(number + 1) % kPieces];
        // (the next Q tiles into L2 while this piece runs)
        if (more_units && leader)
          for (int i = 0; i < wn.halves; ++i)
#pragma unroll
            for (int c = 0; c < C::KB; ++c)
              tma_prefetch_l2_4d(&tm_q, c * 64, wn.hk * share, (wn.rt * (PAIR ? 1 : 2) + i) * rows.tokens, wn.b);
        const int first = more_units ? read_pages(wn, 0) : -1;   // (used behind this piece's last tile)
        for (int j = 0; j < w.n && ok; ++j) {
          const bool in_unit = j + 1 < w.n, more = in_unit || more_units;
          const int sv = ld % C::STAGES, sk = (ld + 1) % C::STAGES;
          const int kj = in_unit ? j + 1 : 0;
          const int nv = boxes(w, j), nk = in_unit ? boxes(w, kj) : more ? boxes(wn, 0) : 0;
          // (the values' pages are those of the keys before)
          const int v_pages = here, v_from = entry(w, j) & 31;
          if (in_unit) {
            if (entry(w, kj) >> 5 != window) {
              ++window;
              here = checked(w, window, ahead);
              ahead = read_pages(w, window + 1);
            }
          } else {
            window = 0;
            here = more ? checked(wn, 0, first) : -1;
            ahead = more ? read_pages(wn, 1) : -1;
          }
          ok = wait_all(bar_empty(sv), ((ld / C::STAGES) & 1) ^ 1, kErrProducer);
          if (ok && more) ok = wait_all(bar_empty(sk), (((ld + 1) / C::STAGES) & 1) ^ 1, kErrProducer);
          if (!ok) break;
          const uint32_t bar = more ? bar_full(sk) : bar_full(sv);
          if (leader) mbar_arrive_expect_tx(bar, (nv + nk) * box * C::ROW);
          __syncwarp();
          ask(&tm_v, sv, bar, w, j, nv, v_pages, v_from);
          if (in_unit)
            ask(&tm_k, sk, bar, w, kj, nk, here, entry(w, kj) & 31);
          else if (more)
            ask(&tm_k, sk, bar, wn, 0, nk, here, 0);
          ld += more ? 2 : 1;
        }
        if (ok && more_units) load_q(wn);
        have = more_units;
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
      // (tests come before the descriptors are built, waits only where a test failed)
      uint32_t g = 0;                // key tiles so far, over all pieces
      uint32_t nq[2] = {0, 0}, np[2] = {1, 1}, nc = 0;
      bool ok = true;
      bool have = take(0, ok, kErrMma);
      // a piece's first scores, query tile by query tile (its K tile is here)
      auto first_qk = [&](const Work& x, uint32_t at) {
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
            if (x.n == 1) mma_commit(bar_qfree(i));
            if (i == x.halves - 1) mma_commit(bar_empty(s));
          }
          __syncwarp();
        }
      };
      if (have) {
        // (tensor memory is free once the piece of nothing is through)
        ok = wait_all(bar_p(0), 0, kErrMma) && wait_all(bar_p(1), 0, kErrMma) && wait_all(bar_full(0), 0, kErrMma);
        if (ok) first_qk(pieces[0], 0);
      }
      for (int number = 0; have && ok; ++number) {
        const bool more_units = take(number + 1, ok, kErrMma);
        if (!ok) break;
        const int n = pieces[number % kPieces].n, drafts = pieces[number % kPieces].drafts;
        const bool two = pieces[number % kPieces].halves == 2;
        for (int j = 0; j < n; ++j, ++g) {
          const bool more = j + 1 < n;
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
          const bool dirty = j >= drafts;
          if (dirty) {
            if (leader) mbar_arrive(bar_dirty);
            __syncwarp();
          }
          // before the tile's first P V
          auto cleaned = [&]() {
            if (!dirty) return true;
            const bool r = wait_all(bar_clean, nc & 1, kErrMma);
            ++nc;
            return r;
          };
          if constexpr (PAIR) {
            const int i = j & 1;
            if (more && leader) {
              // (S_1-i's last P V was issued a step ago)
              tc_fence_after();
              mma_group<C::QK, true>(tmem + (i ^ 1) * kBN, qd, kd, hi, C::IDESC_QK, 0u);
              mma_commit(bar_s(i ^ 1));
              if (j + 2 == n) mma_commit(bar_qfree(0));
              mma_commit(bar_empty(sk));
            }
            __syncwarp();
            ok = cleaned() && wait_all(bar_p(i), np[i] & 1, kErrMma);
            if (!ok) break;
            ++np[i];
#pragma unroll
            for (int kk = 0; kk < C::PV; ++kk) pa[kk] += i * kBN;
            tc_fence_after();
            if (leader) {
              mma_group<C::PV, false>(tmem + C::O_COL + i * D, pa, vd, hi, C::IDESC_PV, j > 1);
              mma_commit(bar_empty(sv));
              if (j + 2 >= n) mma_commit(bar_o(i));
            }
            __syncwarp();
            continue;
          }
          ok = __all_sync(0xffffffffu, p0_now) || wait_all(bar_p(0), np[0] & 1, kErrMma);
          if (!ok || !(ok = cleaned())) break;
          ++np[0];
          const bool p1_now = two && mbar_test(bar_p(1), np[1] & 1);
          tc_fence_after();
          if (leader) {
            mma_group<C::PV, false>(tmem + C::O_COL, pa, vd, hi, C::IDESC_PV, j > 0);
            if (!two) mma_commit(bar_empty(sv));
            if (more) {
              mma_group<C::QK, true>(tmem, qd, kd, hi, C::IDESC_QK, 0u);
              mma_commit(bar_s(0));
              if (j + 2 == n) mma_commit(bar_qfree(0));
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
              if (j + 2 == n) mma_commit(bar_qfree(1));
              mma_commit(bar_empty(sk));
            } else {
              mma_commit(bar_o(1));
            }
          }
          __syncwarp();
        }
        if (ok && more_units) first_qk(pieces[(number + 1) % kPieces], 2 * g);
        have = more_units;
      }
      if (!ok && leader) {
        // let every MMA already issued finish before TMEM is released
        mma_commit(bar_drain);
        mbar_drain(bar_drain, 0, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpWalk) {
      // ----------------------------------------------------------- the walk
      // (one warp's: the others would each fetch its instructions, at the start of a
      // launch from HBM)
      CacheWalk<PAIR ? 128 : 256, kBN> walk;
      walk.start(p);
      for (int number = 0;; ++number) {
        const Work w = next_work<PAIR>(p, walk);
        // (some pieces may have to end, which takes as long as their tiles)
        if (number >= kPieces &&
            !wait_long(bar_done(number % kPieces), (number / kPieces - 1) & 1, tiles_ahead(), kErrWalk))
          break;
        if (leader) {
          if (w.n != 0) cache_note_unit<R, D>(p, w);
          pieces[number % kPieces] = w;
          mbar_arrive(bar_piece(number % kPieces));
        }
        __syncwarp();
        if (w.n == 0) break;
      }
      cache_empty_units<__nv_bfloat16, R, kBN, D>(p, lane, 32);
    } else if (warp == kWarpClean) {
      // -------------------------------------------------------------- cleaner
      uint32_t g = 0, nd = 0;
      bool ok = true;
      for (int number = 0; ok && take(number, ok, kErrClean); ++number) {
        const Work& w = pieces[number % kPieces];
        const int n = w.n;
        g += min(w.drafts, n);
        for (int j = w.drafts; j < n; ++j, ++g) {
          ok = wait_long(bar_dirty, nd & 1, tiles_ahead(), kErrClean);
          if (!ok) break;
          ++nd;
          const int start = w.k0 + j * kBN, valid = min(kBN, w.k1 - start);
          const int from = w.count > 1 ? max(0, w.open - start) : valid;   // (a lone draft: its rows see it)
          uint8_t* tile = smem + (2 + (2 * g + 1) % C::STAGES) * C::TILE;
          // (a value times 0 is not 0 where it is not finite)
          __nv_bfloat162 zero = __float2bfloat162_rn(0.f), acc[2] = {zero, zero};
#pragma unroll 4
          for (int i = from * 8 + lane; i < valid * 8; i += 32)
#pragma unroll
            for (int c = 0; c < C::KB; ++c) {
              const uint4 v = *reinterpret_cast<const uint4*>(tile + c * kBN * 128 + i * 16);
              const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[e % 2] = __hfma2(x[e], zero, acc[e % 2]);
            }
          const float2 sum = __bfloat1622float2(__hadd2(acc[0], acc[1]));
          const bool found = !(sum.x + sum.y == 0.f);
          if (__any_sync(0xffffffffu, found)) {
#pragma unroll 1
            for (int i = from * 8 + lane; i < valid * 8; i += 32)
              for (int c = 0; c < C::KB; ++c) clear_unfinite(reinterpret_cast<uint4*>(tile + c * kBN * 128 + i * 16));
          }
#pragma unroll 4
          for (int i = valid * 8 + lane; i < kBN * 8; i += 32)
#pragma unroll
            for (int c = 0; c < C::KB; ++c) *reinterpret_cast<uint4*>(tile + c * kBN * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          if (found) unclean[number % 8] = number;
          fence_proxy_async_smem();
          __syncwarp();
          if (leader) mbar_arrive(bar_clean);
        }
        if (leader) mbar_arrive(bar_done(number % kPieces));
      }
    }
  } else {
    // ------------------------------------------------------- softmax, output
    regs_increase<kSoftmaxRegs>();
    const int wg = warp / 4, quarter = warp % 4;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + wg * kBN;
    const uint32_t tO = tmem + lane_base + C::O_COL;   // (of the first sum)
    const float sl2 = p.scale_log2;
    uint8_t* stage = staging + warp * 2048;
    uint32_t* path = all_paths + threadIdx.x * kTreeWords;
    const int x = quarter * 32 + lane;                 // this thread's row of its query tile
    const int row_token = rows.token(x);
    int ns = 0, no[2] = {0, 0};
    bool ok = true, ahead = false;
    // First a piece of nothing: a tile of whatever tensor memory holds, of which nothing
    // is kept.  A launch finds this loop's instructions in HBM, and so they arrive while
    // the kernel before this one ends and the first keys are on their way.
    for (int number = -1;; ++number) {
      if (number >= 0) {
        const bool have = take(number, ok, kErrSoftmax);
        // (the two groups stay together, also when a wait has run out)
        if (PAIR) ok = vote_all(ok);
        if (!ok || !have) break;
      }
      const Work& w = pieces[number >= 0 ? number % kPieces : kPieces];
      const bool mine = PAIR || wg < w.halves;
      const int place = (PAIR ? 0 : wg * kBM) + x;
      const int first_token = (PAIR ? w.rt : w.rt * 2 + wg) * rows.tokens;   // of the query tile
      float m = -INFINITY, l = 0.f;
      if (mine && p.parents != nullptr && w.drafts < w.n) {
        // the rows' paths, up from their drafts (this warp's copy of the parents)
        for (int i = lane; i < p.s_q; i += 32) {
          const int32_t* from = p.parents + w.b * p.parents_stride + i;
          copy4(smem_addr(stage) + i * 4, from, CPATTN_IN(p.parents_span, from, 4, p.err));
        }
        copies_commit();
#pragma unroll
        for (int c = 0; c < kTreeWords; c += 4) *reinterpret_cast<uint4*>(path + c) = make_uint4(0u, 0u, 0u, 0u);
        copies_wait<0>();
        __syncwarp();
        const int token = first_token + row_token;
        uint32_t bits = 0u;
        for (int at = row_token >= 0 && token < w.count ? token : -1; at >= 0;) {
          int up = reinterpret_cast<const int*>(stage)[at];
          up = up < at ? up : -1;
          bits |= 1u << (at % 32);
          if (up >> 5 != at >> 5) {   // (none above, or in the word before)
            path[at / 32] = bits;
            bits = 0u;
          }
          at = up;
        }
        __syncwarp();
      }
      const int first = PAIR ? wg : 0;
      // (the second group has no part in pieces with one query tile, and is ahead of them)
      if (ahead && mine) wait_long(bar_s(wg), ns & 1, tiles_ahead(), kErrSoftmax);
      ahead = !mine;
      for (int j = first; mine && j < w.n; j += PAIR ? 2 : 1) {
        ok = wait_all(bar_s(wg), ns & 1, kErrSoftmax);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        uint32_t s[kBN];
        float row_max;
        if (j < w.drafts) {
          tmem_ld_max_x128(tS, s, row_max);
        } else {
          tmem_ld_x128(tS, s);
          const int start = w.k0 + j * kBN, token = first_token + row_token;
          const bool live = row_token >= 0 && token < w.count;
          // what the row sees of 32 keys at a time (seldom: the last tile or two of a unit)
          auto seen = [&](int at) -> uint32_t {
            if (!live) return 0u;
            return static_cast<uint32_t>(p.parents == nullptr ? chain_window(w.len, token, at) : tree_window(path, w.len, at));
          };
          mask_scores<0>(s, seen(start));
          mask_scores<1>(s, seen(start + 32));
          mask_scores<2>(s, seen(start + 64));
          mask_scores<3>(s, seen(start + 96));
          row_max = masked_row_max<kBN>(s, kBN);
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
        if (__any_sync(0xffffffffu, raise)) rescale_o<D>(tO + wg * D, factor);
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
      if (number < 0) {
        launch_wait();
        if (PAIR) ok = vote_all(ok);
        if (!ok) break;
        continue;
      }
      const bool whole = w.whole();
      const int token = first_token + row_token;
      const bool live = row_token >= 0 && token < w.count;
      if (ok && mine) {
        for (int i = 0; i < (PAIR ? 2 : 1); ++i) {
          const int o = PAIR ? i : wg;
          if (PAIR && w.n <= i) continue;
          ok = ok && wait_all(bar_o(o), no[i] & 1, kErrSoftmax);
          ++no[i];
        }
      }
      float own = 1.f, other = 0.f;     // weights of the first sum and the second
      if constexpr (PAIR) {
        sums[wg * kBM + x] = make_float2(m, l);
        ok = vote_all(ok);
        const float2 a = sums[x], b = sums[kBM + x];
        m = fmaxf(a.x, b.x);
        const float base = m == -INFINITY ? 0.f : m;
        own = ex2_approx(a.x - base);
        other = w.n > 1 ? ex2_approx(b.x - base) : 0.f;
        l = a.y * own + b.y * other;
      }
      if (!ok) break;
      tc_fence_after();
      const bool add = live && w.count > 1 && unclean[number % 8] == number;
      // features of the row, 32 at a time, from tensor memory
      const int c_begin = PAIR ? wg * (D / 2) : 0, c_end = PAIR ? c_begin + D / 2 : D;
      auto features = [&](int c0, uint32_t (&o)[32]) {
        tmem_ld_x32(tO + (PAIR ? 0 : wg * D) + c0, o);
        if (PAIR && w.n > 1) {
          uint32_t o2[32];
          tmem_ld_x32(tO + D + c0, o2);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * own + u2f(o2[i]) * other);
        }
        if (__any_sync(0xffffffffu, add)) {
#pragma unroll 1
          for (int i = 0; i < 32 && add; i += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            add_unfinite<__nv_bfloat16>(p, w, token, p.parents != nullptr ? path : nullptr, w.k0, w.k1, c0 + i, v);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e / 4 * 4 == i) o[e] = f2u(u2f(o[e]) + (e % 4 == 0 ? v.x : e % 4 == 1 ? v.y : e % 4 == 2 ? v.z : v.w));
          }
          __syncwarp();
        }
      };
      if (!whole) {
        // not divided by l: a part for the join (rows without a token: only that l is 0)
        const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1);
        if (!PAIR || wg == 0) {
          float2* dl = cache_part_sums<R, D>(p, gridDim.x, part, place);
          if (CPATTN_IN(p.ws_span, dl, 8, p.err)) *dl = live ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
        }
#pragma unroll 1
        for (int c0 = c_begin; c0 < c_end && mine; c0 += 32) {
          uint32_t o[32];
          features(c0, o);
          if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4* dst = cache_part<R, D>(p, part, place, c0 + i);
              if (CPATTN_IN(p.ws_span, dst, 16, p.err))
                *dst = make_float4(u2f(o[i]), u2f(o[i + 1]), u2f(o[i + 2]), u2f(o[i + 3]));
            }
          }
          __syncwarp();
        }
      } else {
        // rows without a token, or all of whose scores are -inf: (0, -inf)
        const bool none = !live || l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
        if ((!PAIR || wg == 0) && row_token >= 0 && token < p.s_q) {
          float* dl = static_cast<float*>(p.lse.data) + w.b * p.lse.s[0] +
                      (w.hk * share + x - row_token * share) * p.lse.s[1] + token * p.lse.s[2];
          if (CPATTN_IN(p.lse.span, dl, 4, p.err)) *dl = none ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        }
        // through the warp's stage, 64 bytes of each of its rows at a time: the lane's
        // four rows there, and its 16 bytes of them
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out.data) + w.b * p.out.s[0] +
                                   w.hk * share * p.out.s[1] + first_token * p.out.s[2] + lane % 4 * 8;
        int64_t to[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int r = quarter * 32 + it * 8 + lane / 4, t = rows.token(r);
          to[it] = t < 0 || first_token + t >= p.s_q ? -1 : (r - t * share) * p.out.s[1] + t * p.out.s[2];
        }
        __syncwarp();
#pragma unroll 1
        for (int c0 = c_begin; c0 < c_end; c0 += 32) {
          uint32_t o[32];
          if (mine) features(c0, o);
          uint4* srow = reinterpret_cast<uint4*>(stage) + lane * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = none ? 0u : pack_bf16x2(u2f(o[8 * i + 2 * e]) * inv, u2f(o[8 * i + 2 * e + 1]) * inv);
            srow[i ^ ((lane >> 1) & 3)] = make_uint4(v[0], v[1], v[2], v[3]);
          }
          __syncwarp();
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int r = it * 8 + lane / 4;
            const uint4 v = reinterpret_cast<const uint4*>(stage)[r * 4 + (lane % 4 ^ ((r >> 1) & 3))];
            __nv_bfloat16* dst = out + to[it] + c0;
            if (to[it] >= 0 && CPATTN_IN(p.out.span, dst, 16, p.err)) *reinterpret_cast<uint4*>(dst) = v;
          }
          __syncwarp();
        }
      }
      if constexpr (PAIR) {
        // (the other group's sum has been read, and so have m and l)
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_done(number % kPieces));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool PAIR>
cudaError_t launch_typed(const CacheMaps& m, const CacheParams& p, int blocks, cudaStream_t stream) {
  auto kernel = cache_fwd_kernel<D, PAIR>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = cross_set_up(kernel, Cfg<D>::SMEM, ready, kLaunchRegs);
  if (e != cudaSuccess) return e;
  e = launch_behind(kernel, dim3(blocks), kThreads, Cfg<D>::SMEM, stream, m.q, m.k, m.v, p);
  if (e != cudaSuccess || !p.split) return e;
  return cache_join<PAIR ? 128 : 256, D, __nv_bfloat16>(p, blocks, stream);
}

}  // namespace

cudaError_t launch_cache_fwd(int head_dim, int places, const CacheMaps& maps, const CacheParams& p, int blocks,
                             cudaStream_t stream) {
  if (head_dim == 64)
    return places == 128 ? launch_typed<64, true>(maps, p, blocks, stream) : launch_typed<64, false>(maps, p, blocks, stream);
  return places == 128 ? launch_typed<128, true>(maps, p, blocks, stream) : launch_typed<128, false>(maps, p, blocks, stream);
}

}  // namespace cpattn
