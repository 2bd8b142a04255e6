// cache.cuh -- the paged key / value cache: where a sequence's tokens are, and the
// parameters of the attention to it (not part of the public ABI).
#pragma once
#include "cross.cuh"
#include "internal.h"
#include "tile_ops.cuh"

namespace cpattn {

struct CachePlace {
  int64_t page;
  int row;
  bool valid;
};

// Tokens of sequence b before this call's, brought into [0, width * page size], and
// its new ones, into [0, most].
__device__ __forceinline__ int cache_length(const PageTable& c, int b, unsigned int* err) {
  const int32_t* at = c.lengths + b;
  const int n = CPATTN_IN(c.lengths_span, at, 4, err) ? *at : 0;
  const int64_t room = static_cast<int64_t>(c.width) << c.shift;
  return max(0, static_cast<int>(min(static_cast<int64_t>(n), room)));
}
__device__ __forceinline__ int cache_count(const PageTable& c, int b, int most, unsigned int* err) {
  if (c.counts == nullptr) return most;
  const int32_t* at = c.counts + b;
  const int n = CPATTN_IN(c.counts_span, at, 4, err) ? *at : 0;
  return max(0, min(n, most));
}

// What the table has for place `at` (a key's number within its sequence) of sequence b,
// not looked at, so that the load need not have ended; and the page that this is: -1, and
// the error word says so, where the pool has no such page.
__device__ __forceinline__ int cache_entry(const PageTable& c, int b, int64_t at, unsigned int* err) {
  const int64_t i = at >> c.shift;
  if (i >= c.width) return -1;
  const int32_t* from = c.table + b * c.stride + i;
  return CPATTN_IN(c.table_span, from, 4, err) ? *from : -1;
}
__device__ __forceinline__ int cache_checked(const PageTable& c, int entry, unsigned int* err) {
  if (entry >= 0 && entry < c.pages) return entry;
  atomicOr(err, kErrBounds);
  return -1;
}
__device__ __forceinline__ int cache_page(const PageTable& c, int b, int64_t at, unsigned int* err) {
  return cache_checked(c, cache_entry(c, b, at, err), err);
}

// Where new token i of sequence b goes (not valid: nowhere).
__device__ __forceinline__ CachePlace cache_place(const PageTable& c, int b, int i, int most, unsigned int* err) {
  CachePlace p = {0, 0, false};
  if (i >= cache_count(c, b, most, err)) return p;
  const int64_t at = static_cast<int64_t>(cache_length(c, b, err)) + i;
  const int page = cache_page(c, b, at, err);
  if (page < 0) return p;
  p.page = page;
  p.row = static_cast<int>(at & ((1 << c.shift) - 1));
  p.valid = true;
  return p;
}

// ------------------------------------------------------------- attention
// S_q new tokens of each sequence against its cache, which holds them already, in
// the places behind lengths[b].  A row is a (token, query head) pair of those that
// share a key head, row = token * share + head % share; a row tile is `tile_rows` of
// them.  Where it is kept they have R places: place r holds row (r / 128) * half_rows
// + r % 128 of the tile, if r % 128 < half_rows (the tensor cores' tiles have 128
// rows, of which whole tokens fill some).
struct CacheParams {
  CrossTensor q, out, lse;    // [B, H, S_q, D], lse [B, H, S_q]
  CrossTensor k, v;           // pages: strides (page, head, row of the page)
  PageTable cache;
  const int32_t* parents;     // [B, S_q], rows `parents_stride` apart, or nullptr: a chain
  int64_t parents_stride;
  Span parents_span;
  float* ws;                  // parts of units, see CacheWalk
  Span ws_span;
  int batch, heads, kv_heads, s_q;
  int row_tiles;              // of a key head
  int tile_rows, half_rows;   // rows of a row tile, and of each 128 places of its storage
  int split;                  // whether units are split over blocks (see CacheWalk)
  float scale_log2;           // softmax scale times log2(e)
  unsigned long long timeout_ns;
  int fault_skip_kv;          // testing: the producer issues no copies
  unsigned int* err;
};

// Asks for what a call reads first -- lengths, counts, the table's beginning, parents --
// while the kernel before it ends (launch_wait() follows; no value is read).
__device__ __forceinline__ void cache_prefetch(const CacheParams& p) {
  auto lines = [&](const int32_t* from, int64_t n) {
    if (from == nullptr) return;
    const int64_t bytes = min(n * 4, static_cast<int64_t>(blockDim.x) * 128);
    if (threadIdx.x * 128 < bytes) prefetch_l2(reinterpret_cast<const char*>(from) + threadIdx.x * 128);
  };
  lines(p.cache.lengths, p.batch);
  lines(p.cache.counts, p.batch);
  lines(p.cache.table, (p.batch - 1) * p.cache.stride + p.cache.width);
  lines(p.parents, p.parents != nullptr ? (p.batch - 1) * p.parents_stride + p.s_q : 0);
}

// Row of (b, hk, rt)'s place r, or -1.
__device__ __forceinline__ int cache_row(const CacheParams& p, int rt, int r) {
  const int x = r % 128, row = rt * p.tile_rows + r / 128 * p.half_rows + x;
  return x < p.half_rows && row < p.s_q * (p.heads / p.kv_heads) ? row : -1;
}

// Key tiles that a block takes at least before another one shares its work, for row
// tiles of `places` and key tiles of `keys` (us; tiles of 64 keys, one token, 8 key
// heads x 1000 keys: at least 2 tiles 11.6, 3 tiles 15.2, 6 tiles 18.0; fp32, tiles of
// 32: 16 rows x 3000 keys 18.2 with 3, 20.7 with 1; 64 rows x 700 keys 20.4 with 3,
// 15.7 with 1).
constexpr int cache_min_tiles(int places, int keys) { return keys >= 64 ? 2 : places > 16 ? 1 : 3; }
// Units a block from which none are split: every block walks over all pairs of sequence
// and row tile to find its stretch, and a split needs tables of the units.  Of equal units
// a round is then at most an eighth of the call; but they are dealt out by number, whatever
// their lengths are, and with unequal ones the busiest block sets the time.  Measured on
// both sides, 8 key heads (us, those of the bytes in brackets; split / whole): one token,
// lengths spread by their logarithm over 100 to 16384, 303 sequences 587 (590) / 304 895
// (590); one of 32768 keys among others of 1000, 303 218 (203) / 512 737 (329); all of
// 3100, 300 564 (563) / 512 928 (960); trees of 27, spread, 151 309 (259) / 152 435 (259).
constexpr int kCacheWholeUnits = 8;

// A piece of work: key tiles t0 .. t1 of row tile rt of (b, hk), which has `tiles`.
struct CachePiece {
  int b, hk, rt;
  int t0, t1, tiles;
  int len, count;             // the sequence's cached and new tokens
  int open;                   // keys before it are seen by every row that has a token
  __device__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// What the beginning and end of a unit cost, in key tiles (us with 0 and with this: tiles
// of 128 keys, 2048 tokens from an empty cache 96.1 / 48.8, trees of 27 x 8192 keys 38.8
// / 37.3; of 64, 8 sequences of 1000 keys 15.7 / 13.9; of 32 13 fp32 rows 24.9 / 20.6).
constexpr int cache_unit_cost(int keys) { return keys >= 128 ? 3 : keys >= 64 ? 2 : 1; }

// Deals the key tiles out to the blocks, evenly, whatever the lengths are.  All (row
// tile, key head) units of all sequences stand in a line, b slowest, then row tile,
// then key head, and each is its key tiles and some that stand for its beginning and
// end; block c takes the c-th of `blocks` stretches of the line's tiles (equal, but for
// one), so its pieces are the end of a unit, whole units, and the beginning of one.  A
// piece that is not a whole unit goes to the workspace: slot 0 of the block if it begins
// inside its unit, slot 1 if it only ends there; the blocks that begin and end a unit
// note themselves for the join kernel.  Not split: whole units, c, c + blocks, ...
// R: places of a row tile, KT: keys of a key tile.  A split line has less than 2^31
// tiles.  Whole warps.
template <int R, int KT>
struct CacheWalk {
  int pos, end;    // tiles of the line (not split: units): the next, one past the last
  int base, x;     // pair (b, row tile) that holds the next; its first tile
  int tiles, len, count;   // of the pair

  // A unit's length in the line.
  __device__ static int length(int tiles) { return tiles > 0 ? tiles + cache_unit_cost(KT) : 0; }

  // Key tiles of pair x.
  __device__ static int tiles_of(const CacheParams& p, int x, int* len, int* count) {
    const int b = x / p.row_tiles, first = (x - b * p.row_tiles) * p.tile_rows, share = p.heads / p.kv_heads;
    *len = cache_length(p.cache, b, p.err);
    *count = cache_count(p.cache, b, p.s_q, p.err);
    if (first / share >= *count) return 0;   // (no row has a token)
    // a chain's rows see nothing past their last token
    const int last = p.parents != nullptr ? *count - 1 : min(*count - 1, (first + p.tile_rows - 1) / share);
    return (*len + last + KT) / KT;
  }
  __device__ void start(const CacheParams& p) {
    pos = blockIdx.x;
    end = p.batch * p.row_tiles * p.kv_heads;
    base = x = tiles = len = count = 0;
    if (!p.split) return;
    const int lane = threadIdx.x % 32, pairs = p.batch * p.row_tiles;
    unsigned total = 0;
    for (int x0 = 0; x0 < pairs; x0 += 32) {
      total += __reduce_add_sync(
          0xffffffffu, x0 + lane < pairs ? static_cast<unsigned>(length(tiles_of(p, x0 + lane, &len, &count)) * p.kv_heads) : 0u);
    }
    unsigned blocks = (total + cache_min_tiles(R, KT) - 1) / cache_min_tiles(R, KT);
    blocks = blocks < gridDim.x ? blocks : gridDim.x;
    pos = end = 0;
    if (blockIdx.x >= blocks) return;
    const unsigned each = total / blocks, more = total - each * blocks;
    pos = blockIdx.x * each + min(blockIdx.x, more);
    end = pos + each + (blockIdx.x < more ? 1 : 0);
    // the pair that holds pos
    for (int x0 = 0; x0 < pairs; x0 += 32) {
      tiles = len = count = 0;
      if (x0 + lane < pairs) tiles = tiles_of(p, x0 + lane, &len, &count);
      const int w = length(tiles) * p.kv_heads;
      int sum = w;
#pragma unroll
      for (int m = 1; m < 32; m *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m) sum += y;
      }
      const unsigned behind = __ballot_sync(0xffffffffu, pos < base + sum);
      if (behind != 0) {
        const int i = __ffs(behind) - 1;
        x = x0 + i;
        base += __shfl_sync(0xffffffffu, sum - w, i);
        tiles = __shfl_sync(0xffffffffu, tiles, i);
        len = __shfl_sync(0xffffffffu, len, i);
        count = __shfl_sync(0xffffffffu, count, i);
        return;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  // The next piece with keys; false: no more.
  __device__ bool next(const CacheParams& p, CachePiece& w) {
    while (pos < end) {
      if (!p.split) {
        x = pos / p.kv_heads;
        w.hk = pos - x * p.kv_heads;
        pos += gridDim.x;
        tiles = tiles_of(p, x, &len, &count);
        if (tiles == 0) continue;
        w.t0 = 0;
        w.t1 = tiles;
      } else {
        const int off = pos - base, unit = length(tiles), all = unit * p.kv_heads;
        if (off >= all) {
          base += all;
          ++x;
          tiles = tiles_of(p, x, &len, &count);
          continue;
        }
        w.hk = off / unit;
        w.t0 = off - w.hk * unit;
        w.t1 = min(w.t0 + end - pos, tiles);
        pos += unit - w.t0;            // (beyond the end, if the piece ends there)
        if (w.t0 >= tiles) continue;   // (what stands for the unit's end)
      }
      w.tiles = tiles;
      w.len = len;
      w.count = count;
      w.b = x / p.row_tiles;
      w.rt = x - w.b * p.row_tiles;
      w.open = w.len + (p.parents != nullptr ? 0 : w.rt * p.tile_rows / (p.heads / p.kv_heads) + 1);
      return true;
    }
    return false;
  }
};

// First and last block of every unit, behind the parts in the workspace.
template <int R, int D>
__device__ __forceinline__ int2* cache_unit_blocks(const CacheParams& p, int most) {
  return reinterpret_cast<int2*>(p.ws + static_cast<int64_t>(most) * 2 * R * (D + 2));
}
// Notes for the join that this block begins or ends the piece's unit (one thread).
template <int R, int D>
__device__ __forceinline__ void cache_note_unit(const CacheParams& p, const CachePiece& w) {
  if (!p.split) return;
  int2* at = cache_unit_blocks<R, D>(p, gridDim.x) + (static_cast<int64_t>(w.b) * p.row_tiles + w.rt) * p.kv_heads + w.hk;
  if (!CPATTN_IN(p.ws_span, at, 8, p.err)) return;
  if (w.t0 == 0) at->x = blockIdx.x;
  if (w.t1 == w.tiles) at->y = blockIdx.x;
}

// Units without keys: (0, -inf) for their rows that exist.  The blocks share the units
// out by their number; thread t of `threads` of a block.
template <typename T, int R, int KT, int D>
__device__ __forceinline__ void cache_empty_units(const CacheParams& p, int t, int threads) {
  if (p.cache.counts == nullptr) return;   // (every sequence has new tokens)
  const int share = p.heads / p.kv_heads;
  const int64_t units = static_cast<int64_t>(p.batch) * p.row_tiles * p.kv_heads;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int x = static_cast<int>(u / p.kv_heads), hk = static_cast<int>(u % p.kv_heads);
    int len, count;
    if (CacheWalk<R, KT>::tiles_of(p, x, &len, &count) != 0) continue;
    const int b = x / p.row_tiles, rt = x - b * p.row_tiles;
    if (p.split && t == 0) {   // (nothing to join)
      int2* at = cache_unit_blocks<R, D>(p, gridDim.x) + u;
      if (CPATTN_IN(p.ws_span, at, 8, p.err)) *at = make_int2(0, 0);
    }
    constexpr int C = D * sizeof(T) / 16;
    for (int i = t; i < R * C; i += threads) {
      const int row = cache_row(p, rt, i / C);
      if (row < 0) continue;
      const int token = row / share, h = hk * share + row % share;
      T* dst = static_cast<T*>(p.out.data) + b * p.out.s[0] + h * p.out.s[1] + token * p.out.s[2] + i % C * (16 / sizeof(T));
      if (CPATTN_IN(p.out.span, dst, 16, p.err)) *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
      float* dl = static_cast<float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + token * p.lse.s[2];
      if (i % C == 0 && CPATTN_IN(p.lse.span, dl, 4, p.err)) *dl = -INFINITY;
    }
  }
}

// A tree's paths: `words` [R][kTreeWords], bit j of row r's: draft j is the row's token
// or above it.  A parent that is not before its draft is none (so a walk ends).
// `parents`: S_q ints of shared memory, loaded.  Thread t of `threads` takes rows t, ...
constexpr int kTreeWords = CPATTN_MAX_TREE / 32;
template <int R>
__device__ __forceinline__ void tree_paths(const CacheParams& p, const int* parents, int rt, int t, int threads,
                                           uint32_t* words) {
  const int share = p.heads / p.kv_heads;
  for (int r = t; r < R; r += threads) {
    uint32_t bits[kTreeWords] = {};
    const int row = cache_row(p, rt, r);
    int j = row < 0 ? -1 : row / share;
    while (j >= 0) {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w)
        if (j / 32 == w) bits[w] |= 1u << (j % 32);
      const int up = parents[j];
      j = up < j ? up : -1;
    }
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) words[r * kTreeWords + w] = bits[w];
  }
}

// What a row sees of the keys start .. start + 63, as bits.  len: the sequence's
// cached tokens; i: the row's token (below its count).
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ unsigned long long chain_window(int len, int i, int start) { return low_bits(len + i + 1 - start); }
__device__ __forceinline__ unsigned long long tree_window(const uint32_t* words, int len, int start) {
  const int cached = len - start;   // of the window
  if (cached >= 64) return ~0ull;
  auto word64 = [&](int w) {        // drafts 32 w .. 32 w + 63
    const unsigned long long lo = w < kTreeWords ? words[w] : 0u, hi = w + 1 < kTreeWords ? words[w + 1] : 0u;
    return lo | hi << 32;
  };
  if (cached >= 0) return low_bits(cached) | (cached == 0 ? word64(0) : word64(0) << cached);
  const int j = -cached, w = j / 32, o = j % 32;
  unsigned long long bits = word64(w) >> o;
  if (o != 0 && w + 2 < kTreeWords) bits |= static_cast<unsigned long long>(words[w + 2]) << (64 - o);
  return bits;
}

// Eight bf16 values: those that are not finite become 0; whether there were any.
__device__ __forceinline__ bool clear_unfinite(uint4* at) {
  uint4 v = *at;
  uint32_t* x = reinterpret_cast<uint32_t*>(&v);
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (x[i] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u, hi = (x[i] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
    found |= (lo | hi) != 0;
    x[i] &= ~(lo | hi);
  }
  if (found) *at = v;
  return found;
}
// Four fp32 values likewise.
__device__ __forceinline__ bool clear_unfinite(float4* at) {
  float4 v = *at;
  float* x = reinterpret_cast<float*>(&v);
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!isfinite(x[i])) {
      x[i] = 0.f;
      found = true;
    }
  if (found) *at = v;
  return found;
}

// Adds to features d .. d + 3 of a row of token i the values that are not finite, of
// the keys k0 .. k1 - 1 from w.open on that it sees (paths: its path, nullptr for a chain).
template <typename T>
__device__ __noinline__ void add_unfinite(const CacheParams& p, const CachePiece& w, int i, const uint32_t* path, int k0,
                                          int k1, int d, float4& sum) {
  for (int key = max(k0, w.open); key < k1; ++key) {
    const int j = key - w.len;
    if (path != nullptr ? !((path[j / 32] >> (j % 32)) & 1u) : j > i) continue;
    const int page = cache_page(p.cache, w.b, key, p.err);
    if (page < 0) continue;
    const T* from = static_cast<const T*>(p.v.data) + page * p.v.s[0] + w.hk * p.v.s[1] +
                    (key & ((1 << p.cache.shift) - 1)) * p.v.s[2] + d;
    if (!CPATTN_IN(p.v.span, from, 4 * sizeof(T), p.err)) continue;
    float* x = reinterpret_cast<float*>(&sum);
    for (int e = 0; e < 4; ++e) {
      const float v = static_cast<float>(from[e]);
      if (!isfinite(v)) x[e] += v;
    }
  }
}

// Four features of a row's result: sum / l and, with feature 0, m ln2 + ln l; (0, -inf)
// where no key had weight.
template <typename T>
__device__ __forceinline__ void cache_write_row(const CacheParams& p, int b, int h, int token, int d, float4 sum, float m,
                                                float l) {
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  if (none) sum = make_float4(0.f, 0.f, 0.f, 0.f);
  T* dst = static_cast<T*>(p.out.data) + b * p.out.s[0] + h * p.out.s[1] + token * p.out.s[2] + d;
  if (CPATTN_IN(p.out.span, dst, 4 * sizeof(T), p.err)) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
    else
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
  }
  if (d != 0) return;
  float* dl = static_cast<float*>(p.lse.data) + b * p.lse.s[0] + h * p.lse.s[1] + token * p.lse.s[2];
  if (CPATTN_IN(p.lse.span, dl, 4, p.err)) *dl = none ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// Where the workspace has features d .. d + 3 of place r of a part ([part][D / 4][R][4]:
// neighbouring places are neighbours in memory), and its m (base 2) and l.  Parts: two
// slots of each of the attention's `most` blocks.
template <int R, int D>
__device__ __forceinline__ float4* cache_part(const CacheParams& p, int64_t part, int r, int d) {
  return reinterpret_cast<float4*>(p.ws + part * R * D) + (d / 4) * R + r;
}
template <int R, int D>
__device__ __forceinline__ float2* cache_part_sums(const CacheParams& p, int most, int64_t part, int r) {
  return reinterpret_cast<float2*>(p.ws + static_cast<int64_t>(most) * 2 * R * D) + part * R + r;
}
template <int R, int D>
__device__ __forceinline__ void cache_write_part(const CacheParams& p, int64_t part, int r, int d, float4 sum, float m,
                                                 float l) {
  float4* dst = cache_part<R, D>(p, part, r, d);
  float2* dl = cache_part_sums<R, D>(p, gridDim.x, part, r);
  if (CPATTN_IN(p.ws_span, dst, 16, p.err)) *dst = sum;
  if (d == 0 && CPATTN_IN(p.ws_span, dl, 8, p.err)) *dl = make_float2(m, l);
}

// Joins the parts of split units (see CacheWalk).  An item is 16 features of a row;
// G threads share an item's parts out, so that all of them are on the way at once,
// and meet in shared memory.  `most`: blocks of the attention's launch.
constexpr int kJoinThreads = 256;
// Items an SM from which a thread has an item's parts to itself (us, from 1024 / never, best
// and median of three runs in turn: 1024 new tokens x 17408 keys 177.7, 184.3 / 178.6, 185.8,
// 2048 tokens from an empty cache 47.8, 51.3 / 49.0, 54.2; from 300: trees of 27 x 8192 keys
// 40.0, 36.6 from 1024).
constexpr int64_t kJoinItems = 1024;
// 2^x: fp32 results take the accurate one.
template <typename T>
__device__ __forceinline__ float power2(float x) {
  if constexpr (sizeof(T) == 4) return exp2f(x);
  return ex2_approx(x);
}
// The factor f for x, sums of one part.  Where it is 0 (the part's maximum is far below
// another's, or it has no weight at all) only values that are not finite are left of x, as
// they are: add_unfinite has put them there for rows that see them, and so they reach the
// result wherever the border of two parts lies, while 0 times an infinity would be NaN.
template <int N>
__device__ __forceinline__ float join_factor(float4 (&x)[N], float f) {
  if (f != 0.f) return f;
#pragma unroll
  for (int e = 0; e < N; ++e)
    x[e] = make_float4(isfinite(x[e].x) ? 0.f : x[e].x, isfinite(x[e].y) ? 0.f : x[e].y, isfinite(x[e].z) ? 0.f : x[e].z,
                       isfinite(x[e].w) ? 0.f : x[e].w);
  return 1.f;
}
template <int R, int D, typename T, int G>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ CacheParams p, int most) {
  constexpr int I = kJoinThreads / G;   // items of a block
  __shared__ float part_sums[G][16][I];
  __shared__ float2 part_ml[G][I];
  const int item = threadIdx.x % I, g = threadIdx.x / I;
  const int hk = blockIdx.x % p.kv_heads, x = blockIdx.x / p.kv_heads;
  const int share = p.heads / p.kv_heads, b = x / p.row_tiles, rt = x - b * p.row_tiles;
  launch_wait();
  launch_next();
  const int2* at_unit = cache_unit_blocks<R, D>(p, most) + blockIdx.x;
  int2 blocks = make_int2(0, 0);
  if (CPATTN_IN(p.ws_span, at_unit, 8, p.err)) blocks = *at_unit;
  const int c0 = blocks.x, c1 = blocks.y;
  // (written by its block; or, behind a wait that ran out, not noted)
  if (c0 < 0 || c0 >= c1 || c1 >= most) return;
  {
    const int i = blockIdx.y * I + item, r = i % R, d = i / R * 16;
    const int row = cache_row(p, rt, r);
    float m = -INFINITY, l = 0.f;
    float4 sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row >= 0 && d < D)
#pragma unroll 2
      for (int c = c0 + g; c <= c1; c += G) {
        // (the first block only ends in the unit's tiles, the others begin in them)
        const int64_t part = static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0);
        const float2* at = cache_part_sums<R, D>(p, most, part, r);
        const float2 a = CPATTN_IN(p.ws_span, at, 8, p.err) ? *at : make_float2(-INFINITY, 0.f);
        float4 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4* o = cache_part<R, D>(p, part, r, d + 4 * e);
          y[e] = CPATTN_IN(p.ws_span, o, 16, p.err) ? *o : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float top = fmaxf(m, a.x), base = top == -INFINITY ? 0.f : top;
        const float f0 = power2<T>(m - base), f1 = power2<T>(a.x - base);
        m = top;
        l = l * f0 + a.y * f1;
        const float g0 = join_factor(sum, f0), g1 = join_factor(y, f1);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum[e] = make_float4(sum[e].x * g0 + y[e].x * g1, sum[e].y * g0 + y[e].y * g1, sum[e].z * g0 + y[e].z * g1,
                               sum[e].w * g0 + y[e].w * g1);
      }
    if constexpr (G == 1) {
      if (row >= 0 && d < D)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          cache_write_row<T>(p, b, hk * share + row % share, row / share, d + 4 * e, sum[e], m, l);
      return;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        part_sums[g][4 * e][item] = sum[e].x;
        part_sums[g][4 * e + 1][item] = sum[e].y;
        part_sums[g][4 * e + 2][item] = sum[e].z;
        part_sums[g][4 * e + 3][item] = sum[e].w;
      }
      part_ml[g][item] = make_float2(m, l);
    }
  }
  __syncthreads();
  // four threads an item, four features each
  for (int t = threadIdx.x; t < I * 4; t += kJoinThreads) {
    const int it = t / 4, i = blockIdx.y * I + it, r = i % R, e = t % 4 * 4, d = i / R * 16 + e;
    const int row = cache_row(p, rt, r);
    if (row < 0 || d >= D) continue;
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < G; ++k) m = fmaxf(m, part_ml[k][it].x);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const float2 a = part_ml[k][it];
      float4 y[1] = {make_float4(part_sums[k][e][it], part_sums[k][e + 1][it], part_sums[k][e + 2][it], part_sums[k][e + 3][it])};
      const float f = power2<T>(a.x - base), g = join_factor(y, f);
      l = fmaf(f, a.y, l);
      sum = make_float4(fmaf(g, y[0].x, sum.x), fmaf(g, y[0].y, sum.y), fmaf(g, y[0].z, sum.z), fmaf(g, y[0].w, sum.w));
    }
    cache_write_row<T>(p, b, hk * share + row % share, row / share, d, sum, m, l);
  }
}

// Launches the join behind an attention of `most` blocks.
template <int R, int D, typename T>
cudaError_t cache_join(const CacheParams& p, int most, cudaStream_t stream) {
  const int units = p.batch * p.row_tiles * p.kv_heads, parts = most / units + 1;
  const int64_t all = static_cast<int64_t>(units) * R * (D / 16);
  const int g = all >= kJoinItems * sm_count() ? 1 : parts <= 2 ? 2 : parts <= 4 ? 4 : 8, items = kJoinThreads / g;
  const dim3 grid(units, (R * (D / 16) + items - 1) / items);
  return launch_behind(g == 1   ? cache_join_kernel<R, D, T, 1>
                       : g == 2 ? cache_join_kernel<R, D, T, 2>
                       : g == 4 ? cache_join_kernel<R, D, T, 4>
                                : cache_join_kernel<R, D, T, 8>,
                       grid, kJoinThreads, 0, stream, p, most);
}

// bf16 inputs, row tiles of 16 or 64 rows, on `blocks` blocks
cudaError_t launch_cache_few(int head_dim, int rows, const CacheParams& p, int blocks, cudaStream_t stream);
// bf16 inputs, row tiles of 128 places (one tile of the tensor cores) or 256 (two)
struct CacheMaps {
  CUtensorMap q, k, v;   // boxes of 64 features: q's of half_rows rows, pages' of `box` rows
};
cudaError_t launch_cache_fwd(int head_dim, int places, const CacheMaps& maps, const CacheParams& p, int blocks,
                             cudaStream_t stream);
// fp32 inputs, row tiles of 16 or 64 rows
constexpr int kCacheF32Keys = 32;
cudaError_t launch_cache_f32(int head_dim, int rows, const CacheParams& p, int blocks, cudaStream_t stream);

}  // namespace cpattn
