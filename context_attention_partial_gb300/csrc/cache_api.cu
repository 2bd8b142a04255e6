// cache_api.cu -- the C ABI of the per-head norms with rotary positions and of the
// paged cache: argument validation and kernel dispatch (host code only).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "args.h"
#include "cache.cuh"
#include "internal.h"

namespace {

using namespace cpattn;

// Positions, axes and frequencies for [B, H, S, D] tensors.
cpattn_status norm_turns(const cpattn_tensor* positions, int axes, const int32_t* axis_dims, double theta,
                         int64_t B, int64_t S, int64_t D, NormParams* p) {
  if (!positions || !axis_dims) return CPATTN_ERR_NULL;
  if (positions->dtype != CPATTN_F32) return CPATTN_ERR_DTYPE;
  if (axes < 1 || axes > CPATTN_MAX_ROTARY_AXES) return CPATTN_ERR_SHAPE;
  const bool per_batch = positions->ndim == 3;
  if (!shape_ok(positions, per_batch ? 3 : 2)) return CPATTN_ERR_SHAPE;
  const int pa = per_batch ? 2 : 1;   // the axis dimension of positions
  if (positions->shape[pa] != axes || positions->shape[pa - 1] != S || (per_batch && positions->shape[0] != B))
    return CPATTN_ERR_SHAPE;
  int64_t turned = 0;
  for (int a = 0; a < axes; ++a) {
    if (axis_dims[a] < 2 || axis_dims[a] % 2 != 0) return CPATTN_ERR_SHAPE;
    turned += axis_dims[a];
  }
  if (turned > D) return CPATTN_ERR_SHAPE;
  if (D > CPATTN_MAX_ROTARY_DIM) return CPATTN_ERR_UNSUPPORTED;
  if (B * S > 0 && !positions->data) return CPATTN_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(positions->data) & 3u) return CPATTN_ERR_LAYOUT;
  for (int i = 0; i < positions->ndim; ++i)
    if (positions->stride[i] < 0) return CPATTN_ERR_LAYOUT;
  p->pos = static_cast<const float*>(positions->data);
  p->pos_sb = per_batch ? positions->stride[0] : 0;
  p->pos_ss = positions->stride[pa - 1];
  p->pos_sa = positions->stride[pa];
  p->pos_span = {positions->data, extent_bytes(positions)};
  fill_turns(*p, axes, axis_dims, theta);
  return CPATTN_OK;
}

// A [D] tensor of weights, or of their gradient.
cpattn_status norm_weight(const cpattn_tensor* w, int32_t dtype, int64_t D) {
  if (w->dtype != dtype || !dtype_known(dtype)) return CPATTN_ERR_DTYPE;
  if (!shape_ok(w, 1) || w->shape[0] != D) return CPATTN_ERR_SHAPE;
  if (D > 0 && !w->data) return CPATTN_ERR_NULL;
  if ((D > 1 && w->stride[0] != 1) || reinterpret_cast<uintptr_t>(w->data) % elem_bytes(dtype) != 0)
    return CPATTN_ERR_LAYOUT;
  return CPATTN_OK;
}

// B, S, D of x[0] for all of x; types, shapes, heads and the sizes that kernels take.
cpattn_status norm_shapes(int n, const cpattn_tensor* x, int64_t* B, int64_t* S, int64_t* D, int64_t* heads) {
  if (!dtype_known(x[0].dtype)) return CPATTN_ERR_DTYPE;
  for (int i = 0; i < n; ++i)
    if (x[i].dtype != x[0].dtype) return CPATTN_ERR_DTYPE;
  for (int i = 0; i < n; ++i)
    if (!shape_ok(&x[i], 4) || x[i].shape[0] != x[0].shape[0] || x[i].shape[2] != x[0].shape[2] ||
        x[i].shape[3] != x[0].shape[3])
      return CPATTN_ERR_SHAPE;
  *B = x[0].shape[0];
  *S = x[0].shape[2];
  *D = x[0].shape[3];
  if (*D < 1) return CPATTN_ERR_SHAPE;
  if (*D > CPATTN_MAX_ROTARY_DIM || (*D * elem_bytes(x[0].dtype)) % 16 != 0) return CPATTN_ERR_UNSUPPORTED;
  *heads = 0;
  for (int i = 0; i < n; ++i) {
    if (x[i].shape[1] > 65535) return CPATTN_ERR_UNSUPPORTED;
    *heads += x[i].shape[1];
  }
  if (*heads > 65535 || *B > 65535 || *S > (int64_t(1) << 30)) return CPATTN_ERR_UNSUPPORTED;
  return CPATTN_OK;
}

// In place only element for element.
bool same_place(const cpattn_tensor* a, const cpattn_tensor* b) {
  for (int j = 0; j < 4; ++j)
    if (a->shape[j] > 1 && a->stride[j] != b->stride[j]) return false;
  return true;
}

void strides(const cpattn_tensor* t, int64_t* s) {
  for (int i = 0; i < 3; ++i) s[i] = t->stride[i];
}

cpattn_status status_of(cudaError_t e) { return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA; }

InDtype type_of(const cpattn_tensor* t) { return t->dtype == CPATTN_BF16 ? InDtype::BF16 : InDtype::F32; }

float eps_of(float eps) { return eps >= 0.f && std::isfinite(eps) ? eps : 1e-6f; }

// Both directions' checks; *run: whether there is a row.
cpattn_status norm_common(int n, const cpattn_tensor* x, const cpattn_tensor* weights, float eps,
                          const cpattn_tensor* positions, int axes, const int32_t* axis_dims, double theta,
                          int interleaved, const cpattn_tensor* y, NormParams* p, bool* run) {
  if (n < 1 || n > kMaxPermuteBatch) return CPATTN_ERR_SHAPE;
  if (!x || !y || !positions || !axis_dims) return CPATTN_ERR_NULL;
  std::memset(p, 0, sizeof(*p));
  int64_t B, S, D, heads;
  cpattn_status st = norm_shapes(n, x, &B, &S, &D, &heads);
  if (st != CPATTN_OK) return st;
  if ((st = norm_turns(positions, axes, axis_dims, theta, B, S, D, p)) != CPATTN_OK) return st;
  const long long shrink = g_check_shrink.load();
  for (int i = 0; i < n; ++i) {
    if (y[i].dtype != x[0].dtype) return CPATTN_ERR_DTYPE;
    if (!shape_ok(&y[i], 4) || !same_shape(&x[i], &y[i], 4)) return CPATTN_ERR_SHAPE;
    NormTensor& t = p->t[i];
    if (weights) {
      if ((st = norm_weight(&weights[i], weights[0].dtype, D)) != CPATTN_OK) return st;
      t.w = weights[i].data;
      t.w_span = {t.w, extent_bytes(&weights[i])};
      p->w_f32 = weights[0].dtype == CPATTN_F32;
    }
    p->head_start[i + 1] = p->head_start[i] + static_cast<int>(x[i].shape[1]);
    t.norm = t.turn = 1;
    if (B * S * x[i].shape[1] == 0) continue;
    if (!x[i].data || !y[i].data) return CPATTN_ERR_NULL;
    if (!layout_ok(&x[i]) || !layout_distinct(&y[i])) return CPATTN_ERR_LAYOUT;
    if (x[i].data == y[i].data && !same_place(&x[i], &y[i])) return CPATTN_ERR_LAYOUT;
    t.x = x[i].data;
    t.y = y[i].data;
    strides(&x[i], t.x_s);
    strides(&y[i], t.y_s);
    t.x_span = {x[i].data, extent_bytes(&x[i])};
    t.y_span = {y[i].data, extent_bytes(&y[i], shrink)};
  }
  p->n = n;
  p->batch = static_cast<int>(B);
  p->seq = static_cast<int>(S);
  p->head_dim = static_cast<int>(D);
  p->interleaved = interleaved != 0;
  p->eps = eps_of(eps);
  p->err = device_error_word();
  *run = B * S * heads > 0;
  return CPATTN_OK;
}

size_t norm_workspace(int n, const cpattn_tensor* x, int64_t B, int64_t S, int64_t D, int64_t heads) {
  return static_cast<size_t>(norm_backward_parts(type_of(x), static_cast<int>(D), B * S, heads)) * n * D * 4;
}

// The cache's pages, table, lengths and counts for B sequences with pages like
// [*, heads, *, D] of `dtype`.  (new tokens: whether any page is touched)
cpattn_status cache_common(const cpattn_tensor* key_pages, const cpattn_tensor* value_pages,
                           const cpattn_tensor* page_table, const cpattn_tensor* lengths, const cpattn_tensor* counts,
                           int32_t dtype, int64_t B, int64_t heads, int64_t D, bool run, PageTable* c) {
  if (!key_pages || !value_pages || !page_table || !lengths) return CPATTN_ERR_NULL;
  if (key_pages->dtype != dtype || value_pages->dtype != dtype || page_table->dtype != CPATTN_I32 ||
      lengths->dtype != CPATTN_I32 || (counts && counts->dtype != CPATTN_I32))
    return CPATTN_ERR_DTYPE;
  if (!shape_ok(key_pages, 4) || !shape_ok(value_pages, 4) || !same_shape(key_pages, value_pages, 4) ||
      !shape_ok(page_table, 2) || !shape_ok(lengths, 1) || (counts && !shape_ok(counts, 1)))
    return CPATTN_ERR_SHAPE;
  if (key_pages->shape[1] != heads || key_pages->shape[3] != D || page_table->shape[0] != B ||
      lengths->shape[0] != B || (counts && counts->shape[0] != B))
    return CPATTN_ERR_SHAPE;
  const int64_t pages = key_pages->shape[0], rows = key_pages->shape[2], width = page_table->shape[1];
  if (rows < CPATTN_MIN_PAGE || rows > CPATTN_MAX_PAGE || (rows & (rows - 1)) != 0) return CPATTN_ERR_UNSUPPORTED;
  if (pages > 0x7fffffff || width * rows > (int64_t(1) << 30)) return CPATTN_ERR_UNSUPPORTED;
  if (run) {
    if (!lengths->data || (counts && !counts->data) || (width > 0 && !page_table->data)) return CPATTN_ERR_NULL;
    if (pages > 0 && (!key_pages->data || !value_pages->data)) return CPATTN_ERR_NULL;
    if (pages > 0 && (!layout_distinct(key_pages) || !layout_distinct(value_pages))) return CPATTN_ERR_LAYOUT;
    for (const cpattn_tensor* t : {lengths, counts})
      if (t && ((B > 1 && t->stride[0] != 1) || (reinterpret_cast<uintptr_t>(t->data) & 3u))) return CPATTN_ERR_LAYOUT;
    if ((width > 1 && page_table->stride[1] != 1) || (B > 1 && page_table->stride[0] < 0) ||
        (reinterpret_cast<uintptr_t>(page_table->data) & 3u))
      return CPATTN_ERR_LAYOUT;
  }
  c->table = static_cast<const int32_t*>(page_table->data);
  c->lengths = static_cast<const int32_t*>(lengths->data);
  c->counts = counts ? static_cast<const int32_t*>(counts->data) : nullptr;
  c->stride = B > 1 ? page_table->stride[0] : 0;
  c->width = static_cast<int>(width);
  c->shift = 0;
  while ((int64_t(1) << c->shift) < rows) ++c->shift;
  c->pages = static_cast<int>(pages);
  c->table_span = {page_table->data, extent_bytes(page_table)};
  c->lengths_span = {lengths->data, extent_bytes(lengths)};
  if (counts) c->counts_span = {counts->data, extent_bytes(counts)};
  return CPATTN_OK;
}

// How an attention to a cache is run; the same for every cache of these sizes, whatever
// its lengths are.
struct CachePlan {
  int places, keys;      // of a row tile (see CacheParams), keys of a key tile
  int tile_rows, half_rows;
  int row_tiles;         // of a key head
  int blocks, split;     // see CacheWalk
  size_t workspace;
};

cpattn_status cache_shape(const cpattn_tensor* q, const cpattn_tensor* key_pages, const cpattn_tensor* page_table) {
  if (!dtype_known(q->dtype) || key_pages->dtype != q->dtype || page_table->dtype != CPATTN_I32) return CPATTN_ERR_DTYPE;
  if (!shape_ok(q, 4) || !shape_ok(key_pages, 4) || !shape_ok(page_table, 2)) return CPATTN_ERR_SHAPE;
  const int64_t B = q->shape[0], H = q->shape[1], S = q->shape[2], D = q->shape[3], Hk = key_pages->shape[1];
  if (key_pages->shape[3] != D || page_table->shape[0] != B || (H > 0 && Hk == 0)) return CPATTN_ERR_SHAPE;
  if (Hk > 0 && H % Hk != 0) return CPATTN_ERR_DIVISIBILITY;
  if (D != 64 && D != 128) return CPATTN_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || Hk > 65535 || S > (int64_t(1) << 24)) return CPATTN_ERR_UNSUPPORTED;
  // (row numbers, and blocks of the join's launch)
  if (S * H > (int64_t(1) << 30) || B * Hk * ((Hk > 0 ? S * (H / Hk) : 0) / 16 + 1) > 0x7fff0000)
    return CPATTN_ERR_UNSUPPORTED;
  return CPATTN_OK;
}

// Whether a bf16 call goes to the tensor cores' 128-row tiles: more than 16 rows a key
// head (us, cache_few.cu's kernel / the tensor cores': 8 sequences x 8 key heads x 8192
// keys, D = 128: 16 rows 49.8 / 50.5, 24 rows 73.8 / 50.7, 64 rows 76.6 / 51.5; one
// sequence of 1000 keys: 4 rows 10.3 / 11.4, 16 rows 11.6 / 11.8, 24 rows 14.9 / 11.8;
// D = 64, 4 sequences x 24 key heads x 4000 keys: 1 row 26.5 / 27.4, 16 rows 29.9 / 27.6,
// 24 rows 46.6 / 27.7, x 16384 keys: 1 row 65.5 / 69.7, 16 rows 68.3 / 69.6).  A token's
// rows have to fit a tile.
bool cache_many(const cpattn_tensor* q, const cpattn_tensor* key_pages) {
  const int64_t share = q->shape[1] / key_pages->shape[1], rows = q->shape[2] * share;
  return rows > 16 && share <= 128 && key_pages->shape[0] > 0;
}

// Queries as the tensor cores' tiles take them: dims (D, H, S, B), boxes of 64 features,
// the heads that share a key head, and `tokens` tokens.
cpattn_status query_map(CUtensorMap* m, const cpattn_tensor* q, int share, int tokens) {
  const EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return CPATTN_ERR_CUDA;
  const int64_t B = q->shape[0], H = q->shape[1], S = q->shape[2], D = q->shape[3];
  const int64_t sh = tma_stride(q, 1, D), ss = tma_stride(q, 2, D), sb = tma_stride(q, 0, D);
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)(sh * 2), (cuuint64_t)(ss * 2), (cuuint64_t)(sb * 2)};
  const cuuint32_t box[4] = {64u, (cuuint32_t)share, (cuuint32_t)tokens, 1u}, step[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q->data, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}

CachePlan cache_plan(const cpattn_tensor* q, const cpattn_tensor* key_pages, const cpattn_tensor* page_table) {
  CachePlan c = {};
  const int64_t B = q->shape[0], H = q->shape[1], S = q->shape[2], D = q->shape[3], Hk = key_pages->shape[1];
  if (B * H * S == 0) return c;
  const int64_t rows = S * (H / Hk);
  // (blocks of an SM: bf16 with D = 64 has room for three; us, three / two: 4 sequences x
  // 24 key heads x 16384 keys, one row 66.1 / 77.2, 16 rows in pages of 16 69.5 / 79.8)
  int64_t slots = (q->dtype == CPATTN_BF16 && D == 64 ? 3 : 2) * static_cast<int64_t>(sm_count());
  if (q->dtype == CPATTN_F32) {
    c.places = rows <= 16 ? 16 : 64;
    c.keys = kCacheF32Keys;
  } else if (cache_many(q, key_pages)) {
    // whole tokens of up to 128 rows, in one or two tiles of the tensor cores
    c.half_rows = static_cast<int>(128 / (H / Hk) * (H / Hk));
    c.places = rows <= c.half_rows ? 128 : 256;
    c.tile_rows = c.places / 128 * c.half_rows;
    c.keys = 128;
    slots = sm_count();
  } else {
    c.places = rows <= 16 ? 16 : 64;
    c.keys = 64;
  }
  if (c.tile_rows == 0) c.tile_rows = c.half_rows = c.places;
  c.row_tiles = static_cast<int>((rows + c.tile_rows - 1) / c.tile_rows);
  const int64_t units = B * c.row_tiles * Hk;
  const int64_t most = (page_table->shape[1] * key_pages->shape[2] + S + c.keys - 1) / c.keys;   // key tiles of a unit
  const int64_t least = cache_min_tiles(c.places, c.keys);
  c.split = most > least && units < kCacheWholeUnits * slots && units * (most + cache_unit_cost(c.keys)) < 0x7fffffff;
  const int64_t want = c.split ? (units * (most + cache_unit_cost(c.keys)) + least - 1) / least : units;
  c.blocks = static_cast<int>(want < slots ? want : slots);
  c.workspace = c.split ? static_cast<size_t>(c.blocks) * 2 * c.places * (D + 2) * 4 + units * 8 : 0;
  return c;
}

CrossTensor cache_tensor(const cpattn_tensor* t, long long shrink = 0) {
  return {t->data, {t->stride[0], t->stride[1], t->stride[2]}, {t->data, extent_bytes(t, shrink)}};
}

}  // namespace

extern "C" {

cpattn_status cpattn_norm_rotary(int n, const cpattn_tensor* x, const cpattn_tensor* weights, float eps,
                                 const cpattn_tensor* positions, int axes, const int32_t* axis_dims, double theta,
                                 int interleaved, cpattn_tensor* y, void* stream) {
  NormParams p;
  bool run = false;
  const cpattn_status st =
      norm_common(n, x, weights, eps, positions, axes, axis_dims, theta, interleaved, y, &p, &run);
  if (st != CPATTN_OK || !run) return st;
  return status_of(launch_norm_rotary(type_of(x), p, static_cast<cudaStream_t>(stream)));
}

size_t cpattn_norm_rotary_backward_workspace_bytes(int n, const cpattn_tensor* x) {
  int64_t B, S, D, heads;
  if (n < 1 || n > kMaxPermuteBatch || !x || norm_shapes(n, x, &B, &S, &D, &heads) != CPATTN_OK) return 0;
  return norm_workspace(n, x, B, S, D, heads);
}

cpattn_status cpattn_norm_rotary_backward(int n, const cpattn_tensor* x, const cpattn_tensor* weights, float eps,
                                          const cpattn_tensor* positions, int axes, const int32_t* axis_dims,
                                          double theta, int interleaved, const cpattn_tensor* dy, cpattn_tensor* dx,
                                          cpattn_tensor* dweights, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  NormParams p;
  bool run = false;
  cpattn_status st = norm_common(n, x, weights, eps, positions, axes, axis_dims, theta, interleaved, dx, &p, &run);
  if (st != CPATTN_OK) return st;
  if (!dy || !weights != !dweights) return CPATTN_ERR_NULL;
  const int64_t B = p.batch, S = p.seq, D = p.head_dim;
  const long long shrink = g_check_shrink.load();
  for (int i = 0; i < n; ++i) {
    if (dy[i].dtype != x[0].dtype) return CPATTN_ERR_DTYPE;
    if (!shape_ok(&dy[i], 4) || !same_shape(&x[i], &dy[i], 4)) return CPATTN_ERR_SHAPE;
    NormTensor& t = p.t[i];
    if (weights) {
      if ((st = norm_weight(&dweights[i], weights[0].dtype, D)) != CPATTN_OK) return st;
      t.dw = dweights[i].data;
      t.dw_span = {t.dw, extent_bytes(&dweights[i], shrink)};
    }
    if (B * S * x[i].shape[1] == 0) continue;
    if (!dy[i].data) return CPATTN_ERR_NULL;
    if (!layout_ok(&dy[i])) return CPATTN_ERR_LAYOUT;
    if (dy[i].data == dx[i].data && !same_place(&dy[i], &dx[i])) return CPATTN_ERR_LAYOUT;
    t.dy = dy[i].data;
    strides(&dy[i], t.dy_s);
    t.dy_span = {dy[i].data, extent_bytes(&dy[i])};
  }
  if (!run && !weights) return CPATTN_OK;
  const size_t need = weights ? norm_workspace(n, x, B, S, D, p.head_start[n]) : 0;
  if (need > 0) {
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return CPATTN_ERR_WORKSPACE;
    p.ws = static_cast<float*>(workspace);
    p.ws_span = {workspace, need > static_cast<size_t>(shrink) ? need - shrink : 0};
  }
  return status_of(launch_norm_backward(type_of(x), p, static_cast<cudaStream_t>(stream)));
}

cpattn_status cpattn_cache_append(const cpattn_tensor* q, const cpattn_tensor* k, const cpattn_tensor* v,
                                  const cpattn_tensor* q_weight, const cpattn_tensor* k_weight, float eps,
                                  const cpattn_tensor* positions, int axes, const int32_t* axis_dims, double theta,
                                  int interleaved, cpattn_tensor* key_pages, cpattn_tensor* value_pages,
                                  const cpattn_tensor* page_table, const cpattn_tensor* lengths,
                                  const cpattn_tensor* counts, cpattn_tensor* q_out, void* stream) {
  if (!k || !v || !q != !q_out) return CPATTN_ERR_NULL;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  // (queries first: where the keys go takes a while to find)
  cpattn_tensor in[3];
  const int n = q ? 3 : 2, key = n - 2;
  if (q) in[0] = *q;
  in[key] = *k;
  in[key + 1] = *v;
  int64_t B, S, D, heads;
  cpattn_status st = norm_shapes(n, in, &B, &S, &D, &heads);
  if (st != CPATTN_OK) return st;
  if (k->shape[1] != v->shape[1]) return CPATTN_ERR_SHAPE;
  if (positions && (st = norm_turns(positions, axes, axis_dims, theta, B, S, D, &p)) != CPATTN_OK) return st;
  const bool run = B * S * heads > 0;
  if ((st = cache_common(key_pages, value_pages, page_table, lengths, counts, k->dtype, B, k->shape[1], D, run,
                         &p.cache)) != CPATTN_OK)
    return st;
  const cpattn_tensor* weights[3] = {};
  cpattn_tensor* out[3] = {};
  if (q) {
    weights[0] = q_weight;
    out[0] = q_out;
  }
  weights[key] = k_weight;
  out[key] = key_pages;
  out[key + 1] = value_pages;
  const long long shrink = g_check_shrink.load();
  for (int i = 0; i < n; ++i) {
    NormTensor& t = p.t[i];
    if (weights[i]) {
      // (of one type, so that one kernel reads them)
      if (i < key && k_weight && q_weight->dtype != k_weight->dtype) return CPATTN_ERR_DTYPE;
      if ((st = norm_weight(weights[i], weights[i]->dtype, D)) != CPATTN_OK) return st;
      t.w = weights[i]->data;
      t.w_span = {t.w, extent_bytes(weights[i])};
      p.w_f32 = weights[i]->dtype == CPATTN_F32;
      t.norm = 1;
    }
    t.turn = i <= key && positions;
    t.paged = i >= key;
    p.head_start[i + 1] = p.head_start[i] + static_cast<int>(in[i].shape[1]);
    if (!t.paged) {
      if (q_out->dtype != q->dtype) return CPATTN_ERR_DTYPE;
      if (!shape_ok(q_out, 4) || !same_shape(q, q_out, 4)) return CPATTN_ERR_SHAPE;
    }
    if (B * S * in[i].shape[1] == 0) continue;
    if (!in[i].data || (!t.paged && !q_out->data)) return CPATTN_ERR_NULL;
    if (!layout_ok(&in[i]) || (!t.paged && !layout_distinct(q_out))) return CPATTN_ERR_LAYOUT;
    if (!t.paged && q->data == q_out->data && !same_place(q, q_out)) return CPATTN_ERR_LAYOUT;
    t.x = in[i].data;
    t.y = out[i]->data;
    strides(&in[i], t.x_s);
    strides(out[i], t.y_s);
    t.x_span = {in[i].data, extent_bytes(&in[i])};
    t.y_span = {out[i]->data, extent_bytes(out[i], shrink)};
  }
  if (!run) return CPATTN_OK;
  if (key_pages->data == value_pages->data && key_pages->data) return CPATTN_ERR_LAYOUT;   // (two writers)
  p.n = n;
  p.batch = static_cast<int>(B);
  p.seq = static_cast<int>(S);
  p.head_dim = static_cast<int>(D);
  p.interleaved = interleaved != 0;
  p.eps = eps_of(eps);
  p.err = device_error_word();
  return status_of(launch_norm_rotary(type_of(k), p, static_cast<cudaStream_t>(stream)));
}

size_t cpattn_cache_attention_workspace_bytes(const cpattn_tensor* q, const cpattn_tensor* key_pages,
                                             const cpattn_tensor* page_table) {
  if (!q || !key_pages || !page_table || cache_shape(q, key_pages, page_table) != CPATTN_OK) return 0;
  return cache_plan(q, key_pages, page_table).workspace;
}

cpattn_status cpattn_cache_attention(const cpattn_tensor* q, const cpattn_tensor* key_pages,
                                     const cpattn_tensor* value_pages, const cpattn_tensor* page_table,
                                     const cpattn_tensor* lengths, const cpattn_tensor* counts,
                                     const cpattn_tensor* parents, float scale, cpattn_tensor* out,
                                     cpattn_tensor* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !key_pages || !value_pages || !page_table || !lengths || !out || !lse) return CPATTN_ERR_NULL;
  if (out->dtype != q->dtype || lse->dtype != CPATTN_F32 || (parents && parents->dtype != CPATTN_I32))
    return CPATTN_ERR_DTYPE;
  cpattn_status st = cache_shape(q, key_pages, page_table);
  if (st != CPATTN_OK) return st;
  if (!shape_ok(out, 4) || !same_shape(out, q, 4) || !shape_ok(lse, 3) || !same_shape(lse, q, 3)) return CPATTN_ERR_SHAPE;
  const int64_t B = q->shape[0], H = q->shape[1], S = q->shape[2], D = q->shape[3];
  const bool run = B * H * S > 0;
  CacheParams p;
  std::memset(&p, 0, sizeof(p));
  if ((st = cache_common(key_pages, value_pages, page_table, lengths, counts, q->dtype, B, key_pages->shape[1], D, run,
                         &p.cache)) != CPATTN_OK)
    return st;
  if (parents) {
    if (!shape_ok(parents, 2) || parents->shape[0] != B || parents->shape[1] != S) return CPATTN_ERR_SHAPE;
    if (S > CPATTN_MAX_TREE) return CPATTN_ERR_UNSUPPORTED;
    if (run && !parents->data) return CPATTN_ERR_NULL;
    if (run && ((S > 1 && parents->stride[1] != 1) || (B > 1 && parents->stride[0] < 0) ||
                (reinterpret_cast<uintptr_t>(parents->data) & 3u)))
      return CPATTN_ERR_LAYOUT;
    p.parents = static_cast<const int32_t*>(parents->data);
    p.parents_stride = B > 1 ? parents->stride[0] : 0;
    p.parents_span = {parents->data, extent_bytes(parents)};
  }
  if (!run) return CPATTN_OK;
  if (!q->data || !out->data || !lse->data) return CPATTN_ERR_NULL;
  if (!layout_distinct(q) || !layout_distinct(out) || !lse_layout_ok(lse)) return CPATTN_ERR_LAYOUT;
  const CachePlan plan = cache_plan(q, key_pages, page_table);
  if (plan.workspace > 0 && (!workspace || workspace_bytes < plan.workspace || !aligned16(workspace)))
    return CPATTN_ERR_WORKSPACE;
  const long long shrink = g_check_shrink.load();
  p.ws = static_cast<float*>(workspace);
  p.ws_span = {workspace, plan.workspace > static_cast<size_t>(shrink) ? plan.workspace - shrink : 0};
  p.q = cache_tensor(q);
  p.k = cache_tensor(key_pages);
  p.v = cache_tensor(value_pages);
  p.out = cache_tensor(out, shrink);
  p.lse = cache_tensor(lse, shrink);
  p.batch = static_cast<int>(B);
  p.heads = static_cast<int>(H);
  p.kv_heads = static_cast<int>(key_pages->shape[1]);
  p.s_q = static_cast<int>(S);
  p.row_tiles = plan.row_tiles;
  p.tile_rows = plan.tile_rows;
  p.half_rows = plan.half_rows;
  p.split = plan.split;
  if (!(scale > 0.f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.timeout_ns = g_timeout_ns.load();
  p.fault_skip_kv = g_fault_skip_kv.load();
  p.err = device_error_word();
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int head_dim = static_cast<int>(D);
  if (q->dtype == CPATTN_F32) return status_of(launch_cache_f32(head_dim, plan.places, p, plan.blocks, cs));
  if (!cache_many(q, key_pages)) return status_of(launch_cache_few(head_dim, plan.places, p, plan.blocks, cs));
  const int share = static_cast<int>(H / key_pages->shape[1]), page = static_cast<int>(key_pages->shape[2]);
  CacheMaps m;
  if ((st = query_map(&m.q, q, share, 128 / share)) != CPATTN_OK) return st;
  if ((st = make_tmap(&m.k, key_pages, page < 128 ? page : 128)) != CPATTN_OK) return st;
  if ((st = make_tmap(&m.v, value_pages, page < 128 ? page : 128)) != CPATTN_OK) return st;
  return status_of(launch_cache_fwd(head_dim, plan.places, m, p, plan.blocks, cs));
}

}  // extern "C"
