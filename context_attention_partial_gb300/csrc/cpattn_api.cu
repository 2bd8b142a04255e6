// cpattn_api.cu -- the C ABI of libcpattn.so: argument validation, the ring
// chunk partition, TMA descriptor encoding and kernel dispatch.  Host code
// only; every step of the computation runs in the kernels.
//
// Validation rules (page title, section):
//   Diffusers "Context parallelism", variants table: Ring needs the sequence
//   length divisible by ring_degree, Ulysses needs the head count divisible
//   by ulysses_degree; "Ring Anything Attention" lifts the first rule and
//   takes no mask.  diffusers _modeling_parallel.py ContextParallelConfig:
//   degrees must be >= 1.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "args.h"
#include "cross.cuh"
#include "internal.h"

namespace cpattn {

std::atomic<unsigned long long> g_timeout_ns{2000000000ull};
std::atomic<int> g_fault_skip_kv{0};
std::atomic<long long> g_check_shrink{0};   // testing: output extents shrunk by this many bytes

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

cpattn_status make_tmap(CUtensorMap* m, const cpattn_tensor* t, int box_rows, bool half_rows) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return CPATTN_ERR_CUDA;
  const int eb = elem_bytes(t->dtype);
  const int64_t B = t->shape[0], H = t->shape[1], S = t->shape[2], D = t->shape[3];
  const int64_t ss = tma_stride(t, 2, D);
  const int64_t sh = tma_stride(t, 1, ss * S);
  const int64_t sb = tma_stride(t, 0, sh * H);
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)S, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)(ss * eb), (cuuint64_t)(sh * eb),
                                 (cuuint64_t)(sb * eb)};
  const cuuint32_t box[4] = {(cuuint32_t)((half_rows ? 64 : 128) / eb), (cuuint32_t)box_rows, 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUtensorMapDataType dt =
      t->dtype == CPATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = enc(m, dt, 4, t->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         half_rows ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CPATTN_OK : CPATTN_ERR_CUDA;
}

}  // namespace cpattn

namespace {

using namespace cpattn;

// Key partition of the ring (plain: S/R each; Ring Anything: the first
// S mod R chunks one longer).
cpattn_status ring_partition(int64_t s_kv, int ring_degree, int ring_anything, int* start) {
  if (ring_degree < 1) return CPATTN_ERR_SHAPE;
  if (ring_degree > CPATTN_MAX_RING_DEGREE) return CPATTN_ERR_UNSUPPORTED;
  if (!ring_anything && s_kv % ring_degree != 0) return CPATTN_ERR_DIVISIBILITY;
  if (ring_anything && ring_degree > s_kv) return CPATTN_ERR_SHAPE;
  const int64_t len = s_kv / ring_degree, longer = s_kv % ring_degree;
  int64_t pos = 0;
  for (int c = 0; c < ring_degree; ++c) {
    start[c] = static_cast<int>(pos);
    pos += len + (c < longer ? 1 : 0);
  }
  start[ring_degree] = static_cast<int>(pos);
  return CPATTN_OK;
}

size_t workspace_bytes_for(int64_t B, int64_t H, int64_t S, int64_t D, int ring_degree) {
  if (ring_degree <= 1) return 0;
  // [B*H*ceil(S/128) query tiles][128 rows][D + 1] floats
  const int64_t rows = B * H * ((S + 127) / 128) * 128;
  return static_cast<size_t>(rows) * static_cast<size_t>(D + 1) * sizeof(float);
}

cpattn_status check_qkv(const cpattn_tensor* q, const cpattn_tensor* k, const cpattn_tensor* v) {
  if (!q || !k || !v) return CPATTN_ERR_NULL;
  if (!dtype_known(q->dtype) || k->dtype != q->dtype || v->dtype != q->dtype)
    return CPATTN_ERR_DTYPE;
  if (!shape_ok(q, 4) || !shape_ok(k, 4) || !shape_ok(v, 4)) return CPATTN_ERR_SHAPE;
  for (int i = 0; i < 4; ++i)
    if (k->shape[i] != v->shape[i]) return CPATTN_ERR_SHAPE;
  if (q->shape[0] != k->shape[0] || q->shape[1] != k->shape[1] || q->shape[3] != k->shape[3])
    return CPATTN_ERR_SHAPE;
  const bool empty_q = q->shape[0] == 0 || q->shape[1] == 0 || q->shape[2] == 0;
  if (!empty_q && k->shape[2] == 0) return CPATTN_ERR_SHAPE;
  if (!empty_q && (!q->data || !k->data || !v->data)) return CPATTN_ERR_NULL;
  return CPATTN_OK;
}

cpattn_status run_attention(const cpattn_tensor* q, const cpattn_tensor* k,
                            const cpattn_tensor* v, float scale, int ring_degree,
                            int ring_anything, cpattn_tensor* out, cpattn_tensor* lse,
                            void* workspace, size_t workspace_bytes, bool out_f32,
                            bool causal, cudaStream_t stream, int group_count = 0,
                            int group_heads = 0) {
  cpattn_status st = check_qkv(q, k, v);
  if (st != CPATTN_OK) return st;
  if (!out || !lse) return CPATTN_ERR_NULL;
  const int32_t want_out = out_f32 ? CPATTN_F32 : q->dtype;
  if (out->dtype != want_out || lse->dtype != CPATTN_F32) return CPATTN_ERR_DTYPE;
  if (!shape_ok(out, 4) || !shape_ok(lse, 3)) return CPATTN_ERR_SHAPE;
  for (int i = 0; i < 4; ++i)
    if (out->shape[i] != q->shape[i]) return CPATTN_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (lse->shape[i] != q->shape[i]) return CPATTN_ERR_SHAPE;
  const int64_t B = q->shape[0], H = q->shape[1], S_q = q->shape[2], S_kv = k->shape[2],
                D = q->shape[3];
  int chunk_start[CPATTN_MAX_RING_DEGREE + 1];
  if (ring_degree < 1) return CPATTN_ERR_SHAPE;
  if (ring_degree > CPATTN_MAX_RING_DEGREE) return CPATTN_ERR_UNSUPPORTED;
  const bool empty_q = B == 0 || H == 0 || S_q == 0;
  if (!empty_q) {
    st = ring_partition(S_kv, ring_degree, ring_anything, chunk_start);
    if (st != CPATTN_OK) return st;
  } else if (!ring_anything && S_kv % ring_degree != 0) {
    return CPATTN_ERR_DIVISIBILITY;
  }
  const bool supported = D == 64 || D == 128;
  if (!supported) return CPATTN_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || S_q > (int64_t(1) << 30) || S_kv > (int64_t(1) << 30))
    return CPATTN_ERR_UNSUPPORTED;
  if (empty_q) return CPATTN_OK;
  if (!out->data || !lse->data) return CPATTN_ERR_NULL;
  if (!layout_ok(q) || !layout_ok(k) || !layout_ok(v) || !layout_ok(out)) return CPATTN_ERR_LAYOUT;
  if (lse->shape[2] > 1 && lse->stride[2] != 1) return CPATTN_ERR_LAYOUT;
  if ((reinterpret_cast<uintptr_t>(lse->data) & 3u) != 0) return CPATTN_ERR_LAYOUT;
  const size_t need = workspace_bytes_for(B, H, S_q, D, ring_degree);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
    return CPATTN_ERR_WORKSPACE;

  const InDtype dt = q->dtype == CPATTN_BF16 ? InDtype::BF16 : InDtype::F32;
  const int kv_rows = cpattn::attn_kv_tile_rows(dt, static_cast<int>(D));
  CUtensorMap tm_q, tm_k, tm_v;
  if ((st = make_tmap(&tm_q, q, 128)) != CPATTN_OK) return st;
  if ((st = make_tmap(&tm_k, k, kv_rows)) != CPATTN_OK) return st;
  if ((st = make_tmap(&tm_v, v, kv_rows)) != CPATTN_OK) return st;

  cpattn::AttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.out = out->data;
  p.out_sb = out->stride[0];
  p.out_sh = out->stride[1];
  p.out_ss = out->stride[2];
  p.lse = static_cast<float*>(lse->data);
  p.lse_sb = lse->stride[0];
  p.lse_sh = lse->stride[1];
  p.lse_ss = lse->stride[2];
  if (need > 0) {
    p.ws_o = static_cast<float*>(workspace);
    p.ws_lse = p.ws_o + B * H * ((S_q + 127) / 128) * 128 * D;
  }
  const long long shrink = g_check_shrink.load();
  p.out_span = {out->data, extent_bytes(out, shrink)};
  p.lse_span = {lse->data, extent_bytes(lse, shrink)};
  p.ws_span = {workspace, need > static_cast<size_t>(shrink) ? need - shrink : 0};
  p.batch = static_cast<int>(B);
  p.heads = static_cast<int>(H);
  p.s_q = static_cast<int>(S_q);
  p.s_kv = static_cast<int>(S_kv);
  if (!(scale > 0.f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.ring_degree = ring_degree;
  p.out_f32 = out->dtype == CPATTN_F32 ? 1 : 0;
  p.timeout_ns = g_timeout_ns.load();
  p.fault_skip_kv = g_fault_skip_kv.load();
  p.causal = causal ? 1 : 0;
  p.group_count = group_count;
  p.group_heads = group_heads;
  for (int c = 0; c <= ring_degree; ++c) p.chunk_start[c] = chunk_start[c];
  p.n_tiles_all = 0;
  for (int c = 0; c < ring_degree; ++c)
    p.n_tiles_all += (chunk_start[c + 1] - chunk_start[c] + kv_rows - 1) / kv_rows;
  const cudaError_t e =
      cpattn::launch_attention(dt, static_cast<int>(D), tm_q, tm_k, tm_v, p, stream);
  return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

// One Ulysses regroup pair x -> y (even: [B,S,H,D] <-> [G,B,S,H/G,D];
// Ulysses Anything: [B,S,H,D] <-> [G,B,S,ceil(H/G),D]).  Fills dims with
// (B, S, H, D) and bytes with the sizes of x and y.
cpattn_status permute_pair_check(const cpattn_tensor* x, const cpattn_tensor* y, int degree,
                                 int dir, bool anything, int64_t* dims, uintptr_t* xbytes,
                                 uintptr_t* ybytes) {
  if (!x || !y) return CPATTN_ERR_NULL;
  if (!dtype_known(x->dtype) || y->dtype != x->dtype) return CPATTN_ERR_DTYPE;
  if (dir != 1 && dir != -1) return CPATTN_ERR_SHAPE;
  if (degree < 1) return CPATTN_ERR_SHAPE;
  const cpattn_tensor* flat = dir == 1 ? x : y;      // [B, S, H, D]
  const cpattn_tensor* grouped = dir == 1 ? y : x;   // [G, B, S, H/G or ceil(H/G), D]
  if (!shape_ok(flat, 4) || !shape_ok(grouped, 5)) return CPATTN_ERR_SHAPE;
  const int64_t B = flat->shape[0], S = flat->shape[1], H = flat->shape[2], D = flat->shape[3];
  if (!anything && H % degree != 0) return CPATTN_ERR_DIVISIBILITY;
  const int64_t hg = anything ? (H + degree - 1) / degree : H / degree;
  if (grouped->shape[0] != degree || grouped->shape[1] != B || grouped->shape[2] != S ||
      grouped->shape[3] != hg || grouped->shape[4] != D)
    return CPATTN_ERR_SHAPE;
  dims[0] = B;
  dims[1] = S;
  dims[2] = H;
  dims[3] = D;
  const int eb = elem_bytes(x->dtype);
  const uintptr_t flat_bytes = static_cast<uintptr_t>(B * S * H * D * eb);
  const uintptr_t grouped_bytes = static_cast<uintptr_t>(degree * B * S * hg * D * eb);
  *xbytes = dir == 1 ? flat_bytes : grouped_bytes;
  *ybytes = dir == 1 ? grouped_bytes : flat_bytes;
  if (B * S * H * D == 0) return CPATTN_OK;
  if (!x->data || !y->data) return CPATTN_ERR_NULL;
  if (!contiguous(x) || !contiguous(y)) return CPATTN_ERR_LAYOUT;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x->data), ya = reinterpret_cast<uintptr_t>(y->data);
  if (xa % eb || ya % eb) return CPATTN_ERR_LAYOUT;
  return CPATTN_OK;
}

bool overlaps(const void* a, uintptr_t an, const void* b, uintptr_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// n regroups of one shape and dtype in one launch; no output may overlap
// any buffer of the call.
cpattn_status permute_batch(int n, const cpattn_tensor* x, int degree, int dir, cpattn_tensor* y,
                            bool anything, cudaStream_t stream) {
  if (n < 1 || n > cpattn::kMaxPermuteBatch) return CPATTN_ERR_SHAPE;
  if (!x || !y) return CPATTN_ERR_NULL;
  int64_t dims[4] = {0, 0, 0, 0};
  uintptr_t xb = 0, yb = 0;
  for (int i = 0; i < n; ++i) {
    int64_t d[4];
    uintptr_t xbi = 0, ybi = 0;
    const cpattn_status st = permute_pair_check(&x[i], &y[i], degree, dir, anything, d, &xbi, &ybi);
    if (st != CPATTN_OK) return st;
    if (i == 0) {
      for (int j = 0; j < 4; ++j) dims[j] = d[j];
      xb = xbi;
      yb = ybi;
    } else {
      if (x[i].dtype != x[0].dtype) return CPATTN_ERR_DTYPE;
      for (int j = 0; j < 4; ++j)
        if (d[j] != dims[j]) return CPATTN_ERR_SHAPE;
    }
  }
  if (dims[0] * dims[1] * dims[2] * dims[3] == 0) return CPATTN_OK;
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      if (overlaps(y[i].data, yb, x[j].data, xb) || (i != j && overlaps(y[i].data, yb, y[j].data, yb)))
        return CPATTN_ERR_LAYOUT;
  cpattn::PermuteParams p;
  p.n = n;
  for (int i = 0; i < n; ++i) {
    p.x[i] = x[i].data;
    p.y[i] = y[i].data;
  }
  p.batch = dims[0];
  p.seq = dims[1];
  p.heads = dims[2];
  p.head_dim = dims[3];
  p.degree = degree;
  p.dir = dir;
  p.elem_bytes = elem_bytes(x[0].dtype);
  const long long shrink = g_check_shrink.load();
  p.x_bytes = xb;
  p.y_bytes = yb > static_cast<uintptr_t>(shrink) ? yb - shrink : 0;
  p.err = cpattn::device_error_word();
  const cudaError_t e =
      anything ? cpattn::launch_permute_anything(p, stream) : cpattn::launch_permute(p, stream);
  return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

cpattn::CrossTensor cross_tensor(const cpattn_tensor* t, long long shrink = 0) {
  return {t->data, {t->stride[0], t->stride[1], t->stride[2]}, {t->data, extent_bytes(t, shrink)}};
}

// q [B, H, S_q, D] against k [B, H_kv, S_kv, D]: types, shapes and sizes.
cpattn_status cross_shape(const cpattn_tensor* q, const cpattn_tensor* k) {
  if (!dtype_known(q->dtype) || k->dtype != q->dtype) return CPATTN_ERR_DTYPE;
  if (!shape_ok(q, 4) || !shape_ok(k, 4)) return CPATTN_ERR_SHAPE;
  if (q->shape[0] != k->shape[0] || q->shape[3] != k->shape[3]) return CPATTN_ERR_SHAPE;
  const int64_t B = q->shape[0], H = q->shape[1], Hk = k->shape[1], D = q->shape[3];
  if (H > 0 && Hk == 0) return CPATTN_ERR_SHAPE;
  if (Hk > 0 && H % Hk != 0) return CPATTN_ERR_DIVISIBILITY;
  if (D != 64 && D != 128) return CPATTN_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || Hk > 65535 || q->shape[2] > (int64_t(1) << 30) ||
      k->shape[2] > (int64_t(1) << 30))
    return CPATTN_ERR_UNSUPPORTED;
  // (blocks of one launch)
  if (B * H * ((q->shape[2] + 63) / 64) > 0x7fffffff || B * Hk * ((k->shape[2] + 63) / 64) > 0x7fffffff)
    return CPATTN_ERR_UNSUPPORTED;
  return CPATTN_OK;
}

// Few query rows a key head: bf16 calls that the key and value read bounds.
// Up to 32 rows the few-rows kernel is as fast as the tensor-core kernel or
// faster; up to 64 only where many query heads share the key head, since the
// other one reads it for each of them (figures in cross_few.cu).
bool cross_few(const cpattn_tensor* q, const cpattn_tensor* k) {
  if (q->dtype != CPATTN_BF16 || k->shape[1] == 0) return false;
  const int64_t share = q->shape[1] / k->shape[1], rows = q->shape[2] * share;
  return rows <= 32 || (rows <= 64 && share >= 8);
}

// Blocks that clusters of `size` of them find room for at once: what is left of an
// SM group (GPC) stays free, and how many SMs a group has differs between chips.
// Asked once per device.  Found on one of 152 SMs, sizes 2 to 8: 152 138 144 140 138
// 105 120 with one block an SM, 304 291 296 290 276 266 288 with two.
int cluster_room(bool few, int size) {
  static std::atomic<int> known[64][2][cpattn::kCrossCluster + 1];   // (0: not asked yet)
  int dev = 0;
  const bool place = cudaGetDevice(&dev) == cudaSuccess && dev < 64;
  if (place) {
    const int n = known[dev][few][size].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  const int clusters = few ? cpattn::cross_few_clusters(size) : cpattn::cross_fwd_clusters(size);
  if (clusters < 0) return cpattn::sm_count() * (few ? 2 : 1);   // (no device: any split is as good)
  if (place && clusters > 0) known[dev][few][size].store(clusters * size, std::memory_order_relaxed);
  return clusters * size;
}

// Parts of the key axis of a forward call: 1 where the query rows fill the
// GPU, else as many as keep it full.  For few rows one round of two CTAs per SM
// (64 key heads x 16384 keys: 4 parts 79 us, 8 parts 82, 16 parts 95), each with
// 192 keys or more (2 key heads x 6000 keys: 8 parts 11.4 us, 16 parts 10.5, 32
// parts 9.0, 128 parts 9.8), above 8 parts whole clusters; two clusters and
// their join gain on one only past some 8000 keys (8 key heads: 4096 keys 9.0 us
// with one, 10.9 with two; 8192 14.9 / 15.2; 16384 25.0 / 22.1).  For 256-row
// units of the tensor-core kernel one per SM, each with 256 keys or more and
// none below 1024 keys (256 queries x 8 heads, D = 128: 1024 keys 15.1 us with
// one part, 13.1 with 4, 14.6 with 8; 512 x 512 x 8 heads at D = 64 8.4 with one,
// 9.6 with 4); for fp32's blocks likewise, each with 128 keys or more.
int cross_splits(const cpattn_tensor* q, const cpattn_tensor* k) {
  const int64_t bh = q->shape[0] * q->shape[1], sm = cpattn::sm_count();
  if (bh == 0 || q->shape[2] == 0 || k->shape[2] == 0) return 1;
  int64_t most, want, units;
  if (cross_few(q, k)) {
    units = q->shape[0] * k->shape[1];
    most = (k->shape[2] + 191) / 192;
    want = 2 * sm / units;
  } else {
    units = (q->shape[2] + 255) / 256 * bh;
    if (q->dtype != CPATTN_BF16) {
      units = (q->shape[2] + 63) / 64 * bh;
      if (!cpattn::cross_f32_rows(units, k->shape[2] * k->shape[3]))
        units = q->shape[2] > 2 ? (q->shape[2] + 7) / 8 * bh : bh;
    }
    most = q->dtype != CPATTN_BF16 ? (k->shape[2] + 127) / 128 : k->shape[2] < 1024 ? 1 : (k->shape[2] + 255) / 256;
    want = sm / units;
  }
  int64_t s = want < most ? want : most;
  if (q->dtype == CPATTN_BF16 && s > cpattn::kCrossCluster) {
    s -= s % cpattn::kCrossCluster;
    if (s < 3 * cpattn::kCrossCluster && k->shape[2] <= 8192) s = cpattn::kCrossCluster;
  }
  // a second round of clusters costs up to half (40 key heads x 8192 keys: 6 parts
  // 28.7 us, 7 parts 41.1)
  if (q->dtype == CPATTN_BF16)
    while (s > 1 && units * s > cluster_room(cross_few(q, k), static_cast<int>(s < 8 ? s : 8))) s -= s > 8 ? 8 : 1;
  return s > 1 ? static_cast<int>(s < 65535 ? s : 65535) : 1;
}

size_t cross_workspace(const cpattn_tensor* q, const cpattn_tensor* k) {
  const int64_t rows = q->shape[0] * q->shape[1] * q->shape[2];
  const int splits = cross_splits(q, k);
  const int parts = q->dtype == CPATTN_BF16 ? splits / cpattn::kCrossCluster : splits;
  return parts > 1 && rows > 0 ? static_cast<size_t>(parts) * rows * (q->shape[3] + 1) * 4 : 0;
}

// Parts of the query axis for dk and dv.
int cross_parts(const cpattn_tensor* q, const cpattn_tensor* k) {
  const int64_t rows = q->shape[0] * q->shape[1] * q->shape[2], keys = k->shape[0] * k->shape[1] * k->shape[2];
  if (rows == 0 || keys == 0) return 1;
  if (q->dtype != CPATTN_BF16)
    return cpattn::cross_f32_parts(k->shape[0] * k->shape[1] * ((k->shape[2] + 63) / 64),
                                   q->shape[1] / k->shape[1] * ((q->shape[2] + 63) / 64));
  return cpattn::cross_backward_parts(k->shape[0] * k->shape[1] * ((k->shape[2] + 127) / 128),
                                      q->shape[1] / k->shape[1] * ((q->shape[2] + 127) / 128));
}

// Floats before the parts' sums: delta of every query row, whole 16-byte vectors.
int64_t cross_delta_floats(const cpattn_tensor* q) {
  return (q->shape[0] * q->shape[1] * q->shape[2] + 3) / 4 * 4;
}

size_t cross_backward_workspace(const cpattn_tensor* q, const cpattn_tensor* k) {
  const int parts = cross_parts(q, k);
  const int64_t keys = k->shape[0] * k->shape[1] * k->shape[2];
  return static_cast<size_t>(cross_delta_floats(q) + (parts > 1 ? 2 * parts * keys * q->shape[3] : 0)) * 4;
}

// What both directions check and fill in; *run stays false where q has no row.
cpattn_status cross_common(const cpattn_tensor* q, const cpattn_tensor* k, const cpattn_tensor* v,
                           const cpattn_tensor* out, const cpattn_tensor* lse,
                           const cpattn_tensor* lengths, float scale, cpattn::CrossParams* p) {
  if (!q || !k || !v || !out || !lse) return CPATTN_ERR_NULL;
  if (v->dtype != q->dtype || out->dtype != q->dtype || lse->dtype != CPATTN_F32) return CPATTN_ERR_DTYPE;
  if (lengths && lengths->dtype != CPATTN_I32) return CPATTN_ERR_DTYPE;
  if (!shape_ok(v, 4) || !shape_ok(out, 4) || !shape_ok(lse, 3)) return CPATTN_ERR_SHAPE;
  if (lengths && (!shape_ok(lengths, 1) || lengths->shape[0] != q->shape[0])) return CPATTN_ERR_SHAPE;
  const cpattn_status st = cross_shape(q, k);
  if (st != CPATTN_OK) return st;
  if (!same_shape(v, k, 4) || !same_shape(out, q, 4) || !same_shape(lse, q, 3)) return CPATTN_ERR_SHAPE;
  const bool rows = q->shape[0] * q->shape[1] * q->shape[2] > 0;
  const bool keys = k->shape[0] * k->shape[1] * k->shape[2] > 0;
  if (rows && (!q->data || !out->data || !lse->data)) return CPATTN_ERR_NULL;
  if (keys && (!k->data || !v->data)) return CPATTN_ERR_NULL;
  if (lengths && q->shape[0] > 0 && !lengths->data) return CPATTN_ERR_NULL;
  if (rows && (!layout_distinct(q) || !layout_distinct(out) || !lse_layout_ok(lse))) return CPATTN_ERR_LAYOUT;
  if (keys && (!layout_distinct(k) || !layout_distinct(v))) return CPATTN_ERR_LAYOUT;
  if (lengths && ((lengths->shape[0] > 1 && lengths->stride[0] != 1) ||
                  (reinterpret_cast<uintptr_t>(lengths->data) & 3u)))
    return CPATTN_ERR_LAYOUT;
  std::memset(p, 0, sizeof(*p));
  p->q = cross_tensor(q);
  p->k = cross_tensor(k);
  p->v = cross_tensor(v);
  p->out = cross_tensor(out);
  p->lse = cross_tensor(lse);
  if (lengths) {
    p->lengths = static_cast<const int32_t*>(lengths->data);
    p->lengths_span = {lengths->data, extent_bytes(lengths)};
  }
  p->batch = static_cast<int>(q->shape[0]);
  p->heads = static_cast<int>(q->shape[1]);
  p->kv_heads = static_cast<int>(k->shape[1]);
  p->s_q = static_cast<int>(q->shape[2]);
  p->s_kv = static_cast<int>(k->shape[2]);
  if (!(scale > 0.f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(q->shape[3]));
  p->scale = scale;
  p->scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p->timeout_ns = g_timeout_ns.load();
  p->fault_skip_kv = g_fault_skip_kv.load();
  p->err = cpattn::device_error_word();
  return CPATTN_OK;
}

cpattn_status cross_workspace_ok(void* workspace, size_t bytes, size_t need, cpattn::CrossParams* p) {
  if (need > 0 && (workspace == nullptr || bytes < need || !aligned16(workspace))) return CPATTN_ERR_WORKSPACE;
  const size_t shrink = static_cast<size_t>(g_check_shrink.load());
  p->ws = static_cast<float*>(workspace);
  p->ws_span = {workspace, need > shrink ? need - shrink : 0};
  return CPATTN_OK;
}

}  // namespace

extern "C" {

cpattn_status cpattn_partial(const cpattn_tensor* q, const cpattn_tensor* k,
                             const cpattn_tensor* v, float scale, cpattn_tensor* out,
                             cpattn_tensor* lse, void* stream) {
  return run_attention(q, k, v, scale, 1, 0, out, lse, nullptr, 0, true, false,
                       static_cast<cudaStream_t>(stream));
}

cpattn_status cpattn_ring(const cpattn_tensor* q, const cpattn_tensor* k, const cpattn_tensor* v,
                          float scale, int ring_degree, int ring_anything, cpattn_tensor* out,
                          cpattn_tensor* lse, void* workspace, size_t workspace_bytes,
                          void* stream) {
  return run_attention(q, k, v, scale, ring_degree, ring_anything, out, lse, workspace,
                       workspace_bytes, false, false, static_cast<cudaStream_t>(stream));
}

cpattn_status cpattn_ring_causal(const cpattn_tensor* q, const cpattn_tensor* k,
                                 const cpattn_tensor* v, float scale, int ring_degree,
                                 int ring_anything, cpattn_tensor* out, cpattn_tensor* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return run_attention(q, k, v, scale, ring_degree, ring_anything, out, lse, workspace,
                       workspace_bytes, false, true, static_cast<cudaStream_t>(stream));
}

size_t cpattn_ring_workspace_bytes(const cpattn_tensor* q, int ring_degree) {
  if (!q || q->ndim != 4) return 0;
  for (int i = 0; i < 4; ++i)
    if (q->shape[i] < 0) return 0;
  return workspace_bytes_for(q->shape[0], q->shape[1], q->shape[2], q->shape[3], ring_degree);
}

cpattn_status cpattn_merge(cpattn_tensor* out_a, cpattn_tensor* lse_a, const cpattn_tensor* out_b,
                           const cpattn_tensor* lse_b, void* stream) {
  if (!out_a || !lse_a || !out_b || !lse_b) return CPATTN_ERR_NULL;
  if (out_a->dtype != CPATTN_F32 || out_b->dtype != CPATTN_F32 || lse_a->dtype != CPATTN_F32 ||
      lse_b->dtype != CPATTN_F32)
    return CPATTN_ERR_DTYPE;
  if (!shape_ok(out_a, 4) || !shape_ok(out_b, 4) || !shape_ok(lse_a, 3) || !shape_ok(lse_b, 3))
    return CPATTN_ERR_SHAPE;
  for (int i = 0; i < 4; ++i)
    if (out_a->shape[i] != out_b->shape[i]) return CPATTN_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (lse_a->shape[i] != out_a->shape[i] || lse_b->shape[i] != out_a->shape[i])
      return CPATTN_ERR_SHAPE;
  const int64_t B = out_a->shape[0], H = out_a->shape[1], S = out_a->shape[2],
                D = out_a->shape[3];
  if (D != 4 && D != 8 && D != 16 && D != 32 && D != 64 && D != 128)
    return CPATTN_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || S > (int64_t(1) << 31)) return CPATTN_ERR_UNSUPPORTED;
  if (B * H * S == 0) return CPATTN_OK;
  if (!out_a->data || !lse_a->data || !out_b->data || !lse_b->data) return CPATTN_ERR_NULL;
  if (!layout_ok(out_a) || !layout_ok(out_b)) return CPATTN_ERR_LAYOUT;
  if ((lse_a->shape[2] > 1 && lse_a->stride[2] != 1) ||
      (lse_b->shape[2] > 1 && lse_b->stride[2] != 1))
    return CPATTN_ERR_LAYOUT;
  if ((reinterpret_cast<uintptr_t>(lse_a->data) & 3u) || (reinterpret_cast<uintptr_t>(lse_b->data) & 3u))
    return CPATTN_ERR_LAYOUT;
  cpattn::MergeParams p;
  p.o_a = static_cast<float*>(out_a->data);
  p.l_a = static_cast<float*>(lse_a->data);
  p.o_b = static_cast<const float*>(out_b->data);
  p.l_b = static_cast<const float*>(lse_b->data);
  p.rows = B * H * S;
  p.head_dim = static_cast<int>(D);
  p.heads = static_cast<int>(H);
  p.seq = static_cast<int>(S);
  for (int i = 0; i < 3; ++i) {
    p.oa_s[i] = out_a->stride[i];
    p.ob_s[i] = out_b->stride[i];
    p.la_s[i] = lse_a->stride[i];
    p.lb_s[i] = lse_b->stride[i];
  }
  p.dense = contiguous(out_a) && contiguous(out_b) && contiguous(lse_a) && contiguous(lse_b);
  const long long shrink = g_check_shrink.load();
  p.oa_span = {out_a->data, extent_bytes(out_a, shrink)};
  p.la_span = {lse_a->data, extent_bytes(lse_a, shrink)};
  p.ob_span = {out_b->data, extent_bytes(out_b)};
  p.lb_span = {lse_b->data, extent_bytes(lse_b)};
  p.err = cpattn::device_error_word();
  const cudaError_t e = cpattn::launch_merge(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

cpattn_status cpattn_ulysses_permute_batch(int n, const cpattn_tensor* x, int degree, int dir,
                                           cpattn_tensor* y, void* stream) {
  return permute_batch(n, x, degree, dir, y, false, static_cast<cudaStream_t>(stream));
}

cpattn_status cpattn_ulysses_permute(const cpattn_tensor* x, int degree, int dir, cpattn_tensor* y,
                                     void* stream) {
  return permute_batch(1, x, degree, dir, y, false, static_cast<cudaStream_t>(stream));
}

cpattn_status cpattn_ulysses_anything_permute_batch(int n, const cpattn_tensor* x, int degree,
                                                    int dir, cpattn_tensor* y, void* stream) {
  return permute_batch(n, x, degree, dir, y, true, static_cast<cudaStream_t>(stream));
}

cpattn_status cpattn_ulysses_anything_permute(const cpattn_tensor* x, int degree, int dir,
                                              cpattn_tensor* y, void* stream) {
  return permute_batch(1, x, degree, dir, y, true, static_cast<cudaStream_t>(stream));
}

cpattn_status cpattn_ulysses_anything_attention(const cpattn_tensor* q, const cpattn_tensor* k,
                                                const cpattn_tensor* v, float scale, int heads,
                                                int is_causal, cpattn_tensor* out,
                                                cpattn_tensor* lse, void* stream) {
  if (!q || !k || !v || !out || !lse) return CPATTN_ERR_NULL;
  const cpattn_tensor* five[4] = {q, k, v, out};
  for (const cpattn_tensor* t : five)
    if (!shape_ok(t, 5)) return CPATTN_ERR_SHAPE;
  if (!shape_ok(lse, 4)) return CPATTN_ERR_SHAPE;
  const int64_t G = q->shape[0], B = q->shape[1], S = q->shape[2], hm = q->shape[3];
  if (heads < 1 || G < 1 || hm != (heads + G - 1) / G) return CPATTN_ERR_SHAPE;
  for (const cpattn_tensor* t : five)
    for (int i = 0; i < 5; ++i)
      if (t->shape[i] != q->shape[i]) return CPATTN_ERR_SHAPE;
  if (lse->shape[0] != G || lse->shape[1] != B || lse->shape[2] != hm || lse->shape[3] != S)
    return CPATTN_ERR_SHAPE;
  // the (group, batch) axes merge into one batch axis of the 4-D view
  for (const cpattn_tensor* t : five)
    if (G > 1 && B > 0 && t->stride[0] != B * t->stride[1]) return CPATTN_ERR_LAYOUT;
  if (G > 1 && B > 0 && lse->stride[0] != B * lse->stride[1]) return CPATTN_ERR_LAYOUT;
  if (G * B > 65535) return CPATTN_ERR_UNSUPPORTED;
  // view [G*B, hm, S, D] (strides: batch, head, token, feature)
  auto view = [&](const cpattn_tensor* t) {
    cpattn_tensor w = *t;
    w.ndim = 4;
    w.shape[0] = G * B; w.shape[1] = hm; w.shape[2] = S; w.shape[3] = t->shape[4];
    w.stride[0] = t->stride[1]; w.stride[1] = t->stride[3]; w.stride[2] = t->stride[2];
    w.stride[3] = t->stride[4];
    w.stride[4] = 0; w.shape[4] = 0;
    return w;
  };
  cpattn_tensor vq = view(q), vk = view(k), vv = view(v), vo = view(out);
  cpattn_tensor vl = *lse;
  vl.ndim = 3;
  vl.shape[0] = G * B; vl.shape[1] = hm; vl.shape[2] = S;
  vl.stride[0] = lse->stride[1]; vl.stride[1] = lse->stride[2]; vl.stride[2] = lse->stride[3];
  vl.shape[3] = vl.shape[4] = 0; vl.stride[3] = vl.stride[4] = 0;
  return run_attention(&vq, &vk, &vv, scale, 1, 0, &vo, &vl, nullptr, 0, false, is_causal != 0,
                       static_cast<cudaStream_t>(stream), static_cast<int>(G), heads);
}

cpattn_status cpattn_rotary(int n, const cpattn_tensor* x, const cpattn_tensor* positions, int axes,
                            const int32_t* axis_dims, double theta, int interleaved, int inverse,
                            cpattn_tensor* y, void* stream) {
  if (n < 1 || n > cpattn::kMaxPermuteBatch) return CPATTN_ERR_SHAPE;
  if (!x || !y || !positions || !axis_dims) return CPATTN_ERR_NULL;
  if (positions->dtype != CPATTN_F32 || !dtype_known(x[0].dtype)) return CPATTN_ERR_DTYPE;
  for (int i = 0; i < n; ++i)
    if (x[i].dtype != x[0].dtype || y[i].dtype != x[0].dtype) return CPATTN_ERR_DTYPE;
  if (axes < 1 || axes > CPATTN_MAX_ROTARY_AXES) return CPATTN_ERR_SHAPE;
  for (int i = 0; i < n; ++i) {
    if (!shape_ok(&x[i], 4) || !shape_ok(&y[i], 4) || !same_shape(&x[i], &y[i], 4)) return CPATTN_ERR_SHAPE;
    if (x[i].shape[0] != x[0].shape[0] || x[i].shape[2] != x[0].shape[2] || x[i].shape[3] != x[0].shape[3])
      return CPATTN_ERR_SHAPE;
  }
  const int64_t B = x[0].shape[0], S = x[0].shape[2], D = x[0].shape[3];
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
  if (D > CPATTN_MAX_ROTARY_DIM || (D * elem_bytes(x[0].dtype)) % 16 != 0) return CPATTN_ERR_UNSUPPORTED;
  int64_t heads = 0;
  for (int i = 0; i < n; ++i) {
    if (x[i].shape[1] > 65535) return CPATTN_ERR_UNSUPPORTED;
    heads += x[i].shape[1];
  }
  if (B > 65535 || S > (int64_t(1) << 30)) return CPATTN_ERR_UNSUPPORTED;
  if (B * S * heads == 0) return CPATTN_OK;
  if (!positions->data) return CPATTN_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(positions->data) & 3u) return CPATTN_ERR_LAYOUT;
  for (int i = 0; i < positions->ndim; ++i)
    if (positions->stride[i] < 0) return CPATTN_ERR_LAYOUT;

  cpattn::RotaryParams p;
  std::memset(&p, 0, sizeof(p));
  const long long shrink = g_check_shrink.load();
  for (int i = 0; i < n; ++i) {
    const bool none = x[i].shape[1] == 0;
    if (!none && (!x[i].data || !y[i].data)) return CPATTN_ERR_NULL;
    if (!none && (!layout_ok(&x[i]) || !layout_distinct(&y[i]))) return CPATTN_ERR_LAYOUT;
    if (!none && x[i].data == y[i].data)   // in place: element for element
      for (int j = 0; j < 4; ++j)
        if (x[i].shape[j] > 1 && x[i].stride[j] != y[i].stride[j]) return CPATTN_ERR_LAYOUT;
    p.x[i] = x[i].data;
    p.y[i] = y[i].data;
    p.x_sb[i] = x[i].stride[0];
    p.x_sh[i] = x[i].stride[1];
    p.x_ss[i] = x[i].stride[2];
    p.y_sb[i] = y[i].stride[0];
    p.y_sh[i] = y[i].stride[1];
    p.y_ss[i] = y[i].stride[2];
    p.head_start[i + 1] = p.head_start[i] + static_cast<int>(x[i].shape[1]);
    p.x_span[i] = {x[i].data, extent_bytes(&x[i])};
    p.y_span[i] = {y[i].data, extent_bytes(&y[i], shrink)};
  }
  p.n = n;
  p.batch = static_cast<int>(B);
  p.seq = static_cast<int>(S);
  p.head_dim = static_cast<int>(D);
  p.pos = static_cast<const float*>(positions->data);
  p.pos_sb = per_batch ? positions->stride[0] : 0;
  p.pos_ss = positions->stride[pa - 1];
  p.pos_sa = positions->stride[pa];
  p.pos_span = {positions->data, extent_bytes(positions)};
  p.interleaved = interleaved != 0;
  p.inverse = inverse != 0;
  p.err = cpattn::device_error_word();
  fill_turns(p, axes, axis_dims, theta);
  const InDtype dt = x[0].dtype == CPATTN_BF16 ? InDtype::BF16 : InDtype::F32;
  return cpattn::launch_rotary(dt, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CPATTN_OK
                                                                                       : CPATTN_ERR_CUDA;
}

size_t cpattn_cross_workspace_bytes(const cpattn_tensor* q, const cpattn_tensor* k) {
  return q && k && cross_shape(q, k) == CPATTN_OK ? cross_workspace(q, k) : 0;
}

size_t cpattn_cross_backward_workspace_bytes(const cpattn_tensor* q, const cpattn_tensor* k) {
  return q && k && cross_shape(q, k) == CPATTN_OK ? cross_backward_workspace(q, k) : 0;
}

cpattn_status cpattn_cross_attention(const cpattn_tensor* q, const cpattn_tensor* k,
                                     const cpattn_tensor* v, const cpattn_tensor* kv_lengths,
                                     float scale, cpattn_tensor* out, cpattn_tensor* lse,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  cpattn::CrossParams p;
  cpattn_status st = cross_common(q, k, v, out, lse, kv_lengths, scale, &p);
  if (st != CPATTN_OK) return st;
  if (q->shape[0] * q->shape[1] * q->shape[2] == 0) return CPATTN_OK;
  const size_t need = cross_workspace(q, k);
  if ((st = cross_workspace_ok(workspace, workspace_bytes, need, &p)) != CPATTN_OK) return st;
  const long long shrink = g_check_shrink.load();
  p.out = cross_tensor(out, shrink);
  p.lse = cross_tensor(lse, shrink);
  const InDtype dt = q->dtype == CPATTN_BF16 ? InDtype::BF16 : InDtype::F32;
  const int D = static_cast<int>(q->shape[3]);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  p.splits = p.s_kv > 0 ? cross_splits(q, k) : 0;
  bool join = p.splits != 1;   // (no parts: the join writes the empty result)
  if (p.splits > 0 && cross_few(q, k)) {
    e = cpattn::launch_cross_few(D, p, cs);
  } else if (p.splits > 0 && dt == InDtype::BF16) {
    CUtensorMap tm_q, tm_k, tm_v, tm_o;
    if ((st = make_tmap(&tm_q, q, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&tm_k, k, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&tm_v, v, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&tm_o, out, 32)) != CPATTN_OK) return st;
    e = cpattn::launch_cross_fwd(D, tm_q, tm_k, tm_v, tm_o, p, cs);
  } else if (p.splits > 0) {
    e = cpattn::launch_cross_simt(D, p, cs);
  }
  if (dt == InDtype::BF16 && p.splits > 0) {   // (a cluster has joined its parts)
    p.splits /= cpattn::kCrossCluster;
    join = p.splits > 1;
  }
  if (e == cudaSuccess && join) e = cpattn::launch_cross_join(dt, D, p, cs);
  return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

cpattn_status cpattn_cross_attention_backward(const cpattn_tensor* q, const cpattn_tensor* k,
                                              const cpattn_tensor* v, const cpattn_tensor* out,
                                              const cpattn_tensor* lse, const cpattn_tensor* dout,
                                              const cpattn_tensor* kv_lengths, float scale,
                                              cpattn_tensor* dq, cpattn_tensor* dk,
                                              cpattn_tensor* dv, void* workspace,
                                              size_t workspace_bytes, void* stream) {
  if (!dout || !dq || !dk || !dv) return CPATTN_ERR_NULL;
  cpattn::CrossParams p;
  cpattn_status st = cross_common(q, k, v, out, lse, kv_lengths, scale, &p);
  if (st != CPATTN_OK) return st;
  const cpattn_tensor* rows4[2] = {dout, dq};
  const cpattn_tensor* keys4[2] = {dk, dv};
  const bool rows = q->shape[0] * q->shape[1] * q->shape[2] > 0;
  const bool keys = k->shape[0] * k->shape[1] * k->shape[2] > 0;
  for (const cpattn_tensor* t : rows4) {
    if (t->dtype != q->dtype) return CPATTN_ERR_DTYPE;
    if (!shape_ok(t, 4) || !same_shape(t, q, 4)) return CPATTN_ERR_SHAPE;
    if (rows && !t->data) return CPATTN_ERR_NULL;
    if (rows && !layout_distinct(t)) return CPATTN_ERR_LAYOUT;
  }
  for (const cpattn_tensor* t : keys4) {
    if (t->dtype != q->dtype) return CPATTN_ERR_DTYPE;
    if (!shape_ok(t, 4) || !same_shape(t, k, 4)) return CPATTN_ERR_SHAPE;
    if (keys && !t->data) return CPATTN_ERR_NULL;
    if (keys && !layout_distinct(t)) return CPATTN_ERR_LAYOUT;
  }
  if (!rows && !keys) return CPATTN_OK;
  const size_t need = cross_backward_workspace(q, k);
  if ((st = cross_workspace_ok(workspace, workspace_bytes, need, &p)) != CPATTN_OK) return st;
  const long long shrink = g_check_shrink.load();
  p.dout = cross_tensor(dout);
  p.dq = cross_tensor(dq, shrink);
  p.dk = cross_tensor(dk, shrink);
  p.dv = cross_tensor(dv, shrink);
  p.splits = cross_parts(q, k);
  const InDtype dt = q->dtype == CPATTN_BF16 ? InDtype::BF16 : InDtype::F32;
  const int D = static_cast<int>(q->shape[3]);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (!rows || !keys) {
    e = cpattn::launch_cross_zeros(dt, D, p, cs);
  } else if (dt == InDtype::BF16) {
    cpattn::CrossBwdMaps m;
    if ((st = make_tmap(&m.q, q, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&m.k, k, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&m.v, v, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&m.out, out, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&m.dout, dout, 128)) != CPATTN_OK) return st;
    if ((st = make_tmap(&m.dq, dq, 32, D == 64)) != CPATTN_OK) return st;
    if ((st = make_tmap(&m.dk, dk, 32)) != CPATTN_OK) return st;
    if ((st = make_tmap(&m.dv, dv, 32)) != CPATTN_OK) return st;
    e = cpattn::launch_cross_bwd(D, m, p, cross_delta_floats(q), cs);
  } else {
    e = cpattn::launch_cross_simt_backward(D, p, cross_delta_floats(q), cs);
  }
  return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

const char* cpattn_status_string(cpattn_status status) {
  switch (status) {
    case CPATTN_OK: return "ok";
    case CPATTN_ERR_NULL: return "null pointer";
    case CPATTN_ERR_DTYPE: return "dtype not allowed";
    case CPATTN_ERR_SHAPE: return "inconsistent shape";
    case CPATTN_ERR_DIVISIBILITY: return "length not divisible by the degree";
    case CPATTN_ERR_LAYOUT: return "layout: inner stride must be 1, strides and data 16-byte aligned";
    case CPATTN_ERR_UNSUPPORTED: return "unsupported size or head dimension";
    case CPATTN_ERR_WORKSPACE: return "workspace missing or too small";
    case CPATTN_ERR_CUDA: return "CUDA runtime error";
    case CPATTN_ERR_TIMEOUT: return "device-side wait timed out";
    case CPATTN_ERR_BOUNDS: return "device-side bounds check failed (check build)";
  }
  return "unknown status";
}

cpattn_status cpattn_last_device_status(void* stream) {
  unsigned int v = 0;
  const cudaError_t e = cpattn::read_and_clear_device_error(&v, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return CPATTN_ERR_CUDA;
  if (v & cpattn::kErrBounds) return CPATTN_ERR_BOUNDS;
  return v ? CPATTN_ERR_TIMEOUT : CPATTN_OK;
}

void cpattn_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns ? ns : 1); }

void cpattn_set_fault_injection(int mode) { g_fault_skip_kv.store(mode == 1 ? 1 : 0); }

void cpattn_set_check_shrink(int64_t bytes) { g_check_shrink.store(bytes > 0 ? bytes : 0); }

int cpattn_is_check_build(void) {
#ifdef CPATTN_CHECK
  return 1;
#else
  return 0;
#endif
}

}  // extern "C"
