// capi_dense.cu -- entry points of the position rotation, the cache extension
// and the attention over a shared prefix: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "capi_common.h"
#include "csa2_internal.cuh"
#include "kernels.h"

using namespace csa2;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

#define CSA2_REQUIRE_I32(p)                                                        \
  do {                                                                             \
    if ((p) == nullptr) return ::csa2::fail(CSA2_ERR_INVALID_ARG, "%s is NULL", #p); \
    if (!aligned4(p))                                                              \
      return ::csa2::fail(CSA2_ERR_ALIGNMENT, "%s is not 4-byte aligned", #p);      \
  } while (0)

csa2_status check_ws(const void* ws, size_t bytes, size_t need) {
  CSA2_REQUIRE_PTR(ws);
  CSA2_REQUIRE(bytes >= need, CSA2_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", bytes,
               need);
  return CSA2_OK;
}

csa2_status check_rope(const csa2_rope& r, const char* what, int ch) {
  CSA2_REQUIRE(aligned16(r.table), CSA2_ERR_ALIGNMENT, "%s.table is not 16-byte aligned", what);
  CSA2_REQUIRE(r.style == CSA2_ROPE_PAIRS || r.style == CSA2_ROPE_HALVES, CSA2_ERR_INVALID_ARG,
               "%s.style = %d", what, r.style);
  CSA2_REQUIRE(r.n_pos >= 1, CSA2_ERR_SHAPE, "%s.n_pos = %d", what, r.n_pos);
  CSA2_REQUIRE(r.dims > 0 && r.dims % 32 == 0 && r.dims <= ch, CSA2_ERR_SHAPE,
               "%s.dims = %d (a multiple of 32 up to %d)", what, r.dims, ch);
  return CSA2_OK;
}

RopeParams rope_params(const csa2_rope& r) {
  if (!r.table) return RopeParams{nullptr, 0, 0, 0};
  return RopeParams{reinterpret_cast<const float2*>(r.table), r.n_pos, r.dims, r.style};
}

// The row map of a cache, without what the decode step alone needs.
csa2_status check_rows(const csa2_kv_view& kv) {
  CSA2_REQUIRE_PTR(kv.codes);
  CSA2_REQUIRE_PTR(kv.scales);
  CSA2_REQUIRE_I32(kv.n_rows);
  CSA2_REQUIRE(kv.pool_rows >= 0 && kv.pool_rows <= (int64_t)0x7FFF0000, CSA2_ERR_SHAPE,
               "pool_rows = %lld", (long long)kv.pool_rows);
  if (kv.page_table) {
    CSA2_REQUIRE_I32(kv.page_table);
    CSA2_REQUIRE(kv.page_rows == 64, CSA2_ERR_SHAPE, "page_rows = %d (must be 64)", kv.page_rows);
    CSA2_REQUIRE(kv.max_pages >= 0, CSA2_ERR_SHAPE, "max_pages = %d", kv.max_pages);
  } else {
    CSA2_REQUIRE(kv.seq_stride >= 0 && kv.seq_stride % 64 == 0, CSA2_ERR_ALIGNMENT,
                 "seq_stride = %lld is not a multiple of 64 rows", (long long)kv.seq_stride);
    CSA2_REQUIRE(kv.seq_stride <= (int64_t)0x7FFF0000, CSA2_ERR_SHAPE, "seq_stride = %lld",
                 (long long)kv.seq_stride);
  }
  return CSA2_OK;
}

csa2_status prefix_params(const csa2_prefix_desc* d, PrefixParams& p) {
  CSA2_REQUIRE(d != nullptr, CSA2_ERR_INVALID_ARG, "desc is NULL");
  const csa2_kv_view& kv = d->kv;
  CSA2_REQUIRE(kv.batch >= 1 && kv.batch <= CSA2_PREFIX_MAX_BATCH, CSA2_ERR_SHAPE,
               "batch = %d outside [1, %d]", kv.batch, (int)CSA2_PREFIX_MAX_BATCH);
  const int nq = d->n_query < 1 ? 1 : d->n_query;
  CSA2_REQUIRE(d->n_query >= 0 && nq <= CSA2_MAX_QUERY && kv.batch * nq <= 65535, CSA2_ERR_SHAPE,
               "n_query = %d with batch = %d", d->n_query, kv.batch);
  CSA2_REQUIRE(kv.max_rows >= 0 && kv.max_rows <= CSA2_MAX_ROWS, CSA2_ERR_SHAPE,
               "max_rows = %d outside [0, %d]", kv.max_rows, (int)CSA2_MAX_ROWS);
  CSA2_REQUIRE(d->prefix_rows >= 0 && d->prefix_rows <= kv.max_rows, CSA2_ERR_SHAPE,
               "prefix_rows = %d outside [0, max_rows = %d]", d->prefix_rows, kv.max_rows);
  p = PrefixParams{};
  p.codes = kv.codes;
  p.scales = kv.scales;
  p.page_table = kv.page_table;
  p.max_pages = kv.max_pages;
  p.max_rows = kv.max_rows;
  p.seq_stride = kv.seq_stride;
  p.pool_rows = kv.pool_rows;
  p.n_rows = kv.n_rows;
  p.batch = kv.batch;
  p.nq = nq;
  p.prefix = d->prefix_rows;
  p.q = d->q;
  p.swa = d->swa;
  p.swa_len = d->swa_len;
  p.swa_rows = CSA2_W + nq - 1;
  p.scale_log2 = d->sm_scale * (1.4426950408889634f / 256);
  p.out = d->out;
  p.grid = prefix_grid(p, num_sms());
  return CSA2_OK;
}

size_t prefix_ws_bytes(const PrefixParams& p) {
  return CSA2_WS_HEADER + prefix_partial_rows(p) * (CSA2_D + 3) * sizeof(float) +
         prefix_image_tiles(p) * (PREFIX_IMAGE + 64);
}

}  // namespace

extern "C" {

csa2_status csa2_rope_rows(const csa2_rope* rope, const uint16_t* x, const int32_t* pos,
                           int64_t rows, int32_t heads, int32_t ch, int32_t inverse, uint16_t* y,
                           void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_REQUIRE(rope != nullptr, CSA2_ERR_INVALID_ARG, "rope is NULL");
  CSA2_REQUIRE(ch > 0 && ch % 8 == 0 && ch <= 65536, CSA2_ERR_SHAPE,
               "ch = %d is not a multiple of 8 up to 65536", ch);
  CSA2_REQUIRE(rows >= 0 && heads >= 0 && heads <= 65536, CSA2_ERR_SHAPE,
               "rows = %lld, heads = %d (up to 65536)", (long long)rows, heads);
  CSA2_REQUIRE_PTR(rope->table);
  csa2_status r = check_rope(*rope, "rope", ch);
  if (r) return r;
  if (rows == 0 || heads == 0) return CSA2_OK;
  CSA2_REQUIRE(rows <= ((int64_t)1 << 40) / ch / heads, CSA2_ERR_SHAPE,
               "rows = %lld x heads = %d x ch = %d", (long long)rows, heads, ch);
  CSA2_REQUIRE_PTR(x);
  CSA2_REQUIRE_PTR(y);
  CSA2_REQUIRE_I32(pos);
  if ((r = check_ws(ws, ws_bytes, CSA2_WS_HEADER))) return r;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  const uintptr_t bytes = (uintptr_t)(rows * heads * ch) * 2;
  CSA2_REQUIRE(a == b || a + bytes <= b || b + bytes <= a, CSA2_ERR_INVALID_ARG,
               "x and y overlap without being the same buffer");
  RopeRowsParams p{};
  p.rope = rope_params(*rope);
  p.x = x;
  p.y = y;
  p.pos = pos;
  p.rows = rows;
  p.heads = heads;
  p.ch = ch;
  p.inverse = inverse != 0;
  p.in_place = a == b;
  p.status = static_cast<uint32_t*>(ws);
  CSA2_CUDA(launch_rope_rows(p, (cudaStream_t)stream));
  trace_mark("end", (cudaStream_t)stream);
  return CSA2_OK;
}

csa2_status csa2_cache_extend(const csa2_extend_desc* d, void* ws, size_t ws_bytes,
                              csa2_stream_t stream) {
  CSA2_REQUIRE(d != nullptr, CSA2_ERR_INVALID_ARG, "desc is NULL");
  const csa2_kv_view& kv = d->kv;
  csa2_status r;
  CSA2_REQUIRE(kv.batch >= 1 && kv.batch <= 65535, CSA2_ERR_SHAPE, "batch = %d", kv.batch);
  CSA2_REQUIRE(d->total >= 0 && d->total < (1 << 24), CSA2_ERR_SHAPE, "total = %d", d->total);
  CSA2_REQUIRE(d->n_layers >= 0 && d->n_layers <= 1024, CSA2_ERR_SHAPE, "n_layers = %d",
               d->n_layers);
  if (d->cu_tokens) {
    CSA2_REQUIRE_I32(d->cu_tokens);
  } else {
    CSA2_REQUIRE(d->total == kv.batch, CSA2_ERR_SHAPE,
                 "total = %d tokens without cu_tokens for batch = %d", d->total, kv.batch);
  }
  if (d->total == 0) return CSA2_OK;
  CSA2_REQUIRE(d->x != nullptr || d->n_layers > 0, CSA2_ERR_INVALID_ARG,
               "neither entries nor window layers");
  CSA2_REQUIRE(aligned4(d->pos), CSA2_ERR_ALIGNMENT, "d->pos is not 4-byte aligned");
  if (d->x) {
    if ((r = check_rows(kv))) return r;
    CSA2_REQUIRE_PTR(kv.idx_k);
    CSA2_REQUIRE_PTR(d->x);
    CSA2_REQUIRE_PTR(d->w_idx);
    if (d->rope.table && (r = check_rope(d->rope, "rope", CSA2_D))) return r;
    if (d->rope_idx.table && (r = check_rope(d->rope_idx, "rope_idx", CSA2_DI))) return r;
  }
  if (d->n_layers > 0) {
    CSA2_REQUIRE_PTR(d->x_swa);
    CSA2_REQUIRE_PTR(d->swa);
    CSA2_REQUIRE_I32(d->swa_pos);
    CSA2_REQUIRE_I32(d->swa_len);
    if (d->rope_swa.table && (r = check_rope(d->rope_swa, "rope_swa", CSA2_D))) return r;
  }
  if ((r = check_ws(ws, ws_bytes, CSA2_WS_HEADER))) return r;
  ExtendParams p{};
  if (d->x) {
    p.codes = const_cast<uint8_t*>(kv.codes);
    p.scales = const_cast<uint8_t*>(kv.scales);
    p.idx_k = const_cast<uint16_t*>(kv.idx_k);
    p.page_table = kv.page_table;
    p.max_pages = kv.max_pages;
    p.seq_stride = kv.seq_stride;
    p.pool_rows = kv.pool_rows;
    p.n_rows = const_cast<int32_t*>(kv.n_rows);
    p.x = d->x;
    p.w_idx = d->w_idx;
    p.rope = rope_params(d->rope);
    p.rope_idx = rope_params(d->rope_idx);
  }
  p.batch = kv.batch;
  p.total = d->total;
  p.cu = d->cu_tokens;
  p.pos = d->pos;
  p.n_layers = d->n_layers;
  if (d->n_layers > 0) {
    p.rope_swa = rope_params(d->rope_swa);
    p.x_swa = d->x_swa;
    p.swa = d->swa;
    p.swa_pos = d->swa_pos;
    p.swa_len = d->swa_len;
  }
  p.status = static_cast<uint32_t*>(ws);
  CSA2_CUDA(launch_extend(p, (cudaStream_t)stream));
  trace_mark("end", (cudaStream_t)stream);
  return CSA2_OK;
}

size_t csa2_prefix_attn_workspace_size(const csa2_prefix_desc* desc) {
  PrefixParams p;
  if (prefix_params(desc, p) != CSA2_OK) return 0;
  return prefix_ws_bytes(p);
}

csa2_status csa2_prefix_attn(const csa2_prefix_desc* d, void* ws, size_t ws_bytes,
                             csa2_stream_t stream) {
  PrefixParams p;
  csa2_status r = prefix_params(d, p);
  if (r) return r;
  if ((r = check_rows(d->kv))) return r;
  if (d->kv.page_table) {
    CSA2_REQUIRE((int64_t)d->kv.max_pages * 64 >= d->kv.max_rows, CSA2_ERR_SHAPE,
                 "max_pages = %d cannot hold max_rows = %d", d->kv.max_pages, d->kv.max_rows);
  } else {
    CSA2_REQUIRE(d->kv.seq_stride >= d->kv.max_rows, CSA2_ERR_SHAPE,
                 "seq_stride = %lld < max_rows = %d", (long long)d->kv.seq_stride,
                 d->kv.max_rows);
  }
  CSA2_REQUIRE_PTR(d->q);
  CSA2_REQUIRE_PTR(d->out);
  if (d->swa || d->swa_len) {
    CSA2_REQUIRE_PTR(d->swa);
    CSA2_REQUIRE_I32(d->swa_len);
  }
  CSA2_REQUIRE(std::isfinite(d->sm_scale), CSA2_ERR_INVALID_ARG, "sm_scale is not finite");
  if ((r = check_ws(ws, ws_bytes, prefix_ws_bytes(p)))) return r;
  const size_t rows = prefix_partial_rows(p);
  p.status = static_cast<uint32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + CSA2_WS_HEADER);
  p.part_ml = p.part_o + rows * CSA2_D;
  p.part_scl = p.part_ml + rows * 2;
  p.image = reinterpret_cast<uint8_t*>(p.part_scl + rows);
  p.image_key = p.image + prefix_image_tiles(p) * PREFIX_IMAGE;
  CSA2_CUDA(launch_prefix_attn(p, (cudaStream_t)stream));
  trace_mark("end", (cudaStream_t)stream);
  return CSA2_OK;
}

}  // extern "C"
