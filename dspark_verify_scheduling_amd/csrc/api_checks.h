// Argument checks that the entry points of the target pass share.
#pragma once

#include "api_status.h"
#include "kv_dev.h"

namespace dspark {

// The cache's own fields; fills `kv`. `layers`: also the strides between layers.
inline dspark_status check_cache(const char* fn, const dspark_kv_cache* c, bool layers,
                          KvView* kv) {
  if (!c) return fail(DSPARK_E_INVALID, "%s: cache is NULL", fn);
  if (c->dtype != DSPARK_BF16 && c->dtype != DSPARK_F16 && c->dtype != DSPARK_E4M3)
    return fail(DSPARK_E_UNSUPPORTED, "%s: unsupported cache dtype %d", fn, (int)c->dtype);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(DSPARK_E_UNSUPPORTED, "%s: head_dim = %d is not 64, 128 or 256", fn, c->head_dim);
  int shift = 0;
  for (int s = 4; s <= 8; ++s) shift = c->block_size == 1 << s ? s : shift;
  if (!shift)
    return fail(DSPARK_E_UNSUPPORTED, "%s: block_size = %d is not 16, 32, 64, 128 or 256", fn,
                c->block_size);
  if (c->num_kv_heads < 1 || c->num_kv_heads > DSPARK_MAX_HEADS)
    return fail(DSPARK_E_INVALID, "%s: num_kv_heads = %d outside [1, %d]", fn, c->num_kv_heads,
                DSPARK_MAX_HEADS);
  if (c->num_blocks < 1)
    return fail(DSPARK_E_INVALID, "%s: num_blocks = %d < 1", fn, c->num_blocks);
  const bool e8 = c->dtype == DSPARK_E4M3;
  const int64_t cb = e8 ? 1 : 2;
  const int64_t tokens = (int64_t)c->num_kv_heads * c->block_size;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v))
    return fail(DSPARK_E_INVALID, "%s: k or v of the cache NULL or not 16-byte aligned", fn);
  if (c->block_stride < tokens * c->head_dim || c->block_stride > (1LL << 40) ||
      c->block_stride * cb % 16 != 0)
    return fail(DSPARK_E_INVALID,
                "%s: block_stride = %lld must be >= %lld elements and a multiple of 16 bytes", fn,
                (long long)c->block_stride, (long long)(tokens * c->head_dim));
  if (e8 && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
             c->scale_block_stride < tokens || c->scale_block_stride > (1LL << 40) ||
             c->scale_block_stride % 16 != 0))
    return fail(DSPARK_E_INVALID,
                "%s: an E4M3 cache needs k_scale and v_scale, 16-byte aligned, and "
                "scale_block_stride >= %lld, a multiple of 16",
                fn, (long long)tokens);
  if (layers) {
    if (c->num_layers < 1 || c->num_layers > DSPARK_MAX_LAYERS)
      return fail(DSPARK_E_INVALID, "%s: num_layers = %d outside [1, %d]", fn, c->num_layers,
                  DSPARK_MAX_LAYERS);
    if (c->num_layers > 1 &&
        (c->layer_stride < tokens * c->head_dim || c->layer_stride > (1LL << 50) ||
         c->layer_stride * cb % 16 != 0 ||
         (e8 && (c->scale_layer_stride < tokens || c->scale_layer_stride > (1LL << 50) ||
                 c->scale_layer_stride % 16 != 0))))
      return fail(DSPARK_E_INVALID,
                  "%s: layers overlap, or their stride is not a multiple of 16 bytes", fn);
  }
  kv->k = static_cast<unsigned char*>(c->k);
  kv->v = static_cast<unsigned char*>(c->v);
  kv->ks = e8 ? c->k_scale : nullptr;
  kv->vs = e8 ? c->v_scale : nullptr;
  kv->page_bytes = c->block_stride * cb;
  kv->scale_page_bytes = e8 ? c->scale_block_stride : 0;
  kv->layer_bytes = layers && c->num_layers > 1 ? c->layer_stride * cb : 0;
  kv->scale_layer_bytes = layers && c->num_layers > 1 && e8 ? c->scale_layer_stride : 0;
  kv->num_layers = layers ? c->num_layers : 1;
  kv->num_blocks = c->num_blocks;
  kv->hkv = c->num_kv_heads;
  kv->page_shift = shift;
  kv->dim = c->head_dim;
  kv->cb = (int)cb;
  return DSPARK_OK;
}

// The requests' arrays (`packed`: with rows of a packed buffer); fills `q`.
inline dspark_status check_requests(const char* fn, bool packed, int32_t B, int32_t gamma, int32_t max_rows,
                             const int32_t* cu, const int32_t* prefix, const int32_t* parents,
                             const int32_t* table, int32_t width, ReqView* q) {
  if (B < 0) return fail(DSPARK_E_INVALID, "%s: B = %d < 0", fn, B);
  if (B > DSPARK_MAX_BATCH)
    return fail(DSPARK_E_UNSUPPORTED, "%s: B = %d exceeds %d", fn, B, DSPARK_MAX_BATCH);
  if (gamma < 1 || gamma > DSPARK_MAX_GAMMA)
    return fail(DSPARK_E_INVALID, "%s: gamma = %d outside [1, %d]", fn, gamma, DSPARK_MAX_GAMMA);
  if (max_rows < 0) return fail(DSPARK_E_INVALID, "%s: max_rows = %d < 0", fn, max_rows);
  if (packed && !cu) return fail(DSPARK_E_INVALID, "%s: cu_seqlens is NULL", fn);
  if (B > 0 && (!prefix || !table))
    return fail(DSPARK_E_INVALID, "%s: an array of the requests is NULL", fn);
  if (B > 0 && width < 1)
    return fail(DSPARK_E_INVALID, "%s: table_width = %d < 1", fn, width);
  *q = {cu, prefix, parents, table, B, gamma, max_rows, width};
  return DSPARK_OK;
}

// The query side of append and attention.
inline dspark_status check_heads(const char* fn, int32_t num_heads, dspark_dtype dt,
                          const dspark_kv_cache* c) {
  if (dt != DSPARK_BF16 && dt != DSPARK_F16)
    return fail(DSPARK_E_UNSUPPORTED, "%s: unsupported dtype %d", fn, (int)dt);
  if (c->dtype != dt && !(c->dtype == DSPARK_E4M3 && dt == DSPARK_BF16))
    return fail(DSPARK_E_UNSUPPORTED, "%s: dtype %d over a cache of dtype %d", fn, (int)dt,
                (int)c->dtype);
  if (num_heads < 1 || num_heads > DSPARK_MAX_HEADS || num_heads % c->num_kv_heads != 0 ||
      num_heads / c->num_kv_heads > DSPARK_MAX_GROUP)
    return fail(DSPARK_E_INVALID,
                "%s: num_heads = %d must be a multiple of num_kv_heads = %d, at most %d times it "
                "and %d",
                fn, num_heads, c->num_kv_heads, DSPARK_MAX_GROUP, DSPARK_MAX_HEADS);
  return DSPARK_OK;
}

// Rows of `heads` dense heads of 16-bit elements.
inline dspark_status check_rows(const char* fn, const char* name, const void* p, int64_t ld,
                         int64_t row_elems, int32_t max_rows) {
  if (max_rows > 0 && (!p || !aligned16(p)))
    return fail(DSPARK_E_INVALID, "%s: %s NULL or not 16-byte aligned", fn, name);
  if (ld < row_elems || ld % 8 != 0 || ld > (1LL << 40))
    return fail(DSPARK_E_INVALID,
                "%s: the row stride %lld of %s must be >= %lld elements and a multiple of 8", fn,
                (long long)ld, name, (long long)row_elems);
  return DSPARK_OK;
}

}  // namespace dspark
