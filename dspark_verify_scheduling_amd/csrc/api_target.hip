// C entry points of the target pass: argument checks on the host, then kernel
// launches on the caller's stream.
#include <float.h>

#include "api_status.h"
#include "kv_dev.h"

using dspark::aligned16;
using dspark::fail;
using dspark::launched;

namespace {

// The cache's own fields; fills `kv`. `layers`: also the strides between layers.
dspark_status check_cache(const char* fn, const dspark_kv_cache* c, bool layers,
                          dspark::KvView* kv) {
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
dspark_status check_requests(const char* fn, bool packed, int32_t B, int32_t gamma, int32_t max_rows,
                             const int32_t* cu, const int32_t* prefix, const int32_t* parents,
                             const int32_t* table, int32_t width, dspark::ReqView* q) {
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
dspark_status check_heads(const char* fn, int32_t num_heads, dspark_dtype dt,
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
dspark_status check_rows(const char* fn, const char* name, const void* p, int64_t ld,
                         int64_t row_elems, int32_t max_rows) {
  if (max_rows > 0 && (!p || !aligned16(p)))
    return fail(DSPARK_E_INVALID, "%s: %s NULL or not 16-byte aligned", fn, name);
  if (ld < row_elems || ld % 8 != 0 || ld > (1LL << 40))
    return fail(DSPARK_E_INVALID,
                "%s: the row stride %lld of %s must be >= %lld elements and a multiple of 8", fn,
                (long long)ld, name, (long long)row_elems);
  return DSPARK_OK;
}

}  // namespace

extern "C" {

dspark_status dspark_kv_append(int32_t B, int32_t gamma, int32_t num_heads, dspark_dtype dt,
                               const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                               const void* v, int64_t v_ld, int32_t max_rows,
                               const int32_t* cu_seqlens, const int32_t* prefix_lens,
                               const int32_t* tree_parents, const int32_t* block_table,
                               int32_t table_width, const void* q_weight, const void* k_weight,
                               float eps, const float* rope, int32_t rope_rows,
                               int32_t rope_dim, int32_t rope_interleaved, void* q_out,
                               int64_t q_out_ld, const dspark_kv_cache* cache,
                               int32_t* append_meta, void* stream) {
  const char* fn = "dspark_kv_append";
  dspark::AppendArgs a;
  dspark_status st = check_cache(fn, cache, false, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, gamma, max_rows, cu_seqlens, prefix_lens, tree_parents,
                      block_table, table_width, &a.req);
  if (st != DSPARK_OK) return st;
  st = check_heads(fn, num_heads, dt, cache);
  if (st != DSPARK_OK) return st;
  const int64_t D = cache->head_dim;
  const struct {
    const char* name;
    const void* p;
    int64_t ld, heads;
  } rows[4] = {{"q", q, q_ld, num_heads},
               {"k", k, k_ld, cache->num_kv_heads},
               {"v", v, v_ld, cache->num_kv_heads},
               {"q_out", q_out, q_out_ld, num_heads}};
  for (const auto& x : rows) {
    st = check_rows(fn, x.name, x.p, x.ld, x.heads * D, B > 0 ? max_rows : 0);
    if (st != DSPARK_OK) return st;
  }
  if (q_out == q && q_out_ld != q_ld)
    return fail(DSPARK_E_INVALID, "%s: q_out is q, but their row strides differ", fn);
  if (!append_meta) return fail(DSPARK_E_INVALID, "%s: append_meta is NULL", fn);
  if (!aligned16(q_weight) || !aligned16(k_weight))
    return fail(DSPARK_E_INVALID, "%s: a weight is not 16-byte aligned", fn);
  if (!(eps >= 0.0f && eps <= FLT_MAX))
    return fail(DSPARK_E_INVALID, "%s: eps must be >= 0 and finite", fn);
  if (rope) {
    if (!aligned16(rope)) return fail(DSPARK_E_INVALID, "%s: rope is not 16-byte aligned", fn);
    if (rope_rows < 1) return fail(DSPARK_E_INVALID, "%s: rope_rows = %d < 1", fn, rope_rows);
    if (rope_dim < 16 || rope_dim % 16 != 0 || rope_dim > D)
      return fail(DSPARK_E_INVALID,
                  "%s: rope_dim = %d must be a multiple of 16 up to head_dim = %d", fn, rope_dim,
                  (int)D);
  }
  a.num_heads = num_heads;
  a.q = static_cast<const unsigned char*>(q);
  a.k = static_cast<const unsigned char*>(k);
  a.v = static_cast<const unsigned char*>(v);
  a.q_ld = 2 * q_ld;
  a.k_ld = 2 * k_ld;
  a.v_ld = 2 * v_ld;
  a.q_out_ld = 2 * q_out_ld;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.rope = rope;
  a.rope_rows = rope ? rope_rows : 0;
  a.rope_dim = rope ? rope_dim : 0;
  a.rope_interleaved = rope_interleaved != 0;
  a.q_out = static_cast<unsigned char*>(q_out);
  a.meta = append_meta;
  return launched(dspark::launch_append(a, dt, (hipStream_t)stream), fn);
}

dspark_status dspark_kv_read(int32_t B, int32_t max_rows, const int32_t* cu_seqlens,
                             const int32_t* starts, const int32_t* block_table,
                             int32_t table_width, const dspark_kv_cache* cache, void* k_out,
                             void* v_out, int64_t out_ld, int32_t* read_meta, void* stream) {
  const char* fn = "dspark_kv_read";
  dspark::ReadArgs a;
  dspark_status st = check_cache(fn, cache, false, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, 1, max_rows, cu_seqlens, starts, nullptr, block_table,
                      table_width, &a.req);
  if (st != DSPARK_OK) return st;
  const int64_t row = (int64_t)cache->num_kv_heads * cache->head_dim;
  st = check_rows(fn, "k_out", k_out, out_ld, row, B > 0 ? max_rows : 0);
  if (st != DSPARK_OK) return st;
  st = check_rows(fn, "v_out", v_out, out_ld, row, B > 0 ? max_rows : 0);
  if (st != DSPARK_OK) return st;
  if (!read_meta) return fail(DSPARK_E_INVALID, "%s: read_meta is NULL", fn);
  a.k_out = static_cast<unsigned char*>(k_out);
  a.v_out = static_cast<unsigned char*>(v_out);
  a.out_ld = 2 * out_ld;
  a.meta = read_meta;
  return launched(dspark::launch_read(a, (hipStream_t)stream), fn);
}

size_t dspark_tree_attention_workspace_size(int32_t B, int32_t gamma, int32_t num_heads,
                                            int32_t num_kv_heads, int32_t head_dim) {
  if (B < 0 || B > DSPARK_MAX_BATCH || gamma < 1 || gamma > DSPARK_MAX_GAMMA ||
      num_kv_heads < 1 || num_kv_heads > DSPARK_MAX_HEADS || num_heads < 1 ||
      num_heads > DSPARK_MAX_HEADS || num_heads % num_kv_heads != 0 ||
      num_heads / num_kv_heads > DSPARK_MAX_GROUP ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  return dspark::attention_workspace(B, gamma, num_heads, num_kv_heads, head_dim);
}

dspark_status dspark_tree_attention(int32_t B, int32_t gamma, int32_t num_heads, dspark_dtype dt,
                                    const void* q, int64_t q_ld, int32_t max_rows,
                                    const int32_t* cu_seqlens, const int32_t* prefix_lens,
                                    const int32_t* tree_parents, const int32_t* block_table,
                                    int32_t table_width, const dspark_kv_cache* cache,
                                    float scale, void* out, int64_t out_ld, float* lse,
                                    int32_t* attention_meta, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const char* fn = "dspark_tree_attention";
  dspark::AttnArgs a;
  dspark_status st = check_cache(fn, cache, false, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, gamma, max_rows, cu_seqlens, prefix_lens, tree_parents,
                      block_table, table_width, &a.req);
  if (st != DSPARK_OK) return st;
  st = check_heads(fn, num_heads, dt, cache);
  if (st != DSPARK_OK) return st;
  const int64_t row = (int64_t)num_heads * cache->head_dim;
  st = check_rows(fn, "q", q, q_ld, row, B > 0 ? max_rows : 0);
  if (st != DSPARK_OK) return st;
  st = check_rows(fn, "out", out, out_ld, row, B > 0 ? max_rows : 0);
  if (st != DSPARK_OK) return st;
  if (!attention_meta) return fail(DSPARK_E_INVALID, "%s: attention_meta is NULL", fn);
  if (!(scale >= -FLT_MAX && scale <= FLT_MAX))
    return fail(DSPARK_E_INVALID, "%s: scale is not finite", fn);
  const size_t need =
      dspark::attention_workspace(B, gamma, num_heads, cache->num_kv_heads, cache->head_dim);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < need)
    return fail(DSPARK_E_WORKSPACE, "%s: workspace needs %zu bytes, 256-byte aligned", fn, need);
  a.num_heads = num_heads;
  a.group = num_heads / cache->num_kv_heads;
  a.q = static_cast<const unsigned char*>(q);
  a.q_ld = 2 * q_ld;
  a.scale = scale;
  a.out = static_cast<unsigned char*>(out);
  a.out_ld = 2 * out_ld;
  a.lse = lse;
  a.meta = attention_meta;
  a.ws = workspace;
  return launched(dspark::launch_attention(a, dt, (hipStream_t)stream), fn);
}

dspark_status dspark_kv_commit(int32_t B, int32_t gamma, const int32_t* path_rows,
                               const int32_t* num_correct, const int32_t* prefix_lens,
                               const int32_t* block_table, int32_t table_width,
                               const dspark_kv_cache* cache, int32_t* commit_meta, void* stream) {
  const char* fn = "dspark_kv_commit";
  dspark::CommitArgs a;
  dspark_status st = check_cache(fn, cache, true, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, false, B, gamma, 0, nullptr, prefix_lens, nullptr, block_table,
                      table_width, &a.req);
  if (st != DSPARK_OK) return st;
  if (B > 0 && (!path_rows || !num_correct))
    return fail(DSPARK_E_INVALID, "%s: path_rows or num_correct is NULL", fn);
  if (!commit_meta) return fail(DSPARK_E_INVALID, "%s: commit_meta is NULL", fn);
  a.path = path_rows;
  a.num_correct = num_correct;
  a.meta = commit_meta;
  return launched(dspark::launch_commit(a, (hipStream_t)stream), fn);
}

}  // extern "C"
