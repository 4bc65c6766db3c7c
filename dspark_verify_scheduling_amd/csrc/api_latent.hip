// C entry points of the target pass over a latent cache: argument checks on the
// host, then kernel launches on the caller's stream.
#include <float.h>

#include "api_checks.h"
#include "latent.h"

using dspark::aligned16;
using dspark::check_requests;
using dspark::check_rows;
using dspark::fail;
using dspark::launched;

namespace {

// The cache's own fields; fills `kv`. `layers`: also the strides between layers.
dspark_status check_latent(const char* fn, const dspark_latent_cache* c, bool layers,
                           dspark::LatentView* kv) {
  if (!c) return fail(DSPARK_E_INVALID, "%s: cache is NULL", fn);
  if (c->dtype != DSPARK_BF16 && c->dtype != DSPARK_F16 && c->dtype != DSPARK_E4M3)
    return fail(DSPARK_E_UNSUPPORTED, "%s: unsupported cache dtype %d", fn, (int)c->dtype);
  if (c->latent_dim != 256 && c->latent_dim != 512)
    return fail(DSPARK_E_UNSUPPORTED, "%s: latent_dim = %d is not 256 or 512", fn, c->latent_dim);
  int shift = 0;
  for (int s = 4; s <= 8; ++s) shift = c->block_size == 1 << s ? s : shift;
  if (!shift)
    return fail(DSPARK_E_UNSUPPORTED, "%s: block_size = %d is not 16, 32, 64, 128 or 256", fn,
                c->block_size);
  if (c->num_blocks < 1)
    return fail(DSPARK_E_INVALID, "%s: num_blocks = %d < 1", fn, c->num_blocks);
  const bool e8 = c->dtype == DSPARK_E4M3;
  struct {
    const char* name;
    const void* p;
    int64_t stride, layer, row, bytes;  // elements, elements, of a token, of an element
  } parts[3] = {{"latent", c->latent, c->block_stride, c->layer_stride, c->latent_dim, e8 ? 1 : 2},
                {"rope", c->rope, c->rope_block_stride, c->rope_layer_stride, DSPARK_LATENT_ROPE, 2},
                {"scale", c->scale, c->scale_block_stride, c->scale_layer_stride,
                 c->latent_dim / DSPARK_LATENT_GROUP, 1}};
  if (layers && (c->num_layers < 1 || c->num_layers > DSPARK_MAX_LAYERS))
    return fail(DSPARK_E_INVALID, "%s: num_layers = %d outside [1, %d]", fn, c->num_layers,
                DSPARK_MAX_LAYERS);
  const bool many = layers && c->num_layers > 1;
  for (int i = 0; i < (e8 ? 3 : 2); ++i) {
    const auto& x = parts[i];
    const int64_t page = x.row * c->block_size;
    if (!x.p || !aligned16(x.p))
      return fail(DSPARK_E_INVALID, "%s: %s of the cache NULL or not 16-byte aligned", fn, x.name);
    if (x.stride < page || x.stride > (1LL << 40) || x.stride * x.bytes % 16 != 0)
      return fail(DSPARK_E_INVALID,
                  "%s: the page stride %lld of %s must be >= %lld elements and a multiple of 16 "
                  "bytes",
                  fn, (long long)x.stride, x.name, (long long)page);
    if (many && (x.layer < page || x.layer > (1LL << 50) || x.layer * x.bytes % 16 != 0))
      return fail(DSPARK_E_INVALID,
                  "%s: layers of %s overlap, or their stride is not a multiple of 16 bytes", fn,
                  x.name);
  }
  kv->latent = static_cast<unsigned char*>(c->latent);
  kv->rope = static_cast<unsigned char*>(c->rope);
  kv->scale = e8 ? c->scale : nullptr;
  kv->page_bytes = c->block_stride * (e8 ? 1 : 2);
  kv->rope_page_bytes = c->rope_block_stride * 2;
  kv->scale_page_bytes = e8 ? c->scale_block_stride : 0;
  kv->layer_bytes = many ? c->layer_stride * (e8 ? 1 : 2) : 0;
  kv->rope_layer_bytes = many ? c->rope_layer_stride * 2 : 0;
  kv->scale_layer_bytes = many && e8 ? c->scale_layer_stride : 0;
  kv->num_layers = layers ? c->num_layers : 1;
  kv->num_blocks = c->num_blocks;
  kv->page_shift = shift;
  kv->dim = c->latent_dim;
  kv->cb = e8 ? 1 : 2;
  return DSPARK_OK;
}

// The query side: `least` heads or more.
dspark_status check_queries(const char* fn, int32_t num_heads, int32_t least, dspark_dtype dt,
                            const dspark_latent_cache* c) {
  if (dt != DSPARK_BF16 && dt != DSPARK_F16)
    return fail(DSPARK_E_UNSUPPORTED, "%s: unsupported dtype %d", fn, (int)dt);
  if (c->dtype != dt && !(c->dtype == DSPARK_E4M3 && dt == DSPARK_BF16))
    return fail(DSPARK_E_UNSUPPORTED, "%s: dtype %d over a cache of dtype %d", fn, (int)dt,
                (int)c->dtype);
  if (num_heads < least || num_heads > DSPARK_LATENT_MAX_HEADS)
    return fail(DSPARK_E_INVALID, "%s: num_heads = %d outside [%d, %d]", fn, num_heads, least,
                DSPARK_LATENT_MAX_HEADS);
  return DSPARK_OK;
}

// Rows whose heads have a stride of their own: a row's heads lie together, or a head's
// rows do (as a product for each head leaves them).
dspark_status check_head_rows(const char* fn, const char* name, const void* p, int64_t ld,
                              int64_t head_ld, int32_t heads, int64_t dim, int32_t max_rows) {
  if (heads <= 1) return check_rows(fn, name, p, ld, dim, max_rows);
  if (head_ld < dim || head_ld % 8 != 0 || head_ld > (1LL << 40))
    return fail(DSPARK_E_INVALID,
                "%s: the head stride %lld of %s must be >= %lld elements and a multiple of 8", fn,
                (long long)head_ld, name, (long long)dim);
  const int64_t row = (heads - 1) * head_ld + dim;
  const bool by_head = ld < row && (max_rows < 2 || ld <= (head_ld - dim) / (max_rows - 1));
  return check_rows(fn, name, p, ld, by_head ? dim : row, max_rows);
}

}  // namespace

extern "C" {

dspark_status dspark_latent_append(int32_t B, int32_t gamma, int32_t num_heads, dspark_dtype dt,
                                   const void* kv, int64_t kv_ld, const void* q_rope,
                                   int64_t q_ld, int64_t q_head_ld, int32_t max_rows,
                                   const int32_t* cu_seqlens, const int32_t* prefix_lens,
                                   const int32_t* tree_parents, const int32_t* block_table,
                                   int32_t table_width, const void* weight, float eps,
                                   const float* rope, int32_t rope_rows, int32_t rope_interleaved,
                                   void* q_rope_out, int64_t q_out_ld, int64_t q_out_head_ld,
                                   const dspark_latent_cache* cache, int32_t* append_meta,
                                   void* stream) {
  const char* fn = "dspark_latent_append";
  dspark::LatentAppendArgs a;
  dspark_status st = check_latent(fn, cache, false, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, gamma == 0 ? 1 : gamma, max_rows, cu_seqlens, prefix_lens,
                      tree_parents, block_table, table_width, &a.req);
  if (st != DSPARK_OK) return st;
  a.req.gamma = gamma;
  if (gamma == 0 && tree_parents)
    return fail(DSPARK_E_INVALID, "%s: tree_parents needs gamma >= 1", fn);
  st = check_queries(fn, num_heads, 0, dt, cache);
  if (st != DSPARK_OK) return st;
  const int32_t rows = B > 0 ? max_rows : 0;
  st = check_rows(fn, "kv", kv, kv_ld, cache->latent_dim + DSPARK_LATENT_ROPE, rows);
  if (st != DSPARK_OK) return st;
  if (num_heads > 0) {
    st = check_head_rows(fn, "q_rope", q_rope, q_ld, q_head_ld, num_heads, DSPARK_LATENT_ROPE, rows);
    if (st != DSPARK_OK) return st;
    st = check_head_rows(fn, "q_rope_out", q_rope_out, q_out_ld, q_out_head_ld, num_heads,
                         DSPARK_LATENT_ROPE, rows);
    if (st != DSPARK_OK) return st;
    if (q_rope_out == q_rope && (q_out_ld != q_ld || (num_heads > 1 && q_out_head_ld != q_head_ld)))
      return fail(DSPARK_E_INVALID, "%s: q_rope_out is q_rope, but their strides differ", fn);
  }
  if (!append_meta) return fail(DSPARK_E_INVALID, "%s: append_meta is NULL", fn);
  if (!aligned16(weight) || !aligned16(rope))
    return fail(DSPARK_E_INVALID, "%s: weight or rope is not 16-byte aligned", fn);
  if (!(eps >= 0.0f && eps <= FLT_MAX))
    return fail(DSPARK_E_INVALID, "%s: eps must be >= 0 and finite", fn);
  if (rope && rope_rows < 1)
    return fail(DSPARK_E_INVALID, "%s: rope_rows = %d < 1", fn, rope_rows);
  a.num_heads = num_heads;
  a.x = static_cast<const unsigned char*>(kv);
  a.q = static_cast<const unsigned char*>(q_rope);
  a.q_out = static_cast<unsigned char*>(q_rope_out);
  a.x_ld = 2 * kv_ld;
  a.q_ld = num_heads > 0 ? 2 * q_ld : 0;
  a.q_head_ld = num_heads > 1 ? 2 * q_head_ld : 0;
  a.q_out_ld = num_heads > 0 ? 2 * q_out_ld : 0;
  a.q_out_head_ld = num_heads > 1 ? 2 * q_out_head_ld : 0;
  a.weight = weight;
  a.eps = eps;
  a.rope = rope;
  a.rope_rows = rope ? rope_rows : 0;
  a.rope_interleaved = rope_interleaved != 0;
  a.meta = append_meta;
  a.first_row = 0;
  return launched(dspark::launch_latent_append(a, dt, (hipStream_t)stream), fn);
}

dspark_status dspark_latent_read(int32_t B, int32_t max_rows, const int32_t* cu_seqlens,
                                 const int32_t* starts, const int32_t* block_table,
                                 int32_t table_width, const dspark_latent_cache* cache,
                                 void* latent_out, int64_t out_ld, void* rope_out,
                                 int64_t rope_out_ld, int32_t* read_meta, void* stream) {
  const char* fn = "dspark_latent_read";
  dspark::LatentReadArgs a;
  dspark_status st = check_latent(fn, cache, false, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, 1, max_rows, cu_seqlens, starts, nullptr, block_table,
                      table_width, &a.req);
  if (st != DSPARK_OK) return st;
  const int32_t rows = B > 0 ? max_rows : 0;
  st = check_rows(fn, "latent_out", latent_out, out_ld, cache->latent_dim, rows);
  if (st != DSPARK_OK) return st;
  st = check_rows(fn, "rope_out", rope_out, rope_out_ld, DSPARK_LATENT_ROPE, rows);
  if (st != DSPARK_OK) return st;
  if (!read_meta) return fail(DSPARK_E_INVALID, "%s: read_meta is NULL", fn);
  a.latent_out = static_cast<unsigned char*>(latent_out);
  a.rope_out = static_cast<unsigned char*>(rope_out);
  a.out_ld = 2 * out_ld;
  a.rope_out_ld = 2 * rope_out_ld;
  a.meta = read_meta;
  a.first_row = 0;
  return launched(dspark::launch_latent_read(a, (hipStream_t)stream), fn);
}

dspark_status dspark_latent_commit(int32_t B, int32_t gamma, const int32_t* path_rows,
                                   const int32_t* num_correct, const int32_t* prefix_lens,
                                   const int32_t* block_table, int32_t table_width,
                                   const dspark_latent_cache* cache, int32_t* commit_meta,
                                   void* stream) {
  const char* fn = "dspark_latent_commit";
  dspark::LatentView kv;
  dspark::CommitArgs a = {};
  dspark_status st = check_latent(fn, cache, true, &kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, false, B, gamma, 0, nullptr, prefix_lens, nullptr, block_table,
                      table_width, &a.req);
  if (st != DSPARK_OK) return st;
  if (B > 0 && (!path_rows || !num_correct))
    return fail(DSPARK_E_INVALID, "%s: path_rows or num_correct is NULL", fn);
  if (!commit_meta) return fail(DSPARK_E_INVALID, "%s: commit_meta is NULL", fn);
  // what the look-up of moves reads of a cache
  a.kv.page_shift = kv.page_shift;
  a.kv.num_blocks = kv.num_blocks;
  a.path = path_rows;
  a.num_correct = num_correct;
  a.meta = commit_meta;
  return launched(dspark::launch_latent_commit(a, kv, (hipStream_t)stream), fn);
}

size_t dspark_latent_attention_workspace_size(int32_t B, int32_t gamma, int32_t num_heads,
                                              int32_t latent_dim) {
  if (B < 0 || B > DSPARK_MAX_BATCH || gamma < 1 || gamma > DSPARK_MAX_GAMMA || num_heads < 1 ||
      num_heads > DSPARK_LATENT_MAX_HEADS || (latent_dim != 256 && latent_dim != 512))
    return 0;
  return dspark::latent_attention_workspace(B, gamma, num_heads, latent_dim);
}

dspark_status dspark_latent_attention(int32_t B, int32_t gamma, int32_t num_heads,
                                      dspark_dtype dt, const void* q_latent, int64_t ql_ld,
                                      int64_t ql_head_ld, const void* q_rope, int64_t qr_ld,
                                      int64_t qr_head_ld, int32_t max_rows,
                                      const int32_t* cu_seqlens, const int32_t* prefix_lens,
                                      const int32_t* tree_parents, const int32_t* block_table,
                                      int32_t table_width, const dspark_latent_cache* cache,
                                      float scale, void* out, int64_t out_ld, float* lse,
                                      int32_t* attention_meta, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  const char* fn = "dspark_latent_attention";
  dspark::LatentAttnArgs a;
  dspark_status st = check_latent(fn, cache, false, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, gamma, max_rows, cu_seqlens, prefix_lens, tree_parents,
                      block_table, table_width, &a.req);
  if (st != DSPARK_OK) return st;
  st = check_queries(fn, num_heads, 1, dt, cache);
  if (st != DSPARK_OK) return st;
  const int32_t rows = B > 0 ? max_rows : 0;
  st = check_head_rows(fn, "q_latent", q_latent, ql_ld, ql_head_ld, num_heads, cache->latent_dim,
                       rows);
  if (st != DSPARK_OK) return st;
  st = check_head_rows(fn, "q_rope", q_rope, qr_ld, qr_head_ld, num_heads, DSPARK_LATENT_ROPE, rows);
  if (st != DSPARK_OK) return st;
  st = check_rows(fn, "out", out, out_ld, (int64_t)num_heads * cache->latent_dim, rows);
  if (st != DSPARK_OK) return st;
  if (!attention_meta) return fail(DSPARK_E_INVALID, "%s: attention_meta is NULL", fn);
  if (!(scale >= -FLT_MAX && scale <= FLT_MAX))
    return fail(DSPARK_E_INVALID, "%s: scale is not finite", fn);
  const size_t need = dspark::latent_attention_workspace(B, gamma, num_heads, cache->latent_dim);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < need)
    return fail(DSPARK_E_WORKSPACE, "%s: workspace needs %zu bytes, 256-byte aligned", fn, need);
  a.num_heads = num_heads;
  a.ql = static_cast<const unsigned char*>(q_latent);
  a.qr = static_cast<const unsigned char*>(q_rope);
  a.ql_ld = 2 * ql_ld;
  a.ql_head_ld = num_heads > 1 ? 2 * ql_head_ld : 0;
  a.qr_ld = 2 * qr_ld;
  a.qr_head_ld = num_heads > 1 ? 2 * qr_head_ld : 0;
  a.scale = scale;
  a.out = static_cast<unsigned char*>(out);
  a.out_ld = 2 * out_ld;
  a.lse = lse;
  a.meta = attention_meta;
  a.ws = workspace;
  return launched(dspark::launch_latent_attention(a, dt, (hipStream_t)stream), fn);
}

size_t dspark_latent_prefill_workspace_size(int32_t B, int32_t max_rows, int32_t max_keys,
                                            int32_t num_heads, int32_t nope, int32_t latent_dim) {
  if (B < 0 || B > DSPARK_MAX_BATCH || max_rows < 0 || max_keys < 0 ||
      max_keys > DSPARK_LATENT_MAX_KEYS || num_heads < 1 ||
      num_heads > DSPARK_LATENT_MAX_HEADS || (nope != 64 && nope != 128) ||
      (latent_dim != 256 && latent_dim != 512))
    return 0;
  return dspark::latent_prefill_workspace(B, max_rows, max_keys, num_heads, nope, latent_dim);
}

dspark_status dspark_latent_prefill(int32_t B, int32_t num_heads, int32_t nope, dspark_dtype dt,
                                    const void* q, int64_t q_ld, const void* w_k,
                                    const void* w_v, int64_t w_head_ld, int32_t max_rows,
                                    int32_t max_keys, const int32_t* cu_seqlens,
                                    const int32_t* prefix_lens, const int32_t* block_table,
                                    int32_t table_width, const dspark_latent_cache* cache,
                                    float scale, void* out, int64_t out_ld, float* lse,
                                    int32_t* prefill_meta, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const char* fn = "dspark_latent_prefill";
  dspark::LatentPrefillArgs a;
  dspark_status st = check_latent(fn, cache, false, &a.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, 1, max_rows, cu_seqlens, prefix_lens, nullptr, block_table,
                      table_width, &a.req);
  if (st != DSPARK_OK) return st;
  st = check_queries(fn, num_heads, 1, dt, cache);
  if (st != DSPARK_OK) return st;
  if (nope != 64 && nope != 128)
    return fail(DSPARK_E_UNSUPPORTED, "%s: nope = %d is not 64 or 128", fn, nope);
  if (max_keys < 0) return fail(DSPARK_E_INVALID, "%s: max_keys = %d < 0", fn, max_keys);
  if (max_keys > DSPARK_LATENT_MAX_KEYS)
    return fail(DSPARK_E_UNSUPPORTED, "%s: max_keys = %d exceeds %d", fn, max_keys,
                DSPARK_LATENT_MAX_KEYS);
  const int32_t rows = B > 0 ? max_rows : 0;
  st = check_rows(fn, "q", q, q_ld, (int64_t)num_heads * (nope + DSPARK_LATENT_ROPE), rows);
  if (st != DSPARK_OK) return st;
  st = check_rows(fn, "out", out, out_ld, (int64_t)num_heads * nope, rows);
  if (st != DSPARK_OK) return st;
  if (!w_k || !w_v || !aligned16(w_k) || !aligned16(w_v))
    return fail(DSPARK_E_INVALID, "%s: w_k or w_v NULL or not 16-byte aligned", fn);
  if (num_heads > 1 && (w_head_ld < (int64_t)nope * cache->latent_dim || w_head_ld % 8 != 0 ||
                        w_head_ld > (1LL << 40)))
    return fail(DSPARK_E_INVALID,
                "%s: the head stride %lld of the weights must be >= %lld elements and a multiple "
                "of 8",
                fn, (long long)w_head_ld, (long long)nope * cache->latent_dim);
  if (!prefill_meta) return fail(DSPARK_E_INVALID, "%s: prefill_meta is NULL", fn);
  if (!(scale >= -FLT_MAX && scale <= FLT_MAX))
    return fail(DSPARK_E_INVALID, "%s: scale is not finite", fn);
  const size_t need = dspark::latent_prefill_workspace(B, max_rows, max_keys, num_heads, nope,
                                                       cache->latent_dim);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < need)
    return fail(DSPARK_E_WORKSPACE, "%s: workspace needs %zu bytes, 256-byte aligned", fn, need);
  a.num_heads = num_heads;
  a.nope = nope;
  a.max_keys = max_keys;
  a.q = static_cast<const unsigned char*>(q);
  a.wk = static_cast<const unsigned char*>(w_k);
  a.wv = static_cast<const unsigned char*>(w_v);
  a.q_ld = 2 * q_ld;
  a.w_head_ld = num_heads > 1 ? 2 * w_head_ld : 0;
  a.scale = scale;
  a.out = static_cast<unsigned char*>(out);
  a.out_ld = 2 * out_ld;
  a.lse = lse;
  a.meta = prefill_meta;
  a.ws = workspace;
  return launched(dspark::launch_latent_prefill(a, dt, (hipStream_t)stream), fn);
}

}  // extern "C"
