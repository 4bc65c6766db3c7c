// C entry points of the target pass: argument checks on the host, then kernel
// launches on the caller's stream.
#include <float.h>

#include "api_checks.h"
#include "latent.h"

using dspark::aligned16;
using dspark::check_cache;
using dspark::check_heads;
using dspark::check_requests;
using dspark::check_rows;
using dspark::fail;
using dspark::launched;

namespace {

// What the two appends to a key/value cache take alike; fills `a`.
dspark_status append_args(const char* fn, int32_t B, int32_t num_heads, const void* q, int64_t q_ld,
                          const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                          int32_t max_rows, const void* q_weight, const void* k_weight, float eps,
                          const float* rope, int32_t rope_rows, int32_t rope_dim,
                          int32_t rope_interleaved, void* q_out, int64_t q_out_ld,
                          const dspark_kv_cache* cache, int32_t* append_meta,
                          dspark::AppendArgs* args) {
  dspark_status st;
  dspark::AppendArgs& a = *args;
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
  st = append_args(fn, B, num_heads, q, q_ld, k, k_ld, v, v_ld, max_rows, q_weight, k_weight, eps,
                   rope, rope_rows, rope_dim, rope_interleaved, q_out, q_out_ld, cache, append_meta,
                   &a);
  if (st != DSPARK_OK) return st;
  return launched(dspark::launch_append(a, dt, (hipStream_t)stream), fn);
}

dspark_status dspark_kv_append_axes(int32_t B, int32_t num_heads, dspark_dtype dt, const void* q,
                                    int64_t q_ld, const void* k, int64_t k_ld, const void* v,
                                    int64_t v_ld, int32_t max_rows, const int32_t* cu_seqlens,
                                    const int32_t* prefix_lens, const int32_t* positions,
                                    int64_t positions_ld, int32_t num_axes,
                                    const int32_t* pair_axis_host, const int32_t* block_table,
                                    int32_t table_width, const void* q_weight,
                                    const void* k_weight, float eps, const float* rope,
                                    int32_t rope_rows, int32_t rope_dim, int32_t rope_interleaved,
                                    void* q_out, int64_t q_out_ld, const dspark_kv_cache* cache,
                                    int32_t* append_meta, void* stream) {
  const char* fn = "dspark_kv_append_axes";
  dspark::AppendAxesArgs a;
  dspark_status st = check_cache(fn, cache, false, &a.base.kv);
  if (st != DSPARK_OK) return st;
  st = check_requests(fn, true, B, 1, max_rows, cu_seqlens, prefix_lens, nullptr, block_table,
                      table_width, &a.base.req);
  if (st != DSPARK_OK) return st;
  st = check_heads(fn, num_heads, dt, cache);
  if (st != DSPARK_OK) return st;
  st = append_args(fn, B, num_heads, q, q_ld, k, k_ld, v, v_ld, max_rows, q_weight, k_weight, eps,
                   rope, rope_rows, rope_dim, rope_interleaved, q_out, q_out_ld, cache, append_meta,
                   &a.base);
  if (st != DSPARK_OK) return st;
  if (!rope) return fail(DSPARK_E_INVALID, "%s: rope is NULL", fn);
  if (num_axes < 1 || num_axes > DSPARK_MAX_AXES)
    return fail(DSPARK_E_INVALID, "%s: num_axes = %d outside [1, %d]", fn, num_axes,
                DSPARK_MAX_AXES);
  if (B > 0 && max_rows > 0 && !positions)
    return fail(DSPARK_E_INVALID, "%s: positions is NULL", fn);
  if (positions_ld < max_rows || positions_ld > (1LL << 40))
    return fail(DSPARK_E_INVALID, "%s: positions_ld = %lld is less than max_rows = %d", fn,
                (long long)positions_ld, max_rows);
  if (!pair_axis_host) return fail(DSPARK_E_INVALID, "%s: pair_axis_host is NULL", fn);
  for (auto& w : a.axis) w = 0;
  for (int i = 0; i < rope_dim / 2; ++i) {
    if (pair_axis_host[i] < 0 || pair_axis_host[i] >= num_axes)
      return fail(DSPARK_E_INVALID, "%s: pair_axis_host[%d] = %d outside [0, %d)", fn, i,
                  pair_axis_host[i], num_axes);
    a.axis[i >> 5] |= (uint64_t)pair_axis_host[i] << (2 * (i & 31));
  }
  a.positions = positions;
  a.positions_ld = positions_ld;
  a.num_axes = num_axes;
  return launched(dspark::launch_append_axes(a, dt, (hipStream_t)stream), fn);
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
