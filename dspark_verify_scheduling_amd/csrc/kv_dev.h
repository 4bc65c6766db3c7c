// Shared by the target-pass kernels (cache append, read and commit, tree
// attention): the device view of the paged cache, the checks of a request's
// rows and tree, and the 8-bit element conversions.
#pragma once

#include "common.h"

namespace dspark {

// dspark_kv_cache with byte strides; passed to kernels by value.
struct KvView {
  unsigned char* k;
  unsigned char* v;
  uint8_t* ks;  // null unless E4M3
  uint8_t* vs;
  int64_t page_bytes;         // from page to page
  int64_t scale_page_bytes;
  int64_t layer_bytes;        // from layer to layer
  int64_t scale_layer_bytes;
  int num_layers, num_blocks, hkv, page_shift, dim;
  int cb;  // bytes of an element
};

// A call's requests: rows, prefixes, trees, page tables.
struct ReqView {
  const int32_t* cu;
  const int32_t* prefix;
  const int32_t* parents;  // [B, gamma] or null (chain)
  const int32_t* table;    // [B, width]
  int B, gamma, max_rows, width;
};

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) unsigned int kv_u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int kv_u32x2;

struct AppendArgs {
  ReqView req;
  KvView kv;
  int num_heads;
  const unsigned char* q;
  const unsigned char* k;
  const unsigned char* v;
  int64_t q_ld, k_ld, v_ld, q_out_ld;  // bytes
  const void* q_weight;
  const void* k_weight;
  float eps;
  const float* rope;
  int rope_rows, rope_dim, rope_interleaved;
  unsigned char* q_out;
  int32_t* meta;
};
hipError_t launch_append(const AppendArgs& a, dspark_dtype dt, hipStream_t s);

struct ReadArgs {
  ReqView req;  // prefix: the first cache index of each request
  KvView kv;
  unsigned char* k_out;
  unsigned char* v_out;
  int64_t out_ld;  // bytes
  int first_row;   // of a launch
  int32_t* meta;
};
hipError_t launch_read(const ReadArgs& a, hipStream_t s);

struct CommitArgs {
  ReqView req;
  KvView kv;
  const int32_t* path;  // [B, gamma + 1]
  const int32_t* num_correct;
  int32_t* meta;
};
hipError_t launch_commit(const CommitArgs& a, hipStream_t s);

struct AttnArgs {
  ReqView req;
  KvView kv;
  int num_heads, group;
  int waves;  // of a workgroup, and so 16-row tiles of a segment, at most
  const unsigned char* q;
  int64_t q_ld;  // bytes
  float scale;
  unsigned char* out;
  int64_t out_ld;  // bytes
  float* lse;
  int32_t* meta;
  void* ws;
};
hipError_t launch_attention(const AttnArgs& a, dspark_dtype dt, hipStream_t s);
size_t attention_workspace(int B, int gamma, int num_heads, int num_kv_heads, int head_dim);

// Rows of request r inside the packed buffer: false if they are not 1..gamma+1
// rows of [0, total_eff).
__device__ inline bool request_rows(const ReqView& q, int r, int total_eff, int* c0, int* len) {
  const int s = q.cu[r], e = q.cu[r + 1];
  *c0 = s;
  // on unsigned words, so that no pair of words overflows
  *len = (int)((unsigned)e - (unsigned)s);
  return s >= 0 && e > s && e <= total_eff && e - s <= q.gamma + 1;
}

__device__ inline int rows_in_use(const ReqView& q, int* total) {
  *total = q.cu[q.B];
  return min(max(*total, 0), q.max_rows);
}

// Status bits of what a request needs before its pages and positions are
// looked at; 0 where it is well formed. For one thread.
__device__ inline int request_status(const ReqView& q, int r, int total_eff) {
  int c0, len;
  if (!request_rows(q, r, total_eff, &c0, &len)) return DSPARK_DATA_BAD_LENS;
  const int prefix = q.prefix[r];
  if (prefix < 0) return DSPARK_DATA_BAD_LENS;
  if (q.parents) {
    const int32_t* p = q.parents + (size_t)r * q.gamma;
    int bad = 0;
    for (int j = 1; j < len; ++j) bad |= p[j - 1] < 0 || p[j - 1] >= j;
    if (bad) return DSPARK_DATA_BAD_TREE;
  }
  return 0;
}

// One power of two in float32, for e in [-126, 127].
__device__ inline float pow2f(int e) { return __builtin_bit_cast(float, (e + 127) << 23); }

// The exponent of an 8-bit row whose largest finite magnitude is `amax`: the
// least e with amax <= 448 * 2^e = 1.75 * 2^(8 + e), in [-100, 119]. The upper
// end keeps 448 * 2^e a finite float32 and bfloat16 number, the lower end keeps
// the smallest code (2^-9) times 2^e normal in both.
__device__ inline int e4m3_exponent(float amax) {
  const uint32_t b = __builtin_bit_cast(uint32_t, amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0.0f ? 0 : min(max(e, -100), 119);
}

__device__ inline bool finite_f32(float x) {
  return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u;
}

// x * 2^-e as the operand of the 8-bit conversion: finite values held to the
// largest code (they pass it only where the exponent was held to 119), others
// to NaN, which the conversion keeps.
__device__ inline float e4m3_operand(float x, float inv) {
  const float y = fminf(fmaxf(x * inv, -448.0f), 448.0f);
  return finite_f32(x) ? y : __builtin_nanf("");
}

}  // namespace dspark
