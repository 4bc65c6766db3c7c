// Shared by the kernels over a latent cache and by the append with positions on
// several axes: the device view of the cache, the calls' arguments, and the
// search for packed rows' requests.
#pragma once

#include "kv_dev.h"
#include "request_search.h"

namespace dspark {

constexpr int kRope = DSPARK_LATENT_ROPE;
constexpr int kLatGroup = DSPARK_LATENT_GROUP;

// dspark_latent_cache with byte strides; passed to kernels by value.
struct LatentView {
  unsigned char* latent;
  unsigned char* rope;
  uint8_t* scale;  // null unless E4M3
  int64_t page_bytes, rope_page_bytes, scale_page_bytes;     // from page to page
  int64_t layer_bytes, rope_layer_bytes, scale_layer_bytes;  // from layer to layer
  int num_layers, num_blocks, page_shift, dim;
  int cb;  // bytes of a latent's element
};

struct AppendAxesArgs {
  AppendArgs base;  // req: gamma 0, no parents
  const int32_t* positions;
  int64_t positions_ld;
  int num_axes;
  uint64_t axis[4];   // two bits a pair, 32 pairs a word
  int64_t first_row;  // of a launch
};
hipError_t launch_append_axes(const AppendAxesArgs& a, dspark_dtype dt, hipStream_t s);

struct LatentAppendArgs {
  ReqView req;  // gamma 0: any number of rows
  LatentView kv;
  int num_heads;
  const unsigned char* x;
  const unsigned char* q;
  unsigned char* q_out;
  int64_t x_ld, q_ld, q_head_ld, q_out_ld, q_out_head_ld;  // bytes
  const void* weight;
  float eps;
  const float* rope;
  int rope_rows, rope_interleaved;
  int32_t* meta;
  int64_t first_row;  // of a launch
};
hipError_t launch_latent_append(const LatentAppendArgs& a, dspark_dtype dt, hipStream_t s);

struct LatentReadArgs {
  ReqView req;  // prefix: the first cache index of each request
  LatentView kv;
  unsigned char* latent_out;
  unsigned char* rope_out;
  int64_t out_ld, rope_out_ld;  // bytes
  int32_t* meta;
  int64_t first_row;  // of a launch
};
hipError_t launch_latent_read(const LatentReadArgs& a, hipStream_t s);

hipError_t launch_latent_commit(const CommitArgs& a, const LatentView& kv, hipStream_t s);

struct LatentAttnArgs {
  ReqView req;
  LatentView kv;
  int num_heads;
  const unsigned char* ql;
  const unsigned char* qr;
  int64_t ql_ld, ql_head_ld, qr_ld, qr_head_ld;  // bytes
  float scale;
  unsigned char* out;
  int64_t out_ld;  // bytes
  float* lse;
  int32_t* meta;
  void* ws;
};
hipError_t launch_latent_attention(const LatentAttnArgs& a, dspark_dtype dt, hipStream_t s);
size_t latent_attention_workspace(int B, int gamma, int num_heads, int latent_dim);

struct LatentPrefillArgs {
  ReqView req;  // gamma 0
  LatentView kv;
  int num_heads, nope, max_keys;
  const unsigned char* q;
  const unsigned char* wk;
  const unsigned char* wv;
  int64_t q_ld, w_head_ld;  // bytes
  float scale;
  unsigned char* out;
  int64_t out_ld;  // bytes
  float* lse;
  int32_t* meta;
  void* ws;
};
hipError_t launch_latent_prefill(const LatentPrefillArgs& a, dspark_dtype dt, hipStream_t s);
size_t latent_prefill_workspace(int B, int max_rows, int max_keys, int num_heads, int nope,
                                int latent_dim);

// The lines of a kernel's first `BYTES` of arguments, read together. The compiler
// reads an argument where it is first used, and each new line is then a round trip
// to where the launch left it, one after the other.
template <size_t BYTES>
__device__ __forceinline__ void fetch_args() {
  typedef __attribute__((address_space(4))) const unsigned u32;
  const u32* p = (const u32*)__builtin_amdgcn_kernarg_segment_ptr();
  constexpr int kLines = (BYTES + 63) / 64;
  unsigned x[kLines];
#pragma unroll
  for (int i = 0; i < kLines; ++i) x[i] = p[i * 16];
#pragma unroll
  for (int i = 0; i < kLines; ++i) asm volatile("" ::"s"(x[i]));
}

// Whether request c's rows are well formed as far as its words say (its tree and
// page ids apart), and where they are. Rows in all: `most`.
__device__ inline bool span_of(const ReqView& q, int c, int total_eff, int64_t reach, int64_t most,
                               int* s, int* e, int* prefix) {
  *s = q.cu[c];
  *e = q.cu[c + 1];
  *prefix = q.prefix[c];
  return *s >= 0 && *e >= *s && *e <= total_eff && *prefix >= 0 &&
         (int64_t)*prefix + (*e - *s) <= reach && *e - *s <= most;
}

// The requests of the packed rows first .. first + N - 1, lane i of the wave for
// row first + i: *r the request, *j the row's index in it, -1 where the row
// belongs to no well-formed one, *prefix the request's. All lanes of the wave call it together. 64
// steps of the search at once and its rows together, so that a batch of up to
// 64 requests costs two memory latencies.
template <int N>
__device__ inline void rows_requests(const ReqView& q, int first, int total_eff, int64_t reach,
                                     int64_t most, int* r, int* j, int* prefix) {
  const int lane = lane_id();
  int lo[N];
#pragma unroll
  for (int i = 0; i < N; ++i) lo[i] = 0;
  for (int n = q.B; n > 1;) {
    const int step = (n + kWave - 1) / kWave;
    int at[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = lo[i] + lane * step;
      at[i] = lane * step < n && c < q.B ? q.cu[c] : 0x7FFFFFFF;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) lo[i] += search_skip(__ballot(at[i] <= first + i), step);
    n = step;
  }
  int req = lo[0];
#pragma unroll
  for (int i = 1; i < N; ++i) req = lane == i ? lo[i] : req;
  const int row = first + lane;
  auto index_in = [&](int c, int x, int* before) {
    int s, e;
    return span_of(q, c, total_eff, reach, most, &s, &e, before) && s <= x && x < e ? x - s : -1;
  };
  *prefix = 0;
  const bool mine = lane < N && row < total_eff;
  int at = mine ? index_in(req, row, prefix) : -1, other;
  // Words out of order mislead the search: rows that it does not find are looked
  // for in every request and go to the first that holds them. (Rows of none are
  // too: those of a malformed request, or before the first.)
  unsigned long long lost = __ballot(mine && at < 0);
  while (lost) {
    const int i = (int)__builtin_ctzll(lost);
    lost &= lost - 1;
    for (int c0 = 0; c0 < q.B; c0 += kWave) {
      const unsigned long long h =
          __ballot(c0 + lane < q.B && index_in(c0 + lane, first + i, &other) >= 0);
      if (!h) continue;
      if (lane == i) {
        req = c0 + (int)__builtin_ctzll(h);
        at = index_in(req, row, prefix);
      }
      break;
    }
  }
  *r = req;
  *j = at;
}

// Status bits of all requests' rows and pages, a share of them to each thread of a
// workgroup: sixteen lanes a request, a lane a page, kAhead requests of a lane at
// once, so that a batch costs two memory latencies.
template <int THREADS>
__device__ inline int spans_status(const ReqView& q, int page_shift, int num_blocks, int total_eff,
                                   int64_t most) {
  constexpr int kLanes = 16, kAhead = 8;
  const int l = threadIdx.x % kLanes;
  const int64_t reach = (int64_t)q.width << page_shift;
  int bits = 0;
  for (int r0 = threadIdx.x / kLanes; r0 < q.B; r0 += kAhead * (THREADS / kLanes)) {
    int s[kAhead], e[kAhead], st[kAhead], id[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = min(r0 + k * (THREADS / kLanes), q.B - 1);
      s[k] = q.cu[r];
      e[k] = q.cu[r + 1];
      st[k] = q.prefix[r];
    }
    int first[kAhead], last[kAhead];  // the lane's pages
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = min(r0 + k * (THREADS / kLanes), q.B - 1);
      first[k] = 0;
      last[k] = -1;
      if (s[k] < 0 || e[k] < s[k] || e[k] > total_eff || st[k] < 0 || e[k] - s[k] > most) {
        bits |= DSPARK_DATA_BAD_LENS;
      } else if (e[k] > s[k]) {
        const int64_t hi = (int64_t)st[k] + (e[k] - s[k]);
        if (hi > reach) {
          bits |= DSPARK_DATA_BAD_PAGE;
        } else {
          first[k] = (st[k] >> page_shift) + l;
          last[k] = (int)((hi - 1) >> page_shift);
        }
      }
      id[k] = 0;
      if (first[k] <= last[k]) id[k] = q.table[(size_t)r * q.width + first[k]];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = min(r0 + k * (THREADS / kLanes), q.B - 1);
      if (first[k] <= last[k] && (id[k] < 0 || id[k] >= num_blocks)) bits |= DSPARK_DATA_BAD_PAGE;
#pragma unroll 4
      for (int p = first[k] + kLanes; p <= last[k]; p += kLanes) {
        const int x = q.table[(size_t)r * q.width + p];
        if (x < 0 || x >= num_blocks) bits |= DSPARK_DATA_BAD_PAGE;
      }
    }
  }
  return bits;
}

// Bits of the workgroup's threads together, and the packed total, as a call's
// status words.
__device__ inline void write_meta(int32_t* meta, int total, int bits, int* all) {
  if (threadIdx.x == 0) *all = 0;
  __syncthreads();
  if (bits) atomicOr(all, bits);
  __syncthreads();
  if (threadIdx.x == 0) {
    meta[0] = total;
    meta[1] = *all;
  }
}

}  // namespace dspark
