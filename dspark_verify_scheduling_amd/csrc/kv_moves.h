// The moves of a commit: which cache rows of each request go where, and the move
// of one column of them.
#pragma once

#include "kv_dev.h"

namespace dspark {

constexpr int kCommitThreads = 256;

// The moves of N requests, L lanes to each: lane l of them has k = l + 1. `r`:
// the request of the lane's group, -1 for none. bits: its status; *src, *dst the
// lane's cache indices, *src = -1 where it moves nothing. N requests cost three
// memory latencies together.
template <int L, int N>
__device__ inline void path_moves(const CommitArgs& a, const int (&r)[N], int lane, int (&bits)[N],
                                  int64_t (&src)[N], int64_t (&dst)[N]) {
  const ReqView& q = a.req;
  const int l = lane & (L - 1);
  const unsigned long long group = (L == 64 ? ~0ull : (1ull << (L & 63)) - 1) << (lane - l);
  const int64_t reach = (int64_t)q.width << a.kv.page_shift;
  int c[N], prefix[N], root[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    c[n] = prefix[n] = root[n] = 0;
    if (r[n] >= 0) {
      c[n] = a.num_correct[r[n]];
      prefix[n] = q.prefix[r[n]];
      root[n] = a.path[(size_t)r[n] * (q.gamma + 1)];
    }
  }
  int here[N], before[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    bits[n] = c[n] < 0 || c[n] > q.gamma || prefix[n] < 0 ? DSPARK_DATA_BAD_LENS : 0;
    here[n] = before[n] = 0;
    if (!bits[n] && l < c[n]) {
      here[n] = a.path[(size_t)r[n] * (q.gamma + 1) + l + 1];
      before[n] = a.path[(size_t)r[n] * (q.gamma + 1) + l];
    }
  }
  int s[N], d[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    src[n] = dst[n] = -1;
    const bool on = !bits[n] && l < c[n];
    const bool ok = root[n] == 0 && (!on || (here[n] > before[n] && here[n] <= q.gamma));
    if ((__ballot(!ok) & group) && !bits[n]) bits[n] = DSPARK_DATA_BAD_TREE;
    if (!bits[n] && on && here[n] != l + 1) {
      src[n] = (int64_t)prefix[n] + here[n];
      dst[n] = (int64_t)prefix[n] + l + 1;
    }
    s[n] = d[n] = 0;
    if (src[n] >= reach) {
      s[n] = -1;
    } else if (src[n] >= 0) {
      s[n] = q.table[(size_t)r[n] * q.width + (src[n] >> a.kv.page_shift)];
      d[n] = q.table[(size_t)r[n] * q.width + (dst[n] >> a.kv.page_shift)];
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const bool good = s[n] >= 0 && s[n] < a.kv.num_blocks && d[n] >= 0 && d[n] < a.kv.num_blocks;
    if (__ballot(!good) & group) {
      src[n] = -1;
      bits[n] = DSPARK_DATA_BAD_PAGE;
    }
  }
}

// Status and number of moves of all requests; one workgroup.
template <int L>
__device__ inline void commit_status(const CommitArgs& a) {
  constexpr int N = 8, kGroups = kCommitThreads / L;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  __shared__ int all, moved;
  if (tid == 0) all = moved = 0;
  __syncthreads();
  int seen = 0, count = 0;
  for (int r0 = 0; r0 < a.req.B; r0 += N * kGroups) {
    int r[N], bits[N];
    int64_t src[N], dst[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int x = r0 + n * kGroups + tid / L;
      r[n] = x < a.req.B ? x : -1;
    }
    path_moves<L, N>(a, r, lane, bits, src, dst);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      seen |= bits[n];
      count += src[n] >= 0;
    }
  }
  if (seen) atomicOr(&all, seen);
  if (count) atomicAdd(&moved, count);
  __syncthreads();
  if (tid == 0) {
    a.meta[0] = moved;
    a.meta[1] = all;
  }
}

// The n moves of one column of T: up to kMoveBatch loads ahead of their stores.
template <typename T>
__device__ inline void move_column(unsigned char* base, int64_t page_bytes, int64_t row_bytes, int n,
                                   const int* s_id, const int* s_off, const int* d_id,
                                   const int* d_off) {
  constexpr int kMoveBatch = 8;
  for (int k0 = 0; k0 < n; k0 += kMoveBatch) {
    T x[kMoveBatch];
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      x[i] = (T){};
      if (k0 + i < n)
        x[i] = *reinterpret_cast<const T*>(base + s_id[k0 + i] * page_bytes +
                                           s_off[k0 + i] * row_bytes);
    }
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      if (k0 + i < n)
        *reinterpret_cast<T*>(base + d_id[k0 + i] * page_bytes + d_off[k0 + i] * row_bytes) = x[i];
    }
  }
}

}  // namespace dspark
