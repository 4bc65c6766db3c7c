// The paged key/value cache of the target pass: append with per-head norms and
// rotation, read back, and the commit of an accepted path.
//
// All three move every byte once and compute next to nothing on it, so they
// are bound by HBM (large calls) or by the latency of a launch and one or two
// dependent reads (small ones). A row of one head is head_dim * 2 bytes; 16-byte
// loads put it on head_dim / 8 lanes, so every reduction of a head (the sum of
// squares, the largest magnitude) stays inside 8, 16 or 32 lanes.
//
// Status words: workgroup 0 of each launch checks every request by itself and
// writes the status; the others repeat the checks of what they touch and leave
// bad requests or rows out.
#include "append_row.h"
#include "kv_moves.h"
#include "request_search.h"

#include <algorithm>

namespace dspark {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ append

// Status of all requests, their pages and positions included; one workgroup. L
// lanes to a request, lane l for its row l + 1 and its l-th page, N requests of
// a lane at once: a batch costs three memory latencies.
template <int L>
__device__ int append_status(const AppendArgs& a, int total_eff) {
  constexpr int N = 4, kGroups = kThreads / L;
  static_assert((DSPARK_MAX_GAMMA + 1) / 16 + 2 <= 16, "pages of a step to a group");
  const ReqView& q = a.req;
  const int lane = threadIdx.x & (kWave - 1), l = lane & (L - 1);
  const unsigned long long group = (L == 64 ? ~0ull : (1ull << (L & 63)) - 1) << (lane - l);
  int all = 0;
  for (int r0 = 0; r0 < q.B; r0 += N * kGroups) {
    int r[N], c0[N], len[N], prefix[N], par[N], id[N];
    bool ok[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      // (past the last: the last once more)
      r[n] = min(r0 + n * kGroups + (int)threadIdx.x / L, q.B - 1);
      ok[n] = request_rows(q, r[n], total_eff, &c0[n], &len[n]);
      prefix[n] = q.prefix[r[n]];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      ok[n] = ok[n] && prefix[n] >= 0;
      if (!ok[n]) all |= DSPARK_DATA_BAD_LENS;
      par[n] = id[n] = 0;
      if (ok[n] && q.parents && l + 1 < len[n]) par[n] = q.parents[(size_t)r[n] * q.gamma + l];
      const int64_t hi = (int64_t)prefix[n] + len[n];  // cache indices [prefix, hi)
      if (ok[n]) {
        const int64_t p = (prefix[n] >> a.kv.page_shift) + l;
        if (hi > ((int64_t)q.width << a.kv.page_shift)) {
          id[n] = -1;
        } else if (p <= (hi - 1) >> a.kv.page_shift) {
          id[n] = q.table[(size_t)r[n] * q.width + p];
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (__ballot(par[n] < 0 || par[n] > l) & group) {
        all |= DSPARK_DATA_BAD_TREE;
      } else if (ok[n]) {
        if (id[n] < 0 || id[n] >= a.kv.num_blocks) all |= DSPARK_DATA_BAD_PAGE;
        const int64_t hi = (int64_t)prefix[n] + len[n];
        if (a.rope && hi > a.rope_rows && hi <= ((int64_t)q.width << a.kv.page_shift)) {
          // a tree's depths may still be small enough
          if (prefix[n] >= a.rope_rows) all |= DSPARK_DATA_BAD_POS;
          if (l + 1 < len[n]) {
            int depth = l + 1;
            if (q.parents) {
              depth = 0;
              for (int m = l + 1; m > 0; m = q.parents[(size_t)r[n] * q.gamma + m - 1]) ++depth;
            }
            if ((int64_t)prefix[n] + depth >= a.rope_rows) all |= DSPARK_DATA_BAD_POS;
          }
        }
      }
    }
  }
  return all;
}

// One workgroup per (request, row): LPH lanes per head take the heads of q, k
// and v in turn (append_row.h). Every row is read and written once. 256 requests of up to 9 rows, 32
// query heads on 8 of 128, into 8 bits: 13 us (27 MB, 2.1 TB/s; 6 us at a copy's
// rate): the arithmetic of a row (about 250 instructions a wave and round) and
// the reads that say where it goes, in one round of workgroups. 128 threads took
// 15.6 us, 512 14.9. A few rows: 3.4 us, latency.
template <typename T, bool E8, int D>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
  constexpr int LPH = D / 8;
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  int total;
  const int total_eff = rows_in_use(q, &total);
  if (blockIdx.x == 0) {
    int bits = total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    bits |= q.gamma <= 16 ? append_status<16>(a, total_eff) : append_status<kWave>(a, total_eff);
    __shared__ int all;
    if (tid == 0) all = 0;
    __syncthreads();
    if (bits) atomicOr(&all, bits);
    __syncthreads();
    if (tid == 0) {
      a.meta[0] = total;
      a.meta[1] = all;
    }
    return;
  }
  const int u = blockIdx.x - 1;
  const int r = u / (q.gamma + 1);
  const int j = u - r * (q.gamma + 1);
  int c0, len;
  if (!request_rows(q, r, total_eff, &c0, &len) || j >= len) return;
  const int prefix = q.prefix[r];
  const int li = lane & (LPH - 1);  // the lane's eight elements: 8 li ..
  // its first heads are loaded with the reads that say where it goes
  RowAppend<T, E8, D, kThreads> row(a, c0 + j);
  if (prefix < 0 || (int64_t)prefix + len > ((int64_t)q.width << a.kv.page_shift)) return;
  const int64_t slot = (int64_t)prefix + j;
  const int id = q.table[(size_t)r * q.width + (slot >> a.kv.page_shift)];
  int depth = j;
  if (q.parents) {
    // lane l holds the parent of row l + 1; every wave walks by itself
    const int par = lane + 1 < len ? q.parents[(size_t)r * q.gamma + lane] : 0;
    if (__ballot(par < 0 || par > lane)) return;
    depth = 0;
    for (int n = j; n > 0; n = __builtin_amdgcn_readlane(par, n - 1)) ++depth;
  }
  if (id < 0 || id >= a.kv.num_blocks) return;
  const int64_t pos = (int64_t)prefix + depth;
  if (a.rope && pos >= a.rope_rows) return;

  const int half = a.rope_dim >> 1;
  // the lane's cosines and sines, the same for every head
  float co[8], si[8];
  bool turned = false;
  int swap = lane;  // lane that holds the other elements of the pairs
  if (a.rope) {
    const float* cs = a.rope + (size_t)pos * a.rope_dim;
    turned = 8 * li < a.rope_dim;
    if (a.rope_interleaved) {
      const int i0 = turned ? 4 * li : 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        co[2 * e] = co[2 * e + 1] = cs[i0 + e];
        si[2 * e + 1] = cs[half + i0 + e];
        si[2 * e] = -si[2 * e + 1];
      }
    } else {
      const bool low = 8 * li < half;
      const int i0 = turned ? (low ? 8 * li : 8 * li - half) : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        co[e] = cs[i0 + e];
        si[e] = low ? -cs[half + i0 + e] : cs[half + i0 + e];
      }
      if (turned) swap = low ? lane + half / 8 : lane - half / 8;
    }
  }
  const int off = (int)(slot & ((1 << a.kv.page_shift) - 1));
  row.finish(id, off, co, si, turned, swap);
}

// ------------------------------------------------------------------ read

constexpr int kReadThreads = 512;
// Rows of a workgroup: few, so that a small call is many workgroups; more where a
// row gives its threads nothing to do (one head of 128: 230 MB in 98 us with 8
// rows, 48 us with 64).
constexpr int kReadFew = 8, kReadMany = 64;
// Workgroups of a launch that have rows, at most: a grid of 2^32 threads or more is
// cut off without an error. More rows are more launches (all in one, a loop over
// its rows in each workgroup, took 108 us for the 437 MB below).
constexpr int64_t kReadWgs = 1 << 20;

// One workgroup per kReadRows rows: a wave finds its rows' requests and pages,
// then 16-byte vectors of (row, head) are copied or widened. Bound by HBM: 437 MB
// (a third of it read) of 16 contexts of an 8-bit cache, 8 heads of 128, in 96 us,
// 4.5 TB/s; a copy of 2 GiB reaches 4.9. Nontemporal both ways (104 us without).
// A few short spans: 4 us.
template <bool E8, int D, int kReadRows>
__global__ __launch_bounds__(kReadThreads) void read_kernel(ReadArgs a) {
  constexpr int EPL = E8 ? 16 : 8;  // elements of a lane, in 16 bytes
  constexpr int LPH = D / EPL, HPP = kReadThreads / LPH;
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  int total;
  const int total_eff = rows_in_use(q, &total);
  const int64_t reach = (int64_t)q.width << a.kv.page_shift;
  if (blockIdx.x == 0) {
    if (a.first_row) return;
    // sixteen lanes per request, a lane per page; kAhead requests of a lane at
    // once, so that a batch costs two memory latencies (256 requests, one by one:
    // 27 us)
    constexpr int kLanes = 16, kAhead = 8;
    __shared__ int all;
    if (tid == 0) all = total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    __syncthreads();
    const int l = tid % kLanes;
    int bits = 0;
    for (int r0 = tid / kLanes; r0 < q.B; r0 += kAhead * (kReadThreads / kLanes)) {
      int s[kAhead], e[kAhead], st[kAhead], id[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = min(r0 + k * (kReadThreads / kLanes), q.B - 1);
        s[k] = q.cu[r];
        e[k] = q.cu[r + 1];
        st[k] = q.prefix[r];
      }
      int first[kAhead], last[kAhead];  // the lane's pages
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = min(r0 + k * (kReadThreads / kLanes), q.B - 1);
        first[k] = 0;
        last[k] = -1;
        if (s[k] < 0 || e[k] < s[k] || e[k] > total_eff || st[k] < 0) {
          bits |= DSPARK_DATA_BAD_LENS;
        } else if (e[k] > s[k]) {
          const int64_t hi = (int64_t)st[k] + (e[k] - s[k]);
          if (hi > reach) {
            bits |= DSPARK_DATA_BAD_PAGE;
          } else {
            first[k] = (st[k] >> a.kv.page_shift) + l;
            last[k] = (int)((hi - 1) >> a.kv.page_shift);
          }
        }
        id[k] = 0;
        if (first[k] <= last[k]) id[k] = q.table[(size_t)r * q.width + first[k]];
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = min(r0 + k * (kReadThreads / kLanes), q.B - 1);
        if (first[k] <= last[k] && (id[k] < 0 || id[k] >= a.kv.num_blocks))
          bits |= DSPARK_DATA_BAD_PAGE;
#pragma unroll 4
        for (int p = first[k] + kLanes; p <= last[k]; p += kLanes) {
          const int x = q.table[(size_t)r * q.width + p];
          if (x < 0 || x >= a.kv.num_blocks) bits |= DSPARK_DATA_BAD_PAGE;
        }
      }
    }
    if (bits) atomicOr(&all, bits);
    __syncthreads();
    if (tid == 0) {
      a.meta[0] = total;
      a.meta[1] = all;
    }
    return;
  }
  __shared__ int page_of[kReadRows], off_of[kReadRows];
  const int row0 = a.first_row + (blockIdx.x - 1) * kReadRows;
  if (row0 >= total_eff) return;
  {
    // the last request that starts at or before each of the wave's rows, 64 steps
    // of the search at once and its rows together
    constexpr int N = kReadRows / (kReadThreads / kWave);
    const int first = row0 + tid / kWave * N;
    int lo[N];
#pragma unroll
    for (int i = 0; i < N; ++i) lo[i] = 0;
    for (int n = q.B; n > 1;) {
      const int step = (n + kWave - 1) / kWave;
      int at[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = lo[i] + lane * step;
        at[i] = lane * step < n && r < q.B ? q.cu[r] : 0x7FFFFFFF;
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        lo[i] += search_skip(__ballot(at[i] <= first + i), step);
      n = step;
    }
    // one row to a lane from here
    int r = lo[0];
#pragma unroll
    for (int i = 1; i < N; ++i) r = lane == i ? lo[i] : r;
    const int row = first + lane;
    // the cache index of packed row x as one of request c's; -1 where it is none of
    // them, or the request is malformed
    auto slot_of = [&](int c, int x) -> int64_t {
      const int s = q.cu[c], e = q.cu[c + 1], st = q.prefix[c];
      const bool ok = s >= 0 && s <= x && x < e && e <= total_eff && st >= 0 &&
                      (int64_t)st + (e - s) <= reach;
      return ok ? (int64_t)st + (x - s) : -1;
    };
    const bool mine = lane < N && row < total_eff;
    int64_t slot = mine ? slot_of(r, row) : -1;
    // Lengths out of order mislead the search: rows that it does not find are
    // looked for in every request, 64 at once, and go to the first that holds them.
    // (Rows of none are too: those of a malformed request, or before the first.)
    unsigned long long lost = __ballot(mine && slot < 0);
    while (lost) {
      const int i = (int)__builtin_ctzll(lost);
      lost &= lost - 1;
      for (int r0 = 0; r0 < q.B; r0 += kWave) {
        const unsigned long long h =
            __ballot(r0 + lane < q.B && slot_of(r0 + lane, first + i) >= 0);
        if (!h) continue;
        if (lane == i) {
          r = r0 + (int)__builtin_ctzll(h);
          slot = slot_of(r, row);
        }
        break;
      }
    }
    if (lane < N) {
      int id = -1;
      if (slot >= 0) id = q.table[(size_t)r * q.width + (slot >> a.kv.page_shift)];
      if (id >= a.kv.num_blocks) id = -1;
      const int off = (int)(slot & ((1 << a.kv.page_shift) - 1));
      page_of[row - row0] = id;
      off_of[row - row0] = off;
    }
  }
  __syncthreads();
  const int li = lane & (LPH - 1);
  const int items = kReadRows * a.kv.hkv;
  // streamed: nothing comes back to either side
#pragma unroll 4
  for (int n = tid / LPH; n < items; n += HPP) {
    const int i = n / a.kv.hkv, h = n - i * a.kv.hkv;
    const int id = page_of[i];
    const bool live = id >= 0;
    const size_t page = (size_t)(live ? id : 0);
    const size_t at = ((size_t)h << a.kv.page_shift) + off_of[i];
    const size_t dst = (size_t)(row0 + i) * a.out_ld + (size_t)(h * D + EPL * li) * 2;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const unsigned char* src = (w ? a.kv.v : a.kv.k) + page * a.kv.page_bytes;
      unsigned char* to = (w ? a.v_out : a.k_out) + dst;
      if constexpr (E8) {
        const kv_u32x4 c = __builtin_nontemporal_load(
            reinterpret_cast<const kv_u32x4*>(src + at * D + EPL * li));
        const float sc =
            pow2f((int)(w ? a.kv.vs : a.kv.ks)[page * a.kv.scale_page_bytes + at] - 127);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          kv_u32x4 o;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            o[2 * g] = __builtin_bit_cast(
                unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * x + g], sc, false));
            o[2 * g + 1] = __builtin_bit_cast(
                unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * x + g], sc, true));
          }
          if (live) __builtin_nontemporal_store(o, reinterpret_cast<kv_u32x4*>(to + 16 * x));
        }
      } else {
        const kv_u32x4 o = __builtin_nontemporal_load(
            reinterpret_cast<const kv_u32x4*>(src + (at * D + EPL * li) * 2));
        if (live) __builtin_nontemporal_store(o, reinterpret_cast<kv_u32x4*>(to));
      }
    }
  }
}

// ------------------------------------------------------------------ commit

// `parts` workgroups per (request, `per` layers), part blockIdx.y % parts; a thread
// owns 16-byte columns of them (one place of one head of a layer's keys or values) or bytes
// of exponents, and moves the path's rows of that column in ascending order.
// Path rows ascend and path[k] >= k, so a move never overwrites the source of a
// later one, and a batch of loads may run ahead of its stores: the rows it
// stores to, k .. k + kMoveBatch - 1, lie below every later source. Bound by HBM:
// 178 MB read and written of 256 requests, 32 layers of 8 heads of 128 in 8 bits,
// in 34 us, 5.2 TB/s. A few requests and layers: 4 us.
__global__ __launch_bounds__(kCommitThreads) void commit_kernel(CommitArgs a, int per, int parts) {
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  if (blockIdx.x == 0) {
    if (blockIdx.y != 0) return;
    if (q.gamma <= 16) {
      commit_status<16>(a);
    } else {
      commit_status<kWave>(a);
    }
    return;
  }
  __shared__ int s_id[DSPARK_MAX_GAMMA], s_off[DSPARK_MAX_GAMMA], d_id[DSPARK_MAX_GAMMA],
      d_off[DSPARK_MAX_GAMMA];
  __shared__ int n_moves;
  if (tid < kWave) {
    const int r[1] = {(int)blockIdx.x - 1};
    int bits[1];
    int64_t src[1], dst[1];
    path_moves<kWave, 1>(a, r, lane, bits, src, dst);
    const unsigned long long m = __ballot(src[0] >= 0);
    if (src[0] >= 0) {
      const int i = __popcll(m & ((1ull << lane) - 1));
      const int mask = (1 << a.kv.page_shift) - 1;
      s_id[i] = q.table[(size_t)r[0] * q.width + (src[0] >> a.kv.page_shift)];
      d_id[i] = q.table[(size_t)r[0] * q.width + (dst[0] >> a.kv.page_shift)];
      s_off[i] = (int)(src[0] & mask);
      d_off[i] = (int)(dst[0] & mask);
    }
    if (lane == 0) n_moves = __popcll(m);
  }
  __syncthreads();
  const int n = n_moves;
  if (n == 0) return;
  const int row_bytes = a.kv.dim * a.kv.cb, row_vecs = row_bytes / 16;
  const int rows = 2 * a.kv.hkv;  // of a layer: keys' heads, then values' heads
  const int cols = rows * row_vecs;
  const int group = blockIdx.y / parts, first = (blockIdx.y - group * parts) * kCommitThreads + tid;
  const int layer0 = group * per;
  const int layers = min(per, a.kv.num_layers - layer0);
  for (int i = first; i < layers * cols; i += parts * kCommitThreads) {
    const int layer = i / cols, col = i - layer * cols;
    const int row = col / row_vecs, w = row >= a.kv.hkv, h = row - w * a.kv.hkv;
    move_column<kv_u32x4>((w ? a.kv.v : a.kv.k) + (layer0 + layer) * a.kv.layer_bytes +
                              ((int64_t)h << a.kv.page_shift) * row_bytes +
                              (col - row * row_vecs) * 16,
                          a.kv.page_bytes, row_bytes, n, s_id, s_off, d_id, d_off);
  }
  if (a.kv.ks) {
    for (int i = first; i < layers * rows; i += parts * kCommitThreads) {
      const int layer = i / rows, row = i - layer * rows;
      const int w = row >= a.kv.hkv, h = row - w * a.kv.hkv;
      move_column<unsigned char>((w ? a.kv.vs : a.kv.ks) +
                                     (layer0 + layer) * a.kv.scale_layer_bytes +
                                     ((int64_t)h << a.kv.page_shift),
                                 a.kv.scale_page_bytes, 1, n, s_id, s_off, d_id, d_off);
    }
  }
}

template <typename T, bool E8>
void append_by_dim(const AppendArgs& a, unsigned grid, hipStream_t s) {
  switch (a.kv.dim) {
    case 64:
      hipLaunchKernelGGL((append_kernel<T, E8, 64>), dim3(grid), dim3(kThreads), 0, s, a);
      break;
    case 128:
      hipLaunchKernelGGL((append_kernel<T, E8, 128>), dim3(grid), dim3(kThreads), 0, s, a);
      break;
    default:
      hipLaunchKernelGGL((append_kernel<T, E8, 256>), dim3(grid), dim3(kThreads), 0, s, a);
  }
}

template <bool E8, int D>
void read_by_rows(const ReadArgs& a, hipStream_t s) {
  const int64_t rows = a.req.B > 0 ? a.req.max_rows : 0;
  const int at_once = kReadFew * a.kv.hkv * (D * a.kv.cb / 16);  // threads with a vector
  const int per = at_once < kReadThreads ? kReadMany : kReadFew;
  ReadArgs part = a;
  int64_t first = 0;
  do {
    part.first_row = (int)first;
    const int64_t wgs = std::min<int64_t>((rows - first + per - 1) / per, kReadWgs);
    const dim3 grid(1u + (unsigned)wgs), block(kReadThreads);
    if (per == kReadMany) {
      hipLaunchKernelGGL((read_kernel<E8, D, kReadMany>), grid, block, 0, s, part);
    } else {
      hipLaunchKernelGGL((read_kernel<E8, D, kReadFew>), grid, block, 0, s, part);
    }
    first += wgs * per;
  } while (first < rows);
}

template <bool E8>
void read_by_dim(const ReadArgs& a, hipStream_t s) {
  switch (a.kv.dim) {
    case 64: return read_by_rows<E8, 64>(a, s);
    case 128: return read_by_rows<E8, 128>(a, s);
    default: read_by_rows<E8, 256>(a, s);
  }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, dspark_dtype dt, hipStream_t s) {
  const unsigned grid = 1u + (unsigned)a.req.B * (unsigned)(a.req.gamma + 1);
  if (a.kv.cb == 1) {
    append_by_dim<__bf16, true>(a, grid, s);
  } else if (dt == DSPARK_BF16) {
    append_by_dim<__bf16, false>(a, grid, s);
  } else {
    append_by_dim<_Float16, false>(a, grid, s);
  }
  return hipGetLastError();
}

hipError_t launch_read(const ReadArgs& a, hipStream_t s) {
  if (a.kv.cb == 1) {
    read_by_dim<true>(a, s);
  } else {
    read_by_dim<false>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_commit(const CommitArgs& a, hipStream_t s) {
  // up to four layers to a workgroup, whose moves are then looked up once; where
  // that leaves few workgroups, fewer layers, and a layer to several (6 requests,
  // 14 layers of 8 heads of 256: 24 workgroups took 29 us, 672 take 8.7)
  constexpr int64_t kEnough = 1024;
  const int64_t pairs = (int64_t)a.req.B * a.kv.num_layers;
  const int per = (int)std::max<int64_t>(1, std::min<int64_t>(4, pairs / kEnough));
  const int groups = (a.kv.num_layers + per - 1) / per;
  const int cols = per * 2 * a.kv.hkv * (a.kv.dim * a.kv.cb / 16);
  const int64_t wgs = std::max<int64_t>(1, (int64_t)a.req.B * groups);
  const int parts = (int)std::max<int64_t>(
      1, std::min<int64_t>((cols + kCommitThreads - 1) / kCommitThreads, kEnough / wgs));
  hipLaunchKernelGGL(commit_kernel, dim3(1u + (unsigned)a.req.B, (unsigned)(groups * parts)),
                     dim3(kCommitThreads), 0, s, a, per, parts);
  return hipGetLastError();
}

}  // namespace dspark
