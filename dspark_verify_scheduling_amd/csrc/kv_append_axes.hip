// Cache append of rows whose rotation takes a position on several axes.
#include "append_row.h"
#include "latent.h"

#include <algorithm>

namespace dspark {

namespace {

constexpr int kThreads = 256;

// Positions of all packed rows on all axes, a share to each thread. Rows before any
// request's, where the first starts late, are nobody's.
__device__ int position_status(const AppendAxesArgs& a, int total_eff) {
  const ReqView& q = a.base.req;
  int bits = 0;
  if (q.B == 0) return bits;
  __shared__ int first;
  if (threadIdx.x == 0) first = total_eff;
  __syncthreads();
  int lo = max(q.cu[0], 0);
  if (lo > 0)  // (words out of order: not the least then)
    for (int r = threadIdx.x; r < q.B; r += kThreads) lo = min(lo, max(q.cu[r], 0));
  atomicMin(&first, lo);
  __syncthreads();
#pragma unroll 4
  for (int64_t n = (int64_t)first + threadIdx.x; n < total_eff; n += kThreads) {
    int p[DSPARK_MAX_AXES];  // all axes' loads before the first is looked at
#pragma unroll
    for (int x = 0; x < DSPARK_MAX_AXES; ++x)
      p[x] = a.positions[min(x, a.num_axes - 1) * a.positions_ld + n];
#pragma unroll
    for (int x = 0; x < DSPARK_MAX_AXES; ++x)
      if (p[x] < 0 || p[x] >= a.base.rope_rows) bits = DSPARK_DATA_BAD_POS;
  }
  return bits;
}

// ROWS packed rows to a workgroup, its waves split between them: a wave finds its
// row's request and page by itself, and a row's waves take its heads in turn. Pair i
// turns by row positions[axis of i] of the table, so a lane gathers its eight
// cosines and sines from up to num_axes table rows, once for all heads.
// Bound by its arithmetic where rows are many, 2,460 vector instructions a row and four
// fifths of a CU's busy cycles: 13,001 rows of 32 + 2 * 8 heads of 128 into an 8-bit
// cache, 81 us, 3.6 TB/s. Bound by dependent reads where they are few: 8 rows 7.1 us.
// (The one workgroup that checks all positions is hidden beside the rows, 256,000 of 1 +
// 2 heads of 64 among them: 215 us with it and without.) A workgroup to a row, or a wave:
// 128 rows of 32 + 2 * 8 heads in 8 bits 15.5 and 16.5 us, of 28 + 2 * 4 in 16 bits 14.8
// and 11.9; 1,024 rows 25.3 and 29, 23.8 and 23.5; 2,048 rows 32.7 and 31.3, 30.3 and
// 26.4. A wave to a row where rows are few takes 12 rounds one after the other; a
// workgroup to a row where they are many has four waves look the same request up (the
// first case: 199 us for the call with the cache's read, 133 with a wave; 96 with two
// rounds under way, nothing in scratch memory and no exchange through LDS).
template <typename T, bool E8, int D, int ROWS>
__global__ __launch_bounds__(kThreads) void append_axes_kernel(AppendAxesArgs a) {
  constexpr int LPH = D / 8, kRowThreads = kThreads / ROWS;
  fetch_args<sizeof(a)>();
  const AppendArgs& b = a.base;
  const ReqView& q = b.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  int total;
  const int total_eff = rows_in_use(q, &total);
  if (blockIdx.x == 0) {
    if (a.first_row) return;
    __shared__ int all;
    int bits = total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    bits |= spans_status<kThreads>(q, b.kv.page_shift, b.kv.num_blocks, total_eff, 0x7FFFFFFF);
    bits |= position_status(a, total_eff);
    write_meta(b.meta, total, bits, &all);
    return;
  }
  const int64_t packed = a.first_row + (int64_t)(blockIdx.x - 1) * ROWS +
                         __builtin_amdgcn_readfirstlane(tid / kRowThreads);
  if (packed >= total_eff) return;
  const int n = (int)packed;
  RowAppend<T, E8, D, kRowThreads, ROWS == 1 ? 1 : 2> row(b, n);
  int pos[DSPARK_MAX_AXES];
  bool bad = false;
#pragma unroll
  for (int x = 0; x < DSPARK_MAX_AXES; ++x) {
    pos[x] = a.positions[min(x, a.num_axes - 1) * a.positions_ld + n];
    bad |= pos[x] < 0 || pos[x] >= b.rope_rows;
  }
  const int li = lane & (LPH - 1), half = b.rope_dim >> 1;
  const bool turned = 8 * li < b.rope_dim;
  const bool low = b.rope_interleaved || 8 * li < half;
  // the lane's first pair; its pairs' axes stand in one word
  const int i0 = !turned ? 0 : b.rope_interleaved ? 4 * li : (low ? 8 * li : 8 * li - half);
  const uint64_t axes = a.axis[i0 >> 5] >> (2 * (i0 & 31));
  int swap = lane;  // lane that holds the other elements of the pairs
  if (turned && !b.rope_interleaved) swap = low ? lane + half / 8 : lane - half / 8;
  int r, j, prefix;
  rows_requests<1>(q, n, total_eff, (int64_t)q.width << b.kv.page_shift, 0x7FFFFFFF, &r, &j, &prefix);
  r = __builtin_amdgcn_readfirstlane(r);
  j = __builtin_amdgcn_readfirstlane(j);
  if (j < 0 || bad) return;
  const int64_t slot = (int64_t)__builtin_amdgcn_readfirstlane(prefix) + j;
  const int id = q.table[(size_t)r * q.width + (slot >> b.kv.page_shift)];

  // the table's entry of a pair
  auto turn = [&](int e, float* c, float* s) {
    const int x = (int)(axes >> (2 * e)) & 3;
    const int p = x < 2 ? (x == 0 ? pos[0] : pos[1]) : (x == 2 ? pos[2] : pos[3]);
    const float* cs = b.rope + (size_t)p * b.rope_dim + i0 + e;
    *c = cs[0];
    *s = cs[half];
  };
  float co[8], si[8];
  if (b.rope_interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      turn(e, &co[2 * e], &si[2 * e + 1]);
      co[2 * e + 1] = co[2 * e];
      si[2 * e] = -si[2 * e + 1];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      turn(e, &co[e], &si[e]);
      si[e] = low ? -si[e] : si[e];
    }
  }
  // after the gather, which then waits along with the table's entry
  if (id < 0 || id >= b.kv.num_blocks) return;
  row.finish(id, (int)(slot & ((1 << b.kv.page_shift) - 1)), co, si, turned, swap);
}

template <typename T, bool E8, int ROWS>
void by_dim(const AppendAxesArgs& a, unsigned grid, hipStream_t s) {
  switch (a.base.kv.dim) {
    case 64:
      hipLaunchKernelGGL((append_axes_kernel<T, E8, 64, ROWS>), dim3(grid), dim3(kThreads), 0, s, a);
      break;
    case 128:
      hipLaunchKernelGGL((append_axes_kernel<T, E8, 128, ROWS>), dim3(grid), dim3(kThreads), 0, s, a);
      break;
    default:
      hipLaunchKernelGGL((append_axes_kernel<T, E8, 256, ROWS>), dim3(grid), dim3(kThreads), 0, s, a);
  }
}

template <int ROWS>
void by_type(const AppendAxesArgs& a, dspark_dtype dt, unsigned rows, hipStream_t s) {
  const unsigned grid = 1u + (rows + ROWS - 1) / ROWS;
  if (a.base.kv.cb == 1) {
    by_dim<__bf16, true, ROWS>(a, grid, s);
  } else if (dt == DSPARK_BF16) {
    by_dim<__bf16, false, ROWS>(a, grid, s);
  } else {
    by_dim<_Float16, false, ROWS>(a, grid, s);
  }
}

}  // namespace

hipError_t launch_append_axes(const AppendAxesArgs& a, dspark_dtype dt, hipStream_t s) {
  // a grid of 2^32 threads or more is cut off without an error
  constexpr int64_t kMostRows = 1 << 20;
  const int64_t rows = a.base.req.B > 0 ? a.base.req.max_rows : 0;
  AppendAxesArgs part = a;
  part.first_row = 0;
  do {
    const unsigned n = (unsigned)std::min<int64_t>(rows - part.first_row, kMostRows);
    // few rows: all waves to one
    if (rows <= 1024) {
      by_type<1>(part, dt, n, s);
    } else {
      by_type<kThreads / kWave>(part, dt, n, s);
    }
    part.first_row += kMostRows;
  } while (part.first_row < rows);
  return hipGetLastError();
}

}  // namespace dspark
