// Causal attention of prompt rows over keys and values expanded from a latent
// cache. Four launches:
//   plan    checks the requests and lays their keys one after the other
//   gather  cached rows, widened to 16 bits, in that order
//   expand  every head's keys and values: a product of the rows with its weights
//   attend  one pass over a head's keys for each tile of prompt rows
#include "latent.h"
#include "lds_dev.h"

#include <algorithm>

namespace dspark {

namespace prefill {

using attn::barrier;
using attn::copy16_shared;
using attn::f32x16;
using attn::kLn2;
using attn::kLog2e;
using attn::lds_columns;
using attn::lds_read;
using attn::lds_u8;
using attn::lds_write;
using attn::settle;
using attn::Types;
using attn::uniform;
using attn::wait_copies;

constexpr int kPlanThreads = 1024;
constexpr int kKeyTile = 64;    // a request's keys are padded to it
constexpr int kDenseTile = 128; // keys of a workgroup of the expansion
constexpr int kRowTile = 128;   // rows of a workgroup of the attention
constexpr int kXcds = 8;

// A request as the plan leaves it; len 0 where it has no rows or is left out (keys
// -1 then if its words of cu_seqlens are out of order).
struct Req {
  int c0, len, prefix, keys;
};

// The workspace.
struct Space {
  Req* req;        // [B]
  int32_t* tile0;  // [B + 1] row tiles before request r
  int32_t* key0;   // [B + 1] dense keys before request r, then all
  int32_t* order;  // [row tiles] those with the most keys first
  unsigned char* lat;     // [dense][L], 16 bits
  unsigned char* turned;  // [dense][kRope]
  unsigned char* kv;      // [num_heads][dense][2 nope]: keys, then values
  int64_t dense;
};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
  size_t tile0, key0, order, lat, turned, kv, bytes;
  int64_t dense;
};

// Row tiles of a call, at most: no two requests that the plan leaves in have a row
// in common.
int most_tiles(int B, int max_rows, int max_keys) {
  const int rows = std::min(max_rows, max_keys);
  return rows / kRowTile + std::min(B, rows);
}

Layout layout(int B, int max_rows, int max_keys, int num_heads, int nope, int L) {
  Layout p;
  // (no more requests than keys have any)
  const int64_t padded = (int64_t)max_keys + (int64_t)(kKeyTile - 1) * std::min(B, max_keys);
  p.dense = (padded + kDenseTile - 1) / kDenseTile * kDenseTile;
  p.tile0 = align256((size_t)B * sizeof(Req));
  p.key0 = p.tile0 + align256((size_t)(B + 1) * sizeof(int32_t));
  p.order = p.key0 + align256((size_t)(B + 1) * sizeof(int32_t));
  p.lat = p.order + align256((size_t)most_tiles(B, max_rows, max_keys) * sizeof(int32_t));
  p.turned = p.lat + align256((size_t)p.dense * L * 2);
  p.kv = p.turned + align256((size_t)p.dense * kRope * 2);
  p.bytes = p.kv + align256((size_t)p.dense * num_heads * 4 * nope);
  return p;
}

// The last of the ascending words at[0 .. n) that is <= x (the first is), by a wave.
__device__ inline int last_at(const int32_t* at, int n, int x) {
  int lo = 0;
  const int all = n;
  while (n > 1) {
    const int step = (n + kWave - 1) / kWave;
    const int c = lo + lane_id() * step;
    const bool le = lane_id() * step < n && c < all && at[c] <= x;
    lo += search_skip(__ballot(le), step);
    n = step;
  }
  return lo;
}

// ------------------------------------------------------------------ plan

// One workgroup: sixteen lanes check a request's words and pages, then the requests'
// tiles and keys are summed. A few requests: three dependent reads, 4.5 us.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(LatentPrefillArgs a, Space w) {
  fetch_args<sizeof(a) + sizeof(w)>();
  const ReqView& q = a.req;
  const int tid = threadIdx.x;
  int total;
  const int total_eff = rows_in_use(q, &total);
  const int64_t reach = (int64_t)q.width << a.kv.page_shift;
  constexpr int kLanes = 16;
  const int l = tid % kLanes;
  const unsigned long long group = 0xFFFFull << (lane_id() - l);
  int bits = total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
  for (int r0 = 0; r0 < q.B; r0 += kPlanThreads / kLanes) {
    const int r = r0 + tid / kLanes;
    int s = 0, e = 0, prefix = 0;
    bool ok = r < q.B;
    if (ok) {
      s = q.cu[r];
      e = q.cu[r + 1];
      prefix = q.prefix[r];
      ok = s >= 0 && e >= s && e <= total_eff && prefix >= 0;
      if (!ok) bits |= DSPARK_DATA_BAD_LENS;
    }
    if (ok && e > s && (int64_t)prefix + (e - s) > reach) {
      bits |= DSPARK_DATA_BAD_PAGE;
      ok = false;
    }
    bool bad = false;
    if (ok && e > s) {
      const int last = (int)(((int64_t)prefix + (e - s) - 1) >> a.kv.page_shift);
#pragma unroll 4
      for (int p = l; p <= last; p += kLanes) {
        const int id = q.table[(size_t)r * q.width + p];
        bad |= id < 0 || id >= a.kv.num_blocks;
      }
    }
    if (__ballot(bad) & group) {
      bits |= DSPARK_DATA_BAD_PAGE;
      ok = false;
    }
    if (l == 0 && r < q.B) {
      // (held to 32 bits: so many keys pass any max_keys)
      const int keys = (int)min((int64_t)prefix + (e - s), (int64_t)0x7FFFFFFF);
      w.req[r] = ok && e > s ? Req{s, e - s, prefix, keys} : Req{0, 0, 0, e < s ? -1 : 0};
    }
  }
  __syncthreads();
  __shared__ int64_t sums[kPlanThreads / kWave];
  const int per = (q.B + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, q.B), r1 = min(r0 + per, q.B);
  // (keys of all requests are less than 2^13 2^31)
  constexpr int64_t kDisorder = (int64_t)1 << 48;
  int64_t mine = 0, all;
  for (int r = r0; r < r1; ++r)
    mine += w.req[r].len ? w.req[r].keys : w.req[r].keys < 0 ? kDisorder : 0;
  int64_t used = block_excl_scan<int64_t, kPlanThreads>(mine, sums, &all);
  // Requests can claim the same rows only where some word is less than the one before
  // it. Then one that has rows of a well-formed request ahead of it is left out: a row
  // has one writer, and the launch and `order` hold all tiles.
  if (__builtin_expect(all >= kDisorder, 0)) {
    unsigned taken = 0;  // bit k: request r0 + k is left out
    static_assert((DSPARK_MAX_BATCH + kPlanThreads - 1) / kPlanThreads <= 32, "bits of a thread");
    for (int r = r0; r < r1; ++r) {
      const Req x = w.req[r];
      for (int p = 0; x.len && p < r; ++p) {
        const Req y = w.req[p];
        if (y.len && y.c0 < x.c0 + x.len && x.c0 < y.c0 + y.len) taken |= 1u << (r - r0);
      }
    }
    __syncthreads();
    mine = 0;
    for (int r = r0; r < r1; ++r) {
      if ((taken >> (r - r0)) & 1) {
        w.req[r] = Req{0, 0, 0, 0};
        bits |= DSPARK_DATA_BAD_LENS;
      }
      mine += w.req[r].len ? w.req[r].keys : 0;
    }
    used = block_excl_scan<int64_t, kPlanThreads>(mine, sums, &all);
  }
  // requests that do not fit any more are left out: sums only grow
  for (int r = r0; r < r1; ++r) {
    if (!w.req[r].len) continue;
    used += w.req[r].keys;
    if (used > a.max_keys) {
      w.req[r] = Req{0, 0, 0, 0};
      bits |= DSPARK_DATA_BAD_LENS;
    }
  }
  __syncthreads();
  // tiles in the high words, padded keys in the low ones
  mine = 0;
  auto units = [&](int r) {
    const Req x = w.req[r];
    return (int64_t)((x.len + kRowTile - 1) / kRowTile) << 32 |
           (int64_t)((x.keys + kKeyTile - 1) & ~(kKeyTile - 1));
  };
  for (int r = r0; r < r1; ++r) mine += units(r);
  int64_t at = block_excl_scan<int64_t, kPlanThreads>(mine, sums, &all);
  for (int r = r0; r < r1; ++r) {
    w.tile0[r] = (int32_t)(at >> 32);
    w.key0[r] = (int32_t)at;
    at += units(r);
  }
  if (tid == 0) {
    w.tile0[q.B] = (int32_t)(all >> 32);
    w.key0[q.B] = (int32_t)all;
  }
  __shared__ int found;
  write_meta(a.meta, total, bits, &found);
  // Tiles in order of their keys, where a thread each can count those before its own:
  // long ones at the end would run alone (a prompt of 4096 rows, 32 heads: 237 us
  // with its tiles head by head, 202 so).
  const int tiles = (int)(all >> 32);
  __shared__ int length[kPlanThreads];
  if (tiles <= kPlanThreads) {
    if (tid < tiles) {
      int lo = 0, hi = q.B;  // the last request that starts at or before the tile
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (w.tile0[mid] <= tid) {
          lo = mid;
        } else {
          hi = mid;
        }
      }
      const Req x = w.req[lo];
      length[tid] = x.prefix + min((w.tile0[lo + 1] - tid) * kRowTile, x.len);
    }
    __syncthreads();
    if (tid < tiles) {
      const int mine = length[tid];
      int before = 0;
      for (int t = 0; t < tiles; ++t) {
        const int other = length[t];
        before += other > mine || (other == mine && t < tid);
      }
      w.order[before] = tid;
    }
  } else {
    for (int t = tid; t < tiles; t += kPlanThreads) w.order[t] = t;
  }
}

// ------------------------------------------------------------------ gather

constexpr int kGatherThreads = 256, kGatherRows = 4;  // rows of a wave

// Dense row d is a cached row of the request that has it, or zeros past its keys. Bound
// by a chain of four reads: 4096 rows 7 us, 20,798 rows of an 8-bit cache 14 us.
template <bool E8, int L>
__global__ __launch_bounds__(kGatherThreads) void gather_kernel(LatentPrefillArgs a, Space w) {
  fetch_args<sizeof(a) + sizeof(w)>();
  constexpr int EPL = E8 ? 16 : 8;  // elements of a lane, in 16 bytes
  constexpr int kLanes = L / EPL;
  const int lane = lane_id();
  const int64_t d0 =
      ((int64_t)blockIdx.x * (kGatherThreads / kWave) + threadIdx.x / kWave) * kGatherRows;
  if (d0 >= w.key0[a.req.B]) return;
  // (requests start at multiples of kKeyTile: the rows of a wave are of one)
  const int r = __builtin_amdgcn_readfirstlane(last_at(w.key0, a.req.B, (int)d0));
  const int first = (int)d0 - w.key0[r], keys = w.req[r].keys;
  const int id =
      a.req.table[(size_t)r * a.req.width + (min(first, keys - 1) >> a.kv.page_shift)];
  const int off = first & ((1 << a.kv.page_shift) - 1);
  kv_u32x4 x[kGatherRows], t[kGatherRows];
  unsigned sc[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    x[i] = t[i] = (kv_u32x4){0, 0, 0, 0};
    sc[i] = 127;
    if (first + i < keys && lane < kLanes) {
      x[i] = *(reinterpret_cast<const kv_u32x4*>(a.kv.latent + id * a.kv.page_bytes +
                                                 (off + i) * (L * a.kv.cb)) + lane);
      if constexpr (E8)
        sc[i] = a.kv.scale[id * a.kv.scale_page_bytes + (off + i) * (L / kLatGroup) +
                           lane / (kLatGroup / EPL)];
    }
    if (first + i < keys && lane < 8)
      t[i] = *(reinterpret_cast<const kv_u32x4*>(a.kv.rope + id * a.kv.rope_page_bytes +
                                                 (off + i) * (kRope * 2)) + lane);
  }
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    kv_u32x4* to = reinterpret_cast<kv_u32x4*>(w.lat + (d0 + i) * (L * 2));
    if constexpr (E8) {
      const float e = __builtin_bit_cast(float, sc[i] << 23);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        kv_u32x4 o;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          o[2 * g] = __builtin_bit_cast(
              unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i][2 * h + g], e, false));
          o[2 * g + 1] = __builtin_bit_cast(
              unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i][2 * h + g], e, true));
        }
        if (lane < kLanes) to[2 * lane + h] = o;
      }
    } else {
      if (lane < kLanes) to[lane] = x[i];
    }
    if (lane < 8) *(reinterpret_cast<kv_u32x4*>(w.turned + (d0 + i) * (kRope * 2)) + lane) = t[i];
  }
}

// Rows of `bytes` in LDS, unpadded: 16-byte chunk c of row r lies at chunk c ^
// swizzle(r), so that the rows which a wave reads at one column, and the eight rows
// whose columns it reads transposed, spread over all banks.
template <int BYTES>
__device__ inline int swizzle(int r) {
  return BYTES >= 256 ? (r & 3) << 2 | ((r >> 2) & 3) : ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
}

// One copy of 1024 bytes: rows of BYTES from row r0 of a tile on, `stride` apart in
// memory; `from` is row r0's.
template <int BYTES>
__device__ inline void copy_rows(const unsigned char* from, int64_t stride, int r0, unsigned to) {
  constexpr int kChunks = BYTES / 16;
  const int r = lane_id() / kChunks, c = lane_id() % kChunks;
  copy16_shared(uniform(from), (unsigned)(r * stride) + ((c ^ swizzle<BYTES>(r0 + r)) << 4),
                to);
}

// ------------------------------------------------------------------ expand

constexpr int kExpandThreads = 256;

// kDenseTile keys of one head: D = W X^T with the weights' rows (keys' part, then
// values') as rows and the dense rows as columns, so that a lane's results are
// four elements in a row of one key; they are turned through LDS into whole lines.
// 32 of the L products to a step, through a ring of three stages, so that two
// workgroups share a CU and one's first loads and last stores run beside the other's
// products. 34 GFLOP (4096 keys, 32 heads) 47 us, 740 TFLOP/s; 349 GFLOP (20,798 keys, 64
// heads) 418 us, 840; 43 % of a CU's busy cycles are products of its SIMDs, with a barrier
// after every 16 of a wave and the turn through LDS at the end. (One workgroup of 256 keys
// to a CU: 62 and 554 us where these took 43 and 404.)
// Keys and values round to the query type here, as a model's own projection leaves
// them; kept in 32 bits they would be twice the reads of attend() and no operand.
template <typename T, int L, int N>
__global__ __launch_bounds__(kExpandThreads, 2) void expand_kernel(LatentPrefillArgs a, Space w) {
  typedef Types<T> TT;
  typedef typename TT::V8 V8;
  typedef typename TT::V4 V4;
  constexpr int kW = 4, kStages = 3, kStep = 32, kRowBytes = kStep * 2;
  constexpr int kX = kDenseTile * kRowBytes, kY = 2 * N * kRowBytes, kStage = kX + kY;
  constexpr int kRows = 1024 / kRowBytes;  // of a copy
  constexpr int kXCopies = kDenseTile / kRows / kW, kYCopies = 2 * N / kRows / kW;
  constexpr int NY = N / 32;  // 32-row tiles of a wave: half of the weights' rows
  constexpr int kOut = 64 * N * 2;  // bytes of a wave's results
  __shared__ __align__(1024) unsigned char
      mem[kStages * kStage > kW * kOut ? kStages * kStage : kW * kOut];
  static_assert(sizeof(mem) <= 163840 / 2 - 256, "two workgroups to a CU");
  const unsigned lds = (unsigned)(uintptr_t)(lds_u8*)mem;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int qi = lane & 31, hi = lane >> 5;
  // where there are heads for all XCDs, each has its share of them: their weights
  // stay in its L2, and the heads of a tile of rows meet there
  int h, tile;
  if (a.num_heads % kXcds == 0) {
    const int own = a.num_heads / kXcds, b = blockIdx.x / kXcds;
    h = blockIdx.x % kXcds + b % own * kXcds;
    tile = b / own;
  } else {
    h = blockIdx.x % a.num_heads;
    tile = blockIdx.x / a.num_heads;
  }
  const int64_t d0 = (int64_t)tile * kDenseTile;
  if (d0 >= w.key0[a.req.B]) return;
  const unsigned char* x = w.lat + d0 * (L * 2);
  const unsigned char* wk = a.wk + h * a.w_head_ld;
  const unsigned char* wv = a.wv + h * a.w_head_ld;
  // (rows of 64 bytes: chunk c of row r at c ^ (r >> 2 & 3))
  auto copy = [&](const unsigned char* from, unsigned to) {
    const int r = lane >> 2;
    copy16_shared(uniform(from), (unsigned)(r * (L * 2)) + (((lane & 3) ^ ((r >> 2) & 3)) << 4), to);
  };
  auto fill = [&](int step) {
    const unsigned at = lds + step % kStages * kStage;
#pragma unroll
    for (int n = 0; n < kXCopies; ++n) {
      const int r = (wave * kXCopies + n) * kRows;
      copy(x + (size_t)r * (L * 2) + step * kRowBytes, at + r * kRowBytes);
    }
#pragma unroll
    for (int n = 0; n < kYCopies; ++n) {
      const int r = (wave * kYCopies + n) * kRows;
      const unsigned char* from = r < N ? wk + (size_t)r * (L * 2) : wv + (size_t)(r - N) * (L * 2);
      copy(from + step * kRowBytes, at + kX + r * kRowBytes);
    }
  };
  f32x16 o[NY][2];
#pragma unroll
  for (int y = 0; y < NY; ++y)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[y][c][e] = 0.0f;
  const int half_y = wave & 1, half_x = wave >> 1;
  const int turn = (hi ^ ((qi >> 2) & 3)) << 4;
  const int x_at = (half_x * 64 + qi) * kRowBytes + turn;
  const int y_at = kX + (half_y * N + qi) * kRowBytes + turn;
  constexpr int kSteps = L / kStep;
  fill(0);
  fill(1);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (i + 1 < kSteps) {
      wait_copies<kXCopies + kYCopies>();
    } else {
      wait_copies<0>();
    }
    barrier();
    if (i + 2 < kSteps) fill(i + 2);
    unsigned xa = lds + i % kStages * kStage + x_at, ya = lds + i % kStages * kStage + y_at;
    settle(xa);
    settle(ya);
#pragma unroll
    for (int f = 0; f < kStep / 16; ++f) {
      V8 xf[2], yf[NY];
#pragma unroll
      for (int c = 0; c < 2; ++c) xf[c] = lds_read<V8>((xa ^ (f << 5)) + c * 32 * kRowBytes);
#pragma unroll
      for (int y = 0; y < NY; ++y) yf[y] = lds_read<V8>((ya ^ (f << 5)) + y * 32 * kRowBytes);
#pragma unroll
      for (int y = 0; y < NY; ++y)
#pragma unroll
        for (int c = 0; c < 2; ++c) o[y][c] = TT::mfma32(yf[y], xf[c], o[y][c]);
    }
  }
  // the wave's 64 keys by N elements, to LDS and out
  barrier();
  const unsigned own = lds + wave * kOut;
  constexpr int kChunks = N * 2 / 16;  // of a key
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int y = 0; y < NY; ++y)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        V4 z;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = (T)o[y][c][4 * g + e];
        const int key = c * 32 + qi, chunk = (y * 4 + g) ^ (key & (kChunks - 1));
        lds_write(own + key * (N * 2) + chunk * 16 + hi * 8, z);
      }
  unsigned char* dst =
      w.kv + (((int64_t)h * w.dense + d0 + half_x * 64) * (2 * N) + half_y * N) * 2;
#pragma unroll
  for (int n = 0; n < kOut / 1024; ++n) {
    const int key = n * (kWave / kChunks) + lane / kChunks, c = lane % kChunks;
    const kv_u32x4 z =
        lds_read<kv_u32x4>(own + key * (N * 2) + ((c ^ (key & (kChunks - 1))) << 4));
    *reinterpret_cast<kv_u32x4*>(dst + (int64_t)key * (4 * N) + c * 16) = z;
  }
}

// ------------------------------------------------------------------ attend

constexpr int kAttendWaves = 4;
constexpr int kStepKeys = 32;  // keys of a step
constexpr int kHalves = kStepKeys / 32;

template <int N>
struct Ring {
  static constexpr int kRow = 2 * N;                     // bytes of a key, or of a value
  static constexpr int kPart = kStepKeys * kRow;          // keys, or values
  static constexpr int kTurned = kStepKeys * kRope * 2;
  static constexpr int kStage = 2 * kPart + kTurned;
  static constexpr int kStages = 3;
  static constexpr int kCopies = kPart / 1024 / kAttendWaves;  // of keys, and of values
  static constexpr int kPerWave = 2 * kCopies + 1;
  static constexpr int kOdd = kStages * kStage;          // values with NaN or infinity, a bit each
  static constexpr int kBytes = kOdd + 16;
  static_assert(kCopies >= 1, "a copy for every wave");
  static_assert(kBytes <= 163840 / 2 - 256, "a CU's LDS");
};

// A tile of kRowTile prompt rows of one head, 32 to a wave, over the head's keys up
// to the tile's last row:
//   S^T = K Q^T, O^T += V^T P^T
// as the other attention kernels have it: a lane holds one row's scores, and its
// weights are in place as the operand of the second product.
// Bound by exponentials and products, which the CU's two workgroups trade, half of its
// busy cycles products: a prompt of 4096 rows at 32 heads (172 GFLOP) 205 us, 840 TFLOP/s;
// chunks of 300 to 1100 rows over up to 8300 keys at 64 heads (563 GFLOP) 524 us, 1,070,
// where 31 % of the look-ups in an L2 miss (the prompt: 16 %). (Tiles of a head side by side, 4, 8, 16 before the next head's: 256, 268, 278
// us instead of 243 for the prompt's whole call, the chunks' 4 % better to 2 % worse.)
template <typename T, int N>
__global__ __launch_bounds__(kAttendWaves * kWave, 2) void attend_kernel(LatentPrefillArgs a,
                                                                         Space w) {
  typedef Types<T> TT;
  typedef typename TT::V8 V8;
  typedef typename TT::V4 V4;
  typedef Ring<N> R;
  constexpr int NK = N / 16, NF = NK + kRope / 16;  // operand chunks of a key
  constexpr int ND = N / 32;                        // 32-column tiles of the output
  __shared__ __align__(1024) unsigned char mem[R::kBytes];
  const unsigned lds = (unsigned)(uintptr_t)(lds_u8*)mem;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int qi = lane & 31, hi = lane >> 5;
  int h, tile;
  if (a.num_heads % kXcds == 0) {
    const int own = a.num_heads / kXcds, b = blockIdx.x / kXcds;
    h = blockIdx.x % kXcds + b % own * kXcds;
    tile = b / own;
  } else {
    h = blockIdx.x % a.num_heads;
    tile = blockIdx.x / a.num_heads;
  }
  const int all = w.tile0[a.req.B];
  if (tile >= all) return;
  tile = w.order[tile];
  const int r = __builtin_amdgcn_readfirstlane(last_at(w.tile0, a.req.B, tile));
  const Req req = w.req[r];
  // (a request's tiles count from its last rows, which have the most keys)
  const int mine = w.tile0[r + 1] - 1 - tile;
  const int j0 = mine * kRowTile, rows = min(kRowTile, req.len - j0);
  const int n_tiles = (req.prefix + j0 + rows + kStepKeys - 1) / kStepKeys;
  const unsigned char* kv = w.kv + ((int64_t)h * w.dense + w.key0[r]) * (4 * N);
  const unsigned char* turned = w.turned + (int64_t)w.key0[r] * (kRope * 2);
  auto fill = [&](int t, int stage) {
    const unsigned at = lds + stage * R::kStage;
    constexpr int kRows = 1024 / R::kRow;  // of a copy
#pragma unroll
    for (int n = 0; n < R::kCopies; ++n) {
      const int x = (wave * R::kCopies + n) * kRows;
      const unsigned char* from = kv + (int64_t)(t * kStepKeys + x) * (4 * N);
      copy_rows<R::kRow>(from, 4 * N, x, at + x * R::kRow);
      copy_rows<R::kRow>(from + 2 * N, 4 * N, x, at + R::kPart + x * R::kRow);
    }
    copy_rows<kRope * 2>(turned + (int64_t)(t * kStepKeys + wave * 8) * (kRope * 2), kRope * 2,
                         wave * 8, at + 2 * R::kPart + wave * 1024);
  };
  fill(0, 0);
  if (n_tiles > 1) fill(1, 1);

  float sl = fminf(fabsf(a.scale) * kLog2e, 3.4028235e38f);
  const bool flat = sl == 0.0f;
  if (flat) sl = 1.0f;
  const unsigned sign = a.scale < 0.0f ? 0x80008000u : 0u;
  const int j = j0 + wave * 32 + qi;  // the lane's row
  const bool live = j < req.len;
  const int last = req.prefix + j;    // the last key that it sees
  // of the wave's rows
  const int wave_last = req.prefix + min(j0 + wave * 32 + 31, req.len - 1);
  const bool rows_here = j0 + wave * 32 < req.len;
  V8 qf[NF];
  {
    const unsigned char* src =
        a.q + (size_t)(req.c0 + j) * a.q_ld + (size_t)h * ((N + kRope) * 2) + hi * 16;
    kv_u32x4 x[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      x[f] = (kv_u32x4){0, 0, 0, 0};
      if (live && !flat) x[f] = *reinterpret_cast<const kv_u32x4*>(src + f * 32) ^ sign;
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      settle(x[f]);
      qf[f] = __builtin_bit_cast(V8, x[f]);
    }
  }
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
  float mx = -__builtin_inff(), l = 0.0f;

  const int key_at = qi * R::kRow + ((hi ^ swizzle<R::kRow>(qi)) << 4);
  const int turned_at = 2 * R::kPart + qi * (kRope * 2) + ((hi ^ swizzle<kRope * 2>(qi)) << 4);
  const int t4 = lane & 15, vrow = hi * 4 + (t4 >> 2);
  const int val_at = R::kPart + vrow * R::kRow +
                     (((((lane >> 4) & 1) * 2 + ((t4 >> 1) & 1)) ^ swizzle<R::kRow>(vrow)) << 4) +
                     (t4 & 1) * 8;

  int stage = 0;
  for (int t = 0; t < n_tiles; ++t) {
    const int key0 = t * kStepKeys;
    if (t + 1 < n_tiles) {
      wait_copies<R::kPerWave>();
    } else {
      wait_copies<0>();
    }
    // some row of the workgroup does not see all of the tile
    const bool edge = key0 + kStepKeys > req.prefix + j0 + 1;
    const unsigned buf = lds + stage * R::kStage;
    if (edge) {
      // NaN and infinity in a value must not meet the zero weight of a row that does
      // not see it: such values become zeros, and rows that see one get a NaN score
      // instead. Eight values to a wave.
      const unsigned at = buf + R::kPart + wave * (8 * R::kRow) + lane * 16;
      unsigned found = 0;
#pragma unroll
      for (int n = 0; n < R::kCopies; ++n) {
        constexpr int kLanes = R::kRow / 16;
        kv_u32x4 x = lds_read<kv_u32x4>(at + n * 1024);
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          bad |= (x[e] & TT::kExpMask) == TT::kExpMask ||
                 (x[e] >> 16 & TT::kExpMask) == TT::kExpMask;
        unsigned long long b = __ballot(bad);
        unsigned here = 0;
        while (b) {
          here |= 1u << (n * (kWave / kLanes) + (int)__builtin_ctzll(b) / kLanes);
          b &= b - 1;
        }
        found |= here;
        if ((here >> (n * (kWave / kLanes) + lane / kLanes)) & 1)
          lds_write(at + n * 1024, (kv_u32x4){0, 0, 0, 0});
      }
      if (lane == 0) lds_write<unsigned char>(lds + R::kOdd + (t & 1) * 4 + wave, (unsigned char)found);
    }
    barrier();
    if (t + 2 < n_tiles) fill(t + 2, stage + 2 >= R::kStages ? stage + 2 - R::kStages : stage + 2);
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    if (!rows_here || key0 > wave_last) continue;
    // Scores
    f32x16 sc[kHalves];
#pragma unroll
    for (int b = 0; b < kHalves; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[b][e] = 0.0f;
    unsigned ka = buf + key_at, ta = buf + turned_at, va = buf + val_at;
    settle(ka);
    settle(ta);
    settle(va);
    constexpr int FB = 4 / kHalves;
    V8 kf[2][FB][kHalves];
    auto read_keys = [&](int f0, int into) {
#pragma unroll
      for (int f = 0; f < FB; ++f)
#pragma unroll
        for (int b = 0; b < kHalves; ++b)
          kf[into][f][b] = f0 + f < NK
                               ? lds_read<V8>((ka ^ ((f0 + f) << 5)) + b * 32 * R::kRow)
                               : lds_read<V8>((ta ^ ((f0 + f - NK) << 5)) + b * 32 * (kRope * 2));
    };
    read_keys(0, 0);
#pragma unroll
    for (int f0 = 0; f0 < NF; f0 += FB) {
      if (f0 + FB < NF) read_keys(f0 + FB, (f0 / FB + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = 0; f < FB; ++f)
#pragma unroll
        for (int b = 0; b < kHalves; ++b)
          sc[b] = TT::mfma32(kf[(f0 / FB) & 1][f][b], qf[f0 + f], sc[b]);
      __builtin_amdgcn_sched_barrier(0);
    }
    V4 vl[2][ND], vh[2][ND];
    auto read_values = [&](int c, int into) {
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        vl[into][d] = lds_columns<V4>((va ^ (d << 6)) + c * 16 * R::kRow);
        vh[into][d] = lds_columns<V4>((va ^ (d << 6) ^ 32) + (c * 16 + 8) * R::kRow);
      }
    };
    // From here to the step's end the wave goes first: its exponentials fill the gaps
    // of the products of the CU's other workgroup (a prompt of 4096 rows, 32 heads, two
    // cards:
    // 245 -> 231, 257 -> 243 us; the scores' products first instead 236).
    __builtin_amdgcn_s_setprio(2);
    read_values(0, 0);
    if (edge) {
      const unsigned odd = lds_read<unsigned>(lds + R::kOdd + (t & 1) * 4);
#pragma unroll
      for (int b = 0; b < kHalves; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = b * 32 + 8 * (e >> 2) + 4 * hi + (e & 3);
          if (key0 + k > last) {
            sc[b][e] = -__builtin_inff();
          } else if ((odd >> k) & 1) {
            sc[b][e] = __builtin_nanf("");
          }
        }
    }
    float top = sc[0][0];
#pragma unroll
    for (int b = 0; b < kHalves; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[b][e]);
    top *= sl;
    if (__any(top - mx > TT::kAbove + TT::kSlack)) {
      float next = fmaxf(top, __shfl_xor(top, 32, kWave));
      // (rows for themselves: what one sees moves no other's weights)
      const bool moves = next - mx > TT::kAbove + TT::kSlack;
      if constexpr (TT::kAbove > 0.0f) {
        // (not where kAbove rounds up to more than a weight may be)
        const float less = next - TT::kAbove;
        next = next - less > TT::kAbove + TT::kSlack ? next : less;
      }
      next = moves ? fmaxf(mx, next) : mx;
      const float fix = next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx - next);
      mx = next;
      l *= fix;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] *= fix;
    }
    const float ref = mx == -__builtin_inff() ? 0.0f : mx;
    // The product with the scale and the maximum in one rounding: the largest weight is
    // then 2^d, d up to half a step of its score. Where that could matter (2^-8 at a
    // score of 2^16), the product rounds first and the largest weight is 1.
    const bool large = __any(fabsf(ref) > 65536.0f);
    // The product takes weights of the query type, each off by up to half its step;
    // their sum takes them as they are.
    V8 pf[2 * kHalves];
    auto weigh = [&](auto exponent) {
#pragma unroll
      for (int b = 0; b < kHalves; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p = __builtin_amdgcn_exp2f(exponent(sc[b][e]));
          l += p;
          pf[2 * b + (e >> 3)][e & 7] = (T)p;
        }
    };
    if (__builtin_expect(large, 0)) {
      weigh([&](float x) { return x * sl - ref; });
    } else {
      weigh([&](float x) { return __builtin_fmaf(x, sl, -ref); });
    }
#pragma unroll
    for (int c = 0; c < 2 * kHalves; ++c) {
      if (c + 1 < 2 * kHalves) read_values(c + 1, (c + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const V8 vf = __builtin_shufflevector(vl[c & 1][d], vh[c & 1][d], 0, 1, 2, 3, 4, 5, 6, 7);
        o[d] = TT::mfma32(vf, pf[c], o[d]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  }
  if (!rows_here) return;
  const float sum = l + __shfl_xor(l, 32, kWave);
  if (!live) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  T* dst = reinterpret_cast<T*>(a.out + (size_t)(req.c0 + j) * a.out_ld) + (size_t)h * N + hi * 4;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      V4 z;
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = (T)(o[d][4 * g + e] * inv);
      *reinterpret_cast<V4*>(dst + d * 32 + g * 8) = z;
    }
  if (a.lse && hi == 0)
    a.lse[(size_t)(req.c0 + j) * a.num_heads + h] =
        sum == 0.0f ? -__builtin_inff() : (mx + __builtin_amdgcn_logf(sum)) * kLn2;
}

// ------------------------------------------------------------------ launch

template <typename T, int N>
void launch_dims(const LatentPrefillArgs& a, const Space& w, int dense_tiles, int row_tiles,
                 hipStream_t s) {
  const unsigned expand = (unsigned)dense_tiles * a.num_heads;
  if (a.kv.dim == 256) {
    hipLaunchKernelGGL((expand_kernel<T, 256, N>), dim3(expand), dim3(kExpandThreads), 0, s, a, w);
  } else {
    hipLaunchKernelGGL((expand_kernel<T, 512, N>), dim3(expand), dim3(kExpandThreads), 0, s, a, w);
  }
  hipLaunchKernelGGL((attend_kernel<T, N>), dim3((unsigned)row_tiles * a.num_heads),
                     dim3(kAttendWaves * kWave), 0, s, a, w);
}

template <bool E8>
void launch_gather(const LatentPrefillArgs& a, const Space& w, hipStream_t s) {
  const unsigned grid =
      (unsigned)(w.dense / (kGatherThreads / kWave * kGatherRows));
  if (a.kv.dim == 256) {
    hipLaunchKernelGGL((gather_kernel<E8, 256>), dim3(grid), dim3(kGatherThreads), 0, s, a, w);
  } else {
    hipLaunchKernelGGL((gather_kernel<E8, 512>), dim3(grid), dim3(kGatherThreads), 0, s, a, w);
  }
}

}  // namespace prefill

size_t latent_prefill_workspace(int B, int max_rows, int max_keys, int num_heads, int nope,
                                int latent_dim) {
  return prefill::layout(B, max_rows, max_keys, num_heads, nope, latent_dim).bytes;
}

hipError_t launch_latent_prefill(const LatentPrefillArgs& a, dspark_dtype dt, hipStream_t s) {
  const prefill::Layout p =
      prefill::layout(a.req.B, a.req.max_rows, a.max_keys, a.num_heads, a.nope, a.kv.dim);
  unsigned char* at = static_cast<unsigned char*>(a.ws);
  prefill::Space w;
  w.req = reinterpret_cast<prefill::Req*>(at);
  w.tile0 = reinterpret_cast<int32_t*>(at + p.tile0);
  w.key0 = reinterpret_cast<int32_t*>(at + p.key0);
  w.order = reinterpret_cast<int32_t*>(at + p.order);
  w.lat = at + p.lat;
  w.turned = at + p.turned;
  w.kv = at + p.kv;
  w.dense = p.dense;
  hipLaunchKernelGGL(prefill::plan_kernel, dim3(1), dim3(prefill::kPlanThreads), 0, s, a, w);
  hipError_t e = hipGetLastError();
  const int rows = std::min(a.req.max_rows, a.max_keys);
  if (e != hipSuccess || a.req.B == 0 || rows == 0) return e;
  if (a.kv.cb == 1) {
    prefill::launch_gather<true>(a, w, s);
  } else {
    prefill::launch_gather<false>(a, w, s);
  }
  const int dense_tiles = (int)(p.dense / prefill::kDenseTile);
  const int row_tiles = prefill::most_tiles(a.req.B, a.req.max_rows, a.max_keys);
  if (dt == DSPARK_BF16) {
    if (a.nope == 64) {
      prefill::launch_dims<__bf16, 64>(a, w, dense_tiles, row_tiles, s);
    } else {
      prefill::launch_dims<__bf16, 128>(a, w, dense_tiles, row_tiles, s);
    }
  } else {
    if (a.nope == 64) {
      prefill::launch_dims<_Float16, 64>(a, w, dense_tiles, row_tiles, s);
    } else {
      prefill::launch_dims<_Float16, 128>(a, w, dense_tiles, row_tiles, s);
    }
  }
  return hipGetLastError();
}

}  // namespace dspark
