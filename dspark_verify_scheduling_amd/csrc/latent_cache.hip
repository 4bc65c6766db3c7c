// The paged latent cache of the target pass: append with norm and rotation, read
// back, and the commit of an accepted path.
//
// All three move every byte once and compute next to nothing on it, so they are
// bound by HBM (large calls) or by the latency of a launch and a few dependent
// reads (small ones). Workgroup 0 of each launch checks every request and writes
// the status; the others leave bad requests or rows out.
#include "append_row.h"
#include "kv_moves.h"
#include "latent.h"

#include <algorithm>

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
// Workgroups of a launch that have rows, at most: a grid of 2^32 threads or more is
// cut off without an error.
constexpr int64_t kMostWgs = 1 << 20;

// ------------------------------------------------------------------ append

// Whether request r's tree is one; L lanes hold it.
__device__ inline bool tree_of(const ReqView& q, int r, int len, int* par) {
  const int lane = lane_id();
  *par = lane + 1 < len ? q.parents[(size_t)r * q.gamma + lane] : 0;
  return __ballot(*par < 0 || *par > lane) == 0;
}

// Trees and positions of all requests; a request to a wave at a time.
__device__ int tree_status(const LatentAppendArgs& a, int total_eff, int64_t most) {
  const ReqView& q = a.req;
  const int64_t reach = (int64_t)q.width << a.kv.page_shift;
  int bits = 0;
  for (int r = threadIdx.x / kWave; r < q.B; r += kWaves) {
    int s, e, prefix, par;
    if (!span_of(q, r, total_eff, reach, most, &s, &e, &prefix)) continue;
    if (!tree_of(q, r, e - s, &par)) {
      bits |= DSPARK_DATA_BAD_TREE;
    } else if (a.rope && (int64_t)prefix + (e - s) > a.rope_rows) {
      // the depths may still be small enough
      int depth = 0;
      for (int m = lane_id() + 1; m > 0 && lane_id() + 1 < e - s;
           m = q.parents[(size_t)r * q.gamma + m - 1])
        ++depth;
      if (e > s && (int64_t)prefix + depth >= a.rope_rows) bits |= DSPARK_DATA_BAD_POS;
    }
  }
  return bits;
}

// A lane's eight elements of a pair-wise rotation over eight lanes (64 elements).
struct Turn {
  float co[8], si[8];
  __device__ __forceinline__ void load(const float* cs, bool interleaved, int lane) {
    const int li = lane & 7;
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        co[2 * e] = co[2 * e + 1] = cs[4 * li + e];
        si[2 * e + 1] = cs[kRope / 2 + 4 * li + e];
        si[2 * e] = -si[2 * e + 1];
      }
    } else {
      const bool low = li < 4;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        co[e] = cs[8 * (li & 3) + e];
        si[e] = cs[kRope / 2 + 8 * (li & 3) + e];
        si[e] = low ? -si[e] : si[e];
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ typename Vec8<T>::type of(const typename Vec8<T>::type& in,
                                                       bool interleaved) const {
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)in[e];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = interleaved ? x[e ^ 1] : lane_xor<4>(x[e]);
    typename Vec8<T>::type out;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = (T)__builtin_fmaf(x[e], co[e], y[e] * si[e]);
    return out;
  }
};

// `per` packed rows to a workgroup, kWaves / per waves to a row: the first takes
// its latent, and the rotated part with the query heads go eight at a time to the
// waves in turn. 16,401 rows of 512 + 64 and 64 query heads into an 8-bit cache: 52
// us, 5.8 TB/s read and written. A few rows: 4.1 us of dependent reads. All waves to a
// row, or a row to each: 1,024 rows at 64 heads and 8 bits 7.7 and 8.7 us, at 20 heads
// 5.4 and 5.3, at 8 heads (L = 256) 5.1 and 4.6; 3,000 rows 15.8 and 13.1, 10.2 and 7.3,
// 9.0 and 5.7; at 128 heads a row to a workgroup is 7 % better there too.
template <typename T, bool E8, int L>
__global__ __launch_bounds__(kThreads) void latent_append_kernel(LatentAppendArgs a, int per) {
  typedef typename Vec8<T>::type T8;
  constexpr int kLanes = L / 8;  // lanes that hold the latent
  fetch_args<sizeof(a) + 4>();
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int64_t most = q.gamma ? q.gamma + 1 : 0x7FFFFFFF;
  const int64_t reach = (int64_t)q.width << a.kv.page_shift;
  int total;
  const int total_eff = rows_in_use(q, &total);
  if (blockIdx.x == 0) {
    if (a.first_row) return;
    __shared__ int all;
    int bits = total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    bits |= spans_status<kThreads>(q, a.kv.page_shift, a.kv.num_blocks, total_eff, most);
    if (q.parents) {
      bits |= tree_status(a, total_eff, most);
    } else if (a.rope) {
#pragma unroll 4
      for (int r = tid; r < q.B; r += kThreads) {
        int s, e, prefix;
        if (span_of(q, r, total_eff, reach, most, &s, &e, &prefix) && e > s &&
            (int64_t)prefix + (e - s) > a.rope_rows)
          bits |= DSPARK_DATA_BAD_POS;
      }
    }
    write_meta(a.meta, total, bits, &all);
    return;
  }
  const int split = kWaves / per, sub = wave % split;
  const int64_t packed = a.first_row + (int64_t)(blockIdx.x - 1) * per + wave / split;
  if (packed >= total_eff) return;
  const unsigned char* x = a.x + (size_t)packed * a.x_ld;
  const unsigned char* heads = a.q + (size_t)packed * a.q_ld;
  // loaded with the reads that say where the row goes
  T8 lat = {}, weight = {}, next[2];
  if (sub == 0 && lane < kLanes) {
    lat = *(reinterpret_cast<const T8*>(x) + lane);
    if (a.weight) weight = *(reinterpret_cast<const T8*>(a.weight) + lane);
  }
  // head -1: the row's own rotated part
  auto load = [&](int h) {
    T8 v = {};
    if (h < a.num_heads)
      v = *(reinterpret_cast<const T8*>(h < 0 ? x + L * 2 : heads + h * a.q_head_ld) + (lane & 7));
    return v;
  };
  int h = sub * 8 + (lane >> 3) - 1;
  next[0] = load(h);
  next[1] = load(h + 8 * split);
  int r, j, prefix;
  rows_requests<1>(q, (int)packed, total_eff, reach, most, &r, &j, &prefix);
  r = __builtin_amdgcn_readfirstlane(r);
  j = __builtin_amdgcn_readfirstlane(j);
  prefix = __builtin_amdgcn_readfirstlane(prefix);
  if (j < 0) return;
  const int64_t slot = (int64_t)prefix + j;
  const int id = q.table[(size_t)r * q.width + (slot >> a.kv.page_shift)];
  int depth = j;
  if (q.parents) {
    int par;
    if (!tree_of(q, r, q.cu[r + 1] - q.cu[r], &par)) return;
    depth = 0;
    for (int n = j; n > 0; n = __builtin_amdgcn_readlane(par, n - 1)) ++depth;
  }
  const int64_t pos = (int64_t)prefix + depth;
  if (a.rope && pos >= a.rope_rows) return;
  Turn turn;
  if (a.rope) turn.load(a.rope + (size_t)pos * kRope, a.rope_interleaved, lane);
  // after the table's rotations, which then wait along with the page's id
  if (id < 0 || id >= a.kv.num_blocks) return;
  const int off = (int)(slot & ((1 << a.kv.page_shift) - 1));

  if (sub == 0) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (float)lat[e];
    if (a.weight) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(y[e], y[e], ss);
      ss = lanes_sum<kLanes>(ss);
      const float rstd = 1.0f / sqrtf(ss * (1.0f / L) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * rstd * (float)weight[e];
    }
    unsigned char* to = a.kv.latent + (size_t)id * a.kv.page_bytes;
    if constexpr (!E8) {
      T8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (T)y[e];
      if (lane < kLanes) *(reinterpret_cast<T8*>(to + (size_t)off * (L * 2)) + lane) = o;
    } else {
      // an exponent for each sixteen lanes
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = finite_f32(y[e]) ? fmaxf(amax, fabsf(y[e])) : amax;
      amax = lanes_max<kLatGroup / 8>(amax);
      const int e8 = e4m3_exponent(amax);
      const float inv = pow2f(-e8);
      kv_u32x2 c;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        int wd = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_operand(y[4 * g], inv),
                                                 e4m3_operand(y[4 * g + 1], inv), 0, false);
        wd = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_operand(y[4 * g + 2], inv),
                                             e4m3_operand(y[4 * g + 3], inv), wd, true);
        c[g] = (unsigned)wd;
      }
      if (lane < kLanes) {
        *(reinterpret_cast<kv_u32x2*>(to + (size_t)off * L) + lane) = c;
        if (lane % (kLatGroup / 8) == 0)
          a.kv.scale[(size_t)id * a.kv.scale_page_bytes + off * (L / kLatGroup) +
                     lane / (kLatGroup / 8)] = (uint8_t)(e8 + 127);
      }
    }
  }
  unsigned char* out = a.q_out + (size_t)packed * a.q_out_ld;
  unsigned char* own = a.kv.rope + (size_t)id * a.kv.rope_page_bytes + (size_t)off * (kRope * 2);
  auto store = [&](int to, const T8& v) {
    if (to < a.num_heads)
      *(reinterpret_cast<T8*>(to < 0 ? own : out + to * a.q_out_head_ld) + (lane & 7)) = v;
  };
  // two loads under way, each in registers of its own
  for (; h - (lane >> 3) < a.num_heads; h += 16 * split) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int to = h + 8 * split * i;
      const T8 v = next[i];
      next[i] = load(to + 16 * split);
      store(to, a.rope ? turn.template of<T>(v, a.rope_interleaved) : v);
    }
  }
}

// ------------------------------------------------------------------ read

constexpr int kReadRows = 4;  // of a wave, under way at once

// kReadRows rows to a wave: their requests and pages are found together, then each
// row is one 16-byte load a lane for the latent and one of eight lanes for the
// rotated part. 16,401 rows of an 8-bit cache: 10.9 us, 2.7 TB/s, of which 4.4 are a
// single row's.
template <bool E8, int L>
__global__ __launch_bounds__(kThreads) void latent_read_kernel(LatentReadArgs a) {
  constexpr int EPL = E8 ? 16 : 8;  // elements of a lane, in 16 bytes
  constexpr int kLanes = L / EPL;
  fetch_args<sizeof(a)>();
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  int total;
  const int total_eff = rows_in_use(q, &total);
  if (blockIdx.x == 0) {
    if (a.first_row) return;
    __shared__ int all;
    int bits = total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    bits |= spans_status<kThreads>(q, a.kv.page_shift, a.kv.num_blocks, total_eff, 0x7FFFFFFF);
    write_meta(a.meta, total, bits, &all);
    return;
  }
  const int64_t row0 = a.first_row + ((int64_t)(blockIdx.x - 1) * kWaves + wave) * kReadRows;
  if (row0 >= total_eff) return;
  int r, j, prefix, id = -1, off = 0;
  rows_requests<kReadRows>(q, (int)row0, total_eff, (int64_t)q.width << a.kv.page_shift,
                           0x7FFFFFFF, &r, &j, &prefix);
  if (j >= 0) {
    const int64_t slot = (int64_t)prefix + j;
    id = q.table[(size_t)r * q.width + (slot >> a.kv.page_shift)];
    if (id >= a.kv.num_blocks) id = -1;
    off = (int)(slot & ((1 << a.kv.page_shift) - 1));
  }
  kv_u32x4 w[kReadRows], p[kReadRows];
  unsigned sc[kReadRows];
  int ids[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    ids[i] = __builtin_amdgcn_readlane(id, i);
    const int o = __builtin_amdgcn_readlane(off, i);
    const size_t page = (size_t)max(ids[i], 0);
    w[i] = p[i] = (kv_u32x4){0, 0, 0, 0};
    sc[i] = 127;
    if (ids[i] >= 0 && lane < kLanes) {
      w[i] = __builtin_nontemporal_load(reinterpret_cast<const kv_u32x4*>(
                 a.kv.latent + page * a.kv.page_bytes + (size_t)o * (L * a.kv.cb)) + lane);
      if constexpr (E8)
        sc[i] = a.kv.scale[page * a.kv.scale_page_bytes + o * (L / kLatGroup) +
                           lane / (kLatGroup / EPL)];
    }
    if (ids[i] >= 0 && lane < 8)
      p[i] = *(reinterpret_cast<const kv_u32x4*>(a.kv.rope + page * a.kv.rope_page_bytes +
                                                 (size_t)o * (kRope * 2)) + lane);
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (ids[i] < 0) continue;
    kv_u32x4* to = reinterpret_cast<kv_u32x4*>(a.latent_out + (size_t)(row0 + i) * a.out_ld);
    if constexpr (E8) {
      const float e = pow2f((int)sc[i] - 127);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        kv_u32x4 o;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          o[2 * g] = __builtin_bit_cast(
              unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i][2 * x + g], e, false));
          o[2 * g + 1] = __builtin_bit_cast(
              unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i][2 * x + g], e, true));
        }
        if (lane < kLanes) __builtin_nontemporal_store(o, to + 2 * lane + x);
      }
    } else {
      if (lane < kLanes) __builtin_nontemporal_store(w[i], to + lane);
    }
    if (lane < 8)
      *(reinterpret_cast<kv_u32x4*>(a.rope_out + (size_t)(row0 + i) * a.rope_out_ld) + lane) = p[i];
  }
}

// ------------------------------------------------------------------ commit

// A workgroup per (request, a few layers), as many as its threads hold; a thread owns
// 16-byte columns of a row's latent and rotated part or one byte of its exponents
// (256 requests, 27 layers, 8 bits, two rows each to move: 10.8 us, 1.6 TB/s; bound by
// the path's look-up, three dependent reads in each of six workgroups of a request),
// and moves the path's rows of that column in ascending order (as commit_kernel of
// the key/value cache does, with the same reason why batches of loads may run
// ahead of their stores).
__global__ __launch_bounds__(kCommitThreads) void latent_commit_kernel(CommitArgs a, LatentView kv) {
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
      const int mask = (1 << kv.page_shift) - 1;
      s_id[i] = q.table[(size_t)r[0] * q.width + (src[0] >> kv.page_shift)];
      d_id[i] = q.table[(size_t)r[0] * q.width + (dst[0] >> kv.page_shift)];
      s_off[i] = (int)(src[0] & mask);
      d_off[i] = (int)(dst[0] & mask);
    }
    if (lane == 0) n_moves = __popcll(m);
  }
  __syncthreads();
  const int n = n_moves;
  if (n == 0) return;
  const int row_bytes = kv.dim * kv.cb, vecs = row_bytes / 16, turned = kRope * 2 / 16;
  const int groups = kv.scale ? kv.dim / kLatGroup : 0;
  const int cols = vecs + turned + groups;
  const int per = kCommitThreads / cols;  // layers of a workgroup
  const int layer = blockIdx.y * per + tid / cols, col = tid % cols;
  if (tid / cols >= per || layer >= kv.num_layers) return;
  if (col < vecs) {
    move_column<kv_u32x4>(kv.latent + layer * kv.layer_bytes + col * 16, kv.page_bytes, row_bytes,
                          n, s_id, s_off, d_id, d_off);
  } else if (col < vecs + turned) {
    move_column<kv_u32x4>(kv.rope + layer * kv.rope_layer_bytes + (col - vecs) * 16,
                          kv.rope_page_bytes, kRope * 2, n, s_id, s_off, d_id, d_off);
  } else {
    move_column<unsigned char>(kv.scale + layer * kv.scale_layer_bytes + (col - vecs - turned),
                               kv.scale_page_bytes, groups, n, s_id, s_off, d_id, d_off);
  }
}

template <typename T, bool E8>
void append_by_dim(const LatentAppendArgs& a, int per, unsigned grid, hipStream_t s) {
  if (a.kv.dim == 256) {
    hipLaunchKernelGGL((latent_append_kernel<T, E8, 256>), dim3(grid), dim3(kThreads), 0, s, a, per);
  } else {
    hipLaunchKernelGGL((latent_append_kernel<T, E8, 512>), dim3(grid), dim3(kThreads), 0, s, a, per);
  }
}

template <bool E8>
void read_by_dim(const LatentReadArgs& a, unsigned grid, hipStream_t s) {
  if (a.kv.dim == 256) {
    hipLaunchKernelGGL((latent_read_kernel<E8, 256>), dim3(grid), dim3(kThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL((latent_read_kernel<E8, 512>), dim3(grid), dim3(kThreads), 0, s, a);
  }
}

}  // namespace

hipError_t launch_latent_append(const LatentAppendArgs& a, dspark_dtype dt, hipStream_t s) {
  const int64_t rows = a.req.B > 0 ? a.req.max_rows : 0;
  // few rows: their heads on all waves
  const int per = rows <= 2048 ? 1 : kWaves;
  LatentAppendArgs part = a;
  part.first_row = 0;
  do {
    const int64_t wgs = std::min<int64_t>((rows - part.first_row + per - 1) / per, kMostWgs);
    const unsigned grid = 1u + (unsigned)wgs;
    if (a.kv.cb == 1) {
      append_by_dim<__bf16, true>(part, per, grid, s);
    } else if (dt == DSPARK_BF16) {
      append_by_dim<__bf16, false>(part, per, grid, s);
    } else {
      append_by_dim<_Float16, false>(part, per, grid, s);
    }
    part.first_row += kMostWgs * per;
  } while (part.first_row < rows);
  return hipGetLastError();
}

hipError_t launch_latent_read(const LatentReadArgs& a, hipStream_t s) {
  const int64_t rows = a.req.B > 0 ? a.req.max_rows : 0;
  constexpr int per = kWaves * kReadRows;
  LatentReadArgs part = a;
  part.first_row = 0;
  do {
    const int64_t wgs = std::min<int64_t>((rows - part.first_row + per - 1) / per, kMostWgs);
    if (a.kv.cb == 1) {
      read_by_dim<true>(part, 1u + (unsigned)wgs, s);
    } else {
      read_by_dim<false>(part, 1u + (unsigned)wgs, s);
    }
    part.first_row += kMostWgs * per;
  } while (part.first_row < rows);
  return hipGetLastError();
}

hipError_t launch_latent_commit(const CommitArgs& a, const LatentView& kv, hipStream_t s) {
  const int cols = kv.dim * kv.cb / 16 + kRope * 2 / 16 + (kv.scale ? kv.dim / kLatGroup : 0);
  const int per = kCommitThreads / cols;
  hipLaunchKernelGGL(latent_commit_kernel,
                     dim3(1u + (unsigned)a.req.B, (unsigned)((kv.num_layers + per - 1) / per)),
                     dim3(kCommitThreads), 0, s, a, kv);
  return hipGetLastError();
}

}  // namespace dspark
