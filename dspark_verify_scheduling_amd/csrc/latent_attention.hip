// Attention of packed verify rows over the latents of a paged cache: launch,
// workspace and the joining kernel. The split kernel is in latent_attention.h.
#include "latent_attention.h"

#include <algorithm>

namespace dspark {

namespace lattn {
namespace {

constexpr int join_threads(bool shared) { return shared ? 512 : 256; }

// One workgroup per (request, share of its blocks of 32 rows by 32 columns): joins
// the parts that several workgroups of the split kernel left of a segment, a wave to
// a block, its parts in order and several at once, a part's statistics and outputs
// together. SHARED: the waves take the parts of one block by turns and meet in LDS,
// for few blocks of many parts (two contexts of 40k and 131k, 20 heads: 11 us
// against 32, 13 with four waves; 32 chains, 128 heads, two or three parts each: 19.6
// against 11.8). By the number of blocks, whole calls over 4k keys and more: 128 blocks
// 33 us shared, 43 not; 512, 36.7 and 35.0; 1,024, 47.5 and 41.6; 2,048, 70 and 58. The
// first workgroup of each request also checks it and its pages.
template <typename T, int L, bool SHARED>
__global__ __launch_bounds__(join_threads(SHARED)) void join_kernel(LatentAttnArgs a, Parts ws,
                                                                    int shares) {
  constexpr int kJoinThreads = join_threads(SHARED);
  constexpr int kBlocks = L / 32, kJoinWaves = kJoinThreads / kWave;
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int share = blockIdx.x % shares, r = blockIdx.x / shares;
  const int64_t units = ws.base[q.B], base = ws.base[r], end = ws.base[r + 1];
  int total;
  const int total_eff = rows_in_use(q, &total);
  int c0, len, prefix;
  const bool good = rows_of(q, a.kv.page_shift, r, total_eff, &c0, &len, &prefix);
  bool tree = true;
  if (good && q.parents) {
    const int up = lane + 1 < len ? q.parents[(size_t)r * q.gamma + lane] : 0;
    tree = __ballot(up < 0 || up > lane) == 0;
  }
  if (share == 0) {
    int bits = 0;
    if (!good) {
      bits = request_status(q, r, total_eff);
      if (!bits) bits = DSPARK_DATA_BAD_PAGE;
    } else if (end == base) {
      bits = DSPARK_DATA_BAD_LENS;  // rows of a request ahead of it
    } else if (!tree) {
      bits = DSPARK_DATA_BAD_TREE;
    } else {
      const int64_t keys = (int64_t)prefix + len;
      for (int64_t p = tid; p <= (keys - 1) >> a.kv.page_shift; p += kJoinThreads) {
        const int id = q.table[(size_t)r * q.width + p];
        if (id < 0 || id >= a.kv.num_blocks) bits = DSPARK_DATA_BAD_PAGE;
      }
    }
    if (bits) atomicOr(a.meta + 1, bits);
  }
  if (!good || !tree || end == base) return;
  const Shape s = shape_of<L>(a.num_heads, c0, len, prefix);
  const int wgs = wgs_in_use(units, ws.wgs);
  const int qi = lane & 31;
  const int wave = tid / kWave;
  // blocks in order over the segments and their row tiles
  constexpr int kStep = SHARED ? 1 : kJoinWaves;
  for (int n = share * kStep + (SHARED ? 0 : wave); n < s.mtiles * kBlocks; n += shares * kStep) {
    const int mtile = n / kBlocks, block = n - mtile * kBlocks;
    const int seg = mtile / s.per;
    const int64_t u0 = base + (int64_t)seg * (s.nku + kSetup), u1 = u0 + s.nku + kSetup;
    // workgroups of the first and the last unit with keys
    const int wa = (int)(((u0 + kSetup + 1) * wgs - 1) / units), wb = (int)((u1 * wgs - 1) / units);
    if (wa == wb) continue;
    const int slot0 = 2 * wa + (wg_start(units, wa, wgs) >= u0 ? 0 : 1);
    const int parts = wb - wa + 1;
    const int tile = mtile - seg * s.per;
    constexpr int kAhead = 4;
    float top = -__builtin_inff(), sum = 0.0f;
    f32x4 y[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) y[x] = (f32x4){0, 0, 0, 0};
    constexpr int kEvery = SHARED ? kJoinWaves : 1;
    for (int p0 = SHARED ? wave : 0; p0 < parts; p0 += kAhead * kEvery) {
      float m[kAhead], l[kAhead];
      f32x4 v[kAhead][4];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int p = p0 + k * kEvery;
        m[k] = -__builtin_inff();
        l[k] = 0.0f;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[k][x] = (f32x4){0, 0, 0, 0};
        if (p < parts) {
          const size_t at = (size_t)(p ? 2 * (wa + p) : slot0) * ws.rows + tile * kRowTile;
          m[k] = ws.m[at + qi];
          l[k] = ws.l[at + qi];
          const float* src = ws.o + at * L + block * (32 * kRowTile) + lane * 4;
#pragma unroll
          for (int x = 0; x < 4; ++x) v[k][x] = *reinterpret_cast<const f32x4*>(src + x * (kWave * 4));
        }
      }
      float next = top;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) next = fmaxf(next, m[k]);
      const bool none = next == -__builtin_inff();  // nothing seen, or NaN scores only
      const float fix = none ? 1.0f : __builtin_amdgcn_exp2f(top - next);
      sum *= fix;
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] *= fix;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float f = none ? 1.0f : __builtin_amdgcn_exp2f(m[k] - next);
        sum += l[k] * f;
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] += v[k][x] * f;
      }
      top = next;
    }
    if constexpr (SHARED) {
      __shared__ float met[kJoinWaves - 1][18][kWave];
      __syncthreads();
      if (wave > 0) {
        met[wave - 1][16][lane] = top;
        met[wave - 1][17][lane] = sum;
#pragma unroll
        for (int e = 0; e < 16; ++e) met[wave - 1][e][lane] = y[e >> 2][e & 3];
      }
      __syncthreads();
      if (wave > 0) continue;
      float next = top;
#pragma unroll
      for (int w = 0; w < kJoinWaves - 1; ++w) next = fmaxf(next, met[w][16][lane]);
      const bool none = next == -__builtin_inff();
      const float fix = none ? 1.0f : __builtin_amdgcn_exp2f(top - next);
      sum *= fix;
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] *= fix;
#pragma unroll
      for (int w = 0; w < kJoinWaves - 1; ++w) {
        const float f = none ? 1.0f : __builtin_amdgcn_exp2f(met[w][16][lane] - next);
        sum += met[w][17][lane] * f;
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e >> 2][e & 3] += met[w][e][lane] * f;
      }
      top = next;
    }
    const int mm = mtile * kRowTile + qi;
    const int j = mm / a.num_heads, head = mm - j * a.num_heads;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    float z[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = y[e >> 2][e & 3] * inv;
    if (mm < s.mrows) {
      store_columns(reinterpret_cast<T*>(a.out + (size_t)(c0 + j) * a.out_ld) + head * L + block * 32,
                    z);
      if (a.lse && block == 0 && lane < 32)
        a.lse[(size_t)(c0 + j) * a.num_heads + head] =
            sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

constexpr int kCus = 256;  // of the card

struct Plan {
  int rows, wgs;  // of a segment, of the split kernel; at most
  size_t m_off, l_off, o_off, bytes;
};

Plan plan(int B, int gamma, int num_heads, int L) {
  Plan p;
  const int mtiles = (num_heads * (gamma + 1) + kRowTile - 1) / kRowTile;
  p.rows = kRowTile * std::min(row_tiles(L), mtiles);
  p.wgs = kCus;
  const size_t stat = align256((size_t)2 * p.wgs * p.rows * sizeof(float));
  p.m_off = align256((size_t)(B + 1) * sizeof(int64_t));
  p.l_off = p.m_off + stat;
  p.o_off = p.l_off + stat;
  p.bytes = p.o_off + align256((size_t)2 * p.wgs * p.rows * L * sizeof(float));
  return p;
}

template <int L>
void launch_join(const LatentAttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  const int tiles = (a.num_heads * (a.req.gamma + 1) + kRowTile - 1) / kRowTile;
  const int blocks = tiles * (L / 32);
  const bool shared = (int64_t)a.req.B * blocks <= 1024;
  const int waves = join_threads(shared) / kWave;
  const int most = shared ? blocks : (blocks + waves - 1) / waves;
  const int shares = std::max(1, std::min(most, 2048 / std::max(a.req.B, 1)));
  const dim3 grid((unsigned)a.req.B * shares), block(join_threads(shared));
  if (dt == DSPARK_BF16) {
    if (shared) {
      hipLaunchKernelGGL((join_kernel<__bf16, L, true>), grid, block, 0, s, a, ws, shares);
    } else {
      hipLaunchKernelGGL((join_kernel<__bf16, L, false>), grid, block, 0, s, a, ws, shares);
    }
  } else {
    if (shared) {
      hipLaunchKernelGGL((join_kernel<_Float16, L, true>), grid, block, 0, s, a, ws, shares);
    } else {
      hipLaunchKernelGGL((join_kernel<_Float16, L, false>), grid, block, 0, s, a, ws, shares);
    }
  }
}

}  // namespace
}  // namespace lattn

size_t latent_attention_workspace(int B, int gamma, int num_heads, int latent_dim) {
  return lattn::plan(B, gamma, num_heads, latent_dim).bytes;
}

hipError_t launch_latent_attention(const LatentAttnArgs& a, dspark_dtype dt, hipStream_t s) {
  int cus = 0;
  hipError_t e = current_cu_count(&cus);
  if (e != hipSuccess) return e;
  const int L = a.kv.dim;
  const lattn::Plan p = lattn::plan(a.req.B, a.req.gamma, a.num_heads, L);
  unsigned char* w = static_cast<unsigned char*>(a.ws);
  lattn::Parts ws;
  ws.base = reinterpret_cast<int64_t*>(w);
  ws.m = reinterpret_cast<float*>(w + p.m_off);
  ws.l = reinterpret_cast<float*>(w + p.l_off);
  ws.o = reinterpret_cast<float*>(w + p.o_off);
  ws.rows = p.rows;
  ws.wgs = std::min(lattn::kCus, cus);
  if (L == 256) {
    lattn::launch_dim256(a, ws, dt, s);
  } else {
    lattn::launch_dim512(a, ws, dt, s);
  }
  e = hipGetLastError();
  if (e != hipSuccess || a.req.B == 0) return e;
  if (L == 256) {
    lattn::launch_join<256>(a, ws, dt, s);
  } else {
    lattn::launch_join<512>(a, ws, dt, s);
  }
  return hipGetLastError();
}

}  // namespace dspark
