// Attention of packed verify rows over the paged cache: launch, workspace and
// the joining kernel. The split kernel is in tree_attention.h.
#include "tree_attention.h"

#include <algorithm>

namespace dspark {

namespace attn {
namespace {

constexpr int kJoinThreads = 256;

// One workgroup per (request, key/value head, share of its rows): joins the
// parts that several workgroups of the split kernel left of a segment, in order,
// D / 8 lanes to a row with eight elements each. A part's statistics and outputs
// are read together, so a row costs about one memory latency. The first
// workgroup of each request also checks it and its pages. Bound by latency (4 to
// 5 us for one token or for 32 chains) and, with many rows, by the parts' bytes:
// 12 us for 64 trees (about 40 MB; 15 us with four parts at once and 4096
// workgroups).
template <typename T, int D>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(AttnArgs a, Parts ws, int shares) {
  typedef typename Types<T>::V8 V8;
  constexpr int kLanes = D / 8, kRows = kJoinThreads / kLanes;
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int share = blockIdx.x % shares, rh = blockIdx.x / shares;
  const int r = rh / a.kv.hkv, h = rh - r * a.kv.hkv;
  const int64_t units = ws.base[q.B], base = ws.base[r];
  int total;
  const int total_eff = rows_in_use(q, &total);
  int c0, len, prefix;
  const bool good = rows_of(a, r, total_eff, &c0, &len, &prefix);
  bool tree = true;
  if (good && q.parents) {
    const int up = lane + 1 < len ? q.parents[(size_t)r * q.gamma + lane] : 0;
    tree = __ballot(up < 0 || up > lane) == 0;
  }
  if (h == 0 && share == 0) {
    int bits = 0;
    if (!good) {
      bits = request_status(q, r, total_eff);
      if (!bits) bits = DSPARK_DATA_BAD_PAGE;
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
  if (!good || !tree) return;
  const Shape s = shape_of<D>(a, c0, len, prefix);
  const int wgs = wgs_in_use(units, ws.wgs);
  const SmallDiv by_group(a.group);
  const int col = (tid % kLanes) * 8;
  // rows in order over the segments, kRows of one at a time
  const int steps = (s.per * 16 + kRows - 1) / kRows;
  for (int step = share; step < s.nseg * steps; step += shares) {
    const int seg = step / steps;
    const int64_t u0 = base + ((int64_t)h * s.nseg + seg) * s.nku, u1 = u0 + s.nku;
    // workgroups of the first and the last unit
    const int wa = (int)(((u0 + 1) * wgs - 1) / units), wb = (int)((u1 * wgs - 1) / units);
    if (wa == wb) continue;
    const int slot0 = 2 * wa + (wg_start(units, wa, wgs) == u0 ? 0 : 1);
    const int n = wb - wa + 1;
    const int rows = min(s.per * 16, s.mrows - seg * s.per * 16);
    const int row = (step - seg * steps) * kRows + tid / kLanes;
    if (row < rows) {
      constexpr int kAhead = 8;
      float top = -__builtin_inff(), sum = 0.0f;
      f32x4 y[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
      for (int p0 = 0; p0 < n; p0 += kAhead) {
        float m[kAhead], l[kAhead];
        f32x4 x[kAhead][2];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int p = p0 + k;
          m[k] = -__builtin_inff();
          l[k] = 0.0f;
          x[k][0] = x[k][1] = (f32x4){0, 0, 0, 0};
          if (p < n) {
            const size_t at = (size_t)(p ? 2 * (wa + p) : slot0) * ws.rows + row;
            m[k] = ws.m[at];
            l[k] = ws.l[at];
            x[k][0] = *reinterpret_cast<const f32x4*>(ws.o + at * D + col);
            x[k][1] = *reinterpret_cast<const f32x4*>(ws.o + at * D + col + 4);
          }
        }
        float next = top;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) next = fmaxf(next, m[k]);
        const bool none = next == -__builtin_inff();  // nothing seen, or NaN scores only
        const float fix = none ? 1.0f : __builtin_amdgcn_exp2f(top - next);
        sum *= fix;
        y[0] *= fix;
        y[1] *= fix;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float f = none ? 1.0f : __builtin_amdgcn_exp2f(m[k] - next);
          sum += l[k] * f;
          y[0] += x[k][0] * f;
          y[1] += x[k][1] * f;
        }
        top = next;
      }
      const int mm = seg * s.per * 16 + row;
      const int j = by_group.quo(mm);
      const int head = h * a.group + (mm - j * a.group);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      V8 z;
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = (T)(y[e >> 2][e & 3] * inv);
      *reinterpret_cast<V8*>(reinterpret_cast<T*>(a.out + (size_t)(c0 + j) * a.out_ld) + head * D +
                             col) = z;
      if (a.lse && col == 0)
        a.lse[(size_t)(c0 + j) * a.num_heads + head] =
            sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

constexpr int kCus = 256;  // of the card

struct Plan {
  int rows;
  int wgs;  // workgroups of the split kernel, at most: what its LDS rings leave room for
  size_t m_off, l_off, o_off, bytes;
};

Plan plan(int B, int gamma, int group, int D) {
  Plan p;
  const int mtiles = (group * (gamma + 1) + 15) / 16, waves = waves_for(group * (gamma + 1), D);
  p.rows = 16 * std::min(waves, mtiles);
  p.wgs = kCus * per_cu(D, true, waves);  // (8 bits: the most)
  const size_t stat = align256((size_t)2 * p.wgs * p.rows * sizeof(float));
  p.m_off = align256((size_t)(B + 1) * sizeof(int64_t));
  p.l_off = p.m_off + stat;
  p.o_off = p.l_off + stat;
  p.bytes = p.o_off + align256((size_t)2 * p.wgs * p.rows * D * sizeof(float));
  return p;
}

template <int D>
void launch_join(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  // a workgroup's rows at once, and more workgroups where there are few pairs
  const int pairs = a.req.B * a.kv.hkv;
  const int rows = a.group * (a.req.gamma + 1), at_once = kJoinThreads / (D / 8);
  const int most = (rows + at_once - 1) / at_once;
  const int shares = std::max(1, std::min(most, 1024 / std::max(pairs, 1)));
  const dim3 grid((unsigned)pairs * shares), block(kJoinThreads);
  if (dt == DSPARK_BF16) {
    hipLaunchKernelGGL((join_kernel<__bf16, D>), grid, block, 0, s, a, ws, shares);
  } else {
    hipLaunchKernelGGL((join_kernel<_Float16, D>), grid, block, 0, s, a, ws, shares);
  }
}

}  // namespace
}  // namespace attn

size_t attention_workspace(int B, int gamma, int num_heads, int num_kv_heads, int head_dim) {
  return attn::plan(B, gamma, num_heads / num_kv_heads, head_dim).bytes;
}

hipError_t launch_attention(const AttnArgs& args, dspark_dtype dt, hipStream_t s) {
  AttnArgs a = args;
  a.waves = attn::waves_for(a.group * (a.req.gamma + 1), a.kv.dim);
  int cus = 0;
  hipError_t e = current_cu_count(&cus);
  if (e != hipSuccess) return e;
  const attn::Plan p = attn::plan(a.req.B, a.req.gamma, a.group, a.kv.dim);
  unsigned char* w = static_cast<unsigned char*>(a.ws);
  attn::Parts ws;
  ws.base = reinterpret_cast<int64_t*>(w);
  ws.m = reinterpret_cast<float*>(w + p.m_off);
  ws.l = reinterpret_cast<float*>(w + p.l_off);
  ws.o = reinterpret_cast<float*>(w + p.o_off);
  ws.rows = p.rows;
  ws.wgs = std::min(attn::kCus, cus) * attn::per_cu(a.kv.dim, a.kv.cb == 1, a.waves);
  switch (a.kv.dim) {
    case 64: attn::launch_dim64(a, ws, dt, s); break;
    case 128: attn::launch_dim128(a, ws, dt, s); break;
    default: attn::launch_dim256(a, ws, dt, s);
  }
  e = hipGetLastError();
  if (e != hipSuccess || a.req.B == 0) return e;
  switch (a.kv.dim) {
    case 64: attn::launch_join<64>(a, ws, dt, s); break;
    case 128: attn::launch_join<128>(a, ws, dt, s); break;
    default: attn::launch_join<256>(a, ws, dt, s);
  }
  return hipGetLastError();
}

}  // namespace dspark
