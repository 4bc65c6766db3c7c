// Attention of packed verify rows over the paged cache: launch, workspace and
// the joining kernel. The split kernel is in tree_attention.h.
#include "tree_attention.h"

#include <algorithm>

namespace dspark {

namespace attn {
namespace {

// One workgroup per (request, key/value head, share of its rows): joins the
// parts that several workgroups of the split kernel left of a segment, in order,
// a wave per row. The first of each request also checks it and its pages.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnArgs a, Parts ws, int shares) {
  constexpr int E = D / kWave;
  typedef __attribute__((ext_vector_type(E))) float fE;
  typedef __attribute__((ext_vector_type(E))) T TE;
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int share = blockIdx.x % shares, rh = blockIdx.x / shares;
  const int r = rh / a.kv.hkv, h = rh - r * a.kv.hkv;
  int total;
  const int total_eff = rows_in_use(q, &total);
  Shape s;
  const bool good = shape_of<D>(a, r, total_eff, &s);
  const bool tree =
      !good || !q.parents ||
      !__ballot([&] {
        const int up = lane + 1 < s.len ? q.parents[(size_t)r * q.gamma + lane] : 0;
        return up < 0 || up > lane;
      }());
  if (h == 0 && share == 0) {
    int bits = 0;
    if (!good) {
      bits = request_status(q, r, total_eff);
      if (!bits) bits = DSPARK_DATA_BAD_PAGE;
    } else if (!tree) {
      bits = DSPARK_DATA_BAD_TREE;
    } else {
      for (int64_t p = tid; p <= (s.keys - 1) >> a.kv.page_shift; p += kThreads) {
        const int id = q.table[(size_t)r * q.width + p];
        if (id < 0 || id >= a.kv.num_blocks) bits = DSPARK_DATA_BAD_PAGE;
      }
    }
    if (__any(bits != 0)) {
      if (bits) atomicOr(a.meta + 1, bits);
    }
  }
  if (!good || !tree) return;
  const int64_t units = ws.base[q.B], base = ws.base[r];
  const int wgs = wgs_in_use(units, ws.wgs);
  const SmallDiv by_group(a.group);
  // rows in order over the segments, a wave each
  for (int m = share * kWaves + wave; m < s.mrows; m += shares * kWaves) {
    const int seg = (m >> 4) / s.per;
    const int64_t u0 = base + ((int64_t)h * s.nseg + seg) * s.nku, u1 = u0 + s.nku;
    // workgroups of the first and the last unit
    const int wa = (int)(((u0 + 1) * wgs - 1) / units), wb = (int)((u1 * wgs - 1) / units);
    if (wa == wb) continue;
    const int slot0 = 2 * wa + (wg_start(units, wa, wgs) == u0 ? 0 : 1);
    const int n = wb - wa + 1;
    const int row = m - seg * s.per * 16;
    auto place = [&](int p) { return (size_t)(p ? 2 * (wa + p) : slot0) * ws.rows + row; };
    // the first eight parts are under way while their statistics are looked at
    constexpr int kAhead = 8;
    fE x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      x[k] = *reinterpret_cast<const fE*>(ws.o + place(min(k, n - 1)) * D + lane * E);
    float top = -__builtin_inff();
    for (int p = lane; p < n; p += kWave) top = fmaxf(top, ws.m[place(p)]);
    for (int o = kWave / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
    float sum = 0.0f;
    fE y;
    for (int e = 0; e < E; ++e) y[e] = 0.0f;
    for (int p0 = 0; p0 < n; p0 += kWave) {
      // lane i: the factor of part p0 + i; then the parts in order
      const int p = p0 + lane;
      float f = 0.0f;
      if (p < n) {
        f = top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(ws.m[place(p)] - top);
        sum += ws.l[place(p)] * f;
      }
      const int cnt = min(n - p0, kWave);
      for (int i = 0; i < cnt; i += kAhead) {
        fE z[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          z[k] = x[k];
          if (p0 + i + kAhead < n)
            x[k] = *reinterpret_cast<const fE*>(
                ws.o + place(min(p0 + i + kAhead + k, n - 1)) * D + lane * E);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (i + k < cnt) {
            const float fk = read_lane(f, i + k);
            for (int e = 0; e < E; ++e) y[e] += z[k][e] * fk;
          }
        }
      }
    }
    sum = wave_sum(sum);
    const int j = by_group.quo(m);
    const int head = h * a.group + (m - j * a.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    TE z;
    for (int e = 0; e < E; ++e) z[e] = (T)(y[e] * inv);
    *reinterpret_cast<TE*>(reinterpret_cast<T*>(a.out + (size_t)(s.c0 + j) * a.out_ld) + head * D +
                           lane * E) = z;
    if (a.lse && lane == 0)
      a.lse[(size_t)(s.c0 + j) * a.num_heads + head] =
          sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workgroups of the split kernel, at most: two to a CU (their LDS rings).
constexpr int kMaxWgs = 512;

struct Plan {
  int rows;
  size_t m_off, l_off, o_off, bytes;
};

Plan plan(int B, int gamma, int group, int D) {
  Plan p;
  const int mtiles = (group * (gamma + 1) + 15) / 16;
  p.rows = 16 * std::min(D == 256 ? Size<256>::kTiles : Size<128>::kTiles, mtiles);
  const size_t stat = align256((size_t)2 * kMaxWgs * p.rows * sizeof(float));
  p.m_off = align256((size_t)(B + 1) * sizeof(int64_t));
  p.l_off = p.m_off + stat;
  p.o_off = p.l_off + stat;
  p.bytes = p.o_off + align256((size_t)2 * kMaxWgs * p.rows * D * sizeof(float));
  return p;
}

template <int D>
void launch_join(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  // enough waves to fill the card, and no more than there are rows
  const int pairs = a.req.B * a.kv.hkv;
  const int most = (a.group * (a.req.gamma + 1) + kWaves - 1) / kWaves;
  const int shares = std::max(1, std::min(most, 4096 / std::max(pairs, 1)));
  const dim3 grid((unsigned)pairs * shares), block(kThreads);
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

hipError_t launch_attention(const AttnArgs& a, dspark_dtype dt, hipStream_t s) {
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
  ws.wgs = std::min(attn::kMaxWgs, 2 * cus);
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
