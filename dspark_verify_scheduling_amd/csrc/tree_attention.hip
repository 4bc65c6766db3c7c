// Attention of packed verify rows (a chain or tree of drafts per request) over
// the paged cache.
#include "kv_dev.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

__device__ inline float load_elem(const unsigned char* p, size_t i, int kind, float sc) {
  if (kind == 2) {
    const bf16x2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)p[i], sc, false);
    return (float)w[0];
  }
  if (kind == 1) return (float)reinterpret_cast<const _Float16*>(p)[i];
  return (float)reinterpret_cast<const __bf16*>(p)[i];
}

// One workgroup per (request, row, query head); its waves take every fourth
// key, a lane head_dim / 64 elements, with a running maximum and sum each.
template <typename T, int KIND, int D>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttnArgs a) {
  constexpr int E = D / kWave;
  const ReqView& q = a.req;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int total;
  const int total_eff = rows_in_use(q, &total);
  if (blockIdx.x == 0) {
    __shared__ int all;
    if (tid == 0) all = total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    __syncthreads();
    for (int r = wave; r < q.B; r += kWaves) {
      int bits = request_status(q, r, total_eff);
      if (!bits) {
        const int64_t hi = (int64_t)q.prefix[r] + (q.cu[r + 1] - q.cu[r]);
        if (hi > ((int64_t)q.width << a.kv.page_shift)) {
          bits = DSPARK_DATA_BAD_PAGE;
        } else {
          for (int64_t p = lane; p <= (hi - 1) >> a.kv.page_shift; p += kWave) {
            const int id = q.table[(size_t)r * q.width + p];
            if (id < 0 || id >= a.kv.num_blocks) bits = DSPARK_DATA_BAD_PAGE;
          }
        }
      }
      if (bits) atomicOr(&all, bits);
    }
    __syncthreads();
    if (tid == 0) {
      a.meta[0] = total;
      a.meta[1] = all;
    }
    return;
  }
  const int u = blockIdx.x - 1;
  const int h = u % a.num_heads;
  const int rj = u / a.num_heads;
  const int r = rj / (q.gamma + 1), j = rj - r * (q.gamma + 1);
  int c0, len;
  if (!request_rows(q, r, total_eff, &c0, &len) || j >= len) return;
  const int prefix = q.prefix[r];
  if (prefix < 0 || (int64_t)prefix + len > ((int64_t)q.width << a.kv.page_shift)) return;
  // bit i - 1: row i is row j or one of its ancestors; row 0 always is
  unsigned long long seen = j >= 64 ? ~0ull : (1ull << j) - 1;
  if (q.parents) {
    const int par = lane + 1 < len ? q.parents[(size_t)r * q.gamma + lane] : 0;
    if (__ballot(par < 0 || par > lane)) return;
    seen = 0;
    for (int n = j; n > 0; n = __builtin_amdgcn_readlane(par, n - 1)) seen |= 1ull << (n - 1);
  }
  const int kh = h / a.group;
  float x[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = (float)reinterpret_cast<const T*>(a.q + (size_t)(c0 + j) * a.q_ld)[h * D + lane * E + e];
    o[e] = 0.0f;
  }
  float m = -__builtin_inff(), l = 0.0f;
  for (int k = wave; k < prefix + len; k += kWaves) {
    const int i = k - prefix;
    if (i > 0 && !((seen >> (i - 1)) & 1)) continue;
    const int id = q.table[(size_t)r * q.width + (k >> a.kv.page_shift)];
    if (id < 0 || id >= a.kv.num_blocks) continue;
    const size_t row = ((size_t)kh << a.kv.page_shift) + (k & ((1 << a.kv.page_shift) - 1));
    const size_t at = (size_t)id * a.kv.page_bytes;
    float ksc = 1.0f, vsc = 1.0f;
    if (KIND == 2) {
      ksc = pow2f((int)a.kv.ks[(size_t)id * a.kv.scale_page_bytes + row] - 127);
      vsc = pow2f((int)a.kv.vs[(size_t)id * a.kv.scale_page_bytes + row] - 127);
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      s = __builtin_fmaf(x[e], load_elem(a.kv.k + at, row * D + lane * E + e, KIND, ksc), s);
    s = wave_sum(s) * a.scale;
    const float mn = fmaxf(m, s);
    const float fix = m == mn ? 1.0f : expf(m - mn);
    const float p = s == -__builtin_inff() ? 0.0f : expf(s - mn);
    l = l * fix + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * fix + p * load_elem(a.kv.v + at, row * D + lane * E + e, KIND, vsc);
    m = mn;
  }
  __shared__ float ms[kWaves], ls[kWaves], os[kWaves][D];
  if (lane == 0) {
    ms[wave] = m;
    ls[wave] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) os[wave][lane * E + e] = o[e];
  __syncthreads();
  float mt = ms[0];
  for (int w = 1; w < kWaves; ++w) mt = fmaxf(mt, ms[w]);
  float lt = 0.0f;
  for (int w = 0; w < kWaves; ++w) lt += ms[w] == -__builtin_inff() ? 0.0f : ls[w] * expf(ms[w] - mt);
  for (int d = tid; d < D; d += kThreads) {
    float y = 0.0f;
    for (int w = 0; w < kWaves; ++w)
      y += ms[w] == -__builtin_inff() ? 0.0f : os[w][d] * expf(ms[w] - mt);
    reinterpret_cast<T*>(a.out + (size_t)(c0 + j) * a.out_ld)[h * D + d] =
        (T)(lt == 0.0f ? 0.0f : y / lt);
  }
  if (a.lse && tid == 0)
    a.lse[(size_t)(c0 + j) * a.num_heads + h] = lt == 0.0f ? -__builtin_inff() : mt + logf(lt);
}

template <typename T, int KIND>
void by_dim(const AttnArgs& a, unsigned grid, hipStream_t s) {
  switch (a.kv.dim) {
    case 64:
      hipLaunchKernelGGL((attention_kernel<T, KIND, 64>), dim3(grid), dim3(kThreads), 0, s, a);
      break;
    case 128:
      hipLaunchKernelGGL((attention_kernel<T, KIND, 128>), dim3(grid), dim3(kThreads), 0, s, a);
      break;
    default:
      hipLaunchKernelGGL((attention_kernel<T, KIND, 256>), dim3(grid), dim3(kThreads), 0, s, a);
  }
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, dspark_dtype dt, hipStream_t s) {
  const unsigned grid = 1u + (unsigned)((int64_t)a.req.B * (a.req.gamma + 1) * a.num_heads);
  if (a.kv.cb == 1) {
    by_dim<__bf16, 2>(a, grid, s);
  } else if (dt == DSPARK_BF16) {
    by_dim<__bf16, 0>(a, grid, s);
  } else {
    by_dim<_Float16, 1>(a, grid, s);
  }
  return hipGetLastError();
}

size_t attention_workspace(int, int, int, int, int) { return 256; }

}  // namespace dspark
