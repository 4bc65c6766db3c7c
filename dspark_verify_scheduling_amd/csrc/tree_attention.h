// Attention of packed verify rows (a chain or tree of drafts per request) over
// the paged cache: the split kernel's templates, one translation unit per head
// dimension, and the schedule it shares with the joining kernel.
#pragma once

#include "kv_dev.h"

namespace dspark {
namespace attn {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTileKeys = 32;                      // keys of a wave's step
constexpr int kUnitKeys = kWaves * kTileKeys;      // keys of a unit of work

// What the split kernel leaves for the joining kernel: the schedule's prefix
// sums, and per partial segment the running maximum and sum of each of its rows
// and their unnormalised outputs. Workgroup w has segments 2 w (the one its
// range starts with) and 2 w + 1 (a later one that its range ends in).
struct Parts {
  int64_t* base;  // [B + 1] first unit of each request, then the total
  float* m;       // [2 * wgs][rows]
  float* l;
  float* o;       // [2 * wgs][rows][D]
  int wgs;        // workgroups of the split kernel
  int rows;       // rows of a segment, at most
};

// Rows of a (request, key/value head): m = j * group + g for row j and the g-th
// of the head's queries, in tiles of 16, up to `mt_max` tiles to a segment.
struct Shape {
  int len, prefix, c0;
  int mrows, mtiles;
  int nseg, per;   // segments side by side, tiles of each
  int64_t keys;
  int nku;         // units along the keys
};

__device__ inline bool shape_of(const AttnArgs& a, int r, int total_eff, int mt_max, Shape* s) {
  if (!request_rows(a.req, r, total_eff, &s->c0, &s->len)) return false;
  s->prefix = a.req.prefix[r];
  s->keys = (int64_t)s->prefix + s->len;
  if (s->prefix < 0 || s->keys > ((int64_t)a.req.width << a.kv.page_shift) ||
      s->keys > 0x7FFFFF00LL)  // cache indices in 32 bits, a unit beyond included
    return false;
  s->mrows = a.group * s->len;
  s->mtiles = (s->mrows + 15) >> 4;
  s->nseg = (s->mtiles + mt_max - 1) / mt_max;
  s->per = (s->mtiles + s->nseg - 1) / s->nseg;
  s->nku = (int)((s->keys + kUnitKeys - 1) / kUnitKeys);
  return true;
}

__device__ inline int64_t units_of(const AttnArgs& a, int r, int total_eff, int mt_max) {
  Shape s;
  return shape_of(a, r, total_eff, mt_max, &s) ? (int64_t)a.kv.hkv * s.nseg * s.nku : 0;
}

// Workgroups that get units: never one without.
__device__ inline int wgs_in_use(int64_t total, int wgs) { return (int)min((int64_t)wgs, total); }

// The first unit of workgroup w of n <= total.
__device__ inline int64_t wg_start(int64_t total, int w, int n) { return total * w / n; }

template <typename T>
struct Types;
template <>
struct Types<__bf16> {
  typedef bf16x8 V8;
  typedef bf16x4 V4;
  static constexpr unsigned kExpMask = 0x7F80u;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Types<_Float16> {
  typedef f16x8 V8;
  typedef f16x4 V4;
  static constexpr unsigned kExpMask = 0x7C00u;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// Four rows of sixteen 16-bit elements, transposed: with the 16 lanes of a
// group pointing at the rows' quarters in order, lane i gets column i.
template <typename V4>
__device__ inline V4 lds_columns(const void* p) {
  typedef __attribute__((ext_vector_type(4))) short s16x4;
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(V4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

__device__ inline float group_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, kWave));
  return fmaxf(x, __shfl_xor(x, 32, kWave));
}

__device__ inline float group_sum(float x) {
  x += __shfl_xor(x, 16, kWave);
  return x + __shfl_xor(x, 32, kWave);
}

// Row stride of the value tile in LDS: 32 bytes past the head's, so that the
// four rows of a transposed read lie in different banks.
template <int D>
constexpr int v_stride() {
  return 2 * D + 32;
}

// Row stride (floats) of a 16-row output tile in LDS.
template <int D>
constexpr int o_stride() {
  return D + 4;
}

template <int D>
constexpr int wave_lds() {
  return kTileKeys * v_stride<D>() > 16 * o_stride<D>() * 4 ? kTileKeys * v_stride<D>()
                                                            : 16 * o_stride<D>() * 4;
}

// LDS of a workgroup: the waves' regions, then the queries of its row tiles.
template <int D, int MT>
constexpr int wg_lds() {
  return kWaves * wave_lds<D>() + MT * 16 * D * 2;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's maximum follows its scores only when they pass it by this much (in
// log2): weights then stay below 2^kSlack, and most steps rescale nothing.
constexpr float kSlack = 8.0f;

// One segment: the queries of `MT` 16-row tiles of one (request, key/value
// head) over units [ku0, ku0 + n) of its keys. Each wave takes 32 keys of a
// unit and keeps the statistics and outputs of all the segment's rows:
//   S^T = K Q^T: keys are the rows of the product and queries its columns, so a
//   lane holds 4 + 4 scores of one query (lane & 15), which are in place as the
//   operand of  O^T = V^T P^T.  Keys go straight from memory into operands;
//   values pass through the wave's LDS, where they are read by columns.
template <typename T, bool E8, int D, int MT>
__device__ __forceinline__ void segment(const AttnArgs& a, const Parts& ws, const Shape& s, int r,
                                        int h, int tile0, int64_t ku0, int n, bool whole,
                                        int slot, unsigned char* lds, float (*stat)[2][80]) {
  typedef Types<T> TT;
  typedef typename TT::V8 V8;
  typedef typename TT::V4 V4;
  constexpr int CB = E8 ? 1 : 2;
  constexpr int NF = D / 32;            // operand chunks of a key
  constexpr int ND = D / 16;            // 16-column tiles of the output
  constexpr int NK = E8 ? NF / 2 : NF;  // 16-byte loads of a key's share of a lane
  constexpr int LPR = D * CB / 16;      // lanes of a value row
  constexpr int RPI = kWave / LPR;      // value rows of a load
  constexpr int NV = kTileKeys / RPI;   // loads of a value tile
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int qi = lane & 15, g = lane >> 4;
  const int ps = a.kv.page_shift, pm = (1 << ps) - 1;
  const int len = s.len, prefix = s.prefix;
  const int keys = (int)s.keys;
  unsigned char* vt = lds + wave * wave_lds<D>();

  // the step's own tree: bit l of anc, in lane l, is row l + 1 itself, with its
  // ancestors' bits; row 0 is everybody's
  unsigned long long anc = 0;
  if (a.req.parents) {
    int up = lane + 1 < len ? a.req.parents[(size_t)r * a.req.gamma + lane] : 0;
    if (__ballot(up < 0 || up > lane)) return;  // uniform over the workgroup
    anc = 1ull << lane;
    for (int i = 0; i < 6; ++i) {
      const int from = max(up - 1, 0);
      const unsigned long long more = __shfl(anc, from, kWave);
      const int next = __shfl(up, from, kWave);
      if (up > 0) {
        anc |= more;
        up = next;
      }
    }
  }

  // Scores in units of log2 with a positive factor, so that a masked score stays
  // -infinity under it: the scale's sign and its zero go into the queries.
  float sl = fminf(fabsf(a.scale) * kLog2e, 3.4028235e38f);
  const unsigned sign = a.scale < 0.0f ? 0x80008000u : 0u;
  const bool flat = sl == 0.0f;
  if (flat) sl = 1.0f;
  // the queries in LDS, in operand order: chunk f of tile t is one 16-byte read
  // per lane. A lane's place in a key: of two 8-bit chunks in one load.
  const SmallDiv by_group(a.group);
  V8* qs = reinterpret_cast<V8*>(lds + kWaves * wave_lds<D>());
  for (int c = tid; c < MT * NF * kWave; c += kThreads) {
    const int t = c / (NF * kWave), f = (c / kWave) % NF;
    const int m = (tile0 + t) * 16 + qi;
    const int j = by_group.quo(m);
    const int d = E8 ? (f >> 1) * 64 + g * 16 + (f & 1) * 8 : f * 32 + g * 8;
    V8 x = (V8){0, 0, 0, 0, 0, 0, 0, 0};
    if (m < s.mrows && !flat) {
      kv_u32x4 w = *reinterpret_cast<const kv_u32x4*>(
          a.q + (size_t)(s.c0 + j) * a.q_ld +
          ((size_t)(h * a.group + (m - j * a.group)) * D + d) * 2);
      w ^= sign;
      x = __builtin_bit_cast(V8, w);
    }
    qs[c] = x;
  }
  __syncthreads();

  f32x4 o[MT][ND];
  float mx[MT], l[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    mx[t] = -__builtin_inff();
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[t][d] = (f32x4){0, 0, 0, 0};
  }

  const int32_t* table = a.req.table + (size_t)r * a.req.width;
  const int last_page = (keys - 1) >> ps;
  int ids = 0;       // page ids of the next 32 steps, two 16-key halves each
  int id_first = 0;  // the step of lane 0
  auto fetch_ids = [&](int i) {
    id_first = i;
    const int64_t key = (ku0 + i + (lane >> 1)) * kUnitKeys + wave * kTileKeys + (lane & 1) * 16;
    const int p = (int)min(key >> ps, (int64_t)last_page);
    const int id = table[p];
    ids = id >= 0 && id < a.kv.num_blocks ? id : -1;
  };

  kv_u32x4 kr[2][NK], vr[NV];
  unsigned ksb[2] = {0, 0}, vsb[NV];
  int id0 = 0, id1 = 0;  // pages of the halves in flight
  auto issue = [&](int i) {
    if (i - id_first >= 32) fetch_ids(i);
    id0 = __builtin_amdgcn_readlane(ids, 2 * (i - id_first));
    id1 = __builtin_amdgcn_readlane(ids, 2 * (i - id_first) + 1);
    const int key0 = (int)((ku0 + i) * kUnitKeys) + wave * kTileKeys;
    const unsigned char *kp[2], *vp[2];
    size_t sp[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // a page that is none: any valid address, its keys are masked
      const int64_t id = max(b ? id1 : id0, 0);
      const int64_t row = ((int64_t)h << ps) + ((key0 + 16 * b) & pm);
      kp[b] = a.kv.k + id * a.kv.page_bytes + row * (D * CB);
      vp[b] = a.kv.v + id * a.kv.page_bytes + row * (D * CB);
      if (E8) sp[b] = (size_t)(id * a.kv.scale_page_bytes + row);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int f = 0; f < NK; ++f)
        kr[b][f] = *reinterpret_cast<const kv_u32x4*>(kp[b] + qi * (D * CB) + f * 64 + g * 16);
      if (E8) ksb[b] = a.kv.ks[sp[b] + qi];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int b = (v * RPI) >> 4;
      vr[v] = *reinterpret_cast<const kv_u32x4*>(vp[b] + ((v * RPI) & 15) * (D * CB) + lane * 16);
      if (E8) vsb[v] = a.kv.vs[sp[b] + ((v * RPI) & 15) + lane / LPR];
    }
  };

  // steps of this wave: those whose first key exists
  const int64_t first = ku0 * kUnitKeys + wave * kTileKeys;
  const int steps =
      first >= keys ? 0 : (int)min((int64_t)n, (keys - first + kUnitKeys - 1) / kUnitKeys);
  if (steps > 0) {
    fetch_ids(0);
    issue(0);
  }
  // eight 8-bit elements, widened
  auto widen = [](unsigned lo, unsigned hi, float e) {
    kv_u32x4 w;
    w[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, e, false));
    w[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, e, true));
    w[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, e, false));
    w[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, e, true));
    return w;
  };
  // rows of the step's own tree that a query sees, bit l for row l + 1
  auto seen_by = [&](int t) {
    const int j = by_group.quo((tile0 + t) * 16 + qi);
    if (!a.req.parents) return j >= 64 ? ~0ull : (1ull << j) - 1;
    const unsigned long long path = __shfl(anc, max(j - 1, 0) & 63, kWave);
    return j > 0 ? path : 0ull;
  };

  for (int i = 0; i < steps; ++i) {
    const int key0 = (int)first + i * kUnitKeys;
    const int page0 = id0, page1 = id1;
    // the step holds keys that some query does not see (the request's own rows
    // after its root, keys past its last), or lies on a page that is none
    const bool edge = key0 + kTileKeys > prefix + 1 || page0 < 0 || page1 < 0;
    // scores
    f32x4 sc[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) sc[t][0] = sc[t][1] = (f32x4){0, 0, 0, 0};
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      V8 kf[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if constexpr (E8) {
          kf[b] = __builtin_bit_cast(
              V8, widen(kr[b][f >> 1][(f & 1) * 2], kr[b][f >> 1][(f & 1) * 2 + 1],
                        __builtin_bit_cast(float, ksb[b] << 23)));
        } else {
          kf[b] = __builtin_bit_cast(V8, kr[b][f]);
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const V8 x = qs[(t * NF + f) * kWave + lane];
        sc[t][0] = TT::mfma(kf[0], x, sc[t][0]);
        sc[t][1] = TT::mfma(kf[1], x, sc[t][1]);
      }
    }
    unsigned long long odd = 0;  // rows of the step that hold NaN or infinity
    if (edge) {
      // values of keys that do not exist are anything: zeros in their place.
      // NaN and infinity in a row that some query does not see must not meet
      // its zero weight: such elements are left out here and added below.
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int row = v * RPI + lane / LPR;
        const bool there = key0 + row < keys && (row >> 4 ? page1 : page0) >= 0;
        unsigned strange = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          unsigned w = vr[v][x], out = 0;
#pragma unroll
          for (int y = 0; y < 4 / CB; y += 1) {
            constexpr unsigned E = E8 ? 0x7Fu : TT::kExpMask, all = E8 ? 0xFFu : 0xFFFFu;
            const int at = y * 8 * CB;
            if (((w >> at) & E) == E) out |= all << at;
          }
          strange |= out;
          vr[v][x] = there ? w & ~out : 0;
        }
        unsigned long long found = __ballot(strange && there);
        while (found) {
          odd |= 1ull << (v * RPI + (int)__builtin_ctzll(found) / LPR);
          found &= found - 1;
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const unsigned long long seen = seen_by(t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int rel = key0 + (e >> 2) * 16 + g * 4 + (e & 3) - prefix;
          const bool own = rel < len && ((seen >> ((rel - 1) & 63)) & 1);
          if (((e >> 2) ? page1 : page0) < 0 || (rel > 0 && !own))
            sc[t][e >> 2][e & 3] = -__builtin_inff();
        }
      }
    }
    // values into LDS
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      unsigned char* dst = vt + (v * RPI + lane / LPR) * v_stride<D>() + (lane % LPR) * (32 / CB);
#pragma unroll
      for (int c = 0; c < 3 - CB; ++c) {
        kv_u32x4 w = vr[v];
        if constexpr (E8)
          w = widen(vr[v][2 * c], vr[v][2 * c + 1], __builtin_bit_cast(float, vsb[v] << 23));
        *reinterpret_cast<kv_u32x4*>(dst + 16 * c) = w;
      }
    }
    // the step's loads are used up: the next one's start (the last step's again,
    // unused, after it)
    issue(min(i + 1, steps - 1));

    // weights
    V8 pf[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float top = sc[t][0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, sc[t][e >> 2][e & 3]);
      if (__any(top * sl > mx[t] + kSlack)) {
        const float next = fmaxf(mx[t], group_max(top * sl));
        const float fix =
            next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx[t] - next);
        mx[t] = next;
        l[t] *= fix;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[t][d] *= fix;
      }
      const float ref = mx[t] == -__builtin_inff() ? 0.0f : mx[t];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][e >> 2][e & 3], sl, -ref));
        l[t] += p;
        pf[t][e] = (T)p;
      }
    }
    // O^T += V^T P^T
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const unsigned char* at =
          vt + (g * 4 + (qi >> 2)) * v_stride<D>() + d * 32 + (qi & 3) * 8;
      const V4 lo = lds_columns<V4>(at);
      const V4 hi = lds_columns<V4>(at + 16 * v_stride<D>());
      const V8 vf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int t = 0; t < MT; ++t) o[t][d] = TT::mfma(vf, pf[t], o[t][d]);
    }
    while (odd) {
      // a row with NaN or infinity: they go to the queries that see it
      const int row = (int)__builtin_ctzll(odd);
      odd &= odd - 1;
      const int64_t id = row >> 4 ? page1 : page0;
      const int rel = key0 + row - prefix;
      const int64_t at = ((int64_t)h << ps) + ((key0 + row) & pm);
      const unsigned char* src = a.kv.v + id * a.kv.page_bytes + at * (D * CB);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = d * 16 + g * 4 + e;
          float v;
          if (E8) {
            v = (src[col] & 127) == 127 ? __builtin_nanf("") : 0.0f;
          } else {
            v = (float)reinterpret_cast<const T*>(src)[col];
            v = finite_f32(v) ? 0.0f : v;
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const bool vis = rel <= 0 || ((seen_by(t) >> ((rel - 1) & 63)) & 1);
            if (vis) o[t][d][e] += v;
          }
          asm volatile("" ::: "memory");  // one element at a time: no registers for a rare path
        }
      }
    }
  }

  // the waves' parts, through LDS: statistics first, then a 16-row tile at a time
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    l[t] = group_sum(l[t]);
    if (g == 0) {
      stat[wave][0][t * 16 + qi] = mx[t];
      stat[wave][1][t * 16 + qi] = l[t];
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    float top = stat[0][0][t * 16 + qi];
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, stat[w][0][t * 16 + qi]);
    const float fix = top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx[t] - top);
    float* mine = reinterpret_cast<float*>(vt) + qi * o_stride<D>() + g * 4;
#pragma unroll
    for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(mine + d * 16) = o[t][d] * fix;
    __syncthreads();
    for (int c = tid; c < 16 * (D / 8); c += kThreads) {
      const int row = c / (D / 8), col = (c % (D / 8)) * 8;
      const int m = (tile0 + t) * 16 + row;
      if (m >= s.mrows) continue;
      f32x4 y[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
      float rtop = stat[0][0][t * 16 + row], rsum = 0.0f;
      for (int w = 1; w < kWaves; ++w) rtop = fmaxf(rtop, stat[w][0][t * 16 + row]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float* from =
            reinterpret_cast<const float*>(lds + w * wave_lds<D>()) + row * o_stride<D>() + col;
        y[0] += *reinterpret_cast<const f32x4*>(from);
        y[1] += *reinterpret_cast<const f32x4*>(from + 4);
        rsum += rtop == -__builtin_inff()
                    ? stat[w][1][t * 16 + row]
                    : stat[w][1][t * 16 + row] *
                          __builtin_amdgcn_exp2f(stat[w][0][t * 16 + row] - rtop);
      }
      if (whole) {
        const int j = by_group.quo(m);
        const int head = h * a.group + (m - j * a.group);
        const float inv = rsum == 0.0f ? 0.0f : 1.0f / rsum;
        V8 z;
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = (T)(y[e >> 2][e & 3] * inv);
        *reinterpret_cast<V8*>(a.out + (size_t)(s.c0 + j) * a.out_ld + (size_t)(head * D + col) * 2) =
            z;
        if (a.lse && col == 0)
          a.lse[(size_t)(s.c0 + j) * a.num_heads + head] =
              rsum == 0.0f ? -__builtin_inff() : (rtop + __builtin_amdgcn_logf(rsum)) * kLn2;
      } else {
        const size_t at = (size_t)slot * ws.rows + t * 16 + row;
        f32x4* to = reinterpret_cast<f32x4*>(ws.o + at * D + col);
        to[0] = y[0];
        to[1] = y[1];
        if (col == 0) {
          ws.m[at] = rtop;
          ws.l[at] = rsum;
        }
      }
    }
    __syncthreads();
  }
}

// Persistent over the units of all (request, key/value head, row segment)s in
// order: workgroup w takes the w-th equal share, so ragged contexts balance by
// themselves and a long one is split over many workgroups.
template <typename T, bool E8, int D, int MTMAX>
__global__ __launch_bounds__(kThreads, MTMAX > 3 || D == 256 ? 1 : 2) void split_kernel(AttnArgs a, Parts ws) {
  __shared__ __align__(16) unsigned char lds[wg_lds<D, MTMAX>()];
  __shared__ float stat[kWaves][2][80];
  __shared__ int64_t wsum[kWaves];
  __shared__ int start_r;
  __shared__ int64_t start_off;
  const ReqView& q = a.req;
  const int tid = threadIdx.x;
  int rows_total;
  const int total_eff = rows_in_use(q, &rows_total);
  // every workgroup sums the requests' units by itself
  const int per = (q.B + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, q.B), r1 = min(r0 + per, q.B);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += units_of(a, r, total_eff, MTMAX);
  int64_t total;
  int64_t at = block_excl_scan<int64_t, kThreads>(mine, wsum, &total);
  const int wgs = wgs_in_use(total, gridDim.x);
  if (blockIdx.x == 0) {
    int64_t b = at;
    for (int r = r0; r < r1; ++r) {
      ws.base[r] = b;
      b += units_of(a, r, total_eff, MTMAX);
    }
    if (tid == 0) {
      ws.base[q.B] = total;
      a.meta[0] = rows_total;
      a.meta[1] = rows_total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    }
  }
  if ((int)blockIdx.x >= wgs) return;
  const int64_t u0 = wg_start(total, blockIdx.x, wgs), u1 = wg_start(total, blockIdx.x + 1, wgs);
  if (at <= u0 && u0 < at + mine) {
    for (int r = r0; r < r1; ++r) {
      const int64_t n = units_of(a, r, total_eff, MTMAX);
      if (u0 < at + n) {
        start_r = r;
        start_off = u0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int r = __builtin_amdgcn_readfirstlane(start_r);
  int64_t off = start_off;
  int64_t u = u0;
  while (u < u1) {
    Shape s;
    const int64_t n_r =
        shape_of(a, r, total_eff, MTMAX, &s) ? (int64_t)a.kv.hkv * s.nseg * s.nku : 0;
    if (off >= n_r) {
      ++r;
      off = 0;
      continue;
    }
    const int item = (int)(off / s.nku);
    const int64_t ku0 = off - (int64_t)item * s.nku;
    const int n = (int)min(s.nku - ku0, u1 - u);
    const int h = item / s.nseg, seg = item - h * s.nseg;
    const bool whole = n == s.nku;
    const int slot = 2 * blockIdx.x + (u == u0 ? 0 : 1);
    const int tile0 = seg * s.per, mt = min(s.per, s.mtiles - tile0);
#define DSPARK_SEGMENT(MT)                                                                     \
  case MT:                                                                                     \
    if constexpr (MT <= MTMAX)                                                                 \
      segment<T, E8, D, MT>(a, ws, s, r, h, tile0, ku0, n, whole, slot, lds, stat);            \
    break;
    switch (mt) {
      DSPARK_SEGMENT(1)
      DSPARK_SEGMENT(2)
      DSPARK_SEGMENT(3)
      DSPARK_SEGMENT(4)
      DSPARK_SEGMENT(5)
    }
#undef DSPARK_SEGMENT
    off += n;
    u += n;
  }
}

// 16-row tiles of a segment, at most, for requests of up to `mtiles` of them.
template <int D>
constexpr int most_tiles() {
  return D == 256 ? 3 : 5;
}
inline int segment_tiles(int D, int mtiles) {
  const int most = D == 256 ? 3 : 5;
  return mtiles <= 1 ? 1 : (mtiles <= 3 ? 3 : most);
}

template <typename T, bool E8, int D>
void launch_split(const AttnArgs& a, const Parts& ws, int mt_max, hipStream_t s) {
  const dim3 grid((unsigned)ws.wgs), block(kThreads);
  if (mt_max == 1) {
    hipLaunchKernelGGL((split_kernel<T, E8, D, 1>), grid, block, 0, s, a, ws);
  } else if (mt_max == 3) {
    hipLaunchKernelGGL((split_kernel<T, E8, D, 3>), grid, block, 0, s, a, ws);
  } else {
    hipLaunchKernelGGL((split_kernel<T, E8, D, most_tiles<D>()>), grid, block, 0, s, a, ws);
  }
}

template <int D>
void launch_dim(const AttnArgs& a, const Parts& ws, dspark_dtype dt, int mt_max, hipStream_t s) {
  if (a.kv.cb == 1) {
    launch_split<__bf16, true, D>(a, ws, mt_max, s);
  } else if (dt == DSPARK_BF16) {
    launch_split<__bf16, false, D>(a, ws, mt_max, s);
  } else {
    launch_split<_Float16, false, D>(a, ws, mt_max, s);
  }
}

void launch_dim64(const AttnArgs& a, const Parts& ws, dspark_dtype dt, int mt_max, hipStream_t s);
void launch_dim128(const AttnArgs& a, const Parts& ws, dspark_dtype dt, int mt_max, hipStream_t s);
void launch_dim256(const AttnArgs& a, const Parts& ws, dspark_dtype dt, int mt_max, hipStream_t s);

}  // namespace attn
}  // namespace dspark
