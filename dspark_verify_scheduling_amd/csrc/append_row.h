// One packed row of a cache append: norms, rotation and write of its heads.
#pragma once

#include "kv_dev.h"

#include <type_traits>

namespace dspark {

template <typename T>
struct Vec8;
template <>
struct Vec8<__bf16> { typedef bf16x8 type; };
template <>
struct Vec8<_Float16> { typedef f16x8 type; };

// x of lane ^ M, without a way through LDS where a row of sixteen lanes holds both.
template <int M>
__device__ __forceinline__ float lane_xor(float x) {
  const int v = __builtin_bit_cast(int, x);
  auto moved = [](int y, auto at) {
    return __builtin_amdgcn_update_dpp(y, y, decltype(at)::value, 0xF, 0xF, false);
  };
  int z;
  if constexpr (M == 1) {
    z = moved(v, std::integral_constant<int, 0xB1>{});  // pairs
  } else if constexpr (M == 2) {
    z = moved(v, std::integral_constant<int, 0x4E>{});  // halves of a quad
  } else if constexpr (M == 4) {
    // eight lanes back to front, then each quad
    z = moved(moved(v, std::integral_constant<int, 0x141>{}), std::integral_constant<int, 0x1B>{});
  } else if constexpr (M == 8) {
    z = moved(v, std::integral_constant<int, 0x128>{});  // sixteen lanes, turned by eight
  } else {
    return __shfl_xor(x, M, kWave);
  }
  return __builtin_bit_cast(float, z);
}
// The sum, or largest, of LANES neighbours.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  if constexpr (LANES == 1) {
    return x;
  } else {
    return lanes_sum<LANES / 2>(x + lane_xor<LANES / 2>(x));
  }
}
template <int LANES, int LEAST = 1>
__device__ __forceinline__ float lanes_max(float x) {
  if constexpr (LANES == LEAST) {
    return x;
  } else {
    return lanes_max<LANES / 2, LEAST>(fmaxf(x, lane_xor<LANES / 2>(x)));
  }
}

// A row of THREADS threads, a workgroup or a wave: LPH lanes per head take the heads
// of q, k and v in turn, AHEAD rounds of heads loaded ahead. y = x *
// (mean(x^2) + eps)^(-1/2) * w, then (a, b) -> (a c - b s, b c + a s), in float32;
// 8-bit rows scale by the power of two of their largest magnitude.
template <typename T, bool E8, int D, int THREADS, int AHEAD = 1>
struct RowAppend {
  typedef typename Vec8<T>::type T8;
  static constexpr int LPH = D / 8, HPP = THREADS / LPH;
  const AppendArgs& a;
  const size_t packed;
  const int tid, li;  // of the row; the lane's eight elements: 8 li ..
  const int hq, hkv, heads;
  const unsigned char* rows[3];
  T8 next[AHEAD], weight[2];

  // One of two values; a choice between elements of an array itself would put the
  // array into scratch memory, and each use behind a round trip to it.
  template <typename V>
  static __device__ __forceinline__ V pick(bool first, V x, V y) { return first ? x : y; }

  // of the n-th head of q, k and v in turn
  __device__ __forceinline__ T8 load(int h) const {
    const int hh = h < hq ? h : (h < hq + hkv ? h - hq : h - hq - hkv);
    T8 x = {};
    const unsigned char* row = pick(h < hq, rows[0], pick(h < hq + hkv, rows[1], rows[2]));
    if (h < heads) x = *reinterpret_cast<const T8*>(row + (size_t)(hh * D + 8 * li) * 2);
    return x;
  }

  __device__ __forceinline__ RowAppend(const AppendArgs& args, int packed_row)
      : a(args), packed((size_t)packed_row), tid(threadIdx.x % THREADS), li(threadIdx.x & (LPH - 1)),
        hq(args.num_heads), hkv(args.kv.hkv), heads(args.num_heads + 2 * args.kv.hkv),
        rows{args.q + (size_t)packed_row * args.q_ld, args.k + (size_t)packed_row * args.k_ld,
             args.v + (size_t)packed_row * args.v_ld} {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) next[i] = load(tid / LPH + i * HPP);
    weight[0] = weight[1] = T8{};
    if (a.q_weight) weight[0] = *(reinterpret_cast<const T8*>(a.q_weight) + li);
    if (a.k_weight) weight[1] = *(reinterpret_cast<const T8*>(a.k_weight) + li);
  }

  // The n-th head, which `next` holds; loads the one that takes its place.
  __device__ __forceinline__ void round(int h, T8& next, int id, int off, const float (&co)[8],
                                        const float (&si)[8], bool turned, int swap) {
    const bool live = h < heads;
    const int kind = h < hq ? 0 : (h < hq + hkv ? 1 : 2);
    const int hh = kind == 0 ? h : (kind == 1 ? h - hq : h - hq - hkv);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)next[e];
    next = load(h + AHEAD * HPP);
    if (a.q_weight || a.k_weight) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
      ss = lanes_sum<LPH>(ss);
      if (kind == 0 ? a.q_weight != nullptr : kind == 1 && a.k_weight) {
        const float rstd = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
        const T8 ww = pick(kind == 0, weight[0], weight[1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * (float)ww[e];
      }
    }
    if (a.rope) {
      float y[8];
      // the pair's other element: a neighbour, or the same place of another lane
      if (a.rope_interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
      } else if (a.rope_dim == D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = lane_xor<LPH / 2>(x[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __shfl(x[e], swap, kWave);
      }
      if (turned && kind < 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __builtin_fmaf(x[e], co[e], y[e] * si[e]);
      }
    }
    int e8 = 0;
    float inv = 1.0f;
    if (E8 && __any(live && kind != 0)) {
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));  // NaN apart
      if (__any(!finite_f32(amax))) {
        amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = finite_f32(x[e]) ? fmaxf(amax, fabsf(x[e])) : amax;
      }
      amax = lanes_max<LPH>(amax);
      e8 = e4m3_exponent(amax);
      inv = pow2f(-e8);
    }
    if (!live) return;
    if (kind == 0 || !E8) {
      T8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (T)x[e];
      unsigned char* dst;
      if (kind == 0) {
        dst = a.q_out + packed * a.q_out_ld + (size_t)(hh * D + 8 * li) * 2;
      } else {
        dst = (kind == 1 ? a.kv.k : a.kv.v) + (size_t)id * a.kv.page_bytes +
              ((((size_t)hh << a.kv.page_shift) + off) * D + 8 * li) * 2;
      }
      *reinterpret_cast<T8*>(dst) = o;
    } else {
      kv_u32x2 c;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        int wd = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_operand(x[4 * g], inv),
                                                 e4m3_operand(x[4 * g + 1], inv), 0, false);
        wd = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_operand(x[4 * g + 2], inv),
                                             e4m3_operand(x[4 * g + 3], inv), wd, true);
        c[g] = (unsigned)wd;
      }
      const size_t row = ((size_t)hh << a.kv.page_shift) + off;
      *reinterpret_cast<kv_u32x2*>((kind == 1 ? a.kv.k : a.kv.v) + (size_t)id * a.kv.page_bytes +
                                   row * D + 8 * li) = c;
      if (li == 0) {
        (kind == 1 ? a.kv.ks : a.kv.vs)[(size_t)id * a.kv.scale_page_bytes + row] =
            (uint8_t)(e8 + 127);
      }
    }
  }

  // Into token `off` of page `id`. co, si: the lane's cosines and sines, the same
  // for every head (si negated on a pair's first element); `turned`: whether its
  // elements turn; `swap`: the lane that holds their pairs' other elements.
  __device__ __forceinline__ void finish(int id, int off, const float (&co)[8],
                                         const float (&si)[8], bool turned, int swap) {
    for (int h0 = 0; h0 < heads; h0 += AHEAD * HPP) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (i > 0 && h0 + i * HPP >= heads) break;
        round(h0 + i * HPP + tid / LPH, next[i], id, off, co, si, turned, swap);
      }
    }
  }
};

}  // namespace dspark
