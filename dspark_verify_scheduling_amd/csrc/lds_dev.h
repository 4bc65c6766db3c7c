// Shared by the attention kernels: the element types with their matrix products
// and softmax ranges, reads and writes of LDS by address, and copies of memory
// straight into LDS.
#pragma once

#include "kv_dev.h"

namespace dspark {
namespace attn {

typedef __attribute__((ext_vector_type(16))) float f32x16;

// The weights of a row are 2^(score - m), m its running maximum (in log2) less
// kAbove. m follows the scores only when they pass it by kAbove + kSlack, so most
// steps rescale nothing, and the weights stay below 2^(kAbove + kSlack).
// bfloat16 has float32's exponents and needs no kAbove. float16 holds 2^15 to
// 2^-24: with kAbove a weight counts down to 2^-36 of the largest, 25 below it in
// e; with the largest at 1 it would end at 2^-25, and the tail of a long context
// under one large weight with it.
template <typename T>
struct Types;
template <>
struct Types<__bf16> {
  static constexpr float kSlack = 8.0f, kAbove = 0.0f;
  typedef bf16x8 V8;
  typedef bf16x4 V4;
  static constexpr unsigned kExpMask = 0x7F80u;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ f32x16 mfma32(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Types<_Float16> {
  static constexpr float kSlack = 4.0f, kAbove = 11.0f;
  typedef f16x8 V8;
  typedef f16x4 V4;
  static constexpr unsigned kExpMask = 0x7C00u;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ f32x16 mfma32(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

typedef __attribute__((address_space(3))) unsigned char lds_u8;

// Four rows of sixteen 16-bit elements, transposed: with the 16 lanes of a
// group pointing at the rows' quarters in order, lane i gets column i.
template <typename V4>
__device__ inline V4 lds_columns(unsigned at) {
  typedef __attribute__((ext_vector_type(4))) short s16x4;
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(V4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at));
}

// The same for bytes: sixteen lanes read 8 bytes each, lanes 2 i and 2 i + 1 the halves
// of row i's sixteen, and lane l gets column l of the eight rows.
typedef int lds_i32x2 __attribute__((ext_vector_type(2)));
__device__ inline lds_i32x2 lds_columns8(unsigned at) {
  typedef __attribute__((address_space(3))) lds_i32x2 there;
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((there*)(uintptr_t)at);
}

template <typename X>
__device__ inline X lds_read(unsigned at) {
  return *(__attribute__((address_space(3))) const X*)(uintptr_t)at;
}
template <typename X>
__device__ inline void lds_write(unsigned at, X x) {
  *(__attribute__((address_space(3))) X*)(uintptr_t)at = x;
}

// Memory straight into LDS, 16 (or 4) bytes a lane at lds_at + 16 (4) * lane.
// `from` and `lds_at` are wave-uniform; M0 holds lds_at (nothing else here uses
// it). As inline assembly, the compiler's waits do not see the copies: its own
// waits for loads only become more conservative by them, and wait_copies()
// waits for the copies.
__device__ inline void copy16(const unsigned char* from, unsigned lane_bytes, unsigned lds_at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
               :
               : "v"(lane_bytes), "s"(from), "s"(__builtin_amdgcn_readfirstlane((int)lds_at))
               : "memory");
}
// The same for memory that other workgroups read too.
__device__ inline void copy16_shared(const unsigned char* from, unsigned lane_bytes,
                                     unsigned lds_at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(lane_bytes), "s"(from), "s"(__builtin_amdgcn_readfirstlane((int)lds_at))
               : "memory");
}
__device__ inline void copy4(const unsigned char* from, unsigned lane_bytes, unsigned lds_at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(lane_bytes), "s"(from), "s"(__builtin_amdgcn_readfirstlane((int)lds_at))
               : "memory");
}
// A loaded value has arrived here. Without it, the wait for a load from before
// a loop stands at its first use inside, and there waits for the copies of
// every step.
template <typename X>
__device__ inline void settle(X& x) {
  asm volatile("" : "+v"(x));
}
// All but the last `N` loads of the wave are done (they end in order).
template <int N>
__device__ inline void wait_copies() {
  static_assert(N >= 0 && N < 64, "the counter's width");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ inline void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

template <typename X>
__device__ inline X* uniform(X* p) {
  const uint64_t u = (uint64_t)p;
  return (X*)(((uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32) |
              (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)u));
}

__device__ inline float group_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, kWave));
  return fmaxf(x, __shfl_xor(x, 32, kWave));
}

__device__ inline float group_sum(float x) {
  x += __shfl_xor(x, 16, kWave);
  return x + __shfl_xor(x, 32, kWave);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace attn
}  // namespace dspark
