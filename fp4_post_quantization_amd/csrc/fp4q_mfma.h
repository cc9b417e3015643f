// Pieces that the matrix-core kernels share: operand types, rounding to
// bfloat16, direct global-to-LDS loads, their waits and the swizzle of staged
// rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "fp4q_device.h"

namespace fp4q_gemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float float2v __attribute__((ext_vector_type(2)));

// f(std::integral_constant<int, I>) for I = 0, 1, ..., N-1, unrolled at compile time.
template <typename F, int... I>
__device__ __forceinline__ void unroll(std::integer_sequence<int, I...>, F &&f) {
  (f(std::integral_constant<int, I>{}), ...);
}

// float32 -> bfloat16, round to nearest even, two values per instruction (v_cvt_pk_bf16_f32: lo in
// the low half).  On every float32 pattern, in both halves, it gives what the integer rounding
// (b + 0x7FFF + lsb) >> 16 gives, and a NaN gives (b >> 16) | 0x40 (checked on the device over all
// 2^32 patterns).
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((fp4q::f32x2{lo, hi}), bf16x2v));
}
__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) { return (uint16_t)f32x2_to_bf16x2(f, 0.0f); }

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t *p, float v) { *p = f32_to_bf16_rne(v); }

// Staged rows are stored unpadded, with 16-byte chunk c of row r at position c ^ swz(r): the rows that
// 16 lanes read together fall on distinct banks.
template <int ROWB>
__device__ __forceinline__ int swz(int r) {
  if constexpr (ROWB == 64) return (r >> 2) & 3;  // 16 rows of 64 B cover all 64 banks 4 times
  else return (r >> 1) & 7;                       // 128-byte rows: 8 chunks, rows pair up per bank half
}

// This lane's index in its wave, opaque to the optimiser (values derived from it are computed
// where they are used rather than hoisted out of loops).
__device__ __forceinline__ int opaque_lane() {
  int l = (int)(threadIdx.x & 63);
  __asm__ volatile("" : "+v"(l));
  return l;
}

// s_waitcnt with only the vector-memory counter (expcnt, lgkmcnt at their maxima)
template <int VM>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(VM >= 0 && VM < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((VM & 0xF) | ((VM >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// s_waitcnt lgkmcnt(0) alone (vmcnt and expcnt at their maxima)
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4)); }

__device__ __forceinline__ void load_lds16(const void *g, void *l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)g,
                                   (__attribute__((address_space(3))) void *)l, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const void *g, void *l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)g,
                                   (__attribute__((address_space(3))) void *)l, 4, 0, 0);
}

}  // namespace fp4q_gemm
