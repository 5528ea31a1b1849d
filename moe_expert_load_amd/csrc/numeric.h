// bf16 conversions and float reductions of the kernels that compute on what they move, and the
// overlap check of the calls whose outputs may not touch their inputs.
#pragma once

#include <initializer_list>

#include "common.h"

namespace uep {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// nearest-even fp32 -> bf16; a NaN becomes a quiet NaN with its sign
__device__ __forceinline__ uint32_t f32_to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7F800000u) == 0x7F800000u && (u & 0x007FFFFFu) != 0u) return ((u >> 16) | 0x40u) & 0xFFFFu;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// Two of them in one word, by the instruction that does the same to every input (compared
// over all 2^32).
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Wave-wide sum in a fixed order, uniform result: DPP butterflies inside each row of 16
// lanes (xor 1, xor 2, then the mirrored halves and rows, whose lanes are all alike by
// then), the four rows by readlane.  Every lane of the wave must be active.
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));
  const int b = __float_as_int(v);
  return (__int_as_float(readlane(b, 0)) + __int_as_float(readlane(b, 16))) +
         (__int_as_float(readlane(b, 32)) + __int_as_float(readlane(b, 48)));
}

}  // namespace uep

// Whether a buffer shares a byte with one of the others (absent ones are NULL).
struct UepBytes {
  const void* p;
  int64_t n;
};
static inline bool uep_overlap(UepBytes a, std::initializer_list<UepBytes> others) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p);
  for (const UepBytes& b : others) {
    const uintptr_t y = reinterpret_cast<uintptr_t>(b.p);
    if (x && y && a.n > 0 && b.n > 0 && x < y + (uintptr_t)b.n && y < x + (uintptr_t)a.n)
      return true;
  }
  return false;
}
