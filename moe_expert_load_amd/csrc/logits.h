// Router logits: masks, scores, and rows of any length by vectors (the gate and the balance
// loss read them alike).
#pragma once

#include "common.h"
#include "numeric.h"

namespace uep {

__device__ __forceinline__ bool gt_finite(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// NaN or +infinity: flagged (-infinity is a mask)
__device__ __forceinline__ bool gt_bad(float x) {
  return !gt_finite(x) && __float_as_uint(x) != 0xFF800000u;
}

// exp(x); in units of 2^-24 the argument, rounded twice, is 2 |x| off, exp2 two more.
__device__ __forceinline__ float gt_exp(float x) {
  return __builtin_amdgcn_exp2f(1.44269504f * x);
}

// Sigmoid by exp2 and the hardware's reciprocal instead of an exact division (4 instead of about
// 20 instructions for each of the E experts).  In units of 2^-24: the exponential's
// argument, rounded once, is |x| off and exp2 two more, together at most
// s (1 - s)(|x| + 2) < 0.8 of the score; 1 + e is rounded once and the reciprocal within 1.6:
// under 4 in all.
__device__ __forceinline__ float gt_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

template <typename T>
struct GtLoose;                                       // 16 bytes aligned as one element
template <>
struct GtLoose<float> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct GtLoose<uint16_t> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};

// 16 bytes of a row of E elements (at least as many as they hold) from element e0 on, -infinity
// past its end.  Rows start at any element: the memory takes vector accesses at the
// alignment of one.  kRagged: where the row ends inside the 16 bytes its last 16 are read
// and shifted down; otherwise it ends at none.
template <bool kRagged, typename T>
__device__ __forceinline__ u32x4 gt_load16(const T* p, int e0, int E) {
  constexpr uint32_t kFill = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
  constexpr int kCe = 16 / sizeof(T);
  u32x4 w = {kFill, kFill, kFill, kFill};
  const int at = kRagged ? min(e0, E - kCe) : e0;
  if (e0 < E) w = *reinterpret_cast<const typename GtLoose<T>::type*>(p + at);
  if (kRagged) {
    const int shift = e0 < E ? (e0 - at) * (int)sizeof(T) : 0;   // bytes
    w = shift & 8 ? u32x4{w[2], w[3], kFill, kFill} : w;
    w = shift & 4 ? u32x4{w[1], w[2], w[3], kFill} : w;
    if (sizeof(T) == 2) {
      const int bits = shift & 2 ? 16 : 0;
      w = u32x4{__builtin_amdgcn_alignbit(w[1], w[0], bits),
                __builtin_amdgcn_alignbit(w[2], w[1], bits),
                __builtin_amdgcn_alignbit(w[3], w[2], bits),
                __builtin_amdgcn_alignbit(kFill, w[3], bits)};
    }
  }
  return w;
}
template <typename T>
__device__ __forceinline__ float gt_element(u32x4 w, int j) {
  if (sizeof(T) == 4) return __uint_as_float(w[j & 3]);
  return j & 1 ? bf16_hi(w[j / 2 & 3]) : bf16_lo(w[j / 2 & 3]);
}

}  // namespace uep
