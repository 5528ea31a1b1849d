// AdamW over many tensors in one launch, states in fp32 or 8 bits (uep.h: AdamW).
//
// Every element's parameter, gradient and states are read once and written once.  The plan
// lists the work as tiles of 1024 or 4096 elements of one tensor each; a 256-thread workgroup
// takes one tile, each wave one or four chunks of 256 consecutive elements (four per lane:
// 16-byte accesses for fp32, 8 for bf16, 4 for the codes).  A chunk is a block of the 8-bit
// states, so a block's largest level is one reduction over a wave.
//
// Measured on MI355X, 302 M elements in 16 tensors: fp32 states, fp32 parameters and gradients
// with bf16 copies (30 bytes an element) 1520-1650 us by the buffers' placement, 5.5-5.9 TB/s,
// bound by HBM: a large copy reaches 5.65.  bf16 parameters and gradients with 8-bit states
// (10 bytes an element) 556-614 us, bound by its instructions: 77 for every element, of which
// the random words take 10, the codes' way in 12 and out 20.  The decode 325 us, 5.6 TB/s.
// Non-temporal accesses are worth 5 % with fp32 states (1700 -> 1610 us, each byte is used
// once a step), one chunk per wave against four 1-2 % there and 28 % of a small call
// (1.5 M elements in 96 tensors 13.9 -> 9.9 us); with 8-bit states four chunks per wave against
// one 12 % (1084 -> 954 us with the decode), since a tile's own work counts beside them.
#include <stdlib.h>

#include "common.h"
#include "numeric.h"

namespace uep {

constexpr int kAwThreads = 256;
constexpr int kAwWaves = kAwThreads / kWave;
constexpr int kAwChunk = 4 * kWave;               // elements of a wave's chunk = state block
// Chunks per wave of a long tile, and the elements from which on 8-bit states take them.  Four
// chunks against one, bf16 parameters and gradients: 64 K elements 7.2 against 4.9 us, 2 M 9.8 /
// 9.2, 4 M 13.9 / 14.1, 8 M 21.0 / 24.2, 32 M 68.9 / 80.6.
constexpr int kAwLong = 4;
constexpr int64_t kAwLongFrom = 4ll << 20;
constexpr int32_t kAwMagic = 0x41645757;
constexpr int kAwMaxLevel = 0x7F7;                // largest finite: exponent 254, mantissa 7
constexpr int64_t kAwMaxElems = 1ll << 33;
constexpr int kAwMaxTensors = 65535;

struct AwHeader {
  int32_t magic, count, param_dtype, grad_dtype, state_bits, n_tiles, unroll, pad;
};
struct AwTensor {
  uep_adamw_tensor t;
  int64_t first_tile;
  int32_t vec, pad;                               // vec: four elements are aligned everywhere
};
// plan: AwHeader, AwTensor[count], int32 tensor of each tile

struct AwArgs {                                   // scalars of one step
  float b1, ob1, b2, ob2, eps;
  double log_b1, log_b2;                          // -inf for a beta of 0
  uint32_t seed;
};

__device__ __forceinline__ uint32_t aw_mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B9u;                               // 2^32 / golden ratio
  x ^= x >> 15;
  x *= 0xBB67AE85u;                               // fraction of sqrt(3)
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t aw_next(uint32_t x) {   // xorshift32 (Marsaglia 2003)
  x ^= x << 13;
  x ^= x >> 17;
  return x ^ (x << 5);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The tensors' pointers come out of the plan, where the compiler cannot see that they are
// global memory: said here, since flat accesses, which it would make, cost more.
template <typename T>
using Global = __attribute__((address_space(1))) T*;

// Four consecutive elements of an array, as loaded; kFull: all there and aligned for one access.
// Accesses are non-temporal: every byte is used once a step.
template <bool kFull, typename T>
__device__ __forceinline__ void aw_load(Global<const T> p, int left, T (&v)[4]) {
  if constexpr (kFull) {
    typedef T vec __attribute__((ext_vector_type(4)));
    const vec x = __builtin_nontemporal_load((Global<const vec>)p);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = x[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < left ? p[j] : T(0);
  }
}
template <bool kFull, typename T>
__device__ __forceinline__ void aw_store(Global<T> p, int left, const T (&v)[4]) {
  if constexpr (kFull) {
    typedef T vec __attribute__((ext_vector_type(4)));
    vec x;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = v[j];
    __builtin_nontemporal_store(x, (Global<vec>)p);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) p[j] = v[j];
  }
}
// bf16 and codes travel as words: two or four elements of one register.
template <bool kFull>
__device__ __forceinline__ void aw_load(Global<const uint16_t> p, int left, uint32_t (&w)[2]) {
  if constexpr (kFull) {
    const u32x2 x = __builtin_nontemporal_load((Global<const u32x2>)p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    uint16_t v[4];
    aw_load<false>(p, left, v);
    w[0] = v[0] | (uint32_t)v[1] << 16;
    w[1] = v[2] | (uint32_t)v[3] << 16;
  }
}
template <bool kFull>
__device__ __forceinline__ void aw_store(Global<uint16_t> p, int left, const uint32_t (&w)[2]) {
  if constexpr (kFull) {
    __builtin_nontemporal_store(u32x2{w[0], w[1]}, (Global<u32x2>)p);
  } else {
    const uint16_t v[4] = {(uint16_t)w[0], (uint16_t)(w[0] >> 16), (uint16_t)w[1],
                           (uint16_t)(w[1] >> 16)};
    aw_store<false>(p, left, v);
  }
}
template <bool kFull>
__device__ __forceinline__ uint32_t aw_load_codes(Global<const uint8_t> p, int left) {
  if constexpr (kFull) return __builtin_nontemporal_load((Global<const uint32_t>)p);
  uint8_t v[4];
  aw_load<false>(p, left, v);
  return v[0] | (uint32_t)v[1] << 8 | (uint32_t)v[2] << 16 | (uint32_t)v[3] << 24;
}
template <bool kFull>
__device__ __forceinline__ void aw_store_codes(Global<uint8_t> p, int left, uint32_t w) {
  if constexpr (kFull) {
    __builtin_nontemporal_store(w, (Global<uint32_t>)p);
  } else {
    const uint8_t v[4] = {(uint8_t)w, (uint8_t)(w >> 8), (uint8_t)(w >> 16), (uint8_t)(w >> 24)};
    aw_store<false>(p, left, v);
  }
}

// What a lane holds of one chunk, as loaded: fp32 as it is, bf16 in words.
template <typename T>
struct AwFour {
  float x[4];
  template <bool kFull>
  __device__ __forceinline__ void load(const void* p, int64_t chunk, uint32_t at, int left) {
    aw_load<kFull>((Global<const float>)p + chunk + at, left, x);
  }
  __device__ __forceinline__ float at(int j) const { return x[j]; }
};
template <>
struct AwFour<uint16_t> {
  uint32_t w[2];
  template <bool kFull>
  __device__ __forceinline__ void load(const void* p, int64_t chunk, uint32_t at, int left) {
    aw_load<kFull>((Global<const uint16_t>)p + chunk + at, left, w);
  }
  __device__ __forceinline__ float at(int j) const {
    return j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
  }
};
template <typename P, typename G, bool k8>
struct AwChunk {
  AwFour<P> p;
  AwFour<G> g;
  AwFour<float> m, v;                             // fp32 states
  uint32_t mc, vc;                                // 8-bit states
  int tops;
  template <bool kFull>
  __device__ __forceinline__ void load(const AwTensor& t, int64_t chunk, uint32_t at, int left) {
    p.template load<kFull>(t.t.param, chunk, at, left);
    g.template load<kFull>(t.t.grad, chunk, at, left);
    if constexpr (k8) {
      mc = aw_load_codes<kFull>((Global<const uint8_t>)t.t.m + chunk + at, left);
      vc = aw_load_codes<kFull>((Global<const uint8_t>)t.t.v + chunk + at, left);
      tops = ((Global<const int32_t>)t.t.tops)[chunk / kAwChunk];
    } else {
      m.template load<kFull>(t.t.m, chunk, at, left);
      v.template load<kFull>(t.t.v, chunk, at, left);
    }
  }
};

// x + 16 * half, or x + half, of a random word's lower or upper half, in one instruction (a
// mask or shift of its own for the half would be a tenth of what an element costs).
template <bool kUpper>
__device__ __forceinline__ uint32_t aw_add16(uint32_t word, uint32_t x) {
  uint32_t d;
  if (kUpper) asm("v_mad_u32_u16 %0, %1, 16, %2 op_sel:[1,0,0,0]" : "=v"(d) : "v"(word), "v"(x));
  else asm("v_mad_u32_u16 %0, %1, 16, %2" : "=v"(d) : "v"(word), "v"(x));
  return d;
}
template <bool kUpper>
__device__ __forceinline__ uint32_t aw_add(uint32_t word, uint32_t x) {
  uint32_t d;
  if (kUpper) asm("v_mad_u32_u16 %0, %1, 1, %2 op_sel:[1,0,0,0]" : "=v"(d) : "v"(word), "v"(x));
  else asm("v_mad_u32_u16 %0, %1, 1, %2" : "=v"(d) : "v"(word), "v"(x));
  return d;
}

// Value of code j of a word: its level (size - span + top), cut at 0; code 0 is zero.  kPlain:
// the block's window lies above level 0 and the code is not 0.
template <bool kPlain>
__device__ __forceinline__ float aw_decode_m(uint32_t codes, int j, int top) {
  const int size = (codes >> (8 * j)) & 127;
  int x = (size << 20) + ((top - 127) << 20);
  if (!kPlain) x = size ? max(x, 0) : 0;
  return __uint_as_float((uint32_t)x | ((codes << (24 - 8 * j)) & 0x80000000u));
}
template <bool kPlain>
__device__ __forceinline__ float aw_decode_v(uint32_t codes, int j, int top) {
  const int size = (codes >> (8 * j)) & 255;
  int x = (size << 20) + ((top - 255) << 20);
  if (!kPlain) x = size ? max(x, 0) : 0;
  return __uint_as_float((uint32_t)x);
}
// Whether all four m and v codes are above zero: adding 127 to a byte's lower seven bits sets
// its top bit unless they are 0.
__device__ __forceinline__ bool aw_no_zero(uint32_t mc, uint32_t vc) {
  const uint32_t m = (mc & 0x7F7F7F7Fu) + 0x7F7F7F7Fu;
  const uint32_t v = ((vc & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | vc;
  return (m & v & 0x80808080u) == 0x80808080u;
}
// The wave's four m and v each; true where the block is an ordinary one: no zeros, and every v
// at least 2^-125 (level 16), so that one step leaves it a normal number.
__device__ __forceinline__ bool aw_decode(uint32_t mc, uint32_t vc, int tops, float (&m)[4],
                                          float (&v)[4]) {
  const int top_m = tops & 0xFFFF, top_v = tops >> 16;
  const bool plain = top_m >= 127 && top_v >= 255 + 16 && ballot(!aw_no_zero(mc, vc)) == 0;
  if (plain) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = aw_decode_m<true>(mc, j, top_m);
      v[j] = aw_decode_v<true>(vc, j, top_v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = aw_decode_m<false>(mc, j, top_m);
      v[j] = aw_decode_v<false>(vc, j, top_v);
    }
  }
  return plain;
}

// Codes of four new m and v and their block's tops; the whole wave calls it with its chunk.
// Levels come from the random words r; the common case, in which both windows lie above
// level 0 and below infinity, needs no check of zeros (their code comes out as 0 by the
// saturated difference) and no clamp.
__device__ __forceinline__ int aw_encode(const float (&m)[4], const float (&v)[4],
                                         const uint32_t* r, int left, uint32_t* mc, uint32_t* vc) {
  uint32_t bm[4], bv[4], xm[4], xv[4], max_m = 0, max_v = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool on = j < left;
    bm[j] = on ? __float_as_uint(m[j]) & 0x7FFFFFFFu : 0u;
    bv[j] = on ? __float_as_uint(v[j]) : 0u;      // v >= +0
    xm[j] = aw_add16<false>(r[j], bm[j]);         // the level is x >> 20
    xv[j] = aw_add16<true>(r[j], bv[j]);
    max_m = max(max_m, xm[j]);
    max_v = max(max_v, xv[j]);
  }
  int top_m = wave_max((int)max_m) >> 20, top_v = wave_max((int)max_v) >> 20;
  uint32_t cm[4], cv[4];
  if (top_m > 127 && top_v > 255 && max(top_m, top_v) <= kAwMaxLevel) {
    const uint32_t low_m = (uint32_t)(top_m - 127) << 20, low_v = (uint32_t)(top_v - 255) << 20;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cm[j] = __builtin_elementwise_sub_sat(xm[j], low_m) >> 20;
      cv[j] = max(__builtin_elementwise_sub_sat(xv[j], low_v) >> 20, min(bv[j], 1u));
    }
  } else {
    top_m = min(top_m, kAwMaxLevel);
    top_v = min(top_v, kAwMaxLevel);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int lm = min((int)(xm[j] >> 20), kAwMaxLevel), lv = min((int)(xv[j] >> 20), kAwMaxLevel);
      cm[j] = bm[j] ? (uint32_t)max(lm - top_m + 127, 0) : 0u;
      cv[j] = bv[j] ? (uint32_t)max(lv - top_v + 255, 1) : 0u;
    }
  }
  *mc = *vc = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t signed_code = cm[j] | (__float_as_uint(m[j]) >> 24 & 128u);
    *mc |= (cm[j] ? signed_code : 0u) << (8 * j);
    *vc |= cv[j] << (8 * j);
  }
  return top_m | top_v << 16;
}

struct AwScalars {
  float decay, rate, root2, scale;                // 1 - lr wd, lr / bc1, 1 / sqrt(bc2), sched[1]
};

// 1 - beta^t from t log beta <= 0 in double (in fp32, 1 - 0.999^1 would be good to 5 digits):
// with y = k ln 2 + r, 1 - e^y = (1 - 2^k) - 2^k (e^r - 1), e^r - 1 by its series, whose first
// term left out is r^11 / 11! < 4e-13.
__device__ __forceinline__ float aw_correction(double y) {
  if (y < -700.0) return 1.0f;                    // also beta = 0
  const double k = __builtin_rint(y * 1.4426950408889634);
  const double r = fma(k, -0.6931471805599453, y);
  double s = 1.0 / 3628800.0;
  s = fma(s, r, 1.0 / 362880.0);
  s = fma(s, r, 1.0 / 40320.0);
  s = fma(s, r, 1.0 / 5040.0);
  s = fma(s, r, 1.0 / 720.0);
  s = fma(s, r, 1.0 / 120.0);
  s = fma(s, r, 1.0 / 24.0);
  s = fma(s, r, 1.0 / 6.0);
  s = fma(s, r, 0.5);
  s = fma(s * r, r, r);
  const double p = __builtin_amdgcn_ldexp(1.0, (int)k);
  return (float)((1.0 - p) - p * s);
}

// One chunk: step, round, store.
template <typename P, typename G, bool k8, bool kFull>
__device__ __forceinline__ bool aw_chunk(const AwTensor& t, const AwChunk<P, G, k8>& in,
                                         int64_t chunk, uint32_t at, int left, const AwScalars& c,
                                         const AwArgs& a, uint32_t key) {
#pragma clang fp contract(off)
  const uint32_t lane_mul = (threadIdx.x % kWave) * 0x9E3779B9u;
  float g[4], m[4], v[4], w[4], root[4];
  bool bad = false, tiny = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    g[j] = in.g.at(j) * c.scale;
    bad |= (__float_as_uint(g[j]) & 0x7F800000u) == 0x7F800000u;
  }
  if (ballot(bad))
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((__float_as_uint(g[j]) & 0x7F800000u) == 0x7F800000u) g[j] = 0.0f;
  bool normal = false;                            // no new v can be subnormal
  if constexpr (k8) {
    normal = aw_decode(in.mc, in.vc, __builtin_amdgcn_readfirstlane(in.tops), m, v) &&
             a.b2 >= 0.5f;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = in.m.at(j);
      v[j] = in.v.at(j);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = m[j] * a.b1 + g[j] * a.ob1;
    v[j] = v[j] * a.b2 + g[j] * g[j] * a.ob2;
    // root and reciprocal by the hardware's approximations, each within a unit in the last
    // place; the root takes a subnormal number for 0, so those go the long way
    root[j] = __builtin_amdgcn_sqrtf(v[j]);
  }
  if (!normal) {
#pragma unroll
    for (int j = 0; j < 4; ++j) tiny |= __builtin_amdgcn_classf(v[j], 1 << 7);
    if (ballot(tiny))
#pragma unroll
      for (int j = 0; j < 4; ++j) root[j] = sqrtf(v[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float q = m[j] * __builtin_amdgcn_rcpf(fmaf(root[j], c.root2, a.eps));
    w[j] = fmaf(-c.rate, q, in.p.at(j) * c.decay);
  }
  uint32_t r[6] = {0};
  if constexpr (k8 || sizeof(P) == 2) {
    // the group's number times the constant, the chunk's part of it uniform
    r[0] = aw_mix(((uint32_t)(chunk >> 2) * 0x9E3779B9u + lane_mul) ^ key);
#pragma unroll
    for (int j = 1; j < (k8 ? 6 : 2); ++j) r[j] = aw_next(r[j - 1]);
  }
  if constexpr (sizeof(P) == 2) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t bits = __float_as_uint(w[j]);
      o[j] = j & 1 ? aw_add<true>(r[j / 2], bits) : aw_add<false>(r[j / 2], bits);
      // a NaN is cut as it is.  With 8-bit states it needs no check: it was made here, came from
      // a bf16 parameter or is the learning rate's, so its lower half is zero and nothing carries
      if (!k8 && (bits & 0x7FFFFFFFu) > 0x7F800000u) o[j] = bits;
    }
    const uint32_t word[2] = {o[0] >> 16 | (o[1] & 0xFFFF0000u), o[2] >> 16 | (o[3] & 0xFFFF0000u)};
    aw_store<kFull>((Global<uint16_t>)t.t.param + chunk + at, left, word);
  } else {
    aw_store<kFull>((Global<float>)t.t.param + chunk + at, left, w);
    if (t.t.copy) {
      const uint32_t word[2] = {pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3])};
      aw_store<kFull>((Global<uint16_t>)t.t.copy + chunk + at, left, word);
    }
  }
  if constexpr (k8) {
    uint32_t mc, vc;
    const int tops = aw_encode(m, v, r + 2, kFull ? 4 : left, &mc, &vc);
    aw_store_codes<kFull>((Global<uint8_t>)t.t.m + chunk + at, left, mc);
    aw_store_codes<kFull>((Global<uint8_t>)t.t.v + chunk + at, left, vc);
    if (threadIdx.x % kWave == 0) ((Global<int32_t>)t.t.tops)[chunk / kAwChunk] = tops;
  } else {
    aw_store<kFull>((Global<float>)t.t.m + chunk + at, left, m);
    aw_store<kFull>((Global<float>)t.t.v + chunk + at, left, v);
  }
  return bad;
}

// A tile of kU chunks for each wave, the loads of a full one all issued before the first is
// stepped.
template <typename P, typename G, bool k8, int kU, bool kFull>
__device__ __forceinline__ bool aw_tile(const AwTensor& t, int64_t base, const AwScalars& c,
                                        const AwArgs& a, uint32_t key) {
  const uint32_t at = threadIdx.x % kWave * 4;    // the lane's elements in a chunk
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  bool bad = false;
  constexpr int kAhead = kFull ? kU : 1;
  for (int u = 0; u < kU; u += kAhead) {
    AwChunk<P, G, k8> in[kAhead];
    if (!kFull && base + (int64_t)(u * kAwWaves + wave) * kAwChunk >= t.t.n) break;
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int64_t chunk = base + (int64_t)((u + h) * kAwWaves + wave) * kAwChunk;
      in[h].template load<kFull>(t, chunk, at, (int)min((int64_t)4, t.t.n - chunk - at));
    }
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int64_t chunk = base + (int64_t)((u + h) * kAwWaves + wave) * kAwChunk;
      bad |= aw_chunk<P, G, k8, kFull>(t, in[h], chunk, at,
                                       (int)min((int64_t)4, t.t.n - chunk - at), c, a, key);
    }
  }
  return bad;
}

template <typename P, typename G, bool k8, int kU>
__device__ __forceinline__ bool aw_step(const AwTensor& t, int64_t tile, const AwScalars& c,
                                        const AwArgs& a, uint32_t key) {
  constexpr int kTile = kU * kAwWaves * kAwChunk;
  const int64_t base = (tile - t.first_tile) * kTile;
  return t.vec && base + kTile <= t.t.n ? aw_tile<P, G, k8, kU, true>(t, base, c, a, key)
                                        : aw_tile<P, G, k8, kU, false>(t, base, c, a, key);
}

template <typename P, typename G, bool k8>
__global__ __launch_bounds__(kAwThreads) void adamw_kernel(const char* __restrict__ plan,
                                                           int32_t n_tiles, int32_t types,
                                                           const int32_t* __restrict__ step,
                                                           const float* __restrict__ sched,
                                                           AwArgs a, int32_t* err) {
  const AwHeader& h = *reinterpret_cast<const AwHeader*>(plan);
  const int t = step[0];
  if (h.magic != kAwMagic || h.n_tiles != n_tiles || t < 1 ||
      (h.param_dtype | h.grad_dtype << 8 | h.state_bits << 16) != types) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_err(err, UEP_ERR_PLAN);
    return;
  }
  const AwTensor* tensors = reinterpret_cast<const AwTensor*>(plan + sizeof(AwHeader));
  const int32_t* tiles = reinterpret_cast<const int32_t*>(tensors + h.count);
  const int q = tiles[blockIdx.x];
  const AwTensor& x = tensors[q];
  float lr = sched[0] * x.t.lr_scale;
  // any NaN as the one whose lower half is zero, which the random cut of bf16 parameters keeps
  if (lr != lr) lr = __builtin_nanf("");
  // both corrections at once: even lanes the first, odd lanes the second
  const float bc = aw_correction(t * (threadIdx.x & 1 ? a.log_b2 : a.log_b1));
  const float bc1 = __int_as_float(readlane(__float_as_int(bc), 0));
  const float bc2 = __int_as_float(readlane(__float_as_int(bc), 1));
  AwScalars c;
  c.decay = 1.0f - lr * x.t.weight_decay;
  c.rate = lr / bc1;
  c.root2 = 1.0f / sqrtf(bc2);
  c.scale = sched[1];
  const uint32_t key = aw_mix(aw_mix((uint32_t)t * 0x9E3779B9u + a.seed) ^ (uint32_t)(q + 1));
  bool bad;
  if (k8 && h.unroll == kAwLong) bad = aw_step<P, G, k8, kAwLong>(x, blockIdx.x, c, a, key);
  else bad = aw_step<P, G, k8, 1>(x, blockIdx.x, c, a, key);
  if (ballot(bad) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_GRAD);
}

// Four elements per thread; kVec: every pointer is aligned for them.
template <typename T>
__global__ __launch_bounds__(kAwThreads) void adamw_decode_kernel(
    const uint8_t* __restrict__ mc, const uint8_t* __restrict__ vc,
    const int32_t* __restrict__ tops, int64_t n, int vec, T* __restrict__ m, T* __restrict__ v) {
  const int64_t i = ((int64_t)blockIdx.x * kAwThreads + threadIdx.x) * 4;
  if (i >= n) return;
  const int top = tops[i / kAwChunk], left = (int)min((int64_t)4, n - i);
  const bool full = vec && left == 4;
  const uint32_t cm = full ? aw_load_codes<true>((Global<const uint8_t>)mc + i, 4)
                           : aw_load_codes<false>((Global<const uint8_t>)mc + i, left);
  const uint32_t cv = full ? aw_load_codes<true>((Global<const uint8_t>)vc + i, 4)
                           : aw_load_codes<false>((Global<const uint8_t>)vc + i, left);
  float a[4], b[4];
  aw_decode(cm, cv, __builtin_amdgcn_readfirstlane(top), a, b);   // a wave is one block
  if constexpr (sizeof(T) == 4) {
    if (full) {
      aw_store<true>((Global<T>)m + i, 4, a);
      aw_store<true>((Global<T>)v + i, 4, b);
    } else {
      aw_store<false>((Global<T>)m + i, left, a);
      aw_store<false>((Global<T>)v + i, left, b);
    }
  } else {
    const uint32_t wa[2] = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
    const uint32_t wb[2] = {pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3])};
    if (full) {
      aw_store<true>((Global<T>)m + i, 4, wa);
      aw_store<true>((Global<T>)v + i, 4, wb);
    } else {
      aw_store<false>((Global<T>)m + i, left, wa);
      aw_store<false>((Global<T>)v + i, left, wb);
    }
  }
}

// Elements of a tile: one chunk per wave; four with 8-bit states from 4 M elements on, where the
// step is bound by its instructions and a tile's own (its tensor, the corrections) count.
static int64_t aw_tile_elems(int32_t state_bits, int64_t elems) {
  return (int64_t)kAwChunk * kAwWaves * (state_bits == 8 && elems >= kAwLongFrom ? kAwLong : 1);
}

// Host table check: UEP_OK with all elements and the tiles they make, or why not.
static uep_status aw_count(const uep_adamw_tensor* t, int32_t count, int32_t state_bits,
                           int64_t* tile, int64_t* tiles) {
  if (count < 0 || (count > 0 && !t)) return UEP_EINVAL;
  if (count > kAwMaxTensors) return UEP_EGEOM;
  int64_t elems = 0;
  for (int32_t q = 0; q < count; ++q) {
    if (t[q].n < 0) return UEP_EINVAL;
    if (t[q].n > kAwMaxElems) return UEP_EGEOM;
    elems += t[q].n;
  }
  *tile = aw_tile_elems(state_bits, elems);
  *tiles = 0;
  for (int32_t q = 0; q < count; ++q) *tiles += (t[q].n + *tile - 1) / *tile;
  return UEP_OK;
}

static size_t aw_bytes(int32_t count, int64_t tiles) {
  return sizeof(AwHeader) + sizeof(AwTensor) * (size_t)count + sizeof(int32_t) * (size_t)tiles;
}

}  // namespace uep

using namespace uep;

extern "C" size_t uep_adamw_plan_size(const uep_adamw_tensor* tensors_host, int32_t count) {
  int64_t tile, tiles;                            // one chunk per wave: the most tiles
  return aw_count(tensors_host, count, 32, &tile, &tiles) == UEP_OK ? aw_bytes(count, tiles) : 0;
}

extern "C" uep_status uep_adamw_prepare(const uep_adamw_tensor* tensors_host, int32_t count,
                                        int32_t param_dtype, int32_t grad_dtype,
                                        int32_t state_bits, void* plan, size_t plan_bytes,
                                        int64_t* n_tiles, void* stream) {
  int64_t tile = 0, tiles = 0;
  const uep_status st = aw_count(tensors_host, count, state_bits, &tile, &tiles);
  if (st != UEP_OK) return st;
  if (tiles >= (1 << 24)) return UEP_EGEOM;         // a launch holds below 2^32 threads
  if ((param_dtype != UEP_F32 && param_dtype != UEP_BF16) ||
      (grad_dtype != UEP_F32 && grad_dtype != UEP_BF16) || (state_bits != 8 && state_bits != 32) ||
      !plan || !n_tiles)
    return UEP_EINVAL;
  const uintptr_t p_size = param_dtype == UEP_F32 ? 4 : 2, g_size = grad_dtype == UEP_F32 ? 4 : 2;
  const uintptr_t s_size = state_bits / 8;
  for (int32_t q = 0; q < count; ++q) {
    const uep_adamw_tensor& t = tensors_host[q];
    if (!(t.weight_decay > -__builtin_inff() && t.weight_decay < __builtin_inff()) ||
        !(t.lr_scale > -__builtin_inff() && t.lr_scale < __builtin_inff()))
      return UEP_EINVAL;
    if (t.copy && param_dtype != UEP_F32) return UEP_EINVAL;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && !t.tops)) return UEP_EINVAL;
    if ((uintptr_t)t.param % p_size || (uintptr_t)t.grad % g_size || (uintptr_t)t.m % s_size ||
        (uintptr_t)t.v % s_size || (uintptr_t)t.tops % 4 || (uintptr_t)t.copy % 2)
      return UEP_EGEOM;
  }
  const size_t bytes = aw_bytes(count, tiles);
  if (plan_bytes < bytes) return UEP_EWORKSPACE;
  if ((uintptr_t)plan % 8) return UEP_EGEOM;
  char* w = static_cast<char*>(calloc(1, bytes));
  if (!w) return UEP_EHIP;
  AwHeader* h = reinterpret_cast<AwHeader*>(w);
  h->magic = kAwMagic;
  h->count = count;
  h->param_dtype = param_dtype;
  h->grad_dtype = grad_dtype;
  h->state_bits = state_bits;
  h->n_tiles = (int32_t)tiles;
  h->unroll = (int32_t)(tile / (kAwChunk * kAwWaves));
  AwTensor* d = reinterpret_cast<AwTensor*>(w + sizeof(AwHeader));
  int32_t* tensor_of = reinterpret_cast<int32_t*>(d + count);
  int64_t at = 0;
  for (int32_t q = 0; q < count; ++q) {
    const uep_adamw_tensor& t = tensors_host[q];
    d[q].t = t;
    d[q].first_tile = at;
    d[q].vec = (uintptr_t)t.param % (4 * p_size) == 0 && (uintptr_t)t.grad % (4 * g_size) == 0 &&
               (uintptr_t)t.m % (4 * s_size) == 0 && (uintptr_t)t.v % (4 * s_size) == 0 &&
               (uintptr_t)t.copy % 8 == 0;
    for (int64_t k = (t.n + tile - 1) / tile; k > 0; --k) tensor_of[at++] = q;
  }
  hipStream_t s = uep_stream(stream);
  hipError_t e = hipMemcpyAsync(plan, w, bytes, hipMemcpyHostToDevice, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  free(w);
  if (e != hipSuccess) return UEP_EHIP;
  *n_tiles = tiles;
  return UEP_OK;
}

extern "C" uep_status uep_adamw(const void* plan, int64_t n_tiles, int32_t param_dtype,
                                int32_t grad_dtype, int32_t state_bits, const int32_t* step,
                                const float* sched, double beta1, double beta2, double eps,
                                uint32_t seed, int32_t* err, void* stream) {
  if (n_tiles < 0 || (param_dtype != UEP_F32 && param_dtype != UEP_BF16) ||
      (grad_dtype != UEP_F32 && grad_dtype != UEP_BF16) || (state_bits != 8 && state_bits != 32))
    return UEP_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0) ||
      !(eps >= 0x1p-126 && eps <= 0x1p126))    // a normal fp32 number
    return UEP_EINVAL;
  if (n_tiles >= (1 << 24)) return UEP_EGEOM;
  if (n_tiles == 0) return UEP_OK;
  if (!plan || !step || !sched) return UEP_EINVAL;
  AwArgs a;
  a.b1 = (float)beta1;
  a.ob1 = (float)(1.0 - beta1);
  a.b2 = (float)beta2;
  a.ob2 = (float)(1.0 - beta2);
  a.eps = (float)eps;
  a.log_b1 = __builtin_log(beta1);
  a.log_b2 = __builtin_log(beta2);
  a.seed = seed;
  const char* p = static_cast<const char*>(plan);
  const int32_t types = param_dtype | grad_dtype << 8 | state_bits << 16;
  auto kernel = state_bits == 32
      ? (param_dtype == UEP_F32 ? (grad_dtype == UEP_F32 ? adamw_kernel<float, float, false>
                                                         : adamw_kernel<float, uint16_t, false>)
                                : (grad_dtype == UEP_F32 ? adamw_kernel<uint16_t, float, false>
                                                         : adamw_kernel<uint16_t, uint16_t, false>))
      : (param_dtype == UEP_F32 ? (grad_dtype == UEP_F32 ? adamw_kernel<float, float, true>
                                                         : adamw_kernel<float, uint16_t, true>)
                                : (grad_dtype == UEP_F32 ? adamw_kernel<uint16_t, float, true>
                                                         : adamw_kernel<uint16_t, uint16_t, true>));
  hipLaunchKernelGGL(kernel, dim3((unsigned)n_tiles), dim3(kAwThreads), 0, uep_stream(stream), p,
                     (int32_t)n_tiles, types, step, sched, a, err);
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}

extern "C" uep_status uep_adamw_decode(const uint8_t* m_codes, const uint8_t* v_codes,
                                       const int32_t* tops, int64_t n, int32_t dtype, void* m,
                                       void* v, void* stream) {
  if (n < 0 || (dtype != UEP_F32 && dtype != UEP_BF16)) return UEP_EINVAL;
  if (n == 0) return UEP_OK;
  if (!m_codes || !v_codes || !tops || !m || !v) return UEP_EINVAL;
  const int64_t blocks = (n + 4 * kAwThreads - 1) / (4 * kAwThreads);
  if (blocks >= (1 << 24)) return UEP_EGEOM;
  const uintptr_t align = dtype == UEP_F32 ? 16 : 8;
  const int vec = ((uintptr_t)m_codes | (uintptr_t)v_codes) % 4 == 0 &&
                  ((uintptr_t)m | (uintptr_t)v) % align == 0;
  hipStream_t s = uep_stream(stream);
  if (dtype == UEP_F32)
    hipLaunchKernelGGL(adamw_decode_kernel<float>, dim3((unsigned)blocks), dim3(kAwThreads), 0, s,
                       m_codes, v_codes, tops, n, vec, static_cast<float*>(m),
                       static_cast<float*>(v));
  else
    hipLaunchKernelGGL(adamw_decode_kernel<uint16_t>, dim3((unsigned)blocks), dim3(kAwThreads), 0,
                       s, m_codes, v_codes, tops, n, vec, static_cast<uint16_t*>(m),
                       static_cast<uint16_t*>(v));
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}
