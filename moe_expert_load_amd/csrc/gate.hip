// Router gate and its gradient (uep.h: uep_gate, uep_gate_grad).
//
// Gate.  A token's logits are read once; the selection compares distinct keys that order by
// (rank, lowest id), so that one maximum names both the winner and its id.  A large call has
// to move few bytes (262144 tokens of 128 fp32 logits 151 MB, 27 us at the 5.65 TB/s of a
// large copy) and to compare many numbers: K rounds of a wave maximum per token took 273 us
// there, the sorting networks below take 30.  With a bias on sigmoid scores the instructions bound
// it: 262144 tokens of 256 bf16 logits 302 -> 47.5 us, 27 of them memory, 90 instructions a token
// or 23 for every expert, of which 9 sort; ranked by the logits, without a bias, 36.3.  A small
// call is one launch's latency (2.3 us).
//
// Gradient.  Bound by its stores, 134 MB in 34 us for the first of those layers.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "numeric.h"

namespace uep {

constexpr int kGtThreads = 256;
constexpr int kGtTokPerBlock = kGtThreads / kWave;
constexpr int kGtMaxE = 4096;
constexpr int kGtSortE = 1024;        // most experts of the kernel that sorts in registers
// Up to this many tokens a call is bound by its latency and takes 16 lanes per token (the
// shortest chain); above, by its instructions and takes as few lanes as hold the experts (a
// merge across lanes is done by all of them).  16 lanes against few, in a graph: 64 tokens
// 4.1 against 4.9 us (E = 128), 4.9 against 7.4 (E = 256, sigmoid); 8192 tokens 4.7 / 5.2 and
// 6.0 / 7.7; 16384 tokens 5.7 / 5.4 and 8.1 / 7.9; 32768 tokens 8.3 / 6.6 and 11.9 / 10.4.
constexpr int64_t kGtFew = 8192;

template <typename T>
__device__ __forceinline__ float gt_load(const T* p, int64_t i);
template <>
__device__ __forceinline__ float gt_load<float>(const float* p, int64_t i) { return p[i]; }
template <>
__device__ __forceinline__ float gt_load<uint16_t>(const uint16_t* p, int64_t i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}

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

// Keys order by (rank, lowest id), rank an fp32 number that is finite, or -infinity for an
// expert that is not eligible.  Key64: a double with the rank's bits above and the inverted id
// below (its complement under a negative rank, where larger magnitudes are smaller), so that
// one v_max_f64 / v_min_f64 compares both; 64-bit integers have no such instruction, a
// compare and two selects.  The rank's exponent is never all of the double's, so no key is a
// NaN.  Key32: bf16 logits leave the lower half of the word for the id; unsigned order.
constexpr int kGtInv = 0xFFFF;                      // inverted id = kGtInv - id
constexpr float kGtMasked = -__builtin_inff();

struct Key64 {
  typedef double type;
  // of expert e ^ f; inv = kGtInv ^ f is a constant, kept in a scalar register so that one
  // three-way xor makes the lower word
  static __device__ __forceinline__ double make(float rank, int inv, int e) {
    const int u = __float_as_int(rank);
    int low;
    asm("v_bitop3_b32 %0, %1, %2, %3 bitop3:0x96" : "=v"(low) : "v"(u >> 31), "s"(inv), "v"(e));
    return __hiloint2double(u, low);
  }
  static __device__ __forceinline__ double hi(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
  static __device__ __forceinline__ double lo(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
  static __device__ __forceinline__ float rank(double k) {
    return __int_as_float(__double2hiint(k));
  }
  static __device__ __forceinline__ int id(double k) {
    return kGtInv - ((__double2loint(k) ^ (__double2hiint(k) >> 31)) & 0xFFFF);
  }
  template <int kDpp>
  static __device__ __forceinline__ double moved(double k) {
    return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(k), kDpp, 0xF, 0xF, true),
                            __builtin_amdgcn_mov_dpp(__double2loint(k), kDpp, 0xF, 0xF, true));
  }
};
struct Key32 {
  typedef uint32_t type;
  static __device__ __forceinline__ uint32_t make(float rank, int inv, int e) {
    const uint32_t u = __float_as_uint(rank);
    const uint32_t o = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return (o & 0xFFFF0000u) | (uint32_t)(inv ^ e);
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) { return min(a, b); }
  static __device__ __forceinline__ float rank(uint32_t k) {
    return __uint_as_float((k & 0x80000000u ? k ^ 0x80000000u : ~k) & 0xFFFF0000u);
  }
  static __device__ __forceinline__ int id(uint32_t k) { return kGtInv - (int)(k & 0xFFFFu); }
  template <int kDpp>
  static __device__ __forceinline__ uint32_t moved(uint32_t k) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)k, kDpp, 0xF, 0xF, true);
  }
};

// ---------------------------------------------------------------------------------------
// Few slots and experts: kL lanes per token, kPer experts per lane, a running list of the
// kN >= K best.  Sorting networks on registers: every kN experts are sorted (Batcher's
// odd-even mergesort), merged into the list (the larger of list[i] and sorted[kN - 1 - i]
// are the kN best and bitonic; a bitonic merge sorts them), and the kL lanes' lists are
// merged the same way with DPP moves.
template <typename KY, int kN>
__device__ __forceinline__ void gt_order_pair(typename KY::type (&a)[kN], int i, int j) {
  const typename KY::type x = KY::hi(a[i], a[j]), y = KY::lo(a[i], a[j]);
  a[i] = x;
  a[j] = y;
}
template <typename KY, int kN>
__device__ __forceinline__ void gt_sort(typename KY::type (&a)[kN]) {
#pragma unroll
  for (int p = 1; p < kN; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < kN; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < kN && (i + j) / (2 * p) == (i + j + k) / (2 * p))
            gt_order_pair<KY>(a, i + j, i + j + k);
}
template <typename KY, int kN>
__device__ __forceinline__ void gt_merge(typename KY::type (&a)[kN], const typename KY::type (&b)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) a[i] = KY::hi(a[i], b[kN - 1 - i]);
#pragma unroll
  for (int s = kN / 2; s >= 1; s /= 2)
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (!(i & s)) gt_order_pair<KY>(a, i, i + s);
}
template <typename KY, int kDpp, int kN>
__device__ __forceinline__ void gt_merge_lanes(typename KY::type (&a)[kN]) {
  typename KY::type b[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) b[i] = KY::template moved<kDpp>(a[i]);
  gt_merge<KY>(a, b);
}

// sum over the kL lanes of a token
template <int kL>
__device__ __forceinline__ float gt_lanes_sum(float v) {
  auto add = [](float a, int b) { return a + __int_as_float(b); };
  v = add(v, __builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));   // xor 1
  v = add(v, __builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));   // xor 2
  if (kL >= 8) v = add(v, __builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));
  if (kL >= 16) v = add(v, __builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));
  return v;
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

// kBias: ranked by sigmoid score plus bias; otherwise by the logits, whose order is that of
// either score (fp32 scores of different logits can be the same number: 1 above a logit of 17).
template <typename T, typename KY, bool kBias, int kL, int kN, int kPer>
__global__ __launch_bounds__(kGtThreads) void gate_sort_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ batch_size, int64_t n_tok, int tok_per_rank, int E, int K,
    int score, int renorm, float scale, int32_t* __restrict__ topk_ids,
    float* __restrict__ gate_w, int32_t* err) {
  typedef typename KY::type key_t;
  constexpr int kCe = 16 / sizeof(T);                 // experts of one 16-byte load
  constexpr int kChunks = kPer / kCe;
  const int lane = threadIdx.x % kL;
  const int64_t g = (int64_t)blockIdx.x * (kGtThreads / kL) + threadIdx.x / kL;
  bool live = g < n_tok;
  if (live && batch_size) live = (int)(g % tok_per_rank) < batch_size[g / tok_per_rank];
  const T* row = logits + (live ? g : 0) * (int64_t)E;
  const int e_end = live ? E : 0;
  u32x4 raw[kChunks];
  if (E % kCe == 0) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      raw[c] = gt_load16<false>(row, (c * kL + lane) * kCe, e_end);
  } else {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      raw[c] = gt_load16<true>(row, (c * kL + lane) * kCe, e_end);
  }
  bool bad = false, odd_bias = false;
  __shared__ __attribute__((aligned(16))) float bias_lds[kBias ? kL * kPer : 4];
  if (kBias) {
    for (int e = threadIdx.x; e < kL * kPer; e += kGtThreads) {
      const float y = e < E ? bias[e] : 0.0f;
      bad |= gt_bad(y);
      bias_lds[e] = y;
    }
    odd_bias = __syncthreads_or(bad);
  }
  key_t best[kN];
#pragma unroll
  for (int q = 0; q < kPer / kN; ++q) {
    if (q > 0 && q * kN / kCe * kCe * kL >= E) break; // uniform: no lane has such experts
    float f[kN];
    bool odd = odd_bias;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int n = q * kN + i;
      f[i] = gt_element<T>(raw[n / kCe], n % kCe);
      // by logits: NaN and +infinity (bits 0, 1, 9); -infinity is ranked as it is
      odd |= kBias ? !gt_finite(f[i]) : __builtin_amdgcn_classf(f[i], 0x203);
    }
    if (kBias) {
      float y[kN];
#pragma unroll
      for (int h = 0; h < kN; h += 4) {
        const int n = q * kN + h, e = (n / kCe * kL + lane) * kCe + n % kCe;
        const f32x4 w = *reinterpret_cast<const f32x4*>(bias_lds + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[h + j] = w[j];
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) y[i] += gt_sigmoid(f[i]);
      if (ballot(odd))
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          bad |= gt_bad(f[i]);
          if (!gt_finite(f[i]) || !gt_finite(y[i])) y[i] = kGtMasked;
        }
#pragma unroll
      for (int i = 0; i < kN; ++i) f[i] = y[i];
    } else {
      if (ballot(odd))
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          bad |= gt_bad(f[i]);
          if (!gt_finite(f[i])) f[i] = kGtMasked;
        }
#pragma unroll
      for (int i = 0; i < kN; ++i) f[i] += 0.0f;      // -0 ties with +0
    }
    key_t a[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      // the expert is n / kCe * kL * kCe + lane * kCe + n % kCe, three separate bit fields
      const int n = q * kN + i;
      a[i] = KY::make(f[i], kGtInv ^ (n / kCe * kL * kCe + n % kCe), lane * kCe);
    }
    gt_sort<KY>(a);
    if (q == 0) {
#pragma unroll
      for (int i = 0; i < kN; ++i) best[i] = a[i];
    } else {
      gt_merge<KY>(best, a);
    }
  }
  if (ballot(bad) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_LOGIT);
  gt_merge_lanes<KY, 0xB1>(best);                     // xor 1
  gt_merge_lanes<KY, 0x4E>(best);                     // xor 2
  if (kL >= 8) gt_merge_lanes<KY, 0x141>(best);       // the other half of 8 (row_half_mirror)
  if (kL >= 16) gt_merge_lanes<KY, 0x140>(best);      // the other half of 16 (row_mirror)

  constexpr int kSlots = kN > kL ? kN / kL : 1;       // a lane's slots, consecutive
  const float top = KY::rank(best[0]);                // by logits: the largest
  int id[kSlots];
  float s[kSlots], mine = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    key_t k = best[i];
#pragma unroll
    for (int l = 1; l < kL && l * kSlots + i < kN; ++l)
      if (lane == l) k = best[l * kSlots + i];
    const float f = KY::rank(k);
    const bool on = f > kGtMasked && lane * kSlots + i < K;
    id[i] = on ? KY::id(k) : -1;
    s[i] = 0.0f;
    if (on) s[i] = kBias ? gt_sigmoid(gt_load(row, id[i])) : score ? gt_sigmoid(f) : gt_exp(f - top);
    mine += s[i];
  }
  float total = 1.0f;
  if (renorm) {
    total = gt_lanes_sum<kL>(mine);
  } else if (!kBias && !score) {
    float z = 0.0f;
#pragma unroll
    for (int n = 0; n < kPer; ++n) {
      const float f = gt_element<T>(raw[n / kCe], n % kCe);
      z += gt_finite(f) ? gt_exp(f - top) : 0.0f;
    }
    total = gt_lanes_sum<kL>(z);
  }
  // sums of sigmoids go down to 2^-126: the reciprocal before the scale, which could overflow it
  const float norm = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = lane * kSlots + i;
    if (g < n_tok && k < K) {
      topk_ids[g * K + k] = id[i];
      gate_w[g * K + k] = s[i] * norm * scale;
    }
  }
}

// ---------------------------------------------------------------------------------------
// Any size: one wave per token, kVpt experts per lane (expert j * 64 + lane); K rounds of a
// wave maximum over the keys left.
__device__ __forceinline__ double gt_wave_max(double v) {
  v = Key64::hi(v, Key64::moved<0xB1>(v));            // xor 1, xor 2, mirrored halves and rows
  v = Key64::hi(v, Key64::moved<0x4E>(v));
  v = Key64::hi(v, Key64::moved<0x141>(v));
  v = Key64::hi(v, Key64::moved<0x140>(v));
  double r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __hiloint2double(readlane(__double2hiint(v), 16 * i),
                            readlane(__double2loint(v), 16 * i));
  return Key64::hi(Key64::hi(r[0], r[1]), Key64::hi(r[2], r[3]));
}
template <typename T, int kVpt>
__global__ __launch_bounds__(kGtThreads) void gate_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ batch_size, int64_t g0, int64_t g1, int tok_per_rank, int E,
    int K, int score, int renorm, float scale, int32_t* __restrict__ topk_ids,
    float* __restrict__ gate_w, int32_t* err) {
  const int lane = threadIdx.x % kWave;
  const int64_t g = g0 + (int64_t)blockIdx.x * kGtTokPerBlock + threadIdx.x / kWave;
  if (g >= g1) return;
  if (batch_size && (int)(g % tok_per_rank) >= batch_size[g / tok_per_rank]) {
    if (lane < K) {
      topk_ids[g * K + lane] = -1;
      gate_w[g * K + lane] = 0.0f;
    }
    return;
  }
  const double none = Key64::make(kGtMasked, 0, 0);
  double key[kVpt];
  float val[kVpt];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kVpt; ++j) {
    const int e = j * kWave + lane;
    const float x = e < E ? gt_load(logits, g * E + e) : -__builtin_inff();
    val[j] = x;
    bad |= gt_bad(x);
    float f = x + 0.0f;
    if (bias && e < E) {                              // ranked as in the sorting kernel
      const float y = bias[e];
      bad |= gt_bad(y);
      if (gt_finite(x)) f = gt_sigmoid(x) + y;
    }
    key[j] = gt_finite(f) ? Key64::make(f, kGtInv, e) : none;
  }
  if (ballot(bad) && lane == 0) set_err(err, UEP_ERR_LOGIT);
  int id_mine = -1;
  float top = 0.0f;
  for (int k = 0; k < K; ++k) {
    double m = key[0];
#pragma unroll
    for (int j = 1; j < kVpt; ++j) m = Key64::hi(m, key[j]);
    m = gt_wave_max(m);
    if (m == none) break;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) key[j] = key[j] == m ? none : key[j];
    if (k == 0) top = Key64::rank(m);                 // by logits: the largest
    if (lane == k) id_mine = Key64::id(m);
  }
  const bool on = id_mine >= 0;
  const float l = on ? gt_load(logits, g * E + id_mine) : 0.0f;
  const float s = on ? (score ? gt_sigmoid(l) : gt_exp(l - top)) : 0.0f;
  float total = 1.0f;
  if (renorm) {
    total = wave_sum_f32(s);
  } else if (!score) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) z += gt_finite(val[j]) ? gt_exp(val[j] - top) : 0.0f;
    total = wave_sum_f32(z);
  }
  if (lane < K) {
    topk_ids[g * K + lane] = id_mine;
    gate_w[g * K + lane] = total > 0.0f ? s * (1.0f / total) * scale : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void gt_store(T* p, int64_t i, float v) {
  if constexpr (sizeof(T) == 4) p[i] = v;
  else p[i] = (T)f32_to_bf16(v);
}

// ---------------------------------------------------------------------------------------
// Gradient.  A wave takes 64 / kp tokens, kp the power of two from K up: a lane per slot for
// the coefficients, then the tokens' rows, which are one contiguous stretch of dlogits, in
// windows of kGtWin elements.  The slots' values are scattered into a window in LDS that is
// zero otherwise, the window goes out in 16-byte stores that need no row to be aligned, and
// the slots put their zeros back.  Bound by those stores.
//
// Weights that are not renormalised make the softmax's gradient dense.  Its scores need no
// pass over the row: s_e = u_r exp(l_e - l_r) for any selected slot r, and the slot of the
// largest weight is taken.  (A row whose largest weight is tiny, possible only where a
// caller has dropped slots, sums its exponentials.)
constexpr int kGtWin = 1024;
constexpr float kGtTiny = 1e-20f;
// A sigmoid's 1 - s is the score of -l.  Without renormalisation the weight holds s, to 6 units of
// 2^-24 (4 of the score, 2 of the scale), and the difference saves the gather of the logits: down
// to these, where it is good to 2^-15 for fp32 and to 2^-13 for bf16, whose result is rounded to
// 2^-8.  Always the difference against always the logit, 262144 tokens, K = 8: 25.3 against 42.3 us
// (256 experts, bf16) and 25.1 / 42.2 (128, fp32), and nothing is left from a logit of 17 on.
template <typename T>
constexpr float gt_near_one = sizeof(T) == 4 ? 0x1p-6f : 0x1p-8f;
constexpr int kGtGradBlocks = 256 * 8;    // every CU's fill of them; they step through the tokens

template <typename T, bool kDense>
__global__ __launch_bounds__(kGtThreads) void gate_grad_kernel(
    const float* __restrict__ dgate_w, const T* __restrict__ logits,
    const int32_t* __restrict__ topk_ids, const float* __restrict__ gate_w, int64_t n_tok, int E,
    uint32_t e_magic, int K, int lg_kp, int score, int renorm, float scale, int vec,
    T* __restrict__ dlogits, int32_t* err) {
  constexpr int kCe = 16 / sizeof(T);
  __shared__ __attribute__((aligned(16))) float win_all[kGtThreads / kWave][kGtWin];
  __shared__ __attribute__((aligned(16))) f32x4 par_all[kDense ? kGtThreads / kWave : 1][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  float* win = win_all[wave];
  f32x4* par = par_all[kDense ? wave : 0];
  for (int i = lane * 4; i < kGtWin; i += kWave * 4)
    *reinterpret_cast<f32x4*>(win + i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int kp = 1 << lg_kp, tpw = kWave >> lg_kp;
  const int tok = lane >> lg_kp, k = lane & (kp - 1);
  const int64_t n_grp = (n_tok + tpw - 1) / tpw;
  for (int64_t grp = (int64_t)blockIdx.x * kGtTokPerBlock + wave; grp < n_grp;
       grp += (int64_t)gridDim.x * kGtTokPerBlock) {
    const int64_t g0 = grp * tpw, g = g0 + tok;
    const bool there = k < K && g < n_tok;
    int id = there ? topk_ids[g * K + k] : -1;
    const bool bad = id < -1 || id >= E;
    if (ballot(bad) && lane == 0) set_err(err, UEP_ERR_ID_RANGE);
    if (bad) id = -1;
    const bool on = id >= 0;
    const float gk = on ? scale * dgate_w[g * K + k] : 0.0f;
    const float u = on ? gate_w[g * K + k] / scale : 0.0f;
    const bool far = !kDense && !renorm && u <= 1.0f - gt_near_one<T>;   // u is the score
    const float l = on && (kDense || (score && !far)) ? gt_load(logits, g * E + id) : 0.0f;
    float dot = u * gk;
    for (int o = kp / 2; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
    float d;
    if (kDense) {
      d = gk;
      float ur = on ? u : -1.0f, lr = on ? l : __builtin_inff();   // no slot: every score 0
      for (int o = kp / 2; o > 0; o >>= 1) {
        const float u2 = __shfl_xor(ur, o, kWave), l2 = __shfl_xor(lr, o, kWave);
        if (u2 > ur || (u2 == ur && l2 > lr)) { ur = u2; lr = l2; }
      }
      uint64_t tiny = ballot(k == 0 && ur >= 0.0f && ur < kGtTiny);
      while (tiny) {
        const int at = __ffsll((unsigned long long)tiny) - 1;
        tiny &= tiny - 1;
        const int64_t gr = g0 + (at >> lg_kp);
        float m = -__builtin_inff(), z = 0.0f;
        for (int e = lane; e < E; e += kWave) {
          const float x = gt_load(logits, gr * E + e);
          if (gt_finite(x)) m = fmaxf(m, x);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
        for (int e = lane; e < E; e += kWave) {
          const float x = gt_load(logits, gr * E + e);
          if (gt_finite(x)) z += gt_exp(x - m);
        }
        z = wave_sum_f32(z);
        if (tok == at >> lg_kp) {
          ur = 1.0f / z;
          lr = m;
        }
      }
      if (k == 0) par[tok] = f32x4{lr, fmaxf(ur, 0.0f), dot, 0.0f};
    } else if (score) {
      d = u * (far ? 1.0f - u : gt_sigmoid(-l)) * (renorm ? gk - dot : gk);
    } else {
      d = u * (gk - dot);
    }
    const int total = (int)min((int64_t)tpw, n_tok - g0) * E;
    const int unit = vec ? kCe : 1;
    // the window starts `lead` elements before the stretch, on a 16-byte boundary of dlogits
    const int lead = vec ? (int)((g0 * E) % kCe) : 0;
    const int pos = tok * E + id + lead;
    T* dst = dlogits + g0 * E - lead;
    const T* src = logits + g0 * E - lead;
    const int64_t stretch = n_tok * E - g0 * E + lead;   // elements of src up to its end
    for (int o = 0; o < total + lead; o += kGtWin) {
      const bool mine = on && pos >= o && pos < o + kGtWin;
      // zeros of other lanes (the first ones, or those put back) before values in their places
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (mine) win[pos - o] = d;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int end = min(kGtWin, total + lead - o);
      for (int i = lane * unit; i < end; i += kWave * unit) {
        const int at = o + i;                         // element of the stretch, plus lead
        float v[kCe];
        if (vec) {
#pragma unroll
          for (int j = 0; j < kCe; j += 4)
            *reinterpret_cast<f32x4*>(v + j) = *reinterpret_cast<const f32x4*>(win + i + j);
        } else {
          v[0] = win[i];
        }
        if constexpr (kDense) {
          // a unit holds the end of row r0 and, from element `cut` on, the start of the next
          const int p0 = max(at - lead, 0);
          const int r0 = E == 1 ? p0 : (int)__umulhi((uint32_t)p0, e_magic);
          const int cut = (r0 + 1) * E - (at - lead);
          const f32x4 q0 = par[r0], q1 = par[min(r0 + 1, tpw - 1)];
          float x[kCe];
          if (vec && at + kCe <= stretch) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(src + at);
#pragma unroll
            for (int j = 0; j < kCe; ++j) x[j] = gt_element<T>(w, j);
          } else {                                    // single elements, and the tensor's end
#pragma unroll
            for (int j = 0; j < kCe; ++j)
              x[j] = j < unit && at + j < stretch ? gt_load(src, at + j) : 0.0f;
          }
          auto dense = [](float x, float v, f32x4 q) {
            return gt_finite(x) ? q[1] * gt_exp(x - q[0]) * (v - q[2]) : 0.0f;
          };
          if (E % kCe == 0) {                         // units of one row
#pragma unroll
            for (int j = 0; j < kCe; ++j) v[j] = dense(x[j], v[j], q0);
          } else {
#pragma unroll
            for (int j = 0; j < kCe; ++j) v[j] = dense(x[j], v[j], j < cut ? q0 : q1);
          }
        }
        if (vec && at >= lead && at + kCe <= total + lead) {
          u32x4 w;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = sizeof(T) == 4 ? __float_as_uint(v[j])
                                  : pack_bf16(v[2 * j & (kCe - 1)], v[(2 * j + 1) & (kCe - 1)]);
          *reinterpret_cast<u32x4*>(dst + at) = w;
        } else {
#pragma unroll
          for (int j = 0; j < kCe; ++j)               // single elements, and a stretch's ends
            if (j < unit && at + j >= lead && at + j < total + lead) gt_store(dst, at + j, v[j]);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (mine) win[pos - o] = 0.0f;
    }
  }
}

struct GtCall {
  const void* logits;
  const float* bias;
  const int32_t* batch_size;
  int64_t n_tok;
  int T, E, K, score, renorm;
  float scale;
  int32_t* topk_ids;
  float* gate_w;
  int32_t* err;
  hipStream_t stream;
};

static unsigned gt_blocks(int64_t n_tok, int per) { return (unsigned)((n_tok + per - 1) / per); }

// n_tok < 2^26 tokens, at most 16 lanes each: below the 2^32 threads that a launch holds
template <typename T, typename KY, bool kBias, int kL, int kN, int kPer>
static uep_status gt_sorted(const GtCall& c) {
  const unsigned blocks = gt_blocks(c.n_tok, kGtThreads / kL);
  hipLaunchKernelGGL((gate_sort_kernel<T, KY, kBias, kL, kN, kPer>), dim3(blocks), dim3(kGtThreads),
                     0, c.stream, static_cast<const T*>(c.logits), c.bias, c.batch_size, c.n_tok,
                     c.T, c.E, c.K, c.score, c.renorm, c.scale, c.topk_ids, c.gate_w, c.err);
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}

constexpr int64_t kGtLaunch = 1ll << 25;  // a wave each: half of what a launch holds
template <typename T, int kVpt>
static uep_status gt_general(const GtCall& c) {
  for (int64_t g0 = 0; g0 < c.n_tok; g0 += kGtLaunch) {
    const int64_t g1 = std::min(c.n_tok, g0 + kGtLaunch);
    const unsigned blocks = gt_blocks(g1 - g0, kGtTokPerBlock);
    hipLaunchKernelGGL((gate_kernel<T, kVpt>), dim3(blocks), dim3(kGtThreads), 0, c.stream,
                       static_cast<const T*>(c.logits), c.bias, c.batch_size, g0, g1, c.T, c.E,
                       c.K, c.score, c.renorm, c.scale, c.topk_ids, c.gate_w, c.err);
    UEP_CHECK_LAUNCH();
  }
  return UEP_OK;
}

template <typename T, typename KY, bool kBias, int kL, int kPer>
static uep_status gt_by_slots(const GtCall& c) {
  return c.K <= 4   ? gt_sorted<T, KY, kBias, kL, 4, kPer>(c)
         : c.K <= 8 ? gt_sorted<T, KY, kBias, kL, 8, kPer>(c)
                    : gt_sorted<T, KY, kBias, kL, 16, kPer>(c);
}

template <typename T, typename KY, bool kBias>
static uep_status gt_by_experts(const GtCall& c) {
  if (c.n_tok <= kGtFew && c.E <= 16 * 32) return gt_by_slots<T, KY, kBias, 16, 32>(c);
  if (c.E <= 4 * 32) return gt_by_slots<T, KY, kBias, 4, 32>(c);
  if (c.E <= 4 * 64) return gt_by_slots<T, KY, kBias, 4, 64>(c);
  if (c.E <= 8 * 64) return gt_by_slots<T, KY, kBias, 8, 64>(c);
  return gt_by_slots<T, KY, kBias, 16, 64>(c);
}

template <typename T>
static uep_status gt_launch(const GtCall& c) {
  if (c.K <= 16 && c.E <= kGtSortE && c.E >= 16 / (int)sizeof(T)) {
    if (c.bias) return gt_by_experts<T, Key64, true>(c);
    typedef typename std::conditional<sizeof(T) == 2, Key32, Key64>::type key;
    return gt_by_experts<T, key, false>(c);
  }
  if (c.E <= 256) return gt_general<T, 4>(c);       // over 16 slots
  if (c.E <= 1024) return gt_general<T, 16>(c);
  return gt_general<T, 64>(c);
}

static uep_status gt_check(const void* logits, int32_t dtype, int32_t R, int32_t T, int32_t E,
                           int32_t K, int32_t score, float scale) {
  if (R <= 0 || T < 0 || E <= 0 || K <= 0) return UEP_EINVAL;
  if (dtype != UEP_F32 && dtype != UEP_BF16) return UEP_EINVAL;
  if (score != UEP_GATE_SOFTMAX && score != UEP_GATE_SIGMOID) return UEP_EINVAL;
  if (!(scale > -__builtin_inff() && scale < __builtin_inff()) || scale == 0.0f) return UEP_EINVAL;
  if (R > 64 || E > kGtMaxE || K > 64 || K > E || (int64_t)R * T * K >= (1ll << 31) ||
      (int64_t)R * T >= (1ll << 26))
    return UEP_EGEOM;
  if (T > 0 && !logits) return UEP_EINVAL;
  return UEP_OK;
}

}  // namespace uep

using namespace uep;

extern "C" uep_status uep_gate(const void* logits, int32_t dtype, const float* bias,
                               const int32_t* batch_size, int32_t R, int32_t T, int32_t E,
                               int32_t K, int32_t score, int32_t renorm, float scale,
                               int32_t* topk_ids, float* gate_w, int32_t* err, void* stream) {
  const uep_status st = gt_check(logits, dtype, R, T, E, K, score, scale);
  if (st != UEP_OK) return st;
  if (bias && score != UEP_GATE_SIGMOID) return UEP_EINVAL;
  if (T == 0) return UEP_OK;
  if (!topk_ids || !gate_w) return UEP_EINVAL;
  const int64_t n_tok = (int64_t)R * T;
  const UepBytes rows{logits, n_tok * E * (dtype == UEP_F32 ? 4 : 2)}, lift{bias, E * 4ll};
  const UepBytes sizes{batch_size, R * 4ll}, ids{topk_ids, n_tok * K * 4}, w{gate_w, n_tok * K * 4};
  if (uep_overlap(ids, {rows, lift, sizes, w}) || uep_overlap(w, {rows, lift, sizes}))
    return UEP_EINVAL;
  const GtCall c{logits, bias, batch_size, n_tok, T, E, K, score, renorm, scale, topk_ids, gate_w,
                 err, uep_stream(stream)};
  return dtype == UEP_F32 ? gt_launch<float>(c) : gt_launch<uint16_t>(c);
}

extern "C" uep_status uep_gate_grad(const float* dgate_w, const void* logits, int32_t dtype,
                                    const int32_t* topk_ids, const float* gate_w, int32_t R,
                                    int32_t T, int32_t E, int32_t K, int32_t score,
                                    int32_t renorm, float scale, void* dlogits, int32_t* err,
                                    void* stream) {
  const uep_status st = gt_check(logits, dtype, R, T, E, K, score, scale);
  if (st != UEP_OK) return st;
  if (T == 0) return UEP_OK;
  if (!dgate_w || !topk_ids || !gate_w || !dlogits) return UEP_EINVAL;
  const int64_t n_tok = (int64_t)R * T;
  const int64_t bytes = n_tok * E * (dtype == UEP_F32 ? 4 : 2), slots = n_tok * K * 4;
  if (uep_overlap({dlogits, bytes},
                  {{logits, bytes}, {dgate_w, slots}, {topk_ids, slots}, {gate_w, slots}}))
    return UEP_EINVAL;
  int lg_kp = 0;
  while ((1 << lg_kp) < K) ++lg_kp;
  const int64_t n_grp = (n_tok + (kWave >> lg_kp) - 1) / (kWave >> lg_kp);
  const unsigned blocks = (unsigned)std::min<int64_t>(
      (n_grp + kGtTokPerBlock - 1) / kGtTokPerBlock, kGtGradBlocks);
  const uint32_t e_magic = (uint32_t)(((1ull << 32) + E - 1) / E);
  const bool dense = score == UEP_GATE_SOFTMAX && !renorm;
  const uintptr_t size = dtype == UEP_F32 ? 4 : 2;
  // a dense gradient reads in the units that it writes, of at most two rows each
  const int vec = reinterpret_cast<uintptr_t>(dlogits) % 16 == 0 &&
                  (!dense || (reinterpret_cast<uintptr_t>(logits) % 16 == 0 && E * size >= 16));
  hipStream_t s = uep_stream(stream);
#define UEP_GATE_GRAD(T, DENSE)                                                                  \
  hipLaunchKernelGGL((gate_grad_kernel<T, DENSE>), dim3(blocks), dim3(kGtThreads), 0, s, dgate_w, \
                     static_cast<const T*>(logits), topk_ids, gate_w, n_tok, E, e_magic, K, lg_kp, \
                     score, renorm, scale, vec, static_cast<T*>(dlogits), err)
  if (dtype == UEP_F32) {
    if (dense) UEP_GATE_GRAD(float, true);
    else UEP_GATE_GRAD(float, false);
  } else {
    if (dense) UEP_GATE_GRAD(uint16_t, true);
    else UEP_GATE_GRAD(uint16_t, false);
  }
#undef UEP_GATE_GRAD
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}
