// Router gate and its gradient (uep.h: uep_gate, uep_gate_grad).
//
// Selection runs on 64-bit keys that order by (score, lowest id): an fp32 score widened
// to double is exact and leaves 29 zero mantissa bits, which take the expert id, inverted
// for positive scores (adding low bits to a positive double raises it, to a negative one
// lowers it).  Keys are distinct, so one maximum names both the winner and its id.
#include "common.h"

namespace uep {

constexpr int kGtThreads = 256;
constexpr int kGtTokPerBlock = kGtThreads / kWave;
constexpr int kGtMaxE = 4096;

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

__device__ __forceinline__ float gt_sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

constexpr double kGtNone = -__builtin_inf();

__device__ __forceinline__ double gt_key(float f, int e) {
  const uint64_t u = (uint64_t)__double_as_longlong((double)(f + 0.0f));   // -0 counts as +0
  return __longlong_as_double((long long)(u | ((int64_t)u < 0 ? (uint64_t)e
                                                              : (uint64_t)(kGtMaxE - 1 - e))));
}
__device__ __forceinline__ int gt_key_id(double k) {
  const uint64_t u = (uint64_t)__double_as_longlong(k);
  const int low = (int)(u & (kGtMaxE - 1));
  return (int64_t)u < 0 ? low : kGtMaxE - 1 - low;
}

__device__ __forceinline__ double gt_wave_max(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const double w = __shfl_xor(v, o, kWave);
    v = w > v ? w : v;
  }
  return v;
}
__device__ __forceinline__ float gt_wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// One wave per token, kVpt experts per lane (expert j * 64 + lane); K rounds of a wave
// maximum over the keys left.
template <typename T, int kVpt>
__global__ __launch_bounds__(kGtThreads) void gate_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ batch_size, int64_t n_tok, int tok_per_rank, int E, int K,
    int score, int renorm, float scale, int32_t* __restrict__ topk_ids,
    float* __restrict__ gate_w, int32_t* err) {
  const int lane = threadIdx.x % kWave;
  const int64_t g = (int64_t)blockIdx.x * kGtTokPerBlock + threadIdx.x / kWave;
  if (g >= n_tok) return;
  if (batch_size && (int)(g % tok_per_rank) >= batch_size[g / tok_per_rank]) {
    if (lane < K) {
      topk_ids[g * K + lane] = -1;
      gate_w[g * K + lane] = 0.0f;
    }
    return;
  }
  double key[kVpt];
  float val[kVpt];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kVpt; ++j) {
    const int e = j * kWave + lane;
    const float x = e < E ? gt_load(logits, g * E + e) : -__builtin_inff();
    bad |= gt_bad(x);
    val[j] = x;
    key[j] = kGtNone;
    if (gt_finite(x)) {
      const float f = score ? gt_sigmoid(x) + (bias ? bias[e] : 0.0f) : x;
      bad |= gt_bad(f);
      if (gt_finite(f)) key[j] = gt_key(f, e);
    }
  }
  if (ballot(bad) && lane == 0) set_err(err, UEP_ERR_LOGIT);
  int id_mine = -1;
  float top = 0.0f;
  for (int k = 0; k < K; ++k) {
    double m = key[0];
#pragma unroll
    for (int j = 1; j < kVpt; ++j) m = key[j] > m ? key[j] : m;
    m = gt_wave_max(m);
    if (m == kGtNone) break;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) key[j] = key[j] == m ? kGtNone : key[j];
    if (k == 0) top = (float)m;   // softmax: the largest logit, up to the id bits (a shift)
    if (lane == k) id_mine = gt_key_id(m);
  }
  const bool on = id_mine >= 0;
  const float l = on ? gt_load(logits, g * E + id_mine) : 0.0f;
  float s = on ? (score ? gt_sigmoid(l) : expf(l - top)) : 0.0f;
  float total = 1.0f;
  if (renorm) {
    total = gt_wave_sum(s);
  } else if (!score) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) z += gt_finite(val[j]) ? expf(val[j] - top) : 0.0f;
    total = gt_wave_sum(z);
  }
  if (lane < K) {
    topk_ids[g * K + lane] = id_mine;
    gate_w[g * K + lane] = s > 0.0f ? scale * (s / total) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void gt_store(T* p, int64_t i, float v);
template <>
__device__ __forceinline__ void gt_store<float>(float* p, int64_t i, float v) { p[i] = v; }
template <>
__device__ __forceinline__ void gt_store<uint16_t>(uint16_t* p, int64_t i, float v) {
  p[i] = (uint16_t)f32_to_bf16(v);
}

// One wave per token: lane k holds slot k, then the wave writes the row.
template <typename T>
__global__ __launch_bounds__(kGtThreads) void gate_grad_kernel(
    const float* __restrict__ dgate_w, const T* __restrict__ logits,
    const int32_t* __restrict__ topk_ids, const float* __restrict__ gate_w, int64_t n_tok, int E,
    int K, int score, int renorm, float scale, T* __restrict__ dlogits, int32_t* err) {
  const int lane = threadIdx.x % kWave;
  const int64_t g = (int64_t)blockIdx.x * kGtTokPerBlock + threadIdx.x / kWave;
  if (g >= n_tok) return;
  int id = lane < K ? topk_ids[g * K + lane] : -1;
  const bool bad = id < -1 || id >= E;
  if (ballot(bad) && lane == 0) set_err(err, UEP_ERR_ID_RANGE);
  if (bad) id = -1;
  const float gk = id >= 0 ? scale * dgate_w[g * K + lane] : 0.0f;
  const float u = id >= 0 ? gate_w[g * K + lane] / scale : 0.0f;
  const float dot = gt_wave_sum(u * gk);
  float d;
  if (score)
    d = renorm ? (id >= 0 ? u * (1.0f - gt_sigmoid(gt_load(logits, g * E + id))) * (gk - dot) : 0.0f)
               : u * (1.0f - u) * gk;
  else
    d = renorm ? u * (gk - dot) : gk;
  const bool dense = !score && !renorm;
  float m = -__builtin_inff(), z = 0.0f;
  if (dense && ballot(id >= 0)) {
    for (int e = lane; e < E; e += kWave) {
      const float x = gt_load(logits, g * E + e);
      if (gt_finite(x)) m = fmaxf(m, x);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    for (int e = lane; e < E; e += kWave) {
      const float x = gt_load(logits, g * E + e);
      if (gt_finite(x)) z += expf(x - m);
    }
    z = gt_wave_sum(z);
  }
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int e = e0 + lane;
    float v = 0.0f;
    for (int k = 0; k < K; ++k) {
      const int idk = readlane(id, k);
      const float dk = __int_as_float(readlane(__float_as_int(d), k));
      v = idk == e ? dk : v;
    }
    if (e >= E) continue;
    if (dense && z > 0.0f) {
      const float x = gt_load(logits, g * E + e);
      v = gt_finite(x) ? expf(x - m) / z * (v - dot) : 0.0f;
    }
    gt_store(dlogits, g * E + e, v);
  }
}

static uep_status gt_check(const void* logits, int32_t dtype, int32_t R, int32_t T, int32_t E,
                           int32_t K, int32_t score, float scale) {
  if (R <= 0 || T < 0 || E <= 0 || K <= 0) return UEP_EINVAL;
  if (dtype != UEP_F32 && dtype != UEP_BF16) return UEP_EINVAL;
  if (score != UEP_GATE_SOFTMAX && score != UEP_GATE_SIGMOID) return UEP_EINVAL;
  if (!(scale > -__builtin_inff() && scale < __builtin_inff()) || scale == 0.0f) return UEP_EINVAL;
  if (R > 64 || E > kGtMaxE || K > 64 || K > E || (int64_t)R * T * K >= (1ll << 31))
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
  const unsigned blocks = (unsigned)((n_tok + kGtTokPerBlock - 1) / kGtTokPerBlock);
  hipStream_t s = uep_stream(stream);
#define UEP_GATE(VPT)                                                                         \
  do {                                                                                        \
    if (dtype == UEP_F32)                                                                     \
      hipLaunchKernelGGL((gate_kernel<float, VPT>), dim3(blocks), dim3(kGtThreads), 0, s,      \
                         static_cast<const float*>(logits), bias, batch_size, n_tok, T, E, K,  \
                         score, renorm, scale, topk_ids, gate_w, err);                         \
    else                                                                                      \
      hipLaunchKernelGGL((gate_kernel<uint16_t, VPT>), dim3(blocks), dim3(kGtThreads), 0, s,   \
                         static_cast<const uint16_t*>(logits), bias, batch_size, n_tok, T, E,  \
                         K, score, renorm, scale, topk_ids, gate_w, err);                      \
  } while (0)
  if (E <= 128) UEP_GATE(2);
  else if (E <= 256) UEP_GATE(4);
  else if (E <= 512) UEP_GATE(8);
  else if (E <= 1024) UEP_GATE(16);
  else UEP_GATE(64);
#undef UEP_GATE
  UEP_CHECK_LAUNCH();
  return UEP_OK;
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
  const unsigned blocks = (unsigned)((n_tok + kGtTokPerBlock - 1) / kGtTokPerBlock);
  hipStream_t s = uep_stream(stream);
  if (dtype == UEP_F32)
    hipLaunchKernelGGL(gate_grad_kernel<float>, dim3(blocks), dim3(kGtThreads), 0, s, dgate_w,
                       static_cast<const float*>(logits), topk_ids, gate_w, n_tok, E, K, score,
                       renorm, scale, static_cast<float*>(dlogits), err);
  else
    hipLaunchKernelGGL(gate_grad_kernel<uint16_t>, dim3(blocks), dim3(kGtThreads), 0, s, dgate_w,
                       static_cast<const uint16_t*>(logits), topk_ids, gate_w, n_tok, E, K, score,
                       renorm, scale, static_cast<uint16_t*>(dlogits), err);
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}
