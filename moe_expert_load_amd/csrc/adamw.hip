// AdamW over many tensors in one launch, states in fp32 or 8 bits (uep.h: AdamW).
//
// HBM-bound: every element's parameter, gradient and states are read once and written
// once.  The plan lists the work as tiles of 4096 elements of one tensor each; a
// 256-thread workgroup takes one tile, each wave four chunks of 256 consecutive elements
// (four per lane: 16-byte accesses for fp32, 8 for bf16, 4 for the codes).  A chunk is a
// block of the 8-bit states, so a block's largest level is one reduction over a wave.
#include <stdlib.h>

#include "common.h"

namespace uep {

constexpr int kAwThreads = 256;
constexpr int kAwWaves = kAwThreads / kWave;
constexpr int kAwChunk = 4 * kWave;               // elements of a wave's chunk = state block
constexpr int kAwUnroll = 4;                      // chunks per wave
constexpr int kAwTile = kAwChunk * kAwWaves * kAwUnroll;
constexpr int32_t kAwMagic = 0x41645757;
constexpr int kAwMaxLevel = 0x7F7;                // largest finite: exponent 254, mantissa 7
constexpr int64_t kAwMaxElems = 1ll << 33;
constexpr int kAwMaxTensors = 65535;

struct AwHeader {
  int32_t magic, count, param_dtype, grad_dtype, state_bits, n_tiles, pad[2];
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

// Four consecutive elements; kFull: all there and the pointer aligned for one access.
template <bool kFull, typename T>
__device__ __forceinline__ void aw_load(const T* p, int left, T (&v)[4]) {
  if constexpr (kFull) {
    typedef T vec __attribute__((ext_vector_type(4)));
    const vec x = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = x[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < left ? p[j] : T(0);
  }
}
template <bool kFull, typename T>
__device__ __forceinline__ void aw_store(T* p, int left, const T (&v)[4]) {
  if constexpr (kFull) {
    typedef T vec __attribute__((ext_vector_type(4)));
    vec x;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = v[j];
    *reinterpret_cast<vec*>(p) = x;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) p[j] = v[j];
  }
}

__device__ __forceinline__ float aw_f32(float x) { return x; }
__device__ __forceinline__ float aw_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// Level of |x| after adding `dither` / 2^16 of a step; 0 for x = 0.
__device__ __forceinline__ int aw_level(float x, uint32_t dither) {
  const uint32_t bits = __float_as_uint(x) & 0x7FFFFFFFu;
  const int level = (int)((bits + (dither << 4)) >> 20);
  return bits ? min(level, kAwMaxLevel) : 0;
}
__device__ __forceinline__ float aw_value(int level) {
  return __uint_as_float((uint32_t)max(level, 0) << 20);
}
__device__ __forceinline__ float aw_decode_m(uint32_t code, int top) {
  const int size = code & 127;
  const float x = size ? aw_value(size - 127 + top) : 0.0f;
  return code & 128 ? -x : x;
}
__device__ __forceinline__ float aw_decode_v(uint32_t code, int top) {
  return code ? aw_value((int)code - 255 + top) : 0.0f;
}

struct AwScalars {
  float decay, rate, root2, scale;                // 1 - lr wd, lr / bc1, sqrt(bc2), sched[1]
};

template <typename P, typename G, bool k8, bool kFull>
__device__ __forceinline__ bool aw_tile(const AwTensor& t, int64_t base, const AwScalars& c,
                                        const AwArgs& a, uint32_t key) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const P* p_in = static_cast<const P*>(t.t.param);
  bool bad = false;
  for (int u = 0; u < kAwUnroll; ++u) {
    const int64_t chunk = base + (int64_t)(u * kAwWaves + wave) * kAwChunk;
    if (chunk >= t.t.n) break;
    const int64_t i = chunk + lane * 4;
    const int left = (int)min((int64_t)4, t.t.n - i);     // <= 0: past the end
    P p[4];
    G g[4];
    aw_load<kFull>(p_in + i, left, p);
    aw_load<kFull>(static_cast<const G*>(t.t.grad) + i, left, g);
    float m[4], v[4];
    if constexpr (k8) {
      uint8_t mc[4], vc[4];
      aw_load<kFull>(static_cast<const uint8_t*>(t.t.m) + i, left, mc);
      aw_load<kFull>(static_cast<const uint8_t*>(t.t.v) + i, left, vc);
      const int tops = t.t.tops[chunk / kAwChunk];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = aw_decode_m(mc[j], tops & 0xFFFF);
        v[j] = aw_decode_v(vc[j], tops >> 16);
      }
    } else {
      aw_load<kFull>(static_cast<const float*>(t.t.m) + i, left, m);
      aw_load<kFull>(static_cast<const float*>(t.t.v) + i, left, v);
    }
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float gj = aw_f32(g[j]) * c.scale;
      const bool off = (__float_as_uint(gj) & 0x7F800000u) == 0x7F800000u;
      bad |= off;
      gj = off ? 0.0f : gj;
      m[j] = m[j] * a.b1 + gj * a.ob1;
      v[j] = v[j] * a.b2 + gj * gj * a.ob2;
      w[j] = aw_f32(p[j]) * c.decay - c.rate * (m[j] / (sqrtf(v[j]) / c.root2 + a.eps));
    }
    uint32_t r[6] = {0};
    if constexpr (k8 || sizeof(P) == 2) {
      r[0] = aw_mix((uint32_t)(i >> 2) * 0x9E3779B9u ^ key);
#pragma unroll
      for (int j = 1; j < 6; ++j) r[j] = aw_next(r[j - 1]);
    }
    if constexpr (sizeof(P) == 2) {
      uint16_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t bits = __float_as_uint(w[j]);
        const uint32_t d = j & 1 ? r[j / 2] >> 16 : r[j / 2] & 0xFFFFu;
        // an infinity or NaN is cut as it is (a NaN's upper bits are set)
        o[j] = (uint16_t)(((bits & 0x7F800000u) == 0x7F800000u ? bits : bits + d) >> 16);
      }
      aw_store<kFull>(static_cast<uint16_t*>(t.t.param) + i, left, o);
    } else {
      aw_store<kFull>(static_cast<float*>(t.t.param) + i, left, w);
      if (t.t.copy) {
        uint16_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (uint16_t)f32_to_bf16(w[j]);
        aw_store<kFull>(t.t.copy + i, left, o);
      }
    }
    if constexpr (k8) {
      int lm[4], lv[4], top_m = 0, top_v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool on = kFull || j < left;
        lm[j] = on ? aw_level(m[j], r[2 + j] & 0xFFFFu) : 0;
        lv[j] = on ? aw_level(v[j], r[2 + j] >> 16) : 0;
        top_m = max(top_m, lm[j]);
        top_v = max(top_v, lv[j]);
      }
      top_m = wave_max(top_m);
      top_v = wave_max(top_v);
      uint8_t mc[4], vc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int cm = max(lm[j] - top_m + 127, 0);
        mc[j] = (uint8_t)(m[j] != 0.0f && cm ? cm | (m[j] < 0.0f ? 128 : 0) : 0);
        vc[j] = (uint8_t)(v[j] > 0.0f ? max(lv[j] - top_v + 255, 1) : 0);
      }
      aw_store<kFull>(static_cast<uint8_t*>(t.t.m) + i, left, mc);
      aw_store<kFull>(static_cast<uint8_t*>(t.t.v) + i, left, vc);
      if (lane == 0) t.t.tops[chunk / kAwChunk] = top_m | top_v << 16;
    } else {
      aw_store<kFull>(static_cast<float*>(t.t.m) + i, left, m);
      aw_store<kFull>(static_cast<float*>(t.t.v) + i, left, v);
    }
  }
  return bad;
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
  const int64_t base = ((int64_t)blockIdx.x - x.first_tile) * kAwTile;
  const float lr = sched[0] * x.t.lr_scale;
  // 1 - beta^t = -expm1(t log beta), in double: 1 - 0.999^1 in fp32 is good to 5 digits only
  AwScalars c;
  c.decay = 1.0f - lr * x.t.weight_decay;
  c.rate = lr / (float)-expm1(t * a.log_b1);
  c.root2 = sqrtf((float)-expm1(t * a.log_b2));
  c.scale = sched[1];
  const uint32_t key = aw_mix(aw_mix((uint32_t)t * 0x9E3779B9u + a.seed) ^ (uint32_t)(q + 1));
  const bool full = x.vec && base + kAwTile <= x.t.n;
  const bool bad = full ? aw_tile<P, G, k8, true>(x, base, c, a, key)
                        : aw_tile<P, G, k8, false>(x, base, c, a, key);
  if (ballot(bad) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_GRAD);
}

template <typename T>
__global__ __launch_bounds__(kAwThreads) void adamw_decode_kernel(
    const uint8_t* __restrict__ mc, const uint8_t* __restrict__ vc,
    const int32_t* __restrict__ tops, int64_t n, T* __restrict__ m, T* __restrict__ v) {
  const int64_t i = (int64_t)blockIdx.x * kAwThreads + threadIdx.x;
  if (i >= n) return;
  const int top = tops[i / kAwChunk];
  const float a = aw_decode_m(mc[i], top & 0xFFFF), b = aw_decode_v(vc[i], top >> 16);
  if constexpr (sizeof(T) == 4) {
    m[i] = a;
    v[i] = b;
  } else {
    m[i] = (T)(__float_as_uint(a) >> 16);
    v[i] = (T)(__float_as_uint(b) >> 16);
  }
}

static int64_t aw_tiles(int64_t n) { return (n + kAwTile - 1) / kAwTile; }

// Host table check: UEP_OK and the number of tiles, or why not.
static uep_status aw_count(const uep_adamw_tensor* t, int32_t count, int64_t* tiles) {
  if (count < 0 || (count > 0 && !t)) return UEP_EINVAL;
  if (count > kAwMaxTensors) return UEP_EGEOM;
  *tiles = 0;
  for (int32_t q = 0; q < count; ++q) {
    if (t[q].n < 0) return UEP_EINVAL;
    if (t[q].n > kAwMaxElems) return UEP_EGEOM;
    *tiles += aw_tiles(t[q].n);
  }
  return *tiles < (1 << 24) ? UEP_OK : UEP_EGEOM;   // a launch holds below 2^32 threads
}

static size_t aw_bytes(int32_t count, int64_t tiles) {
  return sizeof(AwHeader) + sizeof(AwTensor) * (size_t)count + sizeof(int32_t) * (size_t)tiles;
}

}  // namespace uep

using namespace uep;

extern "C" size_t uep_adamw_plan_size(const uep_adamw_tensor* tensors_host, int32_t count) {
  int64_t tiles = 0;
  return aw_count(tensors_host, count, &tiles) == UEP_OK ? aw_bytes(count, tiles) : 0;
}

extern "C" uep_status uep_adamw_prepare(const uep_adamw_tensor* tensors_host, int32_t count,
                                        int32_t param_dtype, int32_t grad_dtype,
                                        int32_t state_bits, void* plan, size_t plan_bytes,
                                        int64_t* n_tiles, void* stream) {
  int64_t tiles = 0;
  const uep_status st = aw_count(tensors_host, count, &tiles);
  if (st != UEP_OK) return st;
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
  AwTensor* d = reinterpret_cast<AwTensor*>(w + sizeof(AwHeader));
  int32_t* tile = reinterpret_cast<int32_t*>(d + count);
  int64_t at = 0;
  for (int32_t q = 0; q < count; ++q) {
    const uep_adamw_tensor& t = tensors_host[q];
    d[q].t = t;
    d[q].first_tile = at;
    d[q].vec = (uintptr_t)t.param % (4 * p_size) == 0 && (uintptr_t)t.grad % (4 * g_size) == 0 &&
               (uintptr_t)t.m % (4 * s_size) == 0 && (uintptr_t)t.v % (4 * s_size) == 0 &&
               (uintptr_t)t.copy % 8 == 0;
    for (int64_t k = aw_tiles(t.n); k > 0; --k) tile[at++] = q;
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
      !(eps > 0.0 && eps < __builtin_inf()))
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
  const int64_t blocks = (n + kAwThreads - 1) / kAwThreads;
  if (blocks >= (1 << 24)) return UEP_EGEOM;
  hipStream_t s = uep_stream(stream);
  if (dtype == UEP_F32)
    hipLaunchKernelGGL(adamw_decode_kernel<float>, dim3((unsigned)blocks), dim3(kAwThreads), 0, s,
                       m_codes, v_codes, tops, n, static_cast<float*>(m), static_cast<float*>(v));
  else
    hipLaunchKernelGGL(adamw_decode_kernel<uint16_t>, dim3((unsigned)blocks), dim3(kAwThreads), 0,
                       s, m_codes, v_codes, tops, n, static_cast<uint16_t*>(m),
                       static_cast<uint16_t*>(v));
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}
