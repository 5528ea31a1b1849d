// bf16 rows as 8-bit integers with a scale each (uep.h: uep_quant_rows, uep_permute_quant).
//
// A row is read once into registers: its largest magnitude by packed 16-bit maxima (bf16
// magnitudes order like their bits), then every element by one multiply-add that rounds to the
// nearest integer.  The integer is that of the exact quotient x / scale: the product with the
// reciprocal is off by a few units in the last place, which only shows next to a border, and the
// remainder x - q scale is exact (x has 8 bits and q scale at most 31, of which the subtraction
// leaves no more than 24), so a remainder of half a step or more tells the elements to mend.
// Bound by HBM: 2 bytes read and 1 written per element.
#include <algorithm>

#include "common.h"
#include "numeric.h"

namespace uep {

constexpr int kQrBlock = 256;
constexpr int kQrMaxH = 65536;
constexpr int64_t kQrLaunch = 1ll << 21;         // rows of a launch, at most 1024 threads each
constexpr float kQrMagic = 12582912.0f;          // 1.5 * 2^23: its lowest byte takes an integer
constexpr float kQrLeast = 0x1p-126f;            // smallest scale
constexpr uint32_t kQrInf = 0x7F80u;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t qr_max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}

// largest of the row's magnitudes (bf16 bits) over the kThreads threads of the row
template <int kThreads>
__device__ __forceinline__ uint32_t qr_row_max(uint32_t m2, int32_t (&lds)[16]) {
  int m = (int)max(m2 & 0xFFFFu, m2 >> 16);
  m = wave_max(m);
  if constexpr (kThreads > kWave) {
    __syncthreads();                             // the last use of lds
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) m = max(m, lds[w]);
  }
  return (uint32_t)m;
}

// Threads `sub` of kThreads hold the vectors sub + i * kThreads of 16 elements.
template <int kThreads, int kNV, bool kDispatch>
__global__ __launch_bounds__(kThreads > kQrBlock ? kThreads : kQrBlock) void quant_rows_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ dest_row,
    const int32_t* __restrict__ live_rows, int64_t row0, int64_t row1, int K, int H,
    int8_t* __restrict__ q, float* __restrict__ scale, int64_t q_rows, int32_t* err) {
  constexpr int kBlock = kThreads > kQrBlock ? kThreads : kQrBlock;
  __shared__ int32_t lds[16];
  const int sub = threadIdx.x % kThreads, n_vec = H / 16;
  const int64_t row = row0 + (int64_t)blockIdx.x * (kBlock / kThreads) + threadIdx.x / kThreads;
  // whole waves, and whole blocks where they share a row
  if (row >= row1 || (!kDispatch && live_rows && row >= *live_rows)) return;
  int dest = -1;
  if constexpr (kDispatch) {
    const int k = threadIdx.x % kWave;
    dest = checked_row(k < K ? dest_row[row * K + k] : -1, q_rows, err);
    if (!ballot(dest >= 0)) return;
  }
  u32x4 w[kNV][2];
  const u32x4* src = reinterpret_cast<const u32x4*>(x + row * H);
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int v = sub + i * kThreads;
    w[i][0] = w[i][1] = u32x4{0, 0, 0, 0};
    if (v < n_vec) {
      w[i][0] = src[2 * v];
      w[i][1] = src[2 * v + 1];
    }
  }
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m2 = qr_max2(m2, w[i][j / 4][j % 4] & 0x7FFF7FFFu);
  uint32_t top = qr_row_max<kThreads>(m2, lds);
  const bool odd = top >= kQrInf;                // the row holds a NaN or an infinity
  if (odd) {
    if (sub == 0) set_err(err, UEP_ERR_VALUE);
    m2 = 0;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = w[i][j / 4][j % 4] & 0x7FFF7FFFu;
        m2 = qr_max2(m2, ((a & 0xFFFFu) < kQrInf ? a & 0xFFFFu : 0) |
                             ((a >> 16) < kQrInf ? a & 0xFFFF0000u : 0));
      }
    top = qr_row_max<kThreads>(m2, lds);
  }
  const float s = fmaxf(__uint_as_float(top << 16) / 127.0f, kQrLeast);
  const float inv = 1.0f / s, half = 0.5f * s;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int v = sub + i * kThreads;
    u32x4 code;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4], t[4], off = 0.0f;
#pragma unroll
      for (int l = 0; l < 4; ++l) {
        const int e = 4 * j + l;
        const uint32_t pair = w[i][e / 8][e / 2 % 4];
        f[l] = e & 1 ? bf16_hi(pair) : bf16_lo(pair);
        t[l] = fmaf(f[l], inv, kQrMagic);
        off = fmaxf(off, fabsf(fmaf(kQrMagic - t[l], s, f[l])));
      }
      if (ballot(off >= half) || odd) {          // next to a border, or not finite
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          const float r = fmaf(kQrMagic - t[l], s, f[l]);
          const bool tie = fabsf(r) == half && (__float_as_uint(t[l]) & 1u);
          if (fabsf(r) > half || tie) t[l] += copysignf(1.0f, r);
          if (odd) {
            if (fabsf(f[l]) == __builtin_inff()) t[l] = kQrMagic + copysignf(127.0f, f[l]);
            if (f[l] != f[l]) t[l] = kQrMagic;
          }
        }
      }
      const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[1]), __float_as_uint(t[0]), 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[3]), __float_as_uint(t[2]), 0x0C0C0400u);
      code[j] = lo | (hi << 16);
    }
    if (v >= n_vec) continue;
    if constexpr (kDispatch) {
      for (int k = 0; k < K; ++k) {
        const int d = readlane(dest, k);
        if (d >= 0) *reinterpret_cast<u32x4*>(q + (int64_t)d * H + 16 * v) = code;
      }
    } else {
      *reinterpret_cast<u32x4*>(q + row * H + 16 * v) = code;
    }
  }
  if constexpr (kDispatch) {
    if (sub < kWave && dest >= 0) scale[dest] = s;
  } else {
    if (sub == 0) scale[row] = s;
  }
}

struct QrCall {
  const uint16_t* x;
  const int32_t *dest_row, *live_rows;
  int64_t row0, row1;
  int K, H;
  int8_t* q;
  float* scale;
  int64_t q_rows;
  int32_t* err;
  hipStream_t stream;
};

template <int kThreads, int kNV>
static uep_status qr_launch(const QrCall& c) {
  constexpr int kBlock = kThreads > kQrBlock ? kThreads : kQrBlock;
  constexpr int kRows = kBlock / kThreads;
  for (int64_t a = c.row0; a < c.row1; a += kQrLaunch) {
    const int64_t b = std::min(c.row1, a + kQrLaunch);
    const dim3 grid((unsigned)((b - a + kRows - 1) / kRows));
    if (c.dest_row)
      hipLaunchKernelGGL((quant_rows_kernel<kThreads, kNV, true>), grid, dim3(kBlock), 0, c.stream,
                         c.x, c.dest_row, c.live_rows, a, b, c.K, c.H, c.q, c.scale, c.q_rows,
                         c.err);
    else
      hipLaunchKernelGGL((quant_rows_kernel<kThreads, kNV, false>), grid, dim3(kBlock), 0,
                         c.stream, c.x, c.dest_row, c.live_rows, a, b, c.K, c.H, c.q, c.scale,
                         c.q_rows, c.err);
    UEP_CHECK_LAUNCH();
  }
  return UEP_OK;
}

// As few threads as keep a row in four vectors each: a wave needs no barrier.
static uep_status qr_run(const QrCall& c) {
  const int v = c.H / 16;
  if (v <= 64) return qr_launch<64, 1>(c);
  if (v <= 128) return qr_launch<64, 2>(c);
  if (v <= 256) return qr_launch<256, 1>(c);
  if (v <= 512) return qr_launch<256, 2>(c);
  if (v <= 1024) return qr_launch<256, 4>(c);
  if (v <= 2048) return qr_launch<1024, 2>(c);
  return qr_launch<1024, 4>(c);
}

}  // namespace uep

using namespace uep;

static bool qr_odd(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return true;
  return false;
}

extern "C" uep_status uep_quant_rows(const uint16_t* x, int64_t rows, int32_t H,
                                     const int32_t* live_rows, int8_t* q, float* scale,
                                     int32_t* err, void* stream) {
  if (rows < 0 || H <= 0) return UEP_EINVAL;
  if (H % 16 != 0 || H > kQrMaxH || rows >= (1ll << 31)) return UEP_EGEOM;
  if (rows == 0) return UEP_OK;
  if (!x || !q || !scale) return UEP_EINVAL;
  if (qr_odd({x, q})) return UEP_EGEOM;
  const UepBytes src{x, rows * H * 2}, codes{q, rows * H}, s{scale, rows * 4}, n{live_rows, 4};
  if (uep_overlap(codes, {src, s, n}) || uep_overlap(s, {src, n})) return UEP_EINVAL;
  const QrCall c{x, nullptr, live_rows, 0, rows, 0, H, q, scale, rows, err, uep_stream(stream)};
  return qr_run(c);
}

extern "C" uep_status uep_permute_quant(const uint16_t* x, const int32_t* dest_row, int32_t R,
                                        int32_t T, int32_t K, int32_t H, int32_t r_begin,
                                        int32_t r_end, int8_t* q, float* scale,
                                        int64_t out_rows, int32_t* err, void* stream) {
  if (R <= 0 || T < 0 || K <= 0 || H <= 0 || out_rows < 0 || r_begin < 0 || r_end < r_begin ||
      r_end > R)
    return UEP_EINVAL;
  if (R > 64 || K > 64 || H % 16 != 0 || H > kQrMaxH || (int64_t)R * T * K >= (1ll << 31) ||
      out_rows >= (1ll << 31))
    return UEP_EGEOM;
  if (T == 0 || r_begin == r_end) return UEP_OK;
  if (!x || !dest_row || (out_rows > 0 && (!q || !scale))) return UEP_EINVAL;
  if (qr_odd({x, q})) return UEP_EGEOM;
  const int64_t n = (int64_t)R * T;
  const UepBytes src{x, n * H * 2}, to{dest_row, n * K * 4};
  const UepBytes codes{q, out_rows * H}, s{scale, out_rows * 4};
  if (uep_overlap(codes, {src, to, s}) || uep_overlap(s, {src, to})) return UEP_EINVAL;
  const QrCall c{x, dest_row, nullptr, (int64_t)r_begin * T, (int64_t)r_end * T, K, H, q, scale,
                 out_rows, err, uep_stream(stream)};
  return qr_run(c);
}
