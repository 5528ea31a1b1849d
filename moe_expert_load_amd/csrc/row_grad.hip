// Gradient of the combine (uep.h: uep_combine_grad): every dispatch row gets its token's
// output gradient times its weight, and every weight the dot product of that gradient
// with the expert output in its row,
//   dout[d] = bf16(w[g][k] * dy[g]),   dgate_w[g][k] = <dy[g], out[d]>,   d = dest_row[g][k].
//
// One wave per token on the XCD-aware block map, as in the combine: the token's gradient
// is read once into registers, slice by slice (8 x 16 B per lane, 8 KiB per wave), and
// serves its K rows; lanes 0..K-1 hold rows, weights and the running dot products.  Row k
// of `out` is read before row k of dout is written, by the same wave, so that both may be
// one buffer.
#include "common.h"

namespace uep {

constexpr int kRgThreads = 256;
constexpr int kRgTokPerBlock = kRgThreads / kWave;
constexpr int kRgVec = 8;     // 16-byte vectors per lane per slice
// Up to this many tokens, which leave SIMDs without a wave, a token's slots go to a wave each
// instead of one after the other to one.
constexpr int64_t kRgFew = 512;

// Rows of slot k: the vectors of [v0, v0 + kRgVec * kWave) of `base`'s row d, none if d < 0.
__device__ __forceinline__ span_t rg_row(const u32x4* base, int d, int nvec) {
  return span_of(base + (int64_t)max(d, 0) * nvec, d < 0 ? 0 : (int64_t)nvec * 16);
}

template <bool kDot>
__global__ __launch_bounds__(kRgThreads) void combine_grad_kernel(
    const u32x4* __restrict__ dy, const u32x4* out, const int32_t* __restrict__ dest_row,
    const float* __restrict__ gate_w, u32x4* dout, float* __restrict__ dgate_w, int64_t out_rows,
    int64_t g0, int64_t g1, int K, int nvec, int parts, int32_t* err) {
  const int lane = threadIdx.x % kWave;
  const int64_t b = xcd_block(blockIdx.x, gridDim.x);
  const int64_t wv = b * kRgTokPerBlock + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t g = g0 + (parts == 1 ? wv : (int)wv / parts);
  if (g >= g1) return;
  const int k_begin = parts == 1 ? 0 : (int)wv % parts, k_end = parts == 1 ? K : k_begin + 1;
  const bool mine = lane >= k_begin && lane < k_end;
  const int d_mine = checked_row(mine ? dest_row[g * K + lane] : -1, out_rows, err);
  const int w_mine = mine ? __float_as_int(gate_w[g * K + lane]) : 0;
  const span_t src = span_of(dy + g * nvec, (int64_t)nvec * 16);
  float dot_mine = 0.0f;
  for (int v0 = 0; v0 < nvec; v0 += kRgVec * kWave) {
    u32x4 grad[kRgVec], y[2][kRgVec];
    auto fetch = [&](int k, u32x4 (&to)[kRgVec]) {
      const span_t row = rg_row(out, readlane(d_mine, k), nvec);
#pragma unroll
      for (int u = 0; u < kRgVec; ++u) to[u] = stream_load(row, (v0 + u * kWave + lane) * 16);
    };
    auto slot = [&](int k, const u32x4 (&from)[kRgVec]) {
      const float w = __int_as_float(readlane(w_mine, k));
      if (kDot) {
        float dot = 0.0f;
#pragma unroll
        for (int u = 0; u < kRgVec; ++u)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            dot = fmaf(bf16_lo(grad[u][c]), bf16_lo(from[u][c]), dot);
            dot = fmaf(bf16_hi(grad[u][c]), bf16_hi(from[u][c]), dot);
          }
        dot = wave_sum_f32(dot);
        if (lane == k) dot_mine += dot;
      }
      const span_t dst = rg_row(dout, readlane(d_mine, k), nvec);
#pragma unroll
      for (int u = 0; u < kRgVec; ++u) {
        u32x4 o;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          o[c] = pack_bf16(w * bf16_lo(grad[u][c]), w * bf16_hi(grad[u][c]));
        stream_store(o, dst, (v0 + u * kWave + lane) * 16);
      }
    };
#pragma unroll
    for (int u = 0; u < kRgVec; ++u) grad[u] = stream_load(src, (v0 + u * kWave + lane) * 16);
    if (kDot) fetch(k_begin, y[0]);
    for (int k = k_begin; k < k_end; k += 2) {       // row k + 1 is on its way while k is used
      if (kDot && k + 1 < k_end) fetch(k + 1, y[1]);
      slot(k, y[0]);
      if (k + 1 < k_end) {
        if (kDot && k + 2 < k_end) fetch(k + 2, y[0]);
        slot(k + 1, y[1]);
      }
    }
  }
  // a slot without a row read nothing: 0 (0 times an infinite gradient left a NaN)
  if (kDot && mine) dgate_w[g * K + lane] = d_mine < 0 ? 0.0f : dot_mine;
}

}  // namespace uep

using namespace uep;

extern "C" uep_status uep_combine_grad(const uint16_t* dy, const uint16_t* out, int64_t out_rows,
                                       const int32_t* dest_row, const float* gate_w, int32_t R,
                                       int32_t T, int32_t K, int32_t H, int32_t r_begin,
                                       int32_t r_end, uint16_t* dout, float* dgate_w,
                                       int32_t* err, void* stream) {
  if (R <= 0 || T < 0 || K <= 0 || H <= 0 || out_rows < 0) return UEP_EINVAL;
  if (r_begin < 0 || r_end > R || r_begin > r_end) return UEP_EINVAL;
  if (K > 64 || H % 8 != 0 || H > (1 << 29) || (int64_t)R * T * K >= (1ll << 31))
    return UEP_EGEOM;
  const int64_t g0 = (int64_t)r_begin * T, g1 = (int64_t)r_end * T;
  if (g1 == g0) return UEP_OK;
  if (!dy || !dest_row || !gate_w || !dout || !out != !dgate_w) return UEP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(out) |
       reinterpret_cast<uintptr_t>(dout)) % 16 != 0)
    return UEP_EGEOM;
  const int parts = g1 - g0 <= kRgFew ? K : 1;
  const int64_t blocks = ((g1 - g0) * parts + kRgTokPerBlock - 1) / kRgTokPerBlock;
  auto kernel = out ? combine_grad_kernel<true> : combine_grad_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kRgThreads), 0, uep_stream(stream),
                     reinterpret_cast<const u32x4*>(dy), reinterpret_cast<const u32x4*>(out),
                     dest_row, gate_w, reinterpret_cast<u32x4*>(dout), dgate_w, out_rows, g0, g1,
                     K, H / 8, parts, err);
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}
