// Combine: expert outputs from the per-instance dispatch buffer back to token order
// (Waterfill/LPLB blog, section "背景知识与设计原则": DeepEP's combine brings a
// token's routed-expert outputs back; section "共享专家融合作为启用机制": with shared-
// expert fusion the shared slot is one more column of the same layout and combine).
// The weighted sum with the router weights as input is the standard MoE output:
//   y[g] = bf16( sum over k with dest_row[g][k] >= 0 of  w[g][k] * out[dest_row[g][k]] )
// with each product and each addition rounded in fp32, k ascending from +0.0, no
// fused multiply-add, then nearest-even rounding to bf16.
//
// HBM-bound, the permute in reverse: one wave per output token, 4 tokens per
// 256-thread workgroup on the XCD-aware block map; lanes 0..K-1 hold the token's
// rows and weights, broadcast by readlane.  A row is processed in slices of 4 x 16 B
// per lane (4 KiB per wave); the slices of 4 consecutive k are loaded together
// (non-temporal: every dispatch row is read once; +3 % measured) before they are
// accumulated in order.
//
// uep_permute_grad is the same gather without weights (every copy of a token hands its
// gradient back): the kernel's unweighted form, dx[g] = bf16( sum_k dout[dest_row[g][k]] ).
#include <algorithm>

#include "common.h"
#include "numeric.h"

namespace uep {

constexpr int kCbThreads = 256;
constexpr int kCbTokPerBlock = kCbThreads / kWave;
constexpr int kCbVec = 4;     // 16-byte vectors per lane per slice (8 bf16 each)
// Up to this many tokens, which leave SIMDs without a wave, a token's slices go to up to 16
// waves instead of one after the other to one.  Apart against together (K = 9, 14 KiB rows, in a
// graph): 128 tokens 7.2 against 16.0 us, 512 13.8 / 20.7, 1024 27.8 / 28.6, 2048 58.7 / 56.3.
constexpr int64_t kCbFew = 1024;
constexpr int64_t kCbLaunch = 1ll << 25;   // tokens of one launch, which holds below 2^32 threads

// kVec vectors per lane hold a slice of a row (a whole row where it is shorter than a slice of
// kCbVec); kGroup rows go together: 4, and of short rows (up to 2 KiB) as many as a token has, up
// to 8.  Against four vectors and four rows whatever the row: 65536 tokens of eight 512 B rows
// 120 -> 53 us, of one 1072 B row 52 -> 35; one row at a time of 4 KiB rows loses (91 -> 97).
template <bool kWeighted, int kVec, int kGroup>
__global__ __launch_bounds__(kCbThreads) void combine_kernel(const u32x4* __restrict__ y_disp,
                                                             const int32_t* __restrict__ dest_row,
                                                             const float* __restrict__ gate_w,
                                                             u32x4* __restrict__ y,
                                                             int64_t out_rows, int64_t g0,
                                                             int64_t g1, int K, int nvec,
                                                             int parts, int32_t* err) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x % kWave;
  const int64_t b = xcd_block(blockIdx.x, gridDim.x);
  // the wave's token, uniform (readfirstlane), so the row spans below live in SGPRs
  const int64_t wv = b * kCbTokPerBlock + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t g = g0 + (parts == 1 ? wv : (int)wv / parts);
  const int part = parts == 1 ? 0 : (int)wv % parts;
  if (g >= g1) return;
  const int d_mine = checked_row(lane < K ? dest_row[g * K + lane] : -1, out_rows, err);
  const int w_mine = kWeighted && lane < K ? __float_as_int(gate_w[g * K + lane]) : 0;
  for (int v0 = part * kVec * kWave; v0 < nvec; v0 += parts * kVec * kWave) {
    float acc[kVec * 8];
#pragma unroll
    for (int i = 0; i < kVec * 8; ++i) acc[i] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += kGroup) {
      int dq[kGroup];
      float wq[kGroup];
      u32x4 buf[kGroup][kVec];
#pragma unroll
      for (int q = 0; q < kGroup; ++q) {
        const int k = k0 + q;
        dq[q] = k < K ? readlane(d_mine, k) : -1;
        wq[q] = k < K ? __int_as_float(readlane(w_mine, k)) : 0.0f;
        if (dq[q] >= 0) {          // a span per row: vectors past its end read as zero
          const span_t src = span_of(y_disp + (int64_t)dq[q] * nvec, (int64_t)nvec * 16);
#pragma unroll
          for (int u = 0; u < kVec; ++u) buf[q][u] = stream_load(src, (v0 + u * kWave + lane) * 16);
        }
      }
#pragma unroll
      for (int q = 0; q < kGroup; ++q) {
        if (dq[q] < 0) continue;
        const float w = wq[q];
#pragma unroll
        for (int u = 0; u < kVec; ++u) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float p0 = kWeighted ? w * bf16_lo(buf[q][u][c]) : bf16_lo(buf[q][u][c]);
            const float p1 = kWeighted ? w * bf16_hi(buf[q][u][c]) : bf16_hi(buf[q][u][c]);
            acc[u * 8 + 2 * c] = acc[u * 8 + 2 * c] + p0;
            acc[u * 8 + 2 * c + 1] = acc[u * 8 + 2 * c + 1] + p1;
          }
        }
      }
    }
    const span_t dst = span_of(y + g * nvec, (int64_t)nvec * 16);
#pragma unroll
    for (int u = 0; u < kVec; ++u) {           // past the row's end: not written
      u32x4 o;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        o[c] = pack_bf16(acc[u * 8 + 2 * c], acc[u * 8 + 2 * c + 1]);
      stream_store(o, dst, (v0 + u * kWave + lane) * 16);
    }
  }
}

typedef void (*cb_kernel_t)(const u32x4*, const int32_t*, const float*, u32x4*, int64_t, int64_t,
                            int64_t, int, int, int, int32_t*);
template <bool kWeighted, int kVec>
static cb_kernel_t cb_group(int slots) {
  return slots > 4   ? combine_kernel<kWeighted, kVec, 8>
         : slots > 2 ? combine_kernel<kWeighted, kVec, 4>
         : slots > 1 ? combine_kernel<kWeighted, kVec, 2> : combine_kernel<kWeighted, kVec, 1>;
}
// nv: vectors per lane that a row fills
template <bool kWeighted>
static cb_kernel_t cb_kernel(int nv, int slots) {
  return nv <= 1   ? cb_group<kWeighted, 1>(slots)
         : nv <= 2 ? cb_group<kWeighted, 2>(slots) : combine_kernel<kWeighted, kCbVec, 4>;
}

// The argument checks and the launch that both entry points share.
static uep_status cb_launch(const uint16_t* rows, int64_t out_rows, const int32_t* dest_row,
                            const float* gate_w, bool weighted, int32_t R, int32_t T, int32_t K,
                            int32_t H, int32_t r_begin, int32_t r_end, uint16_t* y, int32_t* err,
                            void* stream) {
  if (R <= 0 || T < 0 || K <= 0 || H <= 0 || out_rows < 0) return UEP_EINVAL;
  if (r_begin < 0 || r_end > R || r_begin > r_end) return UEP_EINVAL;
  if (K > 64 || H % 8 != 0 || H > (1 << 29) || (int64_t)R * T * K >= (1ll << 31))
    return UEP_EGEOM;
  const int64_t g0 = (int64_t)r_begin * T, g1 = (int64_t)r_end * T;
  if (g1 == g0) return UEP_OK;
  if ((!rows && out_rows > 0) || !dest_row || (weighted && !gate_w) || !y) return UEP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(y)) % 16 != 0)
    return UEP_EGEOM;
  const int64_t tok = (int64_t)R * T, used = std::min<int64_t>(out_rows, 1ll << 31);
  if (!weighted && uep_overlap({y, tok * H * 2}, {{rows, used * H * 2}, {dest_row, tok * K * 4}}))
    return UEP_EINVAL;
  const int slices = (H / 8 + kCbVec * kWave - 1) / (kCbVec * kWave);
  const int parts = g1 - g0 <= kCbFew ? std::min(slices, 16) : 1;
  const int nv = (H / 8 + kWave - 1) / kWave;       // vectors per lane of a row
  const cb_kernel_t kernel = weighted ? cb_kernel<true>(nv, K) : cb_kernel<false>(nv, K);
  for (int64_t c0 = g0; c0 < g1; c0 += kCbLaunch) {
    const int64_t c1 = std::min(g1, c0 + kCbLaunch);
    const int64_t blocks = ((c1 - c0) * parts + kCbTokPerBlock - 1) / kCbTokPerBlock;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kCbThreads), 0, uep_stream(stream),
                       reinterpret_cast<const u32x4*>(rows), dest_row, gate_w,
                       reinterpret_cast<u32x4*>(y), out_rows, c0, c1, K, H / 8, parts, err);
    UEP_CHECK_LAUNCH();
  }
  return UEP_OK;
}

}  // namespace uep

using namespace uep;

extern "C" uep_status uep_combine(const uint16_t* y_disp, int64_t out_rows,
                                  const int32_t* dest_row, const float* gate_w, int32_t R,
                                  int32_t T, int32_t K, int32_t H, int32_t r_begin, int32_t r_end,
                                  uint16_t* y, int32_t* err, void* stream) {
  return cb_launch(y_disp, out_rows, dest_row, gate_w, true, R, T, K, H, r_begin, r_end, y, err,
                   stream);
}

extern "C" uep_status uep_permute_grad(const uint16_t* dout, int64_t out_rows,
                                       const int32_t* dest_row, int32_t R, int32_t T, int32_t K,
                                       int32_t H, int32_t r_begin, int32_t r_end, uint16_t* dx,
                                       int32_t* err, void* stream) {
  return cb_launch(dout, out_rows, dest_row, nullptr, false, R, T, K, H, r_begin, r_end, dx, err,
                   stream);
}
