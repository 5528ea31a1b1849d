// Gradient of the combine (uep.h: uep_combine_grad): every dispatch row gets its token's
// output gradient times its weight, and every weight the dot product of that gradient
// with the expert output in its row,
//   dout[d] = bf16(w[g][k] * dy[g]),   dgate_w[g][k] = <dy[g], out[d]>,   d = dest_row[g][k].
//
// One wave per token on the XCD-aware block map, as in the combine: the token's gradient
// is read once into registers, slice by slice, and serves its K rows; lanes 0..K-1 hold
// rows, weights and the running dot products, and the next slots' rows of `out` are on
// their way while one group is used.  A row of `out` is read before the same row of dout
// is written, by the same wave, so that both may be one buffer.
//
// Two phases.  HBM takes a stream of reads and a stream of writes faster one after the
// other than mixed, and the two halves of this operator share only dy.  From kRgPhaseBytes of
// dispatch rows on, the dot products (reads alone) and the scaled rows (writes alone) are
// therefore launches of their own, over chunks of tokens whose dy stays in the 256 MB
// last-level cache from the first to the second; not for K = 1, where dy, read twice, is as
// large as the rows (65536 x 4 KiB in one launch 154 us, in two 164).  Measured on MI355X (two launches per chunk
// against one for both): 65536 tokens, K = 8, 8 KiB rows 1760 -> 1503 us (6.08 TB/s of the
// bytes that have to move; a large copy reaches 5.65), chunks of 16 / 64 / 128 / 224 MB of
// dy / all in one 1692 / 1561 / 1519 / 1503 / 1570 us; 32 MB of rows 16.6 -> 16.0 us
// (1 KiB rows) and 16.1 -> 16.9 (4 KiB), 64 MB 32.4 -> 29.3 (512 B), 29.9 -> 27.6 (8 KiB).
//
// Short rows: with vectors for 8 KiB per wave whatever the row, 65536 tokens of eight 512 B
// rows took 293 us; with a row's own vectors and kRgVec of them in flight 116 (one launch).
// Registers for no more slots than a token has leave room for more waves: 65536 tokens of one
// 1072 B row 77 -> 50 us, of two 512 B rows 57 -> 43.
#include <algorithm>

#include "common.h"
#include "numeric.h"

namespace uep {

constexpr int kRgThreads = 256;
constexpr int kRgTokPerBlock = kRgThreads / kWave;
constexpr int kRgVec = 8;     // 16-byte vectors in flight per lane for each of the two row groups
// Up to this many tokens, which leave SIMDs without a wave, a token's slots go to a wave each
// instead of one after the other to one.  Apart against together (K = 8, 8 KiB rows, in a
// graph): 128 tokens 5.5 against 10.6 us, 512 17.1 / 19.7, 1024 28.7 / 27.0.
constexpr int64_t kRgFew = 512;
constexpr int64_t kRgPhaseBytes = 48ll << 20;
constexpr int64_t kRgChunkBytes = 224ll << 20;
constexpr int64_t kRgLaunch = 1ll << 25;   // tokens of one launch, which holds below 2^32 threads

// Row d of `base`, an empty span if d < 0: its loads read zeros, its stores go nowhere.
__device__ __forceinline__ span_t rg_row(const u32x4* base, int d, int nvec) {
  return span_of(base + (int64_t)max(d, 0) * nvec, d < 0 ? 0 : (int64_t)nvec * 16);
}

// kDot: the dot products (dout is not touched unless kScale); kScale: the scaled rows.
// kVec vectors per lane hold a slice of a row (a whole row where it is shorter than a slice of
// kRgVec), kG slots go together.
template <bool kDot, bool kScale, int kVec, int kG>
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
  for (int v0 = 0; v0 < nvec; v0 += kVec * kWave) {
    u32x4 grad[kVec], y[2][kG][kVec];
    auto row_of = [&](int k) { return k < k_end ? readlane(d_mine, k) : -1; };
    auto fetch = [&](int k0, u32x4 (&to)[kG][kVec]) {
#pragma unroll
      for (int q = 0; q < kG; ++q) {
        const span_t row = rg_row(out, row_of(k0 + q), nvec);
#pragma unroll
        for (int u = 0; u < kVec; ++u) to[q][u] = stream_load(row, (v0 + u * kWave + lane) * 16);
      }
    };
    auto slots = [&](int k0, const u32x4 (&from)[kG][kVec]) {
#pragma unroll
      for (int q = 0; q < kG; ++q) {
        const int k = k0 + q, d = row_of(k);
        if (kDot) {
          float dot = 0.0f;
#pragma unroll
          for (int u = 0; u < kVec; ++u)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              dot = fmaf(bf16_lo(grad[u][c]), bf16_lo(from[q][u][c]), dot);
              dot = fmaf(bf16_hi(grad[u][c]), bf16_hi(from[q][u][c]), dot);
            }
          dot = wave_sum_f32(dot);
          if (lane == k) dot_mine += dot;
        }
        if (!kScale || d < 0) continue;
        const float w = __int_as_float(readlane(w_mine, k));
        const span_t dst = rg_row(dout, d, nvec);
#pragma unroll
        for (int u = 0; u < kVec; ++u) {
          u32x4 o;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            o[c] = pack_bf16(w * bf16_lo(grad[u][c]), w * bf16_hi(grad[u][c]));
          stream_store(o, dst, (v0 + u * kWave + lane) * 16);
        }
      }
    };
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const int at = (v0 + u * kWave + lane) * 16;      // read again by the scaling: kept
      grad[u] = kScale ? stream_load(src, at) : __builtin_amdgcn_raw_buffer_load_b128(src, at, 0, 0);
    }
    if (kDot) fetch(k_begin, y[0]);
    for (int k = k_begin; k < k_end; k += 2 * kG) {  // the next slots are on their way
      if (kDot && k + kG < k_end) fetch(k + kG, y[1]);
      slots(k, y[0]);
      if (k + kG < k_end) {
        if (kDot && k + 2 * kG < k_end) fetch(k + 2 * kG, y[0]);
        slots(k + kG, y[1]);
      }
    }
  }
  // a slot without a row read nothing: 0 (0 times an infinite gradient left a NaN)
  if (kDot && mine) dgate_w[g * K + lane] = d_mine < 0 ? 0.0f : dot_mine;
}

typedef void (*rg_kernel_t)(const u32x4*, const u32x4*, const int32_t*, const float*, u32x4*,
                            float*, int64_t, int64_t, int64_t, int, int, int, int32_t*);
struct RgKernels {
  rg_kernel_t both, dot, scale;
};
template <int kVec, int kG>
static RgKernels rg_group() {
  return {combine_grad_kernel<true, true, kVec, kG>, combine_grad_kernel<true, false, kVec, kG>,
          combine_grad_kernel<false, true, kVec, kG>};
}
// slots together: as many as a token has, up to kRgVec vectors
template <int kVec>
static RgKernels rg_kernels(int slots) {
  if (kRgVec / kVec >= 8 && slots > 4) return rg_group<kVec, kRgVec / kVec >= 8 ? 8 : 1>();
  if (kRgVec / kVec >= 4 && slots > 2) return rg_group<kVec, kRgVec / kVec >= 4 ? 4 : 1>();
  if (kRgVec / kVec >= 2 && slots > 1) return rg_group<kVec, kRgVec / kVec >= 2 ? 2 : 1>();
  return rg_group<kVec, 1>();
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
  // a buffer without rows has no address either: dgate_w says whether its zeros are wanted
  if (!dy || !dest_row || !gate_w || (!dout && out_rows > 0) ||
      (out ? !dgate_w : dgate_w && out_rows > 0))
    return UEP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(out) |
       reinterpret_cast<uintptr_t>(dout)) % 16 != 0)
    return UEP_EGEOM;
  // dgate_w is written while gate_w, dout while dy and the others are still to be read
  const int64_t rows_used = std::min<int64_t>(out_rows, 1ll << 31);     // rows are int32
  const UepBytes grad{dy, (int64_t)R * T * H * 2}, rows{out, rows_used * H * 2};
  const UepBytes row_of{dest_row, (int64_t)R * T * K * 4}, weight{gate_w, (int64_t)R * T * K * 4};
  const UepBytes to{dout, rows.n}, dot{dgate_w, weight.n};
  if (uep_overlap(to, {grad, row_of, weight}) || (out != dout && uep_overlap(to, {rows})) ||
      uep_overlap(dot, {grad, rows, row_of, weight, to}))
    return UEP_EINVAL;
  const int nv = (H / 8 + kWave - 1) / kWave;       // vectors per lane of a row
  const int parts = g1 - g0 <= kRgFew ? K : 1;
  auto launch = [&](rg_kernel_t kernel, int64_t c0, int64_t c1) {
    const int64_t blocks = ((c1 - c0) * parts + kRgTokPerBlock - 1) / kRgTokPerBlock;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kRgThreads), 0, uep_stream(stream),
                       reinterpret_cast<const u32x4*>(dy), reinterpret_cast<const u32x4*>(out),
                       dest_row, gate_w, reinterpret_cast<u32x4*>(dout), dgate_w, out_rows, c0, c1,
                       K, H / 8, parts, err);
    return hipGetLastError() == hipSuccess;
  };
  const int slots = parts == 1 ? K : 1;             // of one wave
  const RgKernels f = nv <= 1 ? rg_kernels<1>(slots) : nv <= 2 ? rg_kernels<2>(slots)
                    : nv <= 4 ? rg_kernels<4>(slots) : rg_kernels<8>(slots);
  const bool phases = dgate_w && K > 1 && (g1 - g0) * K * (int64_t)H * 2 >= kRgPhaseBytes;
  // equal chunks of tokens that a launch holds; in phases, whose gradients stay in the
  // last-level cache
  const int64_t cap = std::min(
      kRgLaunch, phases ? std::max<int64_t>(64, kRgChunkBytes / ((int64_t)H * 2)) : kRgLaunch);
  const int64_t n = (g1 - g0 + cap - 1) / cap, chunk = (g1 - g0 + n - 1) / n;
  for (int64_t c0 = g0; c0 < g1; c0 += chunk) {
    const int64_t c1 = std::min(g1, c0 + chunk);
    if (dgate_w && !phases) {
      if (!launch(f.both, c0, c1)) return UEP_EHIP;
      continue;
    }
    if (dgate_w && !launch(f.dot, c0, c1)) return UEP_EHIP;
    if (!launch(f.scale, c0, c1)) return UEP_EHIP;
  }
  return UEP_OK;
}
