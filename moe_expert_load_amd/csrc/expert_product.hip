// The experts' matrix products in 8-bit integers (uep.h: uep_expert_product).
//
// out = (q . w) w_scale scale over the instances' row blocks: int32 sums by the matrix
// instruction on 64 integers at a time (v_mfma_i32_16x16x64_i8), scales and the SwiGLU in fp32,
// one rounding to bf16.  Operand lane layout: lane l holds 16 consecutive integers, from
// 16 (l / 16) on, of row l % 16; result register r of lane l is channel 4 (l / 16) + r (the
// first operand's row) of row l % 16 (the second's).
#include <algorithm>

#include "common.h"
#include "numeric.h"

namespace uep {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kPrMaxD = 65536;         // 2^16 products of at most 2^14 stay below 2^31
constexpr int kPrFar = (int)0x80000000u;   // a span offset behind any end: reads zeros

struct PrArgs {
  const int8_t* q;
  const float* q_scale;
  int64_t rows;
  const int32_t* offset;               // NULL: one instance with every row
  int n_inst, inst_per_rank, e_loc, slots;
  const int8_t *main_w, *slot_w;
  const float *main_scale, *slot_scale;
  int N, n_out, D;                     // weight rows, outputs (N or N / 2), depth
  uint16_t* out;
  int32_t* err;
};

struct PrTile {
  int inst;
  int64_t row0;
  int n_rows;                          // 0: no such tile
};

__device__ __forceinline__ int pr_tiles(int begin, int end, int rows) {
  const int n = max(end - begin, 0);
  return n / rows + (n % rows != 0);
}

// The t-th tile of at most kRows rows of one instance, the instances in order and without the
// empty ones.  Every lane of the wave calls it; lanes take consecutive instances each.
template <int kRows>
__device__ __forceinline__ PrTile pr_tile(const PrArgs& a, int t) {
  if (!a.offset) {
    const int64_t row0 = (int64_t)t * kRows;
    return {0, row0, (int)max((int64_t)0, min((int64_t)kRows, a.rows - row0))};
  }
  const int lane = threadIdx.x % kWave, per = (a.n_inst + kWave - 1) / kWave;
  const int i0 = min(lane * per, a.n_inst), i1 = min(i0 + per, a.n_inst), most = (int)a.rows;
  int tiles = 0;
  {
    int begin = min(max(a.offset[i0], 0), most);
    for (int i = i0; i < i1; ++i) {
      const int end = min(max(a.offset[i + 1], 0), most);
      tiles += pr_tiles(begin, end, kRows);
      begin = end;
    }
  }
  const int upto = wave_incl_scan(tiles);
  const int owner = first_lane(upto > t);
  if (owner < 0) return {0, 0, 0};
  int left = t - (upto - tiles), inst = 0, row0 = 0, n = 0;
  if (lane == owner) {
    int begin = min(max(a.offset[i0], 0), most);
    for (int i = i0; i < i1; ++i) {
      const int end = min(max(a.offset[i + 1], 0), most);
      const int here = pr_tiles(begin, end, kRows);
      if (left < here) {
        inst = i;
        row0 = begin + left * kRows;
        n = min(kRows, end - row0);
        break;
      }
      left -= here;
      begin = end;
    }
  }
  return {readlane(inst, owner), readlane(row0, owner), readlane(n, owner)};
}

__device__ __forceinline__ int64_t pr_weight(const PrArgs& a, int inst, bool& slot) {
  const int r = inst / a.inst_per_rank, j = inst % a.inst_per_rank;
  slot = j >= a.e_loc;
  return slot ? (int64_t)r * a.slots + (j - a.e_loc) : (int64_t)r * a.e_loc + j;
}

__device__ __forceinline__ void pr_check_offsets(const PrArgs& a) {
  if (!a.offset || !a.err) return;
  for (int i = threadIdx.x; i < a.n_inst; i += blockDim.x)
    if (a.offset[i] < 0 || a.offset[i + 1] < a.offset[i] || a.offset[i + 1] > a.rows)
      set_err(a.err, UEP_ERR_OFFSET);
}

// The channel's scale first: it is moderate, so that only a result out of range leaves the range.
__device__ __forceinline__ float pr_scaled(int acc, float w_scale, float q_scale) {
  return (float)acc * w_scale * q_scale;
}
// gate / (1 + e^-gate) * up; exp2's argument rounded once, hardware exp2 and reciprocal
__device__ __forceinline__ float pr_swiglu(float gate, float up) {
  return gate * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * gate)) * up;
}

// ---------------------------------------------------------------------------------------
// Few rows: weights stream from HBM straight into operands.  A block takes 16 kRB rows and 16 kCB
// channels (SwiGLU: half of them gates, half their ups); its waves share the depth, in pieces of
// 64 kU, and add their sums in LDS.
constexpr int kPrWaves = 4;
template <int kRB, int kCB, int kU, bool kGlu>
__global__ __launch_bounds__(kPrWaves* kWave) void pr_stream_kernel(PrArgs a, int t0,
                                                                   int n_tiles) {
  constexpr int kOut = kGlu ? kCB / 2 : kCB;     // blocks of 16 outputs
  __shared__ i32x4 sums[kPrWaves][kRB * kCB][kWave];
  if (blockIdx.x == 0) pr_check_offsets(a);
  const int64_t id = xcd_block(blockIdx.x, gridDim.x);
  const PrTile tile = pr_tile<16 * kRB>(a, t0 + (int)(id % n_tiles));
  if (tile.n_rows <= 0) return;
  const int c0 = (int)(id / n_tiles) * 16 * kOut;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  bool slot;
  const int64_t at = pr_weight(a, tile.inst, slot);
  const int64_t size = (int64_t)a.N * a.D;
  const span_t ws = span_of((slot ? a.slot_w : a.main_w) + at * size, size);
  const span_t qs = span_of(a.q + tile.row0 * a.D, (int64_t)tile.n_rows * a.D);

  int w_row[kCB], q_row[kRB];
#pragma unroll
  for (int c = 0; c < kCB; ++c) {
    const int ch = c0 + 16 * (c % kOut) + lane % 16;
    w_row[c] = ch < a.n_out ? (ch + c / kOut * a.n_out) * a.D : kPrFar;
  }
#pragma unroll
  for (int r = 0; r < kRB; ++r) q_row[r] = (16 * r + lane % 16) * a.D;
  i32x4 acc[kRB][kCB] = {};
  for (int k0 = wave * 64 * kU; k0 < a.D; k0 += kPrWaves * 64 * kU) {
    i32x4 w[kU][kCB], x[kU][kRB];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + 64 * u + 16 * (lane / 16);
      const bool in = k < a.D;
#pragma unroll
      for (int c = 0; c < kCB; ++c)
        w[u][c] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       ws, in && w_row[c] >= 0 ? w_row[c] + k : kPrFar, 0, 0));
#pragma unroll
      for (int r = 0; r < kRB; ++r)
        x[u][r] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(qs, in ? q_row[r] + k : kPrFar, 0, 0));
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int r = 0; r < kRB; ++r)
#pragma unroll
        for (int c = 0; c < kCB; ++c)
          acc[r][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][c], x[u][r], acc[r][c], 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < kRB; ++r)
#pragma unroll
    for (int c = 0; c < kCB; ++c) sums[wave][r * kCB + c][lane] = acc[r][c];
  __syncthreads();

  const float* w_scale = (slot ? a.slot_scale : a.main_scale) + at * a.N;
  for (int o = threadIdx.x; o < kRB * kOut * kWave; o += kPrWaves * kWave) {
    const int l = o % kWave, f = o / kWave, r = f / kOut, c = f % kOut;
    const int row = 16 * r + l % 16, ch = c0 + 16 * c + 4 * (l / 16);
    if (row >= tile.n_rows || ch >= a.n_out) continue;
    i32x4 z = sums[0][r * kCB + c][l], up = {0, 0, 0, 0};
    if constexpr (kGlu) up = sums[0][r * kCB + kOut + c][l];
#pragma unroll
    for (int w = 1; w < kPrWaves; ++w) {
      z += sums[w][r * kCB + c][l];
      if constexpr (kGlu) up += sums[w][r * kCB + kOut + c][l];
    }
    const float qs1 = a.q_scale[tile.row0 + row];
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = pr_scaled(z[j], w_scale[ch + j], qs1);
      if constexpr (kGlu)
        y[j] = pr_swiglu(y[j], pr_scaled(up[j], w_scale[a.n_out + ch + j], qs1));
    }
    uint2 v = {pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
    *reinterpret_cast<uint2*>(a.out + (tile.row0 + row) * a.n_out + ch) = v;
  }
}

// ---------------------------------------------------------------------------------------
// Many rows: tiles of 256 channels (SwiGLU: 128 gates and their ups) and 256 rows by eight
// waves, two beside each other on every SIMD, each 128 channels and 64 rows (128 registers of
// sums).  The depth goes by steps of 128 through two pairs of LDS buffers that the memory fills by
// itself (buffer loads into LDS); a step's loads have a whole step's time.  Half steps of 64 are
// read from LDS into registers one half ahead of the matrix instructions, so that one barrier a
// step is enough: behind it every wave has the step in registers, its buffers are free for the
// step after next, and the next step has landed.
//
// LDS rows are 128 bytes in eight slots of 16; slot s of row r holds bytes 16 (s ^ r % 8), so that the
// 16 rows that a wave reads together spread over all banks.
constexpr int kPtSide = 256, kPtDepth = 128, kPtThreads = 512;
constexpr int kPtBuf = kPtSide * kPtDepth;          // one buffer of one operand

__device__ __forceinline__ i32x4 pt_span(const int8_t* p, int64_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)u),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32) & 0xFFFF),
               __builtin_amdgcn_readfirstlane((int)bytes), kRsrcWord3};
}

// 64 lanes' 16 bytes from span offset `off` + `more` into the 1 KiB of LDS from `lds` on.  Written
// by hand because the compiler has every later read of LDS wait for all of them.
__device__ __forceinline__ void pt_fetch(i32x4 span, uint32_t lds, int off, int more) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(off), "s"(span), "s"(more)
      : "memory", "m0");
}

template <bool kGlu>
__global__ __launch_bounds__(kPtThreads, 2) void pr_tile_kernel(PrArgs a, int t0, int n_tiles,
                                                                int cols) {
  constexpr int kWide = kGlu ? kPtSide / 2 : kPtSide;   // outputs of a tile
  __shared__ __attribute__((aligned(1024))) char lds[4 * kPtBuf];
  if (blockIdx.x == 0) pr_check_offsets(a);
  // eight row tiles by all columns at a time: what an XCD's 32 workgroups share stays in its L2
  const int id = (int)xcd_block(blockIdx.x, gridDim.x);
  const int band = id / (8 * cols), in_band = id % (8 * cols);
  const int high = min(8, n_tiles - band * 8);
  const PrTile tile = pr_tile<kPtSide>(a, t0 + band * 8 + in_band % high);
  if (tile.n_rows <= 0) return;
  const int c0 = in_band / high * kWide;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  bool slot;
  const int64_t at = pr_weight(a, tile.inst, slot);
  const int64_t size = (int64_t)a.N * a.D;
  const i32x4 ws = pt_span((slot ? a.slot_w : a.main_w) + at * size, size);
  const i32x4 qs = pt_span(a.q + tile.row0 * a.D, (int64_t)tile.n_rows * a.D);
  const uint32_t base = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);

  // a wave fills 32 rows of both operands' buffers, 8 by 8
  const int fetch = (lane / 8) * a.D + ((lane ^ (lane / 8)) % 8) * 16;
  int w_row[4], q_row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = wave * 32 + i * 8, f = r % 128 / 16;
    const int ch = kGlu ? r / 128 * 64 + f / 2 * 16 + r % 16 + f % 2 * a.n_out : r;
    w_row[i] = (c0 + ch) * a.D;
    q_row[i] = r * a.D;
  }
  auto fetch_piece = [&](int step, int i) {             // i: 0..3 weights, 4..7 rows
    const uint32_t to = base + (step % 2) * kPtBuf + wave * 4096 + (i % 4) * 1024;
    if (i < 4) pt_fetch(ws, to, fetch, w_row[i % 4] + step * kPtDepth);
    else pt_fetch(qs, to + 2 * kPtBuf, fetch, q_row[i % 4] + step * kPtDepth);
  };

  const int w_wave = wave % 2 * 128, q_wave = wave / 2 * 64;
  const int part = (lane / 16 ^ lane % 8) * 16;          // of the first half; the second ^ 64
  const char* w_lds = lds + (w_wave + lane % 16) * kPtDepth;
  const char* q_lds = lds + 2 * kPtBuf + (q_wave + lane % 16) * kPtDepth;
  i32x4 acc[8][4] = {};
  i32x4 w[2][8], x[2][4];
  auto read_w = [&](int step, int h, int f) {
    w[h][f] = *reinterpret_cast<const i32x4*>(w_lds + (part ^ h * 64) + step % 2 * kPtBuf +
                                              f * 16 * kPtDepth);
  };
  auto read_x = [&](int step, int h, int f) {
    x[h][f] = *reinterpret_cast<const i32x4*>(q_lds + (part ^ h * 64) + step % 2 * kPtBuf +
                                              f * 16 * kPtDepth);
  };
  auto multiply = [&](int h, int f) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[f][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][f], x[h][j], acc[f][j], 0, 0, 0);
  };

  const int steps = (a.D + kPtDepth - 1) / kPtDepth;
  for (int i = 0; i < 8; ++i) fetch_piece(0, i);
  if (steps > 1) {
    for (int i = 0; i < 8; ++i) fetch_piece(1, i);
    asm volatile("s_waitcnt vmcnt(8)" ::: "memory");     // the first step's
  } else {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int f = 0; f < 8; ++f) {
    if (f < 4) read_x(0, 0, f);
    read_w(0, 0, f);
  }
  auto first_half = [&](int k) {
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      if (f < 4) read_x(k, 1, f);
      read_w(k, 1, f);
      multiply(0, f);
      __builtin_amdgcn_sched_barrier(0);                 // keeps the reads between the products
    }
  };
  auto second_half = [&](int k, bool more) {
    // own reads of this step are in registers, own loads of the next have landed
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      if (more) fetch_piece(k + 2, f);
      if (f < 4) read_x(k + 1, 0, f);
      read_w(k + 1, 0, f);
      multiply(1, f);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int k = 0;
  for (; k < steps - 2; ++k) {
    first_half(k);
    second_half(k, true);
  }
  if (k < steps - 1) {
    first_half(k);
    second_half(k, false);
    ++k;
  }
  // The last step: bytes past the end of the depth are another row's, and count as zeros.
  const int rest = a.D - k * kPtDepth;
  auto cut = [&](int h) {
    const bool in = h * 64 + lane / 16 * 16 < rest;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[h][j][i] = in ? x[h][j][i] : 0;
  };
  cut(0);
  first_half(k);
  cut(1);
#pragma unroll
  for (int f = 0; f < 8; ++f) multiply(1, f);

  const float* w_scale = (slot ? a.slot_scale : a.main_scale) + at * a.N;
  float q_scale[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = q_wave + 16 * j + lane % 16;
    q_scale[j] = row < tile.n_rows ? a.q_scale[tile.row0 + row] : 0.0f;
  }
  constexpr int kStep = kGlu ? 2 : 1;
#pragma unroll
  for (int f = 0; f < 8; f += kStep) {
    const int ch = c0 + (kGlu ? wave % 2 * 64 + f / 2 * 16 : w_wave + f * 16) + lane / 16 * 4;
    if (ch >= a.n_out) continue;
    float s[4], s_up[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = w_scale[ch + i];
      if constexpr (kGlu) s_up[i] = w_scale[a.n_out + ch + i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = q_wave + 16 * j + lane % 16;
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = pr_scaled(acc[f][j][i], s[i], q_scale[j]);
        if constexpr (kGlu) y[i] = pr_swiglu(y[i], pr_scaled(acc[f + 1][j][i], s_up[i], q_scale[j]));
      }
      const uint2 v = {pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
      if (row < tile.n_rows)
        *reinterpret_cast<uint2*>(a.out + (tile.row0 + row) * a.n_out + ch) = v;
    }
  }
}

// Launches of fewer than 2^32 threads each, over ranges of tiles.
template <typename F>
static uep_status pr_launches(const PrArgs& a, int side, int cols, int threads, F launch) {
  const int64_t tiles = std::min(a.rows, a.rows / side + a.n_inst);
  const int64_t most = ((1ll << 32) - 1) / threads / cols;
  for (int64_t t = 0; t < tiles; t += most) {
    launch((int)t, (int)std::min(tiles - t, most));
    UEP_CHECK_LAUNCH();
  }
  return UEP_OK;
}

template <int kRB, int kCB, int kU, bool kGlu>
static uep_status pr_stream(const PrArgs& a, hipStream_t s) {
  constexpr int kWide = 16 * (kGlu ? kCB / 2 : kCB);
  const int cols = (a.n_out + kWide - 1) / kWide;
  return pr_launches(a, 16 * kRB, cols, kPrWaves * kWave, [&](int t, int n) {
    hipLaunchKernelGGL((pr_stream_kernel<kRB, kCB, kU, kGlu>), dim3((unsigned)n * cols),
                       dim3(kPrWaves * kWave), 0, s, a, t, n);
  });
}

template <bool kGlu>
static uep_status pr_tiles_of(const PrArgs& a, hipStream_t s) {
  constexpr int kWide = kGlu ? kPtSide / 2 : kPtSide;
  const int cols = (a.n_out + kWide - 1) / kWide;
  return pr_launches(a, kPtSide, cols, kPtThreads, [&](int t, int n) {
    hipLaunchKernelGGL((pr_tile_kernel<kGlu>), dim3((unsigned)n * cols), dim3(kPtThreads), 0, s, a,
                       t, n, cols);
  });
}

template <bool kGlu>
static uep_status pr_run(const PrArgs& a, hipStream_t s) {
  if (a.rows >= 64ll * a.n_inst) return pr_tiles_of<kGlu>(a, s);
  return pr_stream<4, 4, 2, kGlu>(a, s);
}

}  // namespace uep

using namespace uep;

extern "C" uep_status uep_expert_product(const int8_t* q, const float* q_scale, int64_t rows,
                                         const int32_t* inst_offset, int32_t R, int32_t E,
                                         int32_t S, const int8_t* main_w, const float* main_scale,
                                         const int8_t* slot_w, const float* slot_scale, int32_t N,
                                         int32_t D, int32_t act, uint16_t* out, int32_t* err,
                                         void* stream) {
  if (rows < 0 || R <= 0 || E <= 0 || S < 0 || N <= 0 || D <= 0) return UEP_EINVAL;
  if (act != UEP_PRODUCT_PLAIN && act != UEP_PRODUCT_SWIGLU) return UEP_EINVAL;
  const int n_out = act == UEP_PRODUCT_SWIGLU ? N / 2 : N;
  if (R > 64 || E > 4096 || S > 8 || E % R != 0 || D % 16 != 0 || D > kPrMaxD || N % 8 != 0 ||
      n_out % 8 != 0 || (int64_t)N * D >= (1ll << 31) || rows >= (1ll << 31))
    return UEP_EGEOM;
  const int e_loc = E / R, n_inst = R * (e_loc + S);
  if (!inst_offset && n_inst != 1) return UEP_EINVAL;
  if (rows == 0) return UEP_OK;
  if (!q || !q_scale || !main_w || !main_scale || !out || (S > 0 && (!slot_w || !slot_scale)))
    return UEP_EINVAL;
  for (const void* p : {(const void*)q, (const void*)main_w, (const void*)slot_w, (const void*)out})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return UEP_EGEOM;
  const int64_t slots = (int64_t)R * S, size = (int64_t)N * D;
  if (uep_overlap({out, rows * n_out * 2},
                  {{q, rows * D}, {q_scale, rows * 4}, {inst_offset, (n_inst + 1) * 4ll},
                   {main_w, E * size}, {main_scale, E * (int64_t)N * 4}, {slot_w, slots * size},
                   {slot_scale, slots * N * 4}}))
    return UEP_EINVAL;
  const PrArgs a{q, q_scale, rows, inst_offset, n_inst, e_loc + S, e_loc, S, main_w, slot_w,
                 main_scale, slot_scale, N, n_out, D, out, err};
  hipStream_t s = uep_stream(stream);
  return act == UEP_PRODUCT_SWIGLU ? pr_run<true>(a, s) : pr_run<false>(a, s);
}
