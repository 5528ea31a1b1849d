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
#include "rules.h"

namespace uep {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kPrMaxD = 65536;         // 2^16 products of at most 2^14 stay below 2^31
constexpr int64_t kPrMaxRows = 1ll << 29;
constexpr int kPrLaneTiles = (1 << 25) - 1;  // more than kPrMaxRows make; 64 of them fit an int
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
  int n_rows;
};

__device__ __forceinline__ int pr_tiles(int begin, int end, int rows) {
  const int n = max(end - begin, 0);
  return n / rows + (n % rows != 0);
}

// Tiles of at most kRows rows of one instance each, the instances in order and without the empty
// ones.  Every lane of the wave takes consecutive instances and keeps the tiles up to its last.
// All lanes of the wave make the calls; what is found is the same for all.
template <int kRows>
struct PrMap {
  int upto;

  static __device__ __forceinline__ int row(const PrArgs& a, int i) {
    return min(max(a.offset[i], 0), (int)a.rows);
  }
  static __device__ __forceinline__ int per_lane(const PrArgs& a) {
    return (a.n_inst + kWave - 1) / kWave;
  }
  __device__ __forceinline__ explicit PrMap(const PrArgs& a) {
    const int lane = threadIdx.x % kWave;
    int tiles = 0;
    if (!a.offset) {
      tiles = lane == 0 ? pr_tiles(0, (int)a.rows, kRows) : 0;
    } else {
      const int per = per_lane(a), first = min(lane * per, a.n_inst);
      const int last = min(first + per, a.n_inst);
      for (int i = first, at = row(a, first); i < last; ++i) {
        const int to = row(a, i + 1);
        tiles += pr_tiles(at, to, kRows);
        at = to;
      }
      tiles = min(tiles, kPrLaneTiles);                 // a table that falls may name more
    }
    upto = wave_incl_scan(tiles);
  }
  __device__ __forceinline__ int total() const { return readlane(upto, kWave - 1); }
  // t in [0, total()) and the same in every lane
  __device__ __forceinline__ PrTile find(const PrArgs& a, int t) const {
    const int owner = first_lane(upto > t);
    int left = owner > 0 ? t - readlane(upto, owner - 1) : t;
    int inst = 0, at = 0, to = (int)a.rows;
    if (a.offset) {
      inst = __builtin_amdgcn_readfirstlane(owner * per_lane(a));
      at = row(a, inst);
      to = row(a, inst + 1);
      while (left >= pr_tiles(at, to, kRows)) {
        left -= pr_tiles(at, to, kRows);
        ++inst;
        at = to;
        to = row(a, inst + 1);
      }
    }
    const int64_t row0 = at + (int64_t)left * kRows;
    return {inst, row0, (int)min((int64_t)kRows, to - row0)};
  }
};

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
// gate / (1 + e^-gate) * up; exp2's argument rounded once, hardware exp2 and reciprocal.  Below -87 the
// reciprocal leaves its range (it is 0 from -87.3 on), not the result if the up value is large: such
// gates take e^gate by halves, one to each side.  Where the wave has any: for all of them 32768 rows
// of 32 instances, 4096 x 7168, take 832 us instead of 825.
__device__ __forceinline__ void pr_swiglu(float (&gate)[4], const float (&up)[4]) {
  const bool far = fminf(fminf(gate[0], gate[1]), fminf(gate[2], gate[3])) < -87.0f;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = gate[i] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * gate[i])) * up[i];
  if (ballot(far)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float half = __builtin_amdgcn_exp2f(0.72134752f * gate[i]);
      if (gate[i] < -87.0f) y[i] = gate[i] * half * (up[i] * half);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) gate[i] = y[i];
}

// ---------------------------------------------------------------------------------------
// What the two kernels below share.  The depth goes by steps of 128, and the memory itself fills
// the LDS with them (buffer loads into LDS).  A step's rows are 128 bytes in eight slots of 16;
// slot s of row r holds bytes 16 (s ^ r % 8), so that the 16 rows that a wave reads together spread
// over all banks.

// Rows are D bytes apart, so that workgroups at the same step, of whichever channels, ask the same
// few memory channels where D is a multiple of a high power of two.  They begin at different steps
// instead: part `i` of `n` of the way through those before the last, which keeps its place (the
// rest of the depth is cut off there).  (8192 rows of 32 instances, 4096 channels, depth 4096: 164
// -> 148 us; 1024 rows 123 -> 105; 4096 rows of 4 95 -> 85; depth 7168 the same.)
__device__ __forceinline__ int pt_first(int i, int n, int steps) { return i % n * (steps - 1) / n; }

__device__ __forceinline__ i32x4 pt_span(const void* p, int64_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)u),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32) & 0xFFFF),
               __builtin_amdgcn_readfirstlane((int)bytes), kRsrcWord3};
}

// 64 lanes' 16 (4) bytes from span offset `off` + `more` into the 1 KiB (256 bytes) of LDS from
// `lds` on.  Written by hand because the compiler has every later read of LDS wait for them.
// `off` is checked against what `more` leaves of the span, so that `more` has to lie inside:
// rows that a tile does not have are fetched as its first ones, and count for nothing.
// The scalars may come from vector instructions (a spilled one by v_readlane), which the load may
// follow no sooner than five wait states later; the compiler sees to that for its own loads only.
__device__ __forceinline__ void pt_fetch(i32x4 span, uint32_t lds, int off, int more) {
  asm volatile(
      "s_nop 4\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "{m0}"(lds), "v"(off), "s"(span), "s"(more)
      : "memory");
}
__device__ __forceinline__ void pt_fetch4(i32x4 span, uint32_t lds, int off, int more) {
  asm volatile(
      "s_nop 4\n\t"
      "buffer_load_dword %1, %2, %3 offen lds"
      :
      : "{m0}"(lds), "v"(off), "s"(span), "s"(more)
      : "memory");
}

// Lane's part of 8 rows that one load brings, and of 16 rows that one read takes (first half of the
// step; the second is at ^ 64).
__device__ __forceinline__ int pt_fetch_lane(int lane, int D) {
  return (lane / 8) * D + ((lane ^ (lane / 8)) % 8) * 16;
}
__device__ __forceinline__ int pt_read_lane(int lane) {
  return lane % 16 * kPtDepth + (lane / 16 ^ lane % 8) * 16;
}

// ---------------------------------------------------------------------------------------
// Few rows, or too few tiles of the large kernel to fill the chip: tiles of kCh channels (SwiGLU:
// blocks of 16 gates and their ups in turn) and kRows rows.  kWC by kWR waves share a tile, and
// kGroups such groups share the depth, a step each in turn, and add their sums at the end: a long
// depth is the only axis that a small tile has left to split.  A ring of kStages times kGroups
// steps in LDS is what HBM is asked ahead; one barrier for every kGroups steps, half steps read one
// half ahead of the matrix instructions, as in the large kernel below.
template <int kCh, int kRows, int kWC, int kWR, int kGroups, int kStages, bool kGlu>
__global__ __launch_bounds__(kWC* kWR* kGroups* kWave) void pr_ring_kernel(PrArgs a, int t0,
                                                                           int most, int cols) {
  constexpr int kWide = kGlu ? kCh / 2 : kCh;
  constexpr int kTeam = kWC * kWR;
  constexpr int kLoads = (kCh + kRows) / 8 / kTeam;      // of a wave for one step
  constexpr int kStage = (kCh + kRows) * kPtDepth;
  constexpr int kCB = kCh / 16 / kWC, kRB = kRows / 16 / kWR;   // blocks of 16 of a wave
  static_assert((kCh / 8) % kTeam == 0 && (kRows / 8) % kTeam == 0 && (!kGlu || kCB % 2 == 0), "");
  __shared__ __attribute__((aligned(1024))) char lds[kStages * kGroups * kStage];
  static_assert(sizeof(lds) >= (kGroups - 1) * kCh * kRows * 4, "sums of the groups");
  if (blockIdx.x == 0) pr_check_offsets(a);
  // Workgroups without a tile come last: each takes a place in LDS while it looks (64 rows of 16
  // instances, 4096 channels, depth 2048: 30.3 -> 28.2 us).
  const PrMap<kRows> map(a);
  const int n_tiles = min(map.total() - t0, most);
  if ((int64_t)blockIdx.x >= (int64_t)n_tiles * cols) return;
  const uint32_t id = (uint32_t)xcd_block(blockIdx.x, (int64_t)n_tiles * cols);
  const PrTile tile = map.find(a, t0 + (int)(id % n_tiles));
  const int c0 = (int)(id / n_tiles) * kWide;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) % kTeam;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) / kTeam;
  bool slot;
  const int64_t at = pr_weight(a, tile.inst, slot), size = (int64_t)a.N * a.D;
  const i32x4 ws = pt_span((slot ? a.slot_w : a.main_w) + at * size, size);
  const i32x4 qs = pt_span(a.q + tile.row0 * a.D, (int64_t)tile.n_rows * a.D);
  const uint32_t base = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);
  const int rounds = (a.D + kPtDepth * kGroups - 1) / (kPtDepth * kGroups);
  const int fetch_lane = pt_fetch_lane(lane, a.D);
  int turn = pt_first((int)(id / n_tiles), 16, rounds);  // of the rounds before the last
  // loads past the depth go past the span's end: the same number is on the way at every step
  auto fetch = [&](int round) {
    const int step = (round < rounds - 1 ? turn : round) * kGroups + group;
    turn = turn + 1 < rounds - 1 ? turn + 1 : 0;
    const bool inside = step * kPtDepth < a.D;
    const int off = inside ? fetch_lane : kPrFar, more = inside ? step * kPtDepth : 0;
    const uint32_t to = base + (round % kStages * kGroups + group) * kStage;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int piece = wave + kTeam * i;
      if (kTeam * i < kCh / 8) {
        const int r = piece * 8, f = r / 16;
        const int ch = c0 + (kGlu ? f / 2 * 16 + r % 16 + f % 2 * a.n_out : r);
        pt_fetch(ws, to + piece * 1024, off, (ch < a.N ? ch : 0) * a.D + more);
      } else {
        const int r = piece * 8 - kCh;
        pt_fetch(qs, to + piece * 1024, off, (r < tile.n_rows ? r : 0) * a.D + more);
      }
    }
  };
  const int w_wave = wave % kWC * (kCh / kWC), q_wave = wave / kWC * (kRows / kWR);
  const int read_lane = pt_read_lane(lane);
  i32x4 acc[kCB][kRB] = {}, w[2][kCB], x[2][kRB];
  auto read = [&](int round, int h) {
    const char* stage = lds + (round % kStages * kGroups + group) * kStage;
#pragma unroll
    for (int r = 0; r < kRB; ++r)
      x[h][r] = *reinterpret_cast<const i32x4*>(stage + (kCh + q_wave + 16 * r) * kPtDepth +
                                                (read_lane ^ h * 64));
#pragma unroll
    for (int c = 0; c < kCB; ++c)
      w[h][c] = *reinterpret_cast<const i32x4*>(stage + (w_wave + 16 * c) * kPtDepth +
                                                (read_lane ^ h * 64));
  };
  auto multiply = [&](int h) {
#pragma unroll
    for (int c = 0; c < kCB; ++c)
#pragma unroll
      for (int r = 0; r < kRB; ++r)
        acc[c][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][c], x[h][r], acc[c][r], 0, 0, 0);
  };
  // own reads of the last step are done and own loads of the next have landed; then everyone's (a
  // wave by itself has only its own)
  auto meet = [&]() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"((kStages - 2) * kLoads) : "memory");
    if constexpr (kTeam > 1) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(k);
  meet();
  fetch(kStages - 1);
  read(0, 0);
  int k = 0;
  for (; k < rounds - 1; ++k) {
    read(k, 1);
    multiply(0);
    __builtin_amdgcn_sched_barrier(0);                   // keeps the reads ahead of the products
    meet();
    fetch(k + kStages);
    read(k + 1, 0);
    multiply(1);
    __builtin_amdgcn_sched_barrier(0);
  }
  // The last round: bytes past the end of the depth are another row's, and count as zeros.
  read(k, 1);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool in = (k * kGroups + group) * kPtDepth + h * 64 + lane / 16 * 16 < a.D;
#pragma unroll
    for (int r = 0; r < kRB; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[h][r][i] = in ? x[h][r][i] : 0;
    multiply(h);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // no load into LDS outlives its stage
  if constexpr (kGroups > 1) {
    __syncthreads();
    i32x4(*sums)[kTeam][kCB * kRB][kWave] =
        reinterpret_cast<i32x4(*)[kTeam][kCB * kRB][kWave]>(lds);
    if (group > 0) {
#pragma unroll
      for (int c = 0; c < kCB; ++c)
#pragma unroll
        for (int r = 0; r < kRB; ++r) sums[group - 1][wave][c * kRB + r][lane] = acc[c][r];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g)
#pragma unroll
      for (int c = 0; c < kCB; ++c)
#pragma unroll
        for (int r = 0; r < kRB; ++r) acc[c][r] += sums[g - 1][wave][c * kRB + r][lane];
  }

  const float* w_scale = (slot ? a.slot_scale : a.main_scale) + at * a.N;
#pragma unroll
  for (int r = 0; r < kRB; ++r) {
    const int row = q_wave + 16 * r + lane % 16;
    if (row >= tile.n_rows) continue;
    const float q_scale = a.q_scale[tile.row0 + row];
#pragma unroll
    for (int c = 0; c < kCB; c += kGlu ? 2 : 1) {
      const int ch = c0 + (w_wave + 16 * c) / (kGlu ? 2 : 1) + lane / 16 * 4;
      if (ch >= a.n_out) continue;
      float y[4], up[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = pr_scaled(acc[c][r][i], w_scale[ch + i], q_scale);
        if constexpr (kGlu) up[i] = pr_scaled(acc[c + 1][r][i], w_scale[a.n_out + ch + i], q_scale);
      }
      if constexpr (kGlu) pr_swiglu(y, up);
      *reinterpret_cast<uint2*>(a.out + (tile.row0 + row) * a.n_out + ch) =
          uint2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
    }
  }
}

// ---------------------------------------------------------------------------------------
// Many rows: tiles of 256 channels (SwiGLU: 128 gates and their ups) and 256 rows by eight
// waves, two beside each other on every SIMD, each 128 channels and 64 rows (128 registers of
// sums).  Steps go through two pairs of LDS buffers; a step's loads have a whole step's time.  Half
// steps of 64 are read from LDS into registers one half ahead of the matrix instructions, so that
// one barrier a step is enough: behind it every wave has the step in registers, its buffers are
// free for the step after next, and the next step has landed.  A workgroup stays on its CU and
// takes tile after tile: the next one's first two steps are under way while this one's results go
// out.  Beside the buffers each wave has 4 KiB of LDS of its own: 2 to turn results into whole
// lines, and the scales of this tile and the next.
constexpr int kPtThreads = 512;
constexpr int kPtBuf = kPtSide * kPtDepth;          // one buffer of one operand
constexpr int kPtTurn = 4 * kPtBuf;                 // the waves' own parts
constexpr int kPtScales = 2048, kPtScaleBytes = 768;
constexpr int kPtBand = 8;

// What a workgroup knows of a tile.
struct PtTile {
  i32x4 ws, qs;                        // spans of its weights and rows
  const float* w_scale;
  int64_t row0;
  int n_rows, c0;
};

template <bool kGlu>
__device__ __forceinline__ PtTile pt_tile(const PrArgs& a, const PrMap<kPtSide>& map, int tiles,
                                          int id, int cols) {
  // bands of eight row tiles by all columns: what an XCD's workgroups share stays in its L2
  const int band = id / (kPtBand * cols), in_band = id % (kPtBand * cols);
  const int high = min(kPtBand, tiles - band * kPtBand);
  const PrTile t = map.find(a, band * kPtBand + in_band % high);
  bool slot;
  const int64_t at = pr_weight(a, t.inst, slot), size = (int64_t)a.N * a.D;
  return {pt_span((slot ? a.slot_w : a.main_w) + at * size, size),
          pt_span(a.q + t.row0 * a.D, (int64_t)t.n_rows * a.D),
          (slot ? a.slot_scale : a.main_scale) + at * a.N,
          t.row0,
          t.n_rows,
          in_band / high * (kGlu ? kPtSide / 2 : kPtSide)};
}

template <bool kGlu>
__global__ __launch_bounds__(kPtThreads, 2) void pr_tile_kernel(PrArgs a, int cols, int most) {
  __shared__ __attribute__((aligned(1024))) char lds[kPtTurn + 8 * 4096];
  if (blockIdx.x == 0) pr_check_offsets(a);
  const PrMap<kPtSide> map(a);
  const int tiles = min(map.total(), most), total = tiles * cols;
  // Of every round of gridDim.x tiles an XCD takes consecutive ones, and its share of a last one
  // that is not full.  A last round of no more than half as many tiles as workgroups gives each
  // to two, which take 128 of the 256 channels (`half`): 6000 rows, 4096 channels, depth 4096
  // 100 -> 85 us.
  int taken = 0, half = -1;
  auto next = [&](PtTile& t) {
    const int left = total - taken, grid = gridDim.x;
    const bool halves = 2 * left <= grid;
    const int round = min(halves ? 2 * left : left, grid);
    if ((int)blockIdx.x >= round) return false;
    int at = (int)xcd_block(blockIdx.x, round);
    half = halves ? at % 2 : -1;
    at = halves ? at / 2 : at;
    t = pt_tile<kGlu>(a, map, tiles, taken + at, cols);
    taken += gridDim.x;
    return true;
  };
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t base = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);

  const int steps = (a.D + kPtDepth - 1) / kPtDepth;
  // the XCDs at different steps, unless it is one instance whose rows and weights they share (8192
  // rows, 4096 channels, depth 7168: 172 us, else 177)
  const int first = a.offset ? pt_first((int)blockIdx.x, 8, steps) : 0;
  // a wave fills 32 rows of both operands' buffers, 8 by 8
  const int fetch = pt_fetch_lane(lane, a.D);
  int w_fetch = fetch;                                   // of another's channels nothing
  auto fetch_piece = [&](const PtTile& t, int step, int i) {   // i: 0..3 weights, 4..7 rows
    const uint32_t to = base + (step % 2) * kPtBuf + wave * 4096 + (i % 4) * 1024;
    const int r = wave * 32 + i % 4 * 8, f = r % 128 / 16;
    const int ch = t.c0 + (kGlu ? r / 128 * 64 + f / 2 * 16 + r % 16 + f % 2 * a.n_out : r);
    const int from = step + first < steps - 1 ? step + first : step + first - (steps - 1);
    const int more = (step < steps - 1 ? from : step) * kPtDepth;
    if (i < 4) pt_fetch(t.ws, to, w_fetch, (ch < a.N ? ch : 0) * a.D + more);
    else pt_fetch(t.qs, to + 2 * kPtBuf, fetch, (r < t.n_rows ? r : 0) * a.D + more);
  };
  // The two waves of a SIMD (w and w + 4) differ in channels and in rows, so that half of a tile's
  // rows, or half of its channels, is work for every SIMD.
  const int w_half = wave / 4, w_wave = w_half * 128, q_wave = (wave + 2 * w_half) % 4 * 64;
  // scales of the wave's channels (SwiGLU: gates, then ups) and rows, then the first two steps
  auto begin = [&](const PtTile& t, int odd) {
    const uint32_t to = base + kPtTurn + wave * 4096 + kPtScales + odd * kPtScaleBytes;
    const int ch = t.c0 + (kGlu ? w_half * 64 : w_wave), ch2 = ch + (kGlu ? a.n_out : 64);
    const i32x4 w_scale = pt_span(t.w_scale, a.N * 4ll);
    pt_fetch4(w_scale, to, lane * 4, (ch < a.N ? ch : 0) * 4);
    pt_fetch4(w_scale, to + 256, lane * 4, (ch2 < a.N ? ch2 : 0) * 4);
    pt_fetch4(pt_span(a.q_scale + t.row0, t.n_rows * 4ll), to + 512, lane * 4,
              (q_wave < t.n_rows ? q_wave : 0) * 4);
    for (int i = 0; i < 8; ++i) fetch_piece(t, 0, i);
    if (steps > 1)
      for (int i = 0; i < 8; ++i) fetch_piece(t, 1, i);
  };

  const int part = pt_read_lane(lane);
  const char* w_lds = lds + w_wave * kPtDepth;
  const char* q_lds = lds + 2 * kPtBuf + q_wave * kPtDepth;
  i32x4 acc[8][4], w[2][8], x[2][4];
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
  auto first_half = [&](int k) {
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      if (f < 4) read_x(k, 1, f);
      read_w(k, 1, f);
      multiply(0, f);
      __builtin_amdgcn_sched_barrier(0);                 // keeps the reads between the products
    }
  };
  // Own reads of this step are in registers, own loads of the next have landed; then everyone's.
  // Loads of a tile's first two steps have before it begins, and the last tile's results may still
  // be on their way out (16384 rows, 8192 channels, depth 2048: 227 -> 224 us).
  auto meet = [&](bool loads) {
    if (loads) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto second_half = [&](const PtTile& t, int k, bool more) {
    meet(k > 0);
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      if (more) fetch_piece(t, k + 2, f);
      if (f < 4) read_x(k + 1, 0, f);
      read_w(k + 1, 0, f);
      multiply(1, f);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  PtTile t;
  if (!next(t)) return;
  w_fetch = half < 0 || half == w_half ? fetch : kPrFar;
  begin(t, 0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  for (int odd = 0;; odd ^= 1) {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // a wave whose rows are past the tile's, or whose channels another workgroup has, only fetches:
    // its neighbour has the SIMD to itself
    const bool busy = q_wave < t.n_rows && (half < 0 || half == w_half);
    if (busy) {
#pragma unroll
      for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[f][j] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        if (f < 4) read_x(0, 0, f);
        read_w(0, 0, f);
      }
      int k = 0;
      for (; k < steps - 2; ++k) {
        first_half(k);
        second_half(t, k, true);
      }
      if (k < steps - 1) {
        first_half(k);
        second_half(t, k, false);
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
    } else {
      for (int k = 0; k < steps - 1; ++k) {
        meet(k > 0);
        if (k + 2 < steps)
          for (int i = 0; i < 8; ++i) fetch_piece(t, k + 2, i);
      }
    }
    const PtTile done = t;
    const bool again = next(t);
    if (again) {
      w_fetch = half < 0 || half == w_half ? fetch : kPrFar;
      meet(true);                                        // the buffers are free
      begin(t, odd ^ 1);
    }
    if (!busy) {
      if (!again) break;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      continue;
    }
#pragma unroll
    for (int f = 0; f < 8; ++f) multiply(1, f);

    // Results: 16 rows by 64 channels at a time through the wave's own LDS into whole lines.
    // Rows and channels outside go past the span's end, so that the number of stores is fixed.
    int l = lane;                                        // what is made of it, is made here
    asm volatile("" : "+v"(l));
    char* own = lds + kPtTurn + wave * 4096;
    const float* scales = reinterpret_cast<const float*>(own + kPtScales + odd * kPtScaleBytes);
    const span_t os = span_of(a.out + done.row0 * a.n_out, (int64_t)done.n_rows * a.n_out * 2);
    constexpr int kPasses = kGlu ? 1 : 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q_scale = scales[128 + 16 * j + l % 16];
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
#pragma unroll
        for (int o = 0; o < 4; ++o) {                    // 16 outputs
          const int f = kGlu ? 2 * o : 4 * p + o, at = (4 * p + o) * 16 + l / 16 * 4;
          const f32x4 s = *reinterpret_cast<const f32x4*>(scales + at);
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = pr_scaled(acc[f][j][i], s[i], q_scale);
          if constexpr (kGlu) {
            const f32x4 s_up = *reinterpret_cast<const f32x4*>(scales + 64 + at);
            float up[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) up[i] = pr_scaled(acc[f + 1][j][i], s_up[i], q_scale);
            pr_swiglu(y, up);
          }
          const int piece = (2 * o + l / 32) ^ l % 8;
          *reinterpret_cast<uint2*>(own + l % 16 * 128 + piece * 16 + l / 16 % 2 * 8) =
              uint2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 8 * h + l / 8, row = q_wave + 16 * j + r;
          const int ch = done.c0 + (kGlu ? w_half * 64 : w_wave + 64 * p) + l % 8 * 8;
          const u32x4 v = *reinterpret_cast<const u32x4*>(own + r * 128 + (l % 8 ^ r % 8) * 16);
          const bool in = row < done.n_rows && ch < a.n_out;
          __builtin_amdgcn_raw_buffer_store_b128(v, os, in ? (row * a.n_out + ch) * 2 : kPrFar, 0, 0);
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
    if (!again) break;
    // the loads before those stores, in order
    if constexpr (kGlu) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
  }
}

// Launches of fewer than 2^32 threads each, over ranges of tiles.
template <int kCh, int kRows, int kWC, int kWR, int kGroups, int kStages, bool kGlu>
static uep_status pr_ring(const PrArgs& a, hipStream_t s) {
  constexpr int kWide = kGlu ? kCh / 2 : kCh, kThreads = kWC * kWR * kGroups * kWave;
  const int cols = (a.n_out + kWide - 1) / kWide;
  const int64_t tiles = pr_most_tiles(a.rows, a.n_inst, kRows);
  const int64_t most = ((1ll << 32) - 1) / kThreads / cols;
  for (int64_t t = 0; t < tiles; t += most) {
    const int n = (int)std::min(tiles - t, most);
    hipLaunchKernelGGL((pr_ring_kernel<kCh, kRows, kWC, kWR, kGroups, kStages, kGlu>),
                       dim3((unsigned)n * cols), dim3(kThreads), 0, s, a, (int)t, n, cols);
    UEP_CHECK_LAUNCH();
  }
  return UEP_OK;
}

// One workgroup for every CU; the tiles' number is known on the device only.
template <bool kGlu>
static uep_status pr_tiles_of(const PrArgs& a, hipStream_t s) {
  constexpr int kWide = kGlu ? kPtSide / 2 : kPtSide;
  const int cols = (a.n_out + kWide - 1) / kWide;
  const int64_t tiles = pr_most_tiles(a.rows, a.n_inst, kPtSide);
  // twice the tiles: a tile may be two workgroups' work
  hipLaunchKernelGGL((pr_tile_kernel<kGlu>),
                     dim3((unsigned)std::min<int64_t>(2 * tiles * cols, kPtGroups)),
                     dim3(kPtThreads), 0, s, a, cols, (int)tiles);
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}

template <bool kGlu>
static uep_status pr_run(const PrArgs& a, hipStream_t s) {
  switch (pr_form(a.rows, a.n_inst, a.n_out, a.D, kGlu)) {
    case kPrLarge: return pr_tiles_of<kGlu>(a, s);
    case kPr128x128: return pr_ring<128, 128, 4, 2, 1, 2, kGlu>(a, s);
    case kPr128x128Deep: return pr_ring<128, 128, 4, 2, 1, 4, kGlu>(a, s);
    case kPr64x128: return pr_ring<64, 128, 2, 2, 2, 3, kGlu>(a, s);
    case kPr128x64: return pr_ring<128, 64, 2, 2, 1, 3, kGlu>(a, s);
    case kPr64x64: return pr_ring<64, 64, 2, 2, 2, 4, kGlu>(a, s);
    case kPr64x32Deep: return pr_ring<64, 32, 2, 2, 2, 5, kGlu>(a, s);
    case kPr64x32: return pr_ring<64, 32, 2, 2, 1, 4, kGlu>(a, s);
    case kPr32x16: return pr_ring<32, 16, 1, 1, 8, 3, kGlu>(a, s);
    case kPr16x16:
      if constexpr (!kGlu) return pr_ring<16, 16, 1, 1, 8, 4, kGlu>(a, s);
    default: return pr_ring<32, 32, 1, 2, 1, 8, kGlu>(a, s);
  }
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
      n_out % 8 != 0 || (int64_t)N * D >= (1ll << 31) || rows > kPrMaxRows)
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
