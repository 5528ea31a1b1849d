// Choices that the host makes by sizes alone: plain C++, so that a test can ask which one a call
// takes.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace uep {

// ------------------------------------------------------------------------- balance loss
constexpr int kBlThreads = 256;
constexpr int kBlMaxChunk = 2048;     // tokens of a chunk

// Lanes of a token: as few as hold the experts with 16 each (above 1024 experts 64 each).  With 32
// a lane the sigmoid's gradient takes 226 registers and two waves a SIMD (262144 tokens of 256
// bf16 logits, added to others: 110 us against 104).
static inline int bl_lanes_of(int E, int size) {
  if (E * size < 16) return 8;
  int l = 2;
  while (l < 64 && l * 16 < E) l *= 2;
  return l;
}

// Blocks to aim at.  Where each leaves sums to be joined, four for every CU, or two for fp32 logits
// (half as many scores to a byte, of either kind) while a block has no more than 256 KiB to read.  One
// loss, us a call, by two and by four: 65536 x 128 19.5 and 21.1 (sigmoid 19.9 and 21.3), 262144 x 128
// 40.1 and 40.7 (41.0 and 41.4), 131072 x 256 38.5 and 40.4; past it 393216 x 128 61.5 and 52.2 (63.6 and
// 52.8), 524288 x 128 64.3 and 64.1, 262144 x 256 61.0 and 62.8.  Chunks are powers of two: where 512
// blocks come out as 384, as for 393216 x 32, two are the slower ones below it too, 26.6 and 24.9.
// bf16 (262144 x 256) 39.8 and 33.8 of kernel.  In the gradient sixteen, so that one block's start is behind another's
// stream (262144 x 256 bf16 sigmoid, added to others, with 4, 8 and 16: 104, 91 and 84 us).
constexpr int kBlGradBlocks = 4096;
static inline int bl_sum_blocks(int64_t n_tok, int E, int size) {
  return size == 4 && n_tok * E * size <= 512ll << 18 ? 512 : 1024;
}

// Tokens of a chunk: a token for every group of lanes until there are about `blocks` blocks, then
// more.
static inline int bl_chunk_tokens(int64_t n_tok, int E, int size, int blocks) {
  const int groups = kBlThreads / bl_lanes_of(E, size);
  int passes = 1;
  while (groups * passes * 2 <= kBlMaxChunk && n_tok > (int64_t)groups * passes * blocks) passes *= 2;
  return groups * passes;
}

// Whether several blocks join a sequence of `mean` chunks, each for some of its experts; their parts
// of the loss take a launch of their own then.  One loss, us by one block and by several: 128
// experts, 128 chunks 11.9 and 14.9, 500 chunks 16.3 and 15.0; 1000 experts, 32 chunks 12.1 and 14.5, 64
// 15.2 and 14.9, 128 21.4 and 14.9; 4096 experts, 17 chunks 23.9 and 15.5.  (64 experts, 500 chunks
// are on the wrong side: 17.3 and 15.8.)
constexpr int64_t kBlSliced = 50000;
static inline bool bl_sliced(int64_t mean, int E) { return mean * E >= kBlSliced; }

// ---------------------------------------------------------------------- expert product
constexpr int kPtDepth = 128;                       // a step of the depth
constexpr int kPtSide = 256;                        // rows and channels of a large tile
constexpr int kPtMostOut = 1 << 21;                 // a large tile's outputs are one span
constexpr int kPtGroups = 256;                      // its workgroups: one a CU

// Tiles of `side` rows are at most so many, whatever the table: every instance that has rows at
// all leaves side - 1 of its last one empty.
static inline int64_t pr_most_tiles(int64_t rows, int n_inst, int side) {
  return (rows + std::min<int64_t>(n_inst, rows) * (side - 1)) / side;
}

// Which tile.  Each form's time is a chip load of workgroups (`resident` a CU) times the steps of
// the depth, at what a step was measured to take with one workgroup a CU (`one`) and with all
// (`all`), plus what a load takes beside its steps (`load`: first loads, results; us).  Half a tile is
// left over in every instance.  The two forms of a wave a step take their time by the weights that
// they stream, and are weighed while each workgroup has a CU to itself.  The form that comes out
// least is taken.  Rows past an instance's are loads that bring nothing, but not for nothing: a form
// is weighed from `mean` rows an instance on (4096 channels, depth 4096, 72 rows in each of 32:
// 113 us by 128 x 128, 144 by 128 x 64; 50 rows of 14, most of them in few: 88 us by 128 x 64, 107 by
// 128 x 128; 13 rows of 34, 5840 channels, depth 5360: 75 us by 64 x 32, 89 by 128 x 64).
// Measured, one instance, 4096 channels, depth 7168, us:
//   rows            1    64   128   256   512  1024  8192 (8192 channels, depth 8192)
//   taken         8.0  12.1  15.5  20.3  27.9  38.5   378
//   next larger   9.3  16.0  20.5  27.8  37.5  53.5
//   next smaller    -  17.8  19.4  27.6  38.5  55.2
struct PrForm {
  int ch, rows, mean, resident;
  float one, all, load;
};
enum { kPrLarge, kPr128x128, kPr128x128Deep, kPr64x128, kPr128x64, kPr64x64, kPr64x32Deep,
       kPr64x32, kPr32x32, kPr32x16, kPr16x16, kPrForms };
constexpr PrForm kPrForm[kPrForms] = {
    {256, 256, 96, 1, 1.50f, 1.50f, 5}, {128, 128, 64, 2, 0.93f, 1.09f, 8},
    {128, 128, 80, 1, 0.66f, 0.66f, 5}, {64, 128, 80, 1, 0.47f, 0.47f, 4},
    {128, 64, 24, 2, 0.60f, 0.87f, 6},  {64, 64, 24, 1, 0.34f, 0.34f, 3},
    {64, 32, 0, 1, 0.27f, 0.27f, 2},    {64, 32, 0, 3, 0.32f, 0.65f, 5},
    {32, 32, 0, 2, 0.20f, 0.31f, 3},    {32, 16, 0, 1, 0.055f, 0.14f, 2.2f},
    {16, 16, 0, 1, 0.054f, 0.09f, 0.5f}};

static inline int pr_form(int64_t rows, int n_inst, int n_out, int D, bool glu) {
  const int64_t used = std::min<int64_t>(n_inst, rows);
  const float steps = (float)((D + kPtDepth - 1) / kPtDepth);
  // ids of tiles and offsets in a tile's outputs are 32-bit in the large kernel
  const int64_t ids = pr_most_tiles(rows, n_inst, kPtSide) * (n_out / (kPtSide / 2) + 1ll);
  const bool fits = n_out <= kPtMostOut && ids < (1ll << 31) - kPtGroups;
  int best = kPr32x32;
  float least = 0.0f;
  for (int i = 0; i < kPrForms; ++i) {
    const PrForm& f = kPrForm[i];
    if ((i == kPrLarge && !fits) || rows < f.mean * used || (glu && f.ch < 32)) continue;
    const int wide = glu ? f.ch / 2 : f.ch;
    const int64_t cols = (n_out + wide - 1) / wide;
    const int64_t groups = cols * std::max(used, (rows + f.rows - 1) / f.rows + used / 2);
    const float loads = (float)groups / (256.0f * f.resident);
    float us = f.load / 2 + steps * f.one;               // at most one workgroup a CU
    if (i >= kPr32x16) {                                 // a wave a step: by the weights it reads
      if (groups > 256) continue;
      us = f.load + steps * (f.one + f.all * (float)(cols * used) / 256.0f);
    } else if (i == kPrLarge) {                          // a last round of halves
      const int64_t last = groups % 256;
      us = (float)(groups / 256) + (last > 128 ? 1.0f : last > 0 ? 0.6f : 0.0f);
      us *= steps * f.one + f.load;
    } else if (f.resident == 1) {
      us = (float)((groups + 255) / 256) * (steps * f.one + f.load);
    } else if (groups > 256) {
      us = std::max(us, loads * (steps * f.all + f.load));
    }
    if (least == 0.0f || us < least) least = us, best = i;
  }
  return best;
}

}  // namespace uep
