// Balance loss of the router and its gradient (uep.h: uep_balance_loss, uep_balance_loss_grad).
//
// Loss.  A block takes one chunk of one sequence.  The chunk's ids, read in one piece, give its
// counts and which tokens are present; then every logit is read once: a token's kL lanes make its
// scores, and each lane adds those of its own experts over the tokens that it sees, so that sums
// over tokens stay in registers until the block ends.  The chunks' sums are joined in a second
// launch in a fixed order, without float atomics: a call repeats its bits.
// Gradient.  One pass: the scores again from the logits, one dot product a token with the
// sequence's counts, which a lane keeps in registers.
// Both are bound by HBM, with sigmoid scores by the exponentials and reciprocals beside it.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "logits.h"
#include "numeric.h"
#include "rules.h"

namespace uep {

constexpr int kBlMaxE = 4096;
constexpr int kBlMaxSeq = 65535;      // blocks of the second launch
constexpr int kBlSliceWide = 4;       // threads of a joining block for a slice of the experts

// How the tokens fall into chunks of at most `size` tokens of one sequence each.  Equal
// sequences have `per` chunks each.  Otherwise chunk numbers go by offset[g] / size + g, which
// leaves every sequence as many as it needs and asks for no sum over the sequences before it;
// `outer` adds the tokens before the first and behind the last as two sequences of their own.
struct BlChunks {
  const int32_t* offset;   // [n_seq + 1] or NULL
  int n_tok, n_seq, len;   // len: of equal sequences
  int size, per;
  int outer;
};
struct BlChunk {
  int seq;                 // -1 or n_seq: outside
  int begin, end;          // tokens, empty if the chunk has none
  int index;               // of this chunk in its sequence
};

__device__ __forceinline__ int bl_edge(const BlChunks& c, int i) {
  if (c.outer) {
    if (i == 0) return 0;
    if (i == c.n_seq + 2) return c.n_tok;
    --i;
  }
  return min(max(c.offset[i], 0), c.n_tok);
}

__device__ __forceinline__ void bl_check_edges(const BlChunks& c, int g, int32_t* err) {
  const int a = c.offset[g], z = c.offset[g + 1];
  if (a < 0 || z < a || z > c.n_tok) set_err(err, UEP_ERR_OFFSET);
}

// Every thread of the block calls it.  Where each has an edge of its own at most, one load finds
// the last edge with number <= b; otherwise every wave searches 64 at a time.
__device__ __forceinline__ BlChunk bl_chunk(const BlChunks& c, int b) {
  if (!c.offset) {
    const int g = b / c.per, j = b % c.per, end = (g + 1) * c.len;
    const int begin = g * c.len + j * c.size;
    return {g, begin, min(begin + c.size, end), j};
  }
  int lo = 0, hi = c.n_seq + (c.outer ? 2 : 0), begin, end;
  if (hi < (int)blockDim.x) {
    __shared__ int edge[2];
    const int i = threadIdx.x, at = bl_edge(c, min(i, hi));
    lo = max(__syncthreads_count(i < hi && (i == 0 || at / c.size + i <= b)) - 1, 0);
    if (i == lo || i == lo + 1) edge[i - lo] = at;
    __syncthreads();
    begin = edge[0], end = edge[1];
  } else {
    const int lane = threadIdx.x % kWave;
    while (hi - lo > 1) {
      const int step = (hi - lo + kWave - 1) / kWave, at = lo + lane * step;
      const bool below = at < hi && (at == lo || bl_edge(c, at) / c.size + at <= b);
      const int n = __popcll(ballot(below));
      lo = min(lo + (n - 1) * step, hi - 1);
      hi = min(lo + step, hi);
    }
    begin = bl_edge(c, lo), end = bl_edge(c, lo + 1);
  }
  const int j = b - (begin / c.size + lo);
  BlChunk k;
  k.seq = c.outer ? lo - 1 : lo;
  k.index = j;
  k.begin = j < 0 || end <= begin || j > (end - begin) / c.size ? end : begin + j * c.size;
  k.end = min(k.begin + c.size, end);
  return k;
}

// Calls f(token of the chunk, id) for every id of the chunk in [0, E); true if one is
// neither that nor -1.  k_magic = ceil(2^32 / K), exact for the at most 2^17 ids of a chunk.
template <typename F>
__device__ __forceinline__ bool bl_ids(const int32_t* ids, const BlChunk& c, int E, int K,
                                       uint32_t k_magic, F f) {
  const int n = (c.end - c.begin) * K, step = blockDim.x;
  const int32_t* p = ids + (int64_t)c.begin * K;
  bool bad = false;
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * step) {
    int e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) e[u] = i0 + u * step < n ? p[i0 + u * step] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * step;
      const bool in = e[u] >= 0 && e[u] < E;
      bad |= !in && e[u] != -1;
      if (in) f(K == 1 ? i : (int)__umulhi(i, k_magic), e[u]);
    }
  }
  return bad;
}

// over the kL lanes of a token
template <int kL, typename Op>
__device__ __forceinline__ float bl_lanes(float v, Op op) {
  auto moved = [](float x, auto dpp) {
    return __int_as_float(
        __builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(dpp)::value, 0xF, 0xF, true));
  };
  if (kL >= 2) v = op(v, moved(v, std::integral_constant<int, 0xB1>()));     // xor 1
  if (kL >= 4) v = op(v, moved(v, std::integral_constant<int, 0x4E>()));     // xor 2
  if (kL >= 8) v = op(v, moved(v, std::integral_constant<int, 0x141>()));    // half mirror
  if (kL >= 16) v = op(v, moved(v, std::integral_constant<int, 0x140>()));   // mirror
  if (kL >= 32) v = op(v, __shfl_xor(v, 16, kWave));
  if (kL >= 64) v = op(v, __shfl_xor(v, 32, kWave));
  return v;
}
template <int kL>
__device__ __forceinline__ float bl_lanes_sum(float v) {
  return bl_lanes<kL>(v, [](float a, float b) { return a + b; });
}
template <int kL>
__device__ __forceinline__ float bl_lanes_max(float v) {
  return bl_lanes<kL>(v, [](float a, float b) { return fmaxf(a, b); });
}

// A lane's part of a row: kNV vectors of kCe experts, the vectors of a token's lanes side by
// side.  kVec false (rows shorter than one vector): single experts.
template <typename T, int kL, int kNV, bool kVec>
struct BlRow {
  static constexpr int kCe = kVec ? 16 / (int)sizeof(T) : 1;
  static constexpr int kPer = kNV * kCe;
  static constexpr int kRaw = kVec ? kNV : (kNV + 3) / 4;
  u32x4 raw[kRaw];

  static __device__ __forceinline__ int expert(int lane, int i) {
    return (i / kCe * kL + lane) * kCe + i % kCe;
  }
  // experts at or past E are masked
  __device__ __forceinline__ void load(const T* row, int lane, int E) {
    if constexpr (kVec) {
      if (E % kCe == 0) {
#pragma unroll
        for (int v = 0; v < kNV; ++v) raw[v] = gt_load16<false>(row, (v * kL + lane) * kCe, E);
      } else {
#pragma unroll
        for (int v = 0; v < kNV; ++v) raw[v] = gt_load16<true>(row, (v * kL + lane) * kCe, E);
      }
    } else {
#pragma unroll
      for (int v = 0; v < kNV; ++v) {
        const int e = v * kL + lane;
        uint32_t w = 0xFF800000u;
        if (e < E) {
          if constexpr (sizeof(T) == 4) w = __float_as_uint(row[e]);
          else w = (uint32_t)row[e] << 16;
        }
        raw[v / 4][v % 4] = w;
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (kVec) return gt_element<T>(raw[i / kCe], i % kCe);
    else return __uint_as_float(raw[i / 4][i % 4]);
  }
  // Non-temporal: the logits and what is added stay in the last-level cache (262144 tokens of 256
  // bf16 logits, sigmoid, added to others: 104 -> 81 us; with such loads too 98).
  static __device__ __forceinline__ void store(T* row, int lane, int E, const float (&x)[kPer]) {
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      const int e0 = (v * kL + lane) * kCe;
      if constexpr (kVec) {
        if (e0 + kCe <= E) {
          u32x4 w;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(x[v * kCe + j]);
            else w[j] = pack_bf16(x[v * kCe + 2 * j], x[v * kCe + 2 * j + 1]);
          }
          __builtin_nontemporal_store((typename GtLoose<T>::type)w,
                                      reinterpret_cast<typename GtLoose<T>::type*>(row + e0));
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < kCe; ++j)
        if (e0 + j < E) {
          if constexpr (sizeof(T) == 4) row[e0 + j] = x[v * kCe + j];
          else row[e0 + j] = (T)f32_to_bf16(x[v * kCe + j]);
        }
    }
  }
};

// Scores of one token into s, and the factor that makes them sum to one (0 if none is left).
// Only finite logits have a score; NaN and +infinity are reported in `bad`: a NaN makes the sum
// one, and so does +infinity through the softmax's maximum; a sigmoid is asked for its maximum.
// The sigmoid's 1 - s = e^-l s goes into `rest` where the gradient asks for it (anything finite
// where s is 0).  Scores below 2^-126 are 0.
template <bool kSig, bool kRest, int kL, typename Row>
__device__ __forceinline__ float bl_scores(const Row& row, float (&s)[Row::kPer],
                                           float (&rest)[Row::kPer], bool& bad) {
  float x[Row::kPer];
#pragma unroll
  for (int i = 0; i < Row::kPer; ++i) x[i] = row.at(i);
  float top, total;
  auto score = [&]() {
    top = x[0];
#pragma unroll
    for (int i = 1; i < Row::kPer; ++i) top = fmaxf(top, x[i]);
    total = 0.0f;
    if constexpr (kSig) {
#pragma unroll
      for (int i = 0; i < Row::kPer; ++i) {
        const float t = __builtin_amdgcn_exp2f(-1.44269504f * x[i]);
        s[i] = __builtin_amdgcn_rcpf(1.0f + t);
        if constexpr (kRest) rest[i] = fminf(t, 0x1p126f) * s[i];
        total += s[i];
      }
    } else {
      top = bl_lanes_max<kL>(top);
      const float from = top > -__builtin_inff() ? top : 0.0f;      // every expert masked
#pragma unroll
      for (int i = 0; i < Row::kPer; ++i) {
        s[i] = gt_exp(x[i] - from);
        total += s[i];
      }
    }
  };
  score();
  const bool odd = !gt_finite(total) || (kSig && top == __builtin_inff());
  if (ballot(odd)) {
    bad |= odd;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i)
      if (!gt_finite(x[i])) x[i] = -__builtin_inff();
    score();
  }
  total = bl_lanes_sum<kL>(total);
  return total > 0.0f ? 1.0f / total : 0.0f;
}

// Partial sums of the chunks: rows of `pitch` (E rounded up to whole vectors).
struct BlPartial {
  float* prob;      // [chunks][pitch]
  int32_t* count;   // [chunks][pitch]
  int32_t* tokens;  // [chunks]
  double* loss;     // [n_seq][slices]
};

// What a sequence's sums are worth: E / (K n) * sum_e counts_e sum_e / n.
__device__ __forceinline__ float bl_loss(double dot, int E, int K, int n) {
  return n > 0 ? (float)(dot * E / ((double)K * n * n)) : 0.0f;
}

__device__ __forceinline__ double bl_wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// kWhole: every sequence is one chunk, and the block writes the call's outputs.
template <typename T, bool kSig, int kL, int kNV, bool kVec, bool kWhole>
__global__ __launch_bounds__(kBlThreads) void bl_sum_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ ids, BlChunks chunks, int E, int K,
    uint32_t k_magic, int pitch, BlPartial part, float* __restrict__ loss,
    int32_t* __restrict__ counts, float* __restrict__ prob, int32_t* __restrict__ tokens,
    int32_t* err) {
  typedef BlRow<T, kL, kNV, kVec> Row;
  constexpr int kWaves = kBlThreads / kWave, kCols = kL * Row::kPer;
  __shared__ float sum[kWaves][kCols];
  __shared__ int32_t hist[kCols], present;
  __shared__ uint8_t live[kBlMaxChunk];
  __shared__ double loss_wave[kWaves];
  const int b = blockIdx.x, lane = threadIdx.x % kL, group = threadIdx.x / kL;
  const int groups = blockDim.x / kL, wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
  const BlChunk c = bl_chunk(chunks, b);
  const int n_tok = c.end - c.begin;
  if (!kWhole && n_tok <= 0) return;
  // the first row is on its way while the ids are counted
  constexpr bool kAhead = Row::kPer <= 16;
  Row next;
  const T* first = logits + (int64_t)c.begin * E;
  auto fetch = [&](int t) {
    next.load(first + (int64_t)(t < n_tok ? t : 0) * E, lane, t < n_tok ? E : 0);
  };
  if (kAhead) fetch(group);
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  for (int t = threadIdx.x; t < n_tok; t += blockDim.x) live[t] = 0;
  if (threadIdx.x == 0) present = 0;
  __syncthreads();
  const bool bad_id = bl_ids(ids, c, E, K, k_magic, [&](int t, int e) {
    live[t] = 1;
    atomicAdd(&hist[e], 1);
  });
  __syncthreads();
  int mine = 0;
  for (int t = threadIdx.x; t < n_tok; t += blockDim.x) mine += live[t];
  mine = wave_sum(mine);
  if (threadIdx.x % kWave == 0) atomicAdd(&present, mine);

  float acc[Row::kPer] = {};
  bool bad_logit = false;
  for (int t0 = 0; t0 < n_tok; t0 += groups) {
    const int t = t0 + group;
    if (!kAhead) fetch(t);
    const Row row = next;
    if (kAhead) fetch(t + groups);
    float s[Row::kPer], rest[Row::kPer];
    bool bad = false;
    const float share = bl_scores<kSig, false, kL>(row, s, rest, bad);
    const bool here = t < n_tok && live[t];
    bad_logit |= bad && here;                     // an absent token may hold anything
    const float on = here ? share : 0.0f;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) acc[i] = fmaf(s[i], on, acc[i]);
  }
  if (ballot(bad_logit) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_LOGIT);
  if (ballot(bad_id) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_ID_RANGE);

  // a wave's tokens by butterflies, the waves in order
#pragma unroll
  for (int o = kL; o < kWave; o *= 2)
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) acc[i] += __shfl_xor(acc[i], o, kWave);
  if (threadIdx.x % kWave < kL)
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) sum[wave][Row::expert(lane, i)] = acc[i];
  __syncthreads();
  const int n = present;
  double dot = 0.0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float p = sum[0][e];
    for (int w = 1; w < waves; ++w) p += sum[w][e];
    if constexpr (kWhole) {
      counts[(int64_t)c.seq * E + e] = hist[e];
      prob[(int64_t)c.seq * E + e] = n > 0 ? p / (float)n : 0.0f;
      dot += (double)hist[e] * (double)p;
    } else {
      part.prob[(int64_t)b * pitch + e] = p;
      part.count[(int64_t)b * pitch + e] = hist[e];
    }
  }
  if constexpr (kWhole) {
    dot = bl_wave_sum(dot);
    if (threadIdx.x % kWave == 0) loss_wave[wave] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < waves; ++w) dot += loss_wave[w];
      tokens[c.seq] = n;
      loss[c.seq] = bl_loss(dot, E, K, n);
    }
  } else {
    if (threadIdx.x == 0) part.tokens[b] = n;
  }
}

// Joins the chunks of one sequence in 64 bits: `wide` threads have four experts each, the other
// factor of the block shares the chunks out; rows of sums are added as a tree.  A sequence of many
// chunks is joined by several blocks, for 4 `wide` experts each; their parts of the loss are added
// by a launch of its own.
constexpr int kBlJoin = 1024;
__global__ __launch_bounds__(kBlJoin) void bl_join_kernel(
    BlChunks chunks, int E, int K, int pitch, int wide, BlPartial part, float* __restrict__ loss,
    int32_t* __restrict__ counts, float* __restrict__ prob, int32_t* __restrict__ tokens,
    int32_t* err) {
  __shared__ double p_lds[4][kBlJoin];
  __shared__ int32_t c_lds[4][kBlJoin];
  __shared__ double loss_wave[kBlJoin / kWave];
  __shared__ int32_t present;
  const int g = blockIdx.x, col = threadIdx.x % wide, r = threadIdx.x / wide;
  const int rows = blockDim.x / wide, slices = gridDim.y;
  int64_t first;
  int n_ch;
  if (!chunks.offset) {
    first = (int64_t)g * chunks.per;
    n_ch = chunks.per;
  } else {
    if (threadIdx.x == 0) bl_check_edges(chunks, g, err);
    const int lo = bl_edge(chunks, g), hi = bl_edge(chunks, g + 1);
    first = lo / chunks.size + g;
    n_ch = hi > lo ? (hi - lo + chunks.size - 1) / chunks.size : 0;
  }
  if (threadIdx.x == 0) present = 0;
  __syncthreads();
  int mine = 0;
  for (int j = threadIdx.x; j < n_ch; j += blockDim.x) mine += part.tokens[first + j];
  mine = wave_sum(mine);
  if (threadIdx.x % kWave == 0 && mine) atomicAdd(&present, mine);
  double dot = 0.0;
  for (int q0 = blockIdx.y * wide; 4 * q0 < E; q0 += slices * wide) {
    const int e0 = 4 * (q0 + col);
    double p[4] = {};
    int32_t k[4] = {};
    if (e0 < E) {
#pragma unroll 8
      for (int j = r; j < n_ch; j += rows) {
        const int64_t at = (first + j) * pitch + e0;
        const f32x4 a = *reinterpret_cast<const f32x4*>(part.prob + at);
        const u32x4 c = *reinterpret_cast<const u32x4*>(part.count + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] += a[i], k[i] += (int32_t)c[i];
      }
    }
    __syncthreads();                              // the last round's reads
#pragma unroll
    for (int i = 0; i < 4; ++i) p_lds[i][threadIdx.x] = p[i], c_lds[i][threadIdx.x] = k[i];
    for (int h = rows / 2; h > 0; h /= 2) {
      __syncthreads();
      if (r < h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p_lds[i][threadIdx.x] += p_lds[i][threadIdx.x + h * wide];
          c_lds[i][threadIdx.x] += c_lds[i][threadIdx.x + h * wide];
        }
    }
    __syncthreads();
    const int n = present;
    if (r == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < E) {
          const double s = p_lds[i][col];
          const int32_t c = c_lds[i][col];
          counts[(int64_t)g * E + e0 + i] = c;
          prob[(int64_t)g * E + e0 + i] = n > 0 ? (float)(s / n) : 0.0f;
          dot += s * c;
        }
  }
  dot = bl_wave_sum(dot);
  if (threadIdx.x % kWave == 0) loss_wave[threadIdx.x / kWave] = dot;
  __syncthreads();
  if (threadIdx.x > 0) return;
  for (int w = 1; w < (int)blockDim.x / kWave; ++w) dot += loss_wave[w];
  if (blockIdx.y == 0) tokens[g] = present;
  if (slices == 1) loss[g] = bl_loss(dot, E, K, present);
  else part.loss[(int64_t)g * slices + blockIdx.y] = dot;
}

// A wave for each sequence adds its slices' parts, in an order that their number fixes.
__global__ __launch_bounds__(kWave) void bl_loss_kernel(BlPartial part, int slices, int E, int K,
                                                        const int32_t* __restrict__ tokens,
                                                        float* __restrict__ loss) {
  const int g = blockIdx.x;
  double dot = 0.0;
  for (int i = threadIdx.x; i < slices; i += kWave) dot += part.loss[(int64_t)g * slices + i];
  dot = bl_wave_sum(dot);
  if (threadIdx.x == 0) loss[g] = bl_loss(dot, E, K, tokens[g]);
}

// dl_e = f p_e ((c_e - c_0) - sum_j p_j (c_j - c_0)) [(1 - s_e)].  c_0 is the integer next to
// sum_j p_j c_j: the sum is at most about half, so that the result keeps its digits where one
// expert takes nearly all of p, and where the chosen ones take next to nothing.  Counts are
// subtracted as integers, the first expert's before c_0 is looked for (a whole group's counts are
// past 2^24, and what tells them apart are their last digits).  The factor that makes the scores
// sum to one goes up to 2^126 and meets the scores first: p and what follows stay in range.
__device__ __forceinline__ int32_t bl_minus(int32_t a, int32_t b) {     // wraps
  return (int32_t)((uint32_t)a - (uint32_t)b);
}

template <typename T, bool kSig, bool kAdd, int kL, int kNV, bool kVec>
__global__ __launch_bounds__(kBlThreads) void bl_grad_kernel(
    const float* __restrict__ dloss, const T* __restrict__ logits,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, BlChunks chunks, int E, int K, uint32_t k_magic,
    const T* add, T* dlogits, int32_t* err) {
  typedef BlRow<T, kL, kNV, kVec> Row;
  __shared__ int32_t c_lds[kL * Row::kPer];
  __shared__ uint8_t live[kBlMaxChunk];
  const int lane = threadIdx.x % kL, group = threadIdx.x / kL, groups = blockDim.x / kL;
  if (chunks.offset && blockIdx.x == 0)
    for (int g = threadIdx.x; g < chunks.n_seq; g += blockDim.x) bl_check_edges(chunks, g, err);
  const BlChunk c = bl_chunk(chunks, blockIdx.x);
  const int n_tok = c.end - c.begin;
  if (n_tok <= 0) return;
  const bool inside = c.seq >= 0 && c.seq < chunks.n_seq;
  const int e_read = inside ? E : 0;
  const int64_t first = (int64_t)c.begin * E;
  Row next, next_base;
  auto fetch = [&](int t) {
    const int64_t at = first + (int64_t)(t < n_tok ? t : 0) * E;
    next.load(logits + at, lane, t < n_tok ? e_read : 0);
    if constexpr (kAdd) next_base.load(add + at, lane, t < n_tok ? E : 0);
  };
  constexpr bool kAhead = Row::kPer <= 16;
  if (kAhead) fetch(group);
  for (int t = threadIdx.x; t < n_tok; t += blockDim.x) live[t] = 0;
  if (inside) {
    const int32_t* row = counts + (int64_t)c.seq * E;
    const int32_t some = row[0];
    for (int e = threadIdx.x; e < E; e += blockDim.x) c_lds[e] = bl_minus(row[e], some);
  }
  __syncthreads();
  bool bad_id = false;
  float f = 0.0f;
  if (inside) {
    const double n = tokens[c.seq];
    f = n > 0.0 ? dloss[c.seq] * (float)(E / (K * n * n)) : 0.0f;
    bad_id = bl_ids(ids, c, E, K, k_magic, [&](int t, int) { live[t] = 1; });
  }
  __syncthreads();
  int32_t cnt[Row::kPer];
#pragma unroll
  for (int i = 0; i < Row::kPer; ++i) {
    const int e = Row::expert(lane, i);
    cnt[i] = inside && e < E ? c_lds[e] : 0;
  }
  bool bad_logit = false;
  for (int t0 = 0; t0 < n_tok; t0 += groups) {
    const int t = t0 + group;
    if (!kAhead) fetch(t);
    const Row row = next, base = next_base;
    if (kAhead) fetch(t + groups);
    const bool on = t < n_tok && live[t];
    float s[Row::kPer], rest[Row::kPer], out[Row::kPer];
    bool bad = false;
    const float share = bl_scores<kSig, kSig, kL>(row, s, rest, bad);
    bad_logit |= bad && on;                       // an absent token may hold anything
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) {
      s[i] *= share;
      dot = fmaf(s[i], (float)cnt[i], dot);
    }
    // the largest floats that are int32
    const int32_t c0 = (int32_t)rintf(fminf(fmaxf(bl_lanes_sum<kL>(dot), -0x1p31f), 0x1.fffffep30f));
    dot = 0.0f;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) {
      out[i] = (float)bl_minus(cnt[i], c0);
      dot = fmaf(s[i], out[i], dot);
    }
    dot = bl_lanes_sum<kL>(dot);
    const float h = on && share > 0.0f ? f : 0.0f;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) {
      float d = s[i] * (out[i] - dot) * h;
      if constexpr (kSig) d *= rest[i];
      if constexpr (kAdd) d += base.at(i);
      out[i] = d;
    }
    if (t < n_tok) Row::store(dlogits + first + (int64_t)t * E, lane, E, out);
  }
  if (ballot(bad_logit) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_LOGIT);
  if (ballot(bad_id) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_ID_RANGE);
}

// ---------------------------------------------------------------------------------------
struct BlCall {
  const void* logits;
  const int32_t *ids, *offset;
  int n_tok, n_seq, E, K;
  BlPartial part;
  float* loss;
  int32_t* counts;
  float* prob;
  int32_t* tokens;
  const float* dloss;
  const void* add;
  void* dlogits;
  int32_t* err;
  hipStream_t stream;
};

static int64_t bl_n_chunks(const BlChunks& c) {
  if (!c.offset) return (int64_t)c.n_seq * c.per;
  return (int64_t)c.n_tok / c.size + c.n_seq + (c.outer ? 2 : 0);
}

static BlChunks bl_chunks(const int32_t* offset, int n_tok, int n_seq, int size, bool outer) {
  BlChunks c;
  c.offset = offset;
  c.n_tok = n_tok;
  c.n_seq = n_seq;
  c.len = offset ? 0 : n_tok / n_seq;
  c.size = size;
  c.per = offset ? 0 : std::max(1, (c.len + c.size - 1) / c.size);
  c.outer = offset && outer;
  return c;
}

static uint32_t bl_magic(int K) { return K == 1 ? 0u : (uint32_t)(((1ull << 32) + K - 1) / K); }
static int bl_pitch(int E) { return (E + 3) / 4 * 4; }

template <typename T, bool kSig, int kL, int kNV, bool kVec, bool kWhole>
static void bl_sum(const BlCall& c, const BlChunks& ch) {
  hipLaunchKernelGGL((bl_sum_kernel<T, kSig, kL, kNV, kVec, kWhole>),
                     dim3((unsigned)bl_n_chunks(ch)), dim3(kBlThreads), 0, c.stream,
                     static_cast<const T*>(c.logits), c.ids, ch, c.E, c.K, bl_magic(c.K),
                     bl_pitch(c.E), c.part, c.loss, c.counts, c.prob, c.tokens, c.err);
}

template <typename T, bool kSig, int kL, int kNV, bool kVec>
static uep_status bl_forward(const BlCall& c) {
  const int size =
      bl_chunk_tokens(c.n_tok, c.E, sizeof(T), bl_sum_blocks(c.n_tok, c.E, sizeof(T)));
  // Short sequences: a block each and no second launch, up to eight passes over the block's lanes
  // (or a chunk, of so many tokens).  32 sequences of 4, 8 and 16 passes, E = 128 fp32: 8.5, 9.8 and
  // 15.7 us by one launch, 11.3, 11.1 and 10.8 by two; E = 1000 bf16: 8.5, 10.5 and 17.1, 11.9, 11.9 and 12.5.
  const int len = c.n_tok / c.n_seq;
  constexpr int kMost = 8 * kBlThreads / kL;
  static_assert(kMost <= kBlMaxChunk, "tokens of a chunk");
  if (!c.offset && len <= std::max(size, kMost)) {
    bl_sum<T, kSig, kL, kNV, kVec, true>(
        c, bl_chunks(nullptr, c.n_tok, c.n_seq, std::max(len, 1), false));
    UEP_CHECK_LAUNCH();
    return UEP_OK;
  }
  const BlChunks ch = bl_chunks(c.offset, c.n_tok, c.n_seq, size, false);
  bl_sum<T, kSig, kL, kNV, kVec, false>(c, ch);
  UEP_CHECK_LAUNCH();
  // as many rows of threads as a sequence has chunks on the average
  const int64_t mean = bl_n_chunks(ch) / c.n_seq;
  int wide = kBlSliceWide, slices = 1;
  if (bl_sliced(mean, c.E)) slices = (c.E + 4 * wide - 1) / (4 * wide);
  else
    while (wide < 256 && 4 * wide < c.E) wide *= 2;
  int threads = std::max(wide, kWave);
  while (threads < kBlJoin && threads / wide < mean) threads *= 2;
  hipLaunchKernelGGL(bl_join_kernel, dim3((unsigned)c.n_seq, slices), dim3(threads), 0, c.stream,
                     ch, c.E, c.K, bl_pitch(c.E), wide, c.part, c.loss, c.counts, c.prob,
                     c.tokens, c.err);
  if (slices > 1) {
    UEP_CHECK_LAUNCH();
    hipLaunchKernelGGL(bl_loss_kernel, dim3((unsigned)c.n_seq), dim3(kWave), 0, c.stream, c.part,
                       slices, c.E, c.K, c.tokens, c.loss);
  }
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}

template <typename T, bool kSig, int kL, int kNV, bool kVec>
static uep_status bl_backward(const BlCall& c) {
  const BlChunks ch = bl_chunks(c.offset, c.n_tok, c.n_seq,
                                bl_chunk_tokens(c.n_tok, c.E, sizeof(T), kBlGradBlocks), true);
#define UEP_BL_GRAD(ADD)                                                                        \
  hipLaunchKernelGGL((bl_grad_kernel<T, kSig, ADD, kL, kNV, kVec>),                             \
                     dim3((unsigned)bl_n_chunks(ch)), dim3(kBlThreads), 0, c.stream, c.dloss,    \
                     static_cast<const T*>(c.logits), c.ids, c.counts, c.tokens, ch, c.E, c.K,  \
                     bl_magic(c.K), static_cast<const T*>(c.add), static_cast<T*>(c.dlogits),   \
                     c.err)
  if (c.add) UEP_BL_GRAD(true);
  else UEP_BL_GRAD(false);
#undef UEP_BL_GRAD
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}

template <typename T, bool kSig, int kL, int kNV, bool kVec>
static uep_status bl_either(const BlCall& c) {
  return c.dlogits ? bl_backward<T, kSig, kL, kNV, kVec>(c)
                   : bl_forward<T, kSig, kL, kNV, kVec>(c);
}

template <typename T, bool kSig>
static uep_status bl_by_experts(const BlCall& c) {
  constexpr int kSize = sizeof(T);
  if (c.E * kSize < 16) return bl_either<T, kSig, 8, 1, false>(c);
  switch (bl_lanes_of(c.E, kSize)) {
    case 2: return bl_either<T, kSig, 2, kSize, true>(c);
    case 4: return bl_either<T, kSig, 4, kSize, true>(c);
    case 8: return bl_either<T, kSig, 8, kSize, true>(c);
    case 16: return bl_either<T, kSig, 16, kSize, true>(c);
    case 32: return bl_either<T, kSig, 32, kSize, true>(c);
    default: break;
  }
  if (c.E <= 1024) return bl_either<T, kSig, 64, kSize, true>(c);
  return bl_either<T, kSig, 64, 4 * kSize, true>(c);
}

static uep_status bl_run(const BlCall& c, int dtype, int score) {
  const bool sig = score == UEP_GATE_SIGMOID;
  if (dtype == UEP_F32) return sig ? bl_by_experts<float, true>(c) : bl_by_experts<float, false>(c);
  return sig ? bl_by_experts<uint16_t, true>(c) : bl_by_experts<uint16_t, false>(c);
}

static uep_status bl_check(const void* logits, int32_t dtype, const int32_t* topk_ids,
                           const int32_t* seq_offset, int32_t n_seq, int32_t R, int32_t T,
                           int32_t E, int32_t K, int32_t score) {
  if (R <= 0 || T < 0 || E <= 0 || K <= 0 || n_seq <= 0) return UEP_EINVAL;
  if (dtype != UEP_F32 && dtype != UEP_BF16) return UEP_EINVAL;
  if (score != UEP_GATE_SOFTMAX && score != UEP_GATE_SIGMOID) return UEP_EINVAL;
  if (R > 64 || E > kBlMaxE || K > 64 || n_seq > kBlMaxSeq || (int64_t)n_seq * E >= (1ll << 31) ||
      (int64_t)R * T >= (1ll << 26) || (int64_t)R * T * K >= (1ll << 31))
    return UEP_EGEOM;
  if (!seq_offset && ((int64_t)R * T) % n_seq != 0) return UEP_EGEOM;
  if (T > 0 && (!logits || !topk_ids)) return UEP_EINVAL;
  return UEP_OK;
}

static size_t bl_align(size_t n) { return (n + 255) / 256 * 256; }

// Layout of the workspace; chunks for the smaller of the two dtypes' sizes.
static size_t bl_workspace(char* ws, int64_t n_tok, int64_t n_seq, int E, BlPartial* p) {
  const int64_t size = std::min(bl_chunk_tokens(n_tok, E, 4, bl_sum_blocks(n_tok, E, 4)),
                                bl_chunk_tokens(n_tok, E, 2, bl_sum_blocks(n_tok, E, 2)));
  const size_t chunks = (size_t)(n_tok / size + n_seq);
  const size_t row = bl_align(chunks * bl_pitch(E) * 4), tok = bl_align(chunks * 4);
  // sliced: no more sequences than fill the rule's mean
  const size_t slices = (E + 4 * kBlSliceWide - 1) / (4 * kBlSliceWide);
  const size_t most = std::min<size_t>(n_seq, chunks * E / kBlSliced + 1);
  const size_t sliced = most * slices * sizeof(double);
  if (p) {
    p->loss = reinterpret_cast<double*>(ws + 2 * row + tok);
    p->prob = reinterpret_cast<float*>(ws);
    p->count = reinterpret_cast<int32_t*>(ws + row);
    p->tokens = reinterpret_cast<int32_t*>(ws + 2 * row);
  }
  return 2 * row + tok + bl_align(sliced);
}

}  // namespace uep

using namespace uep;

extern "C" size_t uep_balance_loss_workspace_size(int32_t R, int32_t T, int32_t E,
                                                  int32_t n_seq) {
  if (R <= 0 || R > 64 || T < 0 || E <= 0 || E > kBlMaxE || n_seq <= 0 || n_seq > kBlMaxSeq ||
      (int64_t)R * T >= (1ll << 26))
    return 0;
  return bl_workspace(nullptr, (int64_t)R * T, n_seq, E, nullptr);
}

extern "C" uep_status uep_balance_loss(const void* logits, int32_t dtype,
                                       const int32_t* topk_ids, const int32_t* seq_offset,
                                       int32_t n_seq, int32_t R, int32_t T, int32_t E, int32_t K,
                                       int32_t score, float* loss, int32_t* counts, float* prob,
                                       int32_t* tokens, int32_t* err, void* ws, size_t ws_bytes,
                                       void* stream) {
  const uep_status st = bl_check(logits, dtype, topk_ids, seq_offset, n_seq, R, T, E, K, score);
  if (st != UEP_OK) return st;
  if (!loss || !counts || !prob || !tokens) return UEP_EINVAL;
  const int64_t n_tok = (int64_t)R * T, g = n_seq;
  BlCall c = {};
  if (!ws || ws_bytes < bl_workspace(static_cast<char*>(ws), n_tok, g, E, &c.part))
    return UEP_EWORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return UEP_EGEOM;
  const UepBytes rows{logits, n_tok * E * (dtype == UEP_F32 ? 4 : 2)}, id{topk_ids, n_tok * K * 4};
  const UepBytes ends{seq_offset, (g + 1) * 4}, work{ws, (int64_t)ws_bytes};
  const UepBytes o[4] = {{loss, g * 4}, {counts, g * E * 4}, {prob, g * E * 4}, {tokens, g * 4}};
  if (uep_overlap(work, {rows, id, ends}) || uep_overlap(o[0], {rows, id, ends, work, o[1], o[2], o[3]}) ||
      uep_overlap(o[1], {rows, id, ends, work, o[2], o[3]}) ||
      uep_overlap(o[2], {rows, id, ends, work, o[3]}) || uep_overlap(o[3], {rows, id, ends, work}))
    return UEP_EINVAL;
  c.logits = logits;
  c.ids = topk_ids;
  c.offset = seq_offset;
  c.n_tok = (int)n_tok;
  c.n_seq = n_seq;
  c.E = E;
  c.K = K;
  c.loss = loss;
  c.counts = counts;
  c.prob = prob;
  c.tokens = tokens;
  c.err = err;
  c.stream = uep_stream(stream);
  return bl_run(c, dtype, score);
}

extern "C" uep_status uep_balance_loss_grad(const float* dloss, const void* logits, int32_t dtype,
                                            const int32_t* topk_ids, const int32_t* counts,
                                            const int32_t* tokens, const int32_t* seq_offset,
                                            int32_t n_seq, int32_t R, int32_t T, int32_t E,
                                            int32_t K, int32_t score, const void* add,
                                            void* dlogits, int32_t* err, void* stream) {
  const uep_status st = bl_check(logits, dtype, topk_ids, seq_offset, n_seq, R, T, E, K, score);
  if (st != UEP_OK) return st;
  if (T == 0) return UEP_OK;
  if (!dloss || !counts || !tokens || !dlogits) return UEP_EINVAL;
  const int64_t n_tok = (int64_t)R * T, g = n_seq;
  const int64_t bytes = n_tok * E * (dtype == UEP_F32 ? 4 : 2);
  const UepBytes out{dlogits, bytes};
  if (uep_overlap(out, {{logits, bytes}, {topk_ids, n_tok * K * 4}, {dloss, g * 4},
                        {counts, g * E * 4}, {tokens, g * 4}, {seq_offset, (g + 1) * 4}}) ||
      (add != dlogits && uep_overlap(out, {{add, bytes}})))
    return UEP_EINVAL;
  BlCall c = {};
  c.logits = logits;
  c.ids = topk_ids;
  c.offset = seq_offset;
  c.n_tok = (int)n_tok;
  c.n_seq = n_seq;
  c.E = E;
  c.K = K;
  c.counts = const_cast<int32_t*>(counts);
  c.tokens = const_cast<int32_t*>(tokens);
  c.dloss = dloss;
  c.add = add;
  c.dlogits = dlogits;
  c.err = err;
  c.stream = uep_stream(stream);
  return bl_run(c, dtype, score);
}
