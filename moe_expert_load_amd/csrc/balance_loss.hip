// Balance loss of the router and its gradient (uep.h: uep_balance_loss, uep_balance_loss_grad).
//
// Loss.  Every logit is read once: a token's kL lanes make its scores, and each lane adds the
// scores of its own experts over the tokens that it sees, so the sums over tokens stay in
// registers until a block ends.  A block takes one chunk of one sequence; the chunks' sums are
// joined in a second launch in a fixed order (no float atomics: a call repeats its bits).
// Gradient.  One pass: the scores again from the logits, one dot product a token with the
// sequence's counts, which a block keeps in registers.  Both are bound by HBM.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "logits.h"
#include "numeric.h"

namespace uep {

constexpr int kBlThreads = 256;
constexpr int kBlWaves = kBlThreads / kWave;
constexpr int kBlMaxE = 4096;
constexpr int kBlMaxSeq = 65535;      // a grid's second dimension

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

// Every lane of the wave calls it.  The last edge with number <= b is found 64 at a time.
__device__ __forceinline__ BlChunk bl_chunk(const BlChunks& c, int b) {
  if (!c.offset) {
    const int g = b / c.per, j = b % c.per, end = (g + 1) * c.len;
    const int begin = g * c.len + j * c.size;
    return {g, begin, min(begin + c.size, end), j};
  }
  const int lane = threadIdx.x % kWave;
  int lo = 0, hi = c.n_seq + (c.outer ? 2 : 0);
  while (hi - lo > 1) {
    const int step = (hi - lo + kWave - 1) / kWave, at = lo + lane * step;
    const bool below = at < hi && (at == lo || bl_edge(c, at) / c.size + at <= b);
    const int n = __popcll(ballot(below));
    lo = min(lo + (n - 1) * step, hi - 1);
    hi = min(lo + step, hi);
  }
  const int begin = bl_edge(c, lo), end = bl_edge(c, lo + 1);
  const int j = b - (begin / c.size + lo);
  BlChunk k;
  k.seq = c.outer ? lo - 1 : lo;
  k.index = j;
  k.begin = j < 0 || end <= begin || j > (end - begin) / c.size ? end : begin + j * c.size;
  k.end = min(k.begin + c.size, end);
  return k;
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
          *reinterpret_cast<typename GtLoose<T>::type*>(row + e0) = w;
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
// Only finite logits have a score; NaN and +infinity are reported in `bad`.  The sigmoid's
// 1 - s = e^-l s goes into `rest` where the gradient asks for it.  Scores below 2^-126 are 0.
template <bool kSig, bool kRest, int kL, typename Row>
__device__ __forceinline__ float bl_scores(const Row& row, float (&s)[Row::kPer],
                                           float (&rest)[Row::kPer], bool& bad) {
  float x[Row::kPer];
  bool odd = false;
#pragma unroll
  for (int i = 0; i < Row::kPer; ++i) {
    x[i] = row.at(i);
    odd |= __builtin_amdgcn_classf(x[i], 0x203);      // NaN, +infinity
  }
  if (ballot(odd)) {
    bad |= odd;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i)
      if (!gt_finite(x[i])) x[i] = -__builtin_inff();
  }
  float total = 0.0f;
  if constexpr (kSig) {
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) {
      const float t = __builtin_amdgcn_exp2f(-1.44269504f * x[i]);
      s[i] = __builtin_amdgcn_rcpf(1.0f + t);
      if constexpr (kRest) rest[i] = t < 0x1p100f ? t * s[i] : 1.0f;
      total += s[i];
    }
  } else {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < Row::kPer; ++i) top = fmaxf(top, x[i]);
    top = bl_lanes_max<kL>(top);
    top = gt_finite(top) ? top : 0.0f;                // every expert masked
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) {
      s[i] = gt_exp(x[i] - top);
      total += s[i];
    }
  }
  total = bl_lanes_sum<kL>(total);
  return total > 0.0f ? 1.0f / total : 0.0f;
}

// Partial sums of the chunks, and what joins them.
struct BlPartial {
  float* prob;      // [chunks][E]
  int32_t* count;   // [chunks][E]
  int32_t* tokens;  // [chunks]
  double* loss;     // [n_seq][slices]
  int32_t* ticket;  // [n_seq]
};

__device__ __forceinline__ float bl_factor(double E, double K, double n) {
  return n > 0.0 ? (float)(E / (K * n * n)) : 0.0f;
}

// kWhole: every sequence is one chunk, and the block writes the call's outputs.
template <typename T, bool kSig, int kL, int kNV, bool kVec, bool kWhole>
__global__ __launch_bounds__(kBlThreads) void bl_sum_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ ids, BlChunks chunks, int E, int K,
    BlPartial part, float* __restrict__ loss, int32_t* __restrict__ counts,
    float* __restrict__ prob, int32_t* __restrict__ tokens, int32_t* err) {
  typedef BlRow<T, kL, kNV, kVec> Row;
  constexpr int kGroups = kBlThreads / kL;
  __shared__ float sum[kBlMaxE < kL * Row::kPer ? kBlMaxE : kL * Row::kPer];
  __shared__ int32_t hist[kBlMaxE < kL * Row::kPer ? kBlMaxE : kL * Row::kPer];
  __shared__ int32_t present;
  __shared__ double loss_wave[kBlWaves];
  const int b = blockIdx.x, lane = threadIdx.x % kL, group = threadIdx.x / kL;
  const BlChunk c = bl_chunk(chunks, b);
  if constexpr (!kWhole)
    if (b == 0)
      for (int g = threadIdx.x; g < chunks.n_seq; g += kBlThreads) part.ticket[g] = 0;
  if (!kWhole && c.begin >= c.end) return;
  for (int e = threadIdx.x; e < E; e += kBlThreads) hist[e] = 0, sum[e] = 0.0f;
  if (threadIdx.x == 0) present = 0;
  __syncthreads();

  float acc[Row::kPer] = {};
  bool bad_logit = false, bad_id = false;
  Row next;
  next.load(logits + (int64_t)min(c.begin + group, chunks.n_tok - 1) * E, lane,
            c.begin + group < c.end ? E : 0);
  for (int t0 = c.begin; t0 < c.end; t0 += kGroups) {
    const int t = t0 + group, t1 = t + kGroups;
    const Row row = next;
    next.load(logits + (int64_t)min(t1, chunks.n_tok - 1) * E, lane, t1 < c.end ? E : 0);
    float on = 0.0f;
    if (t < c.end)
      for (int k = lane; k < K; k += kL) {
        const int e = ids[(int64_t)t * K + k];
        const bool in = e >= 0 && e < E;
        bad_id |= !in && e != -1;
        if (in) {
          on = 1.0f;
          atomicAdd(&hist[e], 1);
        }
      }
    on = bl_lanes_max<kL>(on);
    if (on > 0.0f && lane == 0) atomicAdd(&present, 1);
    float s[Row::kPer], rest[Row::kPer];
    bool bad = false;
    const float share = on * bl_scores<kSig, false, kL>(row, s, rest, bad);
    bad_logit |= bad && t < c.end;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) acc[i] = fmaf(s[i], share, acc[i]);
  }
  if (ballot(bad_logit) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_LOGIT);
  if (ballot(bad_id) && threadIdx.x % kWave == 0) set_err(err, UEP_ERR_ID_RANGE);

  // the wave's tokens by butterflies, the waves one after the other
#pragma unroll
  for (int o = kL; o < kWave; o *= 2)
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) acc[i] += __shfl_xor(acc[i], o, kWave);
  for (int w = 0; w < kBlWaves; ++w) {
    if (threadIdx.x / kWave == w && threadIdx.x % kWave < kL)
#pragma unroll
      for (int i = 0; i < Row::kPer; ++i) {
        const int e = Row::expert(lane, i);
        if (e < E) sum[e] += acc[i];
      }
    __syncthreads();
  }
  if constexpr (!kWhole) {
    for (int e = threadIdx.x; e < E; e += kBlThreads) {
      part.prob[(int64_t)b * E + e] = sum[e];
      part.count[(int64_t)b * E + e] = hist[e];
    }
    if (threadIdx.x == 0) part.tokens[b] = present;
    return;
  }
  const int n = present;
  double dot = 0.0;
  for (int e = threadIdx.x; e < E; e += kBlThreads) {
    counts[(int64_t)c.seq * E + e] = hist[e];
    prob[(int64_t)c.seq * E + e] = n > 0 ? sum[e] / (float)n : 0.0f;
    dot += (double)hist[e] * (double)sum[e];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
  if (threadIdx.x % kWave == 0) loss_wave[threadIdx.x / kWave] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kBlWaves; ++w) dot += loss_wave[w];
    tokens[c.seq] = n;
    loss[c.seq] = n > 0 ? (float)(dot * E / ((double)K * n * n)) : 0.0f;
  }
}

// Joins the chunks of one sequence for kBlSlice experts in 64 bits: blockDim.x / kBlSlice
// threads an expert share them out.  The last slice of a sequence adds its loss.
constexpr int kBlSlice = 16;
constexpr int kBlJoinThreads = 1024;
constexpr int kBlJoinRows = kBlJoinThreads / kBlSlice;
__global__ __launch_bounds__(kBlJoinThreads) void bl_join_kernel(
    BlChunks chunks, int E, int K, BlPartial part, float* __restrict__ loss,
    int32_t* __restrict__ counts, float* __restrict__ prob, int32_t* __restrict__ tokens,
    int32_t* err) {
  __shared__ double p_lds[kBlJoinRows][kBlSlice];
  __shared__ int32_t c_lds[kBlJoinRows][kBlSlice], n_lds[kBlJoinRows];
  __shared__ bool last;
  const int g = blockIdx.y, slices = gridDim.x, col = threadIdx.x % kBlSlice;
  const int r = threadIdx.x / kBlSlice, e = blockIdx.x * kBlSlice + col;
  const int rows = blockDim.x / kBlSlice;
  int first, n_ch;
  if (!chunks.offset) {
    first = g * chunks.per;
    n_ch = chunks.per;
  } else {
    if (threadIdx.x == 0) bl_check_edges(chunks, g, err);
    const int lo = bl_edge(chunks, g), hi = bl_edge(chunks, g + 1);
    first = lo / chunks.size + g;
    n_ch = hi > lo ? (hi - lo + chunks.size - 1) / chunks.size : 0;
  }
  double p = 0.0;
  int32_t cnt = 0, n = 0;
#pragma unroll 4
  for (int j = r; j < n_ch; j += rows) {
    const int64_t at = first + j;
    n += part.tokens[at];
    if (e < E) {
      p += part.prob[at * E + e];
      cnt += part.count[at * E + e];
    }
  }
  p_lds[r][col] = p;
  c_lds[r][col] = cnt;
  if (col == 0) n_lds[r] = n;
  __syncthreads();
  for (int h = rows / 2; h > 0; h /= 2) {
    if (r < h) {
      p_lds[r][col] += p_lds[r + h][col];
      c_lds[r][col] += c_lds[r + h][col];
      if (col == 0) n_lds[r] += n_lds[r + h];
    }
    __syncthreads();
  }
  n = n_lds[0];
  if (r == 0 && e < E) {
    counts[(int64_t)g * E + e] = c_lds[0][col];
    prob[(int64_t)g * E + e] = n > 0 ? (float)(p_lds[0][col] / n) : 0.0f;
  }
  if (threadIdx.x == 0) {
    double dot = 0.0;
    for (int i = 0; i < kBlSlice; ++i) dot += p_lds[0][i] * c_lds[0][i];
    __hip_atomic_store(&part.loss[(int64_t)g * slices + blockIdx.x], dot, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(&part.ticket[g], 1, __ATOMIC_ACQ_REL,
                                  __HIP_MEMORY_SCOPE_AGENT) == slices - 1;
  }
  __syncthreads();
  if (!last || threadIdx.x >= kWave) return;
  double dot = 0.0;
  for (int i = threadIdx.x; i < slices; i += kWave)
    dot += __hip_atomic_load(&part.loss[(int64_t)g * slices + i], __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
  if (threadIdx.x == 0) {
    tokens[g] = n;
    loss[g] = n > 0 ? (float)(dot * E / ((double)K * n * n)) : 0.0f;
  }
}

// dl_e = f p_e ((c_e - c_0) - sum_j p_j (c_j - c_0)) [(1 - s_e)].  c_0 is the count of the
// token's first expert, mostly its most likely one: where one expert takes nearly all of p the
// difference then keeps its digits.  Counts enter as floats (exact below 2^24).
template <typename T, bool kSig, bool kAdd, int kL, int kNV, bool kVec>
__global__ __launch_bounds__(kBlThreads) void bl_grad_kernel(
    const float* __restrict__ dloss, const T* __restrict__ logits,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, BlChunks chunks, int E, int K, const T* add, T* dlogits,
    int32_t* err) {
  typedef BlRow<T, kL, kNV, kVec> Row;
  constexpr int kGroups = kBlThreads / kL;
  __shared__ float c_lds[kBlMaxE < kL * Row::kPer ? kBlMaxE : kL * Row::kPer];
  const int lane = threadIdx.x % kL, group = threadIdx.x / kL;
  if (chunks.offset && blockIdx.x == 0)
    for (int g = threadIdx.x; g < chunks.n_seq; g += kBlThreads) bl_check_edges(chunks, g, err);
  const BlChunk c = bl_chunk(chunks, blockIdx.x);
  if (c.begin >= c.end) return;
  const bool inside = c.seq >= 0 && c.seq < chunks.n_seq;
  float f = 0.0f;
  if (inside) {
    f = dloss[c.seq] * bl_factor(E, K, tokens[c.seq]);
    for (int e = threadIdx.x; e < E; e += kBlThreads)
      c_lds[e] = (float)counts[(int64_t)c.seq * E + e];
    __syncthreads();
  }
  float cnt[Row::kPer];
#pragma unroll
  for (int i = 0; i < Row::kPer; ++i) {
    const int e = Row::expert(lane, i);
    cnt[i] = inside && e < E ? c_lds[e] : 0.0f;
  }
  bool bad_logit = false, bad_id = false;
  for (int t0 = c.begin; t0 < c.end; t0 += kGroups) {
    const int t = t0 + group;
    const bool live = t < c.end;
    const int64_t at = (int64_t)(live ? t : c.begin) * E;
    Row row, base;
    row.load(logits + at, lane, live && inside ? E : 0);
    if constexpr (kAdd) base.load(add + at, lane, live ? E : 0);
    float on = 0.0f, c0 = 0.0f;
    if (live && inside) {
      for (int k = lane; k < K; k += kL) {
        const int e = ids[(int64_t)t * K + k];
        const bool in = e >= 0 && e < E;
        bad_id |= !in && e != -1;
        if (in) on = 1.0f;
      }
      const int first = ids[(int64_t)t * K];
      if (first >= 0 && first < E) c0 = c_lds[first];
    }
    on = bl_lanes_max<kL>(on);
    float s[Row::kPer], rest[Row::kPer], out[Row::kPer];
    bool bad = false;
    const float share = bl_scores<kSig, kSig, kL>(row, s, rest, bad);
    bad_logit |= bad;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) dot = fmaf(s[i], cnt[i] - c0, dot);
    dot = bl_lanes_sum<kL>(dot) * share;
    const float h = on > 0.0f && share > 0.0f ? f * share : 0.0f;
#pragma unroll
    for (int i = 0; i < Row::kPer; ++i) {
      float d = h * s[i] * ((cnt[i] - c0) - dot);
      if constexpr (kSig) d *= rest[i];
      if constexpr (kAdd) d += base.at(i);
      out[i] = d;
    }
    if (live) Row::store(dlogits + at, lane, E, out);
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

// Lanes of a token: as few as hold the experts in kNV = 4 vectors each.
static int bl_lanes_of(int E, int size) {
  if (E * size < 16) return 8;
  int l = 2;
  while (l < 64 && l * 64 < E * size) l *= 2;
  return l;
}

// Tokens of a chunk: a block's passes over its kGroups tokens amortise its start and its
// partial sums; about 1024 chunks are enough to fill the chip.
static int bl_chunk_size(int64_t n_tok, int E, int size) {
  const int groups = kBlThreads / bl_lanes_of(E, size);
  int passes = 4;
  while (passes < 64 && n_tok > (int64_t)groups * passes * 1024) passes *= 2;
  return groups * passes;
}

static int64_t bl_n_chunks(const BlChunks& c) {
  if (!c.offset) return (int64_t)c.n_seq * c.per;
  return (int64_t)c.n_tok / c.size + c.n_seq + (c.outer ? 2 : 0);
}

static BlChunks bl_chunks(const int32_t* offset, int n_tok, int n_seq, int E, int size, bool outer) {
  BlChunks c;
  c.offset = offset;
  c.n_tok = n_tok;
  c.n_seq = n_seq;
  c.len = offset ? 0 : n_tok / n_seq;
  c.size = bl_chunk_size(n_tok, E, size);
  c.per = offset ? 0 : std::max(1, (c.len + c.size - 1) / c.size);
  c.outer = offset && outer;
  return c;
}

template <typename T, bool kSig, int kL, int kNV, bool kVec>
static uep_status bl_forward(const BlCall& c) {
  const BlChunks ch = bl_chunks(c.offset, c.n_tok, c.n_seq, c.E, sizeof(T), false);
  const unsigned blocks = (unsigned)bl_n_chunks(ch);
  const T* logits = static_cast<const T*>(c.logits);
  if (!c.offset && ch.per == 1) {
    hipLaunchKernelGGL((bl_sum_kernel<T, kSig, kL, kNV, kVec, true>), dim3(blocks),
                       dim3(kBlThreads), 0, c.stream, logits, c.ids, ch, c.E, c.K, c.part, c.loss,
                       c.counts, c.prob, c.tokens, c.err);
    UEP_CHECK_LAUNCH();
    return UEP_OK;
  }
  hipLaunchKernelGGL((bl_sum_kernel<T, kSig, kL, kNV, kVec, false>), dim3(blocks),
                     dim3(kBlThreads), 0, c.stream, logits, c.ids, ch, c.E, c.K, c.part, c.loss,
                     c.counts, c.prob, c.tokens, c.err);
  UEP_CHECK_LAUNCH();
  const unsigned slices = (unsigned)((c.E + kBlSlice - 1) / kBlSlice);
  int rows = 4;                       // as many as a sequence has chunks on the average
  while (rows < kBlJoinRows && rows * c.n_seq < (int)blocks) rows *= 2;
  hipLaunchKernelGGL(bl_join_kernel, dim3(slices, (unsigned)c.n_seq), dim3(rows * kBlSlice), 0,
                     c.stream, ch, c.E, c.K, c.part, c.loss, c.counts, c.prob, c.tokens, c.err);
  UEP_CHECK_LAUNCH();
  return UEP_OK;
}

template <typename T, bool kSig, int kL, int kNV, bool kVec>
static uep_status bl_backward(const BlCall& c) {
  const BlChunks ch = bl_chunks(c.offset, c.n_tok, c.n_seq, c.E, sizeof(T), true);
  const unsigned blocks = (unsigned)bl_n_chunks(ch);
#define UEP_BL_GRAD(ADD)                                                                        \
  hipLaunchKernelGGL((bl_grad_kernel<T, kSig, ADD, kL, kNV, kVec>), dim3(blocks),               \
                     dim3(kBlThreads), 0, c.stream, c.dloss, static_cast<const T*>(c.logits),   \
                     c.ids, c.counts, c.tokens, ch, c.E, c.K, static_cast<const T*>(c.add),     \
                     static_cast<T*>(c.dlogits), c.err)
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
    case 2: return bl_either<T, kSig, 2, 4, true>(c);
    case 4: return bl_either<T, kSig, 4, 4, true>(c);
    case 8: return bl_either<T, kSig, 8, 4, true>(c);
    case 16: return bl_either<T, kSig, 16, 4, true>(c);
    case 32: return bl_either<T, kSig, 32, 4, true>(c);
    default: break;
  }
  if (c.E * kSize <= 64 * 64) return bl_either<T, kSig, 64, 4, true>(c);
  return bl_either<T, kSig, 64, kBlMaxE * kSize / 16 / 64, true>(c);
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
static size_t bl_workspace(char* ws, int64_t n_tok, int64_t n_seq, int64_t E, BlPartial* p) {
  const int64_t size =
      std::min(bl_chunk_size(n_tok, (int)E, 4), bl_chunk_size(n_tok, (int)E, 2));
  const size_t chunks = (size_t)(n_tok / size + n_seq);
  const size_t slices = (size_t)((E + kBlSlice - 1) / kBlSlice);
  const size_t a = bl_align(n_seq * slices * sizeof(double)), t = bl_align(n_seq * 4);
  const size_t row = bl_align(chunks * E * 4), tok = bl_align(chunks * 4);
  if (p) {
    p->loss = reinterpret_cast<double*>(ws);
    p->ticket = reinterpret_cast<int32_t*>(ws + a);
    p->prob = reinterpret_cast<float*>(ws + a + t);
    p->count = reinterpret_cast<int32_t*>(ws + a + t + row);
    p->tokens = reinterpret_cast<int32_t*>(ws + a + t + 2 * row);
  }
  return a + t + 2 * row + tok;
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
