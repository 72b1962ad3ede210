// A token for each row of logits, by temperature, top-k, top-p and min-p and
// a given random number.
//
// With x the row (NaN as -infinity), M its largest, w = exp((x - M) / T) and
// the order "larger first, of equals the earlier": the first k; of these the
// shortest prefix whose weights reach p of theirs; of these the ones with
// w >= min_p; and of what is left, in the order of the row, the first where
// the running sum of the weights passes u times their sum.
//
// The token must not depend on how sums are ordered, nor lie beside the one
// that exact arithmetic gives: weights are taken in 64 bits (whose vector
// instructions run at the rate of those in 32) and added as integers, in units
// of 2^-S of the largest, S = 62 - ceil(log2 cols): 2^-45 for 131072 logits.
#pragma once

#include "wave.hpp"

namespace ltk {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / kWave;
constexpr int kSampleVec = 8;  // consecutive logits of a thread
constexpr int kSampleTile = kSampleThreads * kSampleVec;
constexpr int kSampleBins = 2048;  // of a digit of 11 bits
constexpr int kMaxCols = 1 << 24;
constexpr int kMaxTiles = kMaxCols / kSampleTile;

// Types of logits, as in include/libtopk.h.
constexpr int kLogBf16 = 0, kLogF16 = 1, kLogF32 = 3;

struct SampleParams {
  const char* x;
  int64_t ld;  // bytes
  int32_t cols;
  int32_t frac;  // S
  // NULL: the number after them holds for every row
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all;
  int32_t top_k_all;
  float top_p_all, min_p_all;
  const float* u;
  int64_t* tokens;
  float* logprobs;
  // Of each row of a batch, [row - row0][chunk]: see sample_chunk_kernel.
  int64_t row0;
  int32_t chunks;
  int32_t rank;
  uint32_t* chunk_max;
  uint32_t* chunk_from;
  uint32_t* chunk_n;
  double* chunk_sum;
  uint64_t* lists;  // [row - row0][chunk][kChunkList]
  // Of rows whose prefix is wide, [row - row0].., see sample_bins_kernel.
  struct WideRow* wide;
  uint64_t* bins;        // [kWideBins]
  uint64_t* chunk_mass;  // [chunk]
  uint64_t* pivots;      // [kMaxList]
  uint64_t* ticket;
  uint32_t epoch;
};

// What a wide prefix has to reach.
enum { kNotWide = 0, kWideMass = 1, kWideCount = 2, kWideAll = 3 };
struct WideRow {
  uint32_t mode;
  uint32_t top;     // the largest logit's key
  uint64_t goal;    // mass or count
  uint32_t pivots;  // listed so far
  uint32_t spare;
};
constexpr int kWideBins = 2048;
constexpr int kWideChunks = kSampleThreads / kWave;  // of a workgroup

constexpr int kChunk = 1024;     // logits of a wave
constexpr int kChunkList = 64;   // listed of them at most
constexpr int kMaxChunks = 1024; // of a row with lists
constexpr int kMaxList = 4096;   // of a row
constexpr uint32_t kKeyNone = 0x007fffffu;  // of -infinity

// What a row asks for.
struct Wanted {
  __device__ bool all() const { return k == 0 && p >= 1.0 && min_w <= 0.0; }

  double inv_t;   // 1 / temperature
  bool greedy;
  int32_t k;      // 0: all
  double p;       // >= 1: all
  double min_w;   // <= 0: all
  double u;
};
__device__ __forceinline__ Wanted wanted(const SampleParams& a, int64_t row) {
  Wanted r;
  const float t = a.temperature ? a.temperature[row] : a.temperature_all;
  r.greedy = !(t > 0.0f);
  r.inv_t = 1.0 / (double)t;
  const int32_t k = a.top_k ? a.top_k[row] : a.top_k_all;
  r.k = k > 0 && k < a.cols ? k : 0;
  const float p = a.top_p ? a.top_p[row] : a.top_p_all;
  r.p = p < 1.0f ? (double)p : 1.0;  // NaN: all
  const float m = a.min_p ? a.min_p[row] : a.min_p_all;
  r.min_w = m > 0.0f ? (double)fminf(m, 1.0f) : 0.0;
  const float u = a.u[row];
  r.u = u > 0.0f ? (double)u : 0.0;
  return r;
}

// Logits in an order of unsigned integers; 0 and -0 are one number.
__device__ __forceinline__ uint32_t logit_key(float x) {
  const int b = __float_as_int(x);
  return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  const int b = (int)k;
  return __int_as_float(b < 0 ? b ^ (int)0x80000000 : ~b);
}

template <int T>
__device__ __forceinline__ float read_logit(const char* row, int64_t i) {
  float x;
  if constexpr (T == kLogF32)
    x = ((const float*)row)[i];
  else if constexpr (T == kLogBf16)
    x = __int_as_float((int)((const uint16_t*)row)[i] << 16);
  else
    x = (float)((const _Float16*)row)[i];
  return x != x ? -INFINITY : x + 0.0f;  // -0 + 0 = 0
}

// Eight consecutive logits from i on; -infinity past the row's end.
template <int T>
__device__ __forceinline__ void read_logits(const char* row, int64_t i,
                                            int32_t cols,
                                            float (&x)[kSampleVec]) {
  typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
  typedef unsigned u32x4a __attribute__((ext_vector_type(4), aligned(2)));
  if (i + kSampleVec <= cols) {
    if constexpr (T == kLogF32) {
      const f32x4a a = *(const f32x4a*)(row + i * 4);
      const f32x4a b = *(const f32x4a*)(row + i * 4 + 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = a[e];
        x[4 + e] = b[e];
      }
    } else {
      const u32x4a a = *(const u32x4a*)(row + i * 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const unsigned h = e % 2 ? a[e / 2] >> 16 : a[e / 2] & 0xffffu;
        if constexpr (T == kLogBf16)
          x[e] = __uint_as_float(h << 16);
        else
          x[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)h);
      }
    }
#pragma unroll
    for (int e = 0; e < kSampleVec; ++e)
      x[e] = x[e] != x[e] ? -INFINITY : x[e] + 0.0f;
  } else {
#pragma unroll
    for (int e = 0; e < kSampleVec; ++e)
      x[e] = i + e < cols ? read_logit<T>(row, i + e) : -INFINITY;
  }
}

// exp(t) for t <= 0: 2^n 2^f with |f| <= 1/2 and the series of 2^f in f ln 2
// to the 11th power, which leaves (ln 2 / 2)^12 / 12! = 6e-15.
__device__ __forceinline__ double exp_neg(double t) {
  constexpr double kL = 0.693147180559945309417;
  const double y = t * 1.44269504088896340736;
  const double n = rint(y);
  const double f = (y - n) * kL;
  double s = 1.0 / 39916800.0;
  s = fma(s, f, 1.0 / 3628800.0);
  s = fma(s, f, 1.0 / 362880.0);
  s = fma(s, f, 1.0 / 40320.0);
  s = fma(s, f, 1.0 / 5040.0);
  s = fma(s, f, 1.0 / 720.0);
  s = fma(s, f, 1.0 / 120.0);
  s = fma(s, f, 1.0 / 24.0);
  s = fma(s, f, 1.0 / 6.0);
  s = fma(s, f, 0.5);
  s = fma(s, f, 1.0);
  s = fma(s, f, 1.0);
  // n is exact as an int from -1100 on; below that nothing is left.
  return t < -740.0 ? 0.0 : ldexp(s, (int)n);
}

// Weight of a logit next to the row's largest, `top`.
__device__ __forceinline__ double weight_of(float x, float top, double inv_t) {
  if (x == top) return 1.0;
  // -infinity for a masked logit, and for all next to an infinite one
  const double d = (double)x - (double)top;
  return d == -INFINITY ? 0.0 : exp_neg(d * inv_t);
}
__device__ __forceinline__ uint64_t fixed(double w, int frac) {
  return (uint64_t)(ldexp(w, frac) + 0.5);
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int from) {
  const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)v, from, kWave);
  const uint32_t hi = (uint32_t)__shfl((int)(uint32_t)(v >> 32), from, kWave);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint64_t w = shfl64(v, lane() - o < 0 ? 0 : lane() - o);
    if (lane() >= o) v += w;
  }
  return v;
}

// LDS of a row.
struct SampleLds {
  union {
    struct {  // passes over the row
      uint64_t mass[kSampleBins];
      uint32_t count[kSampleBins];
      uint64_t tile_mass[kMaxTiles];
      int32_t tile_ties[kMaxTiles];
    };
    struct {  // its list
      uint64_t sorted[kMaxList];
      uint64_t listed[kMaxList];
    };
  };
  uint64_t sums[kSampleWaves];
  uint64_t found[4];
};

// Exclusive prefix of v over the workgroup's threads, and the total.
__device__ __forceinline__ uint64_t scan_block(uint64_t v, SampleLds& s,
                                               uint64_t* total) {
  const uint64_t incl = wave_scan64(v);
  __syncthreads();  // the last call's sums have been read
  if (lane() == kWave - 1) s.sums[threadIdx.x / kWave] = incl;
  __syncthreads();
  uint64_t before = 0, all = 0;
  for (int i = 0; i < kSampleWaves; ++i) {
    const uint64_t x = s.sums[i];
    if (i < (int)threadIdx.x / kWave) before += x;
    all += x;
  }
  *total = all;
  return before + incl - v;
}

__device__ __forceinline__ uint64_t max_block(uint64_t v, SampleLds& s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t w = shfl64(v, lane() ^ o);
    v = w > v ? w : v;
  }
  __syncthreads();
  if (lane() == 0) s.sums[threadIdx.x / kWave] = v;
  __syncthreads();
  for (int i = 0; i < kSampleWaves; ++i) v = s.sums[i] > v ? s.sums[i] : v;
  return v;
}

// A prefix of the order: all logits with a key above `key`, and the first
// `ties` (by index) of those at it.
struct Prefix {
  uint32_t key;
  int64_t ties;
  uint64_t above;  // count or mass of those above the key
};

// The shortest prefix within `in` whose count (MASS false) or mass reaches
// `goal`, by digits of the key from the top: 11, 11 and 10 bits.
template <int T, bool MASS>
__device__ Prefix find_prefix(const SampleParams& a, const char* row, float top,
                              double inv_t, const Prefix& in, uint64_t goal,
                              SampleLds& s) {
  Prefix out = {0, 0, 0};
  const int tid = threadIdx.x;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    const int high = shift + bits;  // bits above: the prefix found so far
    auto inside = [&](uint32_t k) {
      return high == 32 || k >> high == out.key >> high;
    };
    for (int i = tid; i < kSampleBins; i += kSampleThreads) {
      s.count[i] = 0;
      s.mass[i] = 0;
    }
    __syncthreads();
    for (int64_t i = (int64_t)tid * kSampleVec; i < a.cols; i += kSampleTile) {
      float x[kSampleVec];
      read_logits<T>(row, i, a.cols, x);
#pragma unroll
      for (int e = 0; e < kSampleVec; ++e) {
        const uint32_t k = logit_key(x[e]);
        if (i + e >= a.cols || !inside(k) || (MASS && k <= in.key)) continue;
        const int bin = (int)(k >> shift & ((1u << bits) - 1));
        if constexpr (MASS)
          atomicAdd((unsigned long long*)&s.mass[bin],
                    fixed(weight_of(x[e], top, inv_t), a.frac));
        else
          atomicAdd(&s.count[bin], 1u);
      }
    }
    // of the ties at the bound of `in` only its own count
    if (MASS && tid == 0 && in.ties > 0 && inside(in.key))
      atomicAdd((unsigned long long*)
                    &s.mass[in.key >> shift & ((1u << bits) - 1)],
                (uint64_t)in.ties *
                    fixed(weight_of(key_logit(in.key), top, inv_t), a.frac));
    __syncthreads();
    // Thread i takes bins 2 i and 2 i + 1 counted from the top.
    const int b = kSampleBins - 1 - 2 * tid;
    const uint64_t c0 = MASS ? s.mass[b] : s.count[b];
    const uint64_t c1 = MASS ? s.mass[b - 1] : s.count[b - 1];
    uint64_t all;
    const uint64_t before = out.above + scan_block(c0 + c1, s, &all);
    if (before < goal && goal <= before + c0) {
      s.found[0] = (uint64_t)b;
      s.found[1] = before;
    } else if (before + c0 < goal && goal <= before + c0 + c1) {
      s.found[0] = (uint64_t)(b - 1);
      s.found[1] = before + c0;
    }
    __syncthreads();
    out.key |= (uint32_t)s.found[0] << shift;
    out.above = s.found[1];
    __syncthreads();
  }
  uint64_t one = 1;
  if (MASS) one = fixed(weight_of(key_logit(out.key), top, inv_t), a.frac);
  out.ties = (int64_t)((goal - out.above + one - 1) / one);
  return out;
}

// A row by as many passes over it as it takes, in one workgroup.
template <int T>
__device__ void sample_row(const SampleParams& a, int64_t row_i,
                           SampleLds& s) {
  const int tid = threadIdx.x;
  const char* row = a.x + row_i * a.ld;
  const Wanted want = wanted(a, row_i);
  // ---- the largest, and where it comes first
  uint64_t best = 0;
  for (int64_t i = (int64_t)tid * kSampleVec; i < a.cols; i += kSampleTile) {
    float x[kSampleVec];
    read_logits<T>(row, i, a.cols, x);
#pragma unroll
    for (int e = 0; e < kSampleVec; ++e) {
      const uint64_t w = (uint64_t)logit_key(x[e]) << 32 |
                         (uint32_t) ~(uint32_t)(i + e);
      best = w > best && i + e < a.cols ? w : best;
    }
  }
  best = max_block(best, s);
  const float top = key_logit((uint32_t)(best >> 32));
  const bool none = top == -INFINITY;
  if (none || want.greedy) {
    if (tid == 0) {
      a.tokens[row_i] = none ? -1 : (int64_t)(uint32_t) ~(uint32_t)best;
      a.logprobs[row_i] = none ? -INFINITY : 0.0f;
    }
    return;
  }
  // ---- the prefixes
  Prefix in = {0, 0, 0};  // every key is above 0: all
  if (want.k > 0)
    in = find_prefix<T, false>(a, row, top, want.inv_t, in, (uint64_t)want.k,
                               s);
  if (want.p < 1.0) {
    uint64_t mine = 0, all = 0;
    for (int64_t i = (int64_t)tid * kSampleVec; i < a.cols; i += kSampleTile) {
      float x[kSampleVec];
      read_logits<T>(row, i, a.cols, x);
#pragma unroll
      for (int e = 0; e < kSampleVec; ++e)
        if (logit_key(x[e]) > in.key)
          mine += fixed(weight_of(x[e], top, want.inv_t), a.frac);
    }
    scan_block(mine, s, &all);
    all += (uint64_t)in.ties *
           fixed(weight_of(key_logit(in.key), top, want.inv_t), a.frac);
    const double part = ceil(want.p * (double)all);
    const uint64_t goal = part < 1.0 ? 1 : (uint64_t)part;
    in = find_prefix<T, true>(a, row, top, want.inv_t, in,
                              goal < all ? goal : all, s);
  }
  // ---- in the order of the row
  // Thread t of a tile has its elements 8 t .. 8 t + 7.
  auto masses = [&](int64_t tile, int64_t ties, uint64_t (&m)[kSampleVec],
                    int64_t* ties_after) {
    const int64_t i = tile * kSampleTile + (int64_t)tid * kSampleVec;
    float x[kSampleVec];
    read_logits<T>(row, i, a.cols, x);
    int n = 0;
#pragma unroll
    for (int e = 0; e < kSampleVec; ++e)
      n += i + e < a.cols && logit_key(x[e]) == in.key;
    uint64_t all;
    int64_t nth = ties + (int64_t)scan_block((uint64_t)n, s, &all);
    *ties_after = ties + (int64_t)all;
    uint64_t sum = 0;
#pragma unroll
    for (int e = 0; e < kSampleVec; ++e) {
      const uint32_t k = logit_key(x[e]);
      bool kept = k > in.key;
      if (i + e < a.cols && k == in.key) kept = nth++ < in.ties;
      m[e] = 0;
      if (kept) {
        const double w = weight_of(x[e], top, want.inv_t);
        if (w >= want.min_w) m[e] = fixed(w, a.frac);
      }
      sum += m[e];
    }
    return sum;
  };
  const int tiles = (int)((a.cols + (int64_t)kSampleTile - 1) / kSampleTile);
  int64_t ties = 0;
  uint64_t total = 0;
  for (int t = 0; t < tiles; ++t) {
    uint64_t m[kSampleVec], all;
    int64_t after;
    const uint64_t sum = masses(t, ties, m, &after);
    scan_block(sum, s, &all);
    if (tid == 0) {
      s.tile_mass[t] = total;
      s.tile_ties[t] = (int32_t)ties;
    }
    total += all;
    ties = after;
  }
  __syncthreads();
  uint64_t goal = (uint64_t)(want.u * (double)total);
  if (goal >= total) goal = total - 1;
  int t = tiles - 1;
  while (s.tile_mass[t] > goal) --t;
  uint64_t m[kSampleVec], all;
  int64_t after;
  const uint64_t sum = masses(t, s.tile_ties[t], m, &after);
  uint64_t part = s.tile_mass[t] + scan_block(sum, s, &all);
  if (part <= goal && goal < part + sum) {
    int e = 0;
    while (part + m[e] <= goal) part += m[e++];
    const int64_t i = (int64_t)t * kSampleTile + (int64_t)tid * kSampleVec + e;
    a.tokens[row_i] = i;
    a.logprobs[row_i] =
        (float)(log(weight_of(read_logit<T>(row, i), top, want.inv_t)) -
                log(ldexp((double)total, -a.frac)));
  }
}

// ---- lists ------------------------------------------------------------------
// Few of a row's logits decide it as a rule, and one pass over the row finds
// them: every wave reads a chunk of 1024 and leaves
//   the largest, and the sum of the weights next to that (if the row asks);
//   a bound, and the logits from the bound on, at most 64, in the row's order.
// The bound is the rank-th largest of what the 64 lanes have as their largest,
// so that the list has some more than `rank`, whatever the numbers are like.
// Above the largest bound of a row's chunks nothing is missing in its lists:
// a prefix of the order that ends above it is found there, by sorting at most
// 4096 words.  Rows whose prefix goes further are done over.
template <int T>
struct ChunkShape {
  static constexpr int VEC = 16 / (T == kLogF32 ? 4 : 2);  // logits of a load
  static constexpr int LOADS = kChunk / kWave / VEC;
  static constexpr int N = VEC * LOADS;  // of a lane: 16
  // Index in the chunk of a lane's logit e.
  __device__ static int at(int e) {
    return (e / VEC * kWave + lane()) * VEC + e % VEC;
  }
};
// A wave reads a chunk; -infinity for NaN and past the row's end.
template <int T>
__device__ __forceinline__ void read_chunk(const char* row, int first,
                                           int32_t cols,
                                           float (&x)[ChunkShape<T>::N]) {
  typedef ChunkShape<T> S;
#pragma unroll
  for (int j = 0; j < S::LOADS; ++j) {
    const int i = first + (j * kWave + lane()) * S::VEC;
    if (i + S::VEC <= cols) {
      if constexpr (T == kLogF32) {
        typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
        const f32x4a v = *(const f32x4a*)(row + (int64_t)i * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j * 4 + e] = v[e];
      } else {
        typedef unsigned u32x4a __attribute__((ext_vector_type(4), aligned(2)));
        const u32x4a v = *(const u32x4a*)(row + (int64_t)i * 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const unsigned d = v[e / 2];
          const unsigned h = e % 2 ? d >> 16 : d & 0xffffu;
          if constexpr (T == kLogBf16)
            x[j * 8 + e] = __uint_as_float(h << 16);
          else
            x[j * 8 + e] = (float)__builtin_bit_cast(_Float16, (uint16_t)h);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < S::VEC; ++e)
        x[j * S::VEC + e] =
            i + e < cols ? read_logit<T>(row, i + e) : -INFINITY;
    }
  }
#pragma unroll
  for (int e = 0; e < S::N; ++e)
    x[e] = x[e] != x[e] ? -INFINITY : x[e] + 0.0f;
}

template <int T>
__global__ __launch_bounds__(kBlock) void sample_chunk_kernel(SampleParams a) {
  typedef ChunkShape<T> S;
  constexpr int VEC = S::VEC, LOADS = S::LOADS, N = S::N;
  const int wg = (a.chunks + kWaves - 1) / kWaves;
  const int r = (int)(blockIdx.x / (unsigned)wg);
  const int chunk =
      uni((int)(blockIdx.x % (unsigned)wg) * kWaves + (int)threadIdx.x / kWave);
  if (chunk >= a.chunks) return;
  const int64_t row_i = a.row0 + r;
  const char* row = a.x + row_i * a.ld;
  const Wanted want = wanted(a, row_i);
  const int ln = lane();
  const int first = chunk * kChunk;
  float x[N];
  read_chunk<T>(row, first, a.cols, x);
  uint32_t k[N];
  uint32_t mine = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    k[e] = logit_key(x[e]);
    mine = k[e] > mine ? k[e] : mine;
  }
  const int64_t at = (int64_t)r * a.chunks + chunk;
  const int sorted = wave_sort_desc<kWave>(unbias(mine));
  const uint32_t top = bias(__builtin_amdgcn_readlane(sorted, 0));
  const float m = key_logit(top);
  if (ln == 0) a.chunk_max[at] = top;
  if (want.greedy || top == kKeyNone) {
    if (ln == 0) {
      a.chunk_from[at] = kKeyNone + 1;  // lists all above -infinity: none
      a.chunk_n[at] = 0;
      a.chunk_sum[at] = 0.0;
    }
    return;
  }
  if (want.k == 0 && (want.p < 1.0 || want.min_w <= 0.0)) {
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < N; ++e) sum += weight_of(x[e], m, want.inv_t);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    if (ln == 0) a.chunk_sum[at] = sum;
  }
  if (want.all()) return;
  // ---- the list
  uint32_t from = 0;
  int n = 0;
  bool fits = false;
  for (int rank = a.rank; rank > 0 && !fits; rank /= 2) {
    from = bias(__builtin_amdgcn_readlane(sorted, rank - 1));
    // (-infinity is never listed)
    from = from > kKeyNone ? from : kKeyNone + 1;
    n = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) n += popc(ballot(k[e] >= from));
    fits = n <= kChunkList;
  }
  if (!fits) {  // more than 64 of the largest: none is listed
    n = 0;
    from = top + 1;
  }
  if (ln == 0) {
    a.chunk_from[at] = from;
    a.chunk_n[at] = (uint32_t)n;
  }
  uint64_t* list = a.lists + at * kChunkList;
  int before = 0;
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    int c = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) c += k[j * VEC + e] >= from;
    if (ballot(c > 0) == 0) continue;
    const int incl = wave_scan_incl(c);
    int to = before + incl - c;
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (k[j * VEC + e] >= from) {
        const uint32_t i = (uint32_t)(first + (j * kWave + ln) * VEC + e);
        list[to++] = (uint64_t)k[j * VEC + e] << 32 | (uint32_t)~i;
      }
    }
  }
}

// Keeps LDS accesses of a wave in their order (which the hardware keeps).
__device__ __forceinline__ void wave_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// Sorts 1024 E words in LDS, largest first: a bitonic network in which a wave
// keeps to its own 64 E words wherever partners are that near.
template <int E>
__device__ void sort_words(uint64_t* w) {
  constexpr int P = kSampleThreads * E, R = P / kSampleWaves;
  const int ln = lane(), wave = (int)threadIdx.x / kWave;
  __syncthreads();
  for (int size = 2; size <= P; size *= 2) {
    for (int j = size / 2; j > 0; j /= 2) {
      const bool far = 2 * j > R;
      if (far) __syncthreads();
#pragma unroll
      for (int m = 0; m < (E + 1) / 2; ++m) {
        const int i = wave * (R / 2) + m * kWave + ln;
        if (E > 1 || ln < R / 2) {
          const int lo = (i & ~(j - 1)) * 2 + (i & (j - 1));
          const uint64_t x = w[lo], y = w[lo + j];
          if ((x < y) == ((lo & size) == 0)) {
            w[lo] = y;
            w[lo + j] = x;
          }
        }
      }
      if (far)
        __syncthreads();
      else
        wave_fence();
    }
  }
  __syncthreads();
}

// The prefix of a row whose lists are in s.listed (n words, in the row's order)
// and s.sorted: the last word kept, or 0 if the lists do not reach so far.
// Nothing is missing in them from the key `from` on.
template <int E>
__device__ uint64_t list_prefix(const SampleParams& a, const Wanted& want,
                                float top, uint32_t from, double total,
                                SampleLds& s) {
  const int tid = threadIdx.x;
  sort_words<E>(s.sorted);
  uint64_t w[E], m[E], sum = 0;
  int sure = 0, rare = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    w[e] = s.sorted[tid * E + e];
    const uint32_t key = (uint32_t)(w[e] >> 32);
    const double x =
        key > kKeyNone ? weight_of(key_logit(key), top, want.inv_t) : 0.0;
    m[e] = fixed(x, a.frac);
    sum += m[e];
    sure += key >= from && key > kKeyNone;
    rare += key > kKeyNone && x >= want.min_w;
  }
  uint64_t all;
  uint64_t before = scan_block(sum, s, &all);
  uint64_t counts;
  scan_block((uint64_t)sure << 32 | (uint32_t)rare, s, &counts);
  const int n_sure = (int)(counts >> 32);
  const bool whole = from <= kKeyNone + 1;  // all that has weight is listed
  if (n_sure < 1 || (want.k > n_sure && want.p < 1.0 && !whole)) return 0;
  int last = n_sure;  // words kept
  bool ends = false;  // within what is sure
  if (want.k > 0) {
    // (rows of fewer logits above -infinity than k keep them all)
    if (want.k <= n_sure) ends = true;
    last = want.k < last ? want.k : last;
  }
  if (want.p < 1.0) {
    // The sum that p is a part of: of the first k, or of the row.
    if (want.k > 0) {
      uint64_t part = before;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        part += m[e];
        if (tid * E + e == last - 1) s.found[0] = part;
      }
      __syncthreads();
      total = (double)s.found[0];
      __syncthreads();
    } else {
      total = ldexp(total, a.frac);
    }
    const double part = ceil(want.p * total);
    const uint64_t goal = part < 1.0 ? 1 : (uint64_t)part;
    if (tid == 0) s.found[0] = (uint64_t)last;
    __syncthreads();
    uint64_t sum2 = before;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint64_t next = sum2 + m[e];
      if (sum2 < goal && goal <= next && tid * E + e < last)
        s.found[0] = (uint64_t)(tid * E + e + 1) | 1ull << 32;
      sum2 = next;
    }
    __syncthreads();
    if (s.found[0] >> 32) ends = true;
    last = (int)(uint32_t)s.found[0];
    __syncthreads();
  }
  if (want.min_w > 0.0) {
    const int n_rare = (int)(uint32_t)counts;
    if (n_rare < n_sure) ends = true;
    last = n_rare < last ? n_rare : last;
  }
  return (ends || whole) && last > 0 ? s.sorted[last - 1] : 0;
}

// Rows: from their chunks, or over again.
template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_finish_kernel(
    SampleParams a) {
  __shared__ SampleLds s;
  const int tid = threadIdx.x, wave = tid / kWave, ln = lane();
  const int64_t row_i = a.row0 + blockIdx.x;
  const char* row = a.x + row_i * a.ld;
  const Wanted want = wanted(a, row_i);
  const int64_t base = (int64_t)blockIdx.x * a.chunks;
  if (tid == 0 && a.bins) a.wide[blockIdx.x].mode = kNotWide;
  const bool in = tid < a.chunks;
  const bool lists = !want.all() && !want.greedy;
  const uint32_t chunk_top = in ? a.chunk_max[base + tid] : 0;
  const uint32_t chunk_from = in && lists ? a.chunk_from[base + tid] : 0;
  const int n = in && lists ? (int)a.chunk_n[base + tid] : 0;
  const uint32_t top_key =
      (uint32_t)max_block((uint64_t)chunk_top, s);
  const float top = key_logit(top_key);
  if (top_key == kKeyNone) {
    if (tid == 0) {
      a.tokens[row_i] = -1;
      a.logprobs[row_i] = -INFINITY;
    }
    return;
  }
  double mass = 0.0;
  if (in && want.k == 0 && !want.greedy && (want.p < 1.0 || want.min_w <= 0.0))
    mass = a.chunk_sum[base + tid] *
           weight_of(key_logit(chunk_top), top, want.inv_t);
  if (want.greedy || want.all()) {
    // ---- the chunk, and its logit
    // Inclusive sums of the chunks' masses: in a wave, then of the waves.
    double incl = mass;
    for (int o = 1; o < kWave; o <<= 1) {
      const double y = __shfl_up(incl, o, kWave);
      if (ln >= o) incl += y;
    }
    double* sums = (double*)s.sums;
    __syncthreads();  // the maxima have been read
    if (ln == kWave - 1) sums[wave] = incl;
    __syncthreads();
    double before = 0.0, total = 0.0;
    for (int i = 0; i < kSampleWaves; ++i) {
      if (i < wave) before += sums[i];
      total += sums[i];
    }
    incl += before;
    __syncthreads();
    const double goal = want.u * total;
    // The first chunk that passes the goal; where rounding leaves none, the
    // last one that has weight.
    const bool past = want.greedy ? chunk_top == top_key
                                  : mass > 0.0 && incl > goal;
    uint64_t pick = past ? (uint64_t)(2 * kMaxChunks - tid)
                    : mass > 0.0 ? (uint64_t)tid + 1 : 0;
    if (past) pick += kMaxChunks;
    pick = max_block(pick, s);
    const int chunk = pick > 2 * kMaxChunks ? (int)(3 * kMaxChunks - pick)
                      : (int)pick - 1;
    __syncthreads();
    if (tid == chunk) sums[0] = incl - mass;
    __syncthreads();
    if (wave > 0) return;
    double part = sums[0];
    const int64_t i0 = (int64_t)chunk * kChunk + ln * 16;
    float x[16];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float y[kSampleVec];
      read_logits<T>(row, i0 + j * kSampleVec, a.cols, y);
#pragma unroll
      for (int e = 0; e < kSampleVec; ++e) x[j * kSampleVec + e] = y[e];
    }
    if (want.greedy) {
      int at = 16;
#pragma unroll
      for (int e = 15; e >= 0; --e)
        if (logit_key(x[e]) == top_key) at = e;
      const uint64_t have = ballot(at < 16);
      if (ln == __builtin_ctzll(have)) {
        a.tokens[row_i] = i0 + at;
        a.logprobs[row_i] = 0.0f;
      }
      return;
    }
    double w[16], sum = 0.0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      w[e] = weight_of(x[e], top, want.inv_t);
      sum += w[e];
    }
    double upto = sum;
    for (int o = 1; o < kWave; o <<= 1) {
      const double y = __shfl_up(upto, o, kWave);
      if (ln >= o) upto += y;
    }
    const uint64_t over = ballot(sum > 0.0 && part + upto > goal);
    const uint64_t some = ballot(sum > 0.0);
    const int who = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
    if (ln != who) return;
    part += upto - sum;
    int at = 0;
    bool done = false;
    double got = 0.0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      part += w[e];
      if (!done && w[e] > 0.0) {
        at = e;
        got = w[e];
        done = part > goal;
      }
    }
    a.tokens[row_i] = i0 + at;
    a.logprobs[row_i] = (float)(log(got) - log(total));
    return;
  }
  // ---- lists: their words in LDS, in the row's order
  const uint32_t from = (uint32_t)max_block((uint64_t)chunk_from, s);
  uint64_t all;
  const uint64_t to = scan_block((uint64_t)n, s, &all);
  const int count = (int)all;
  double total = mass;
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, kWave);
  __syncthreads();
  if (ln == 0) ((double*)s.sums)[wave] = total;
  __syncthreads();
  total = 0.0;
  for (int i = 0; i < kSampleWaves; ++i) total += ((double*)s.sums)[i];
  uint64_t cut = 0;
  if (count <= kMaxList && count > 0) {
    for (int c = wave * kWave; c < a.chunks; c += kSampleThreads) {
      // a wave's 64 chunks are those of its own threads
      for (int i = 0; i < kWave && c + i < a.chunks; ++i) {
        const int nc = __builtin_amdgcn_readlane(n, i);
        const int tc = __builtin_amdgcn_readlane((int)to, i);
        if (ln < nc) {
          const uint64_t w = a.lists[(base + c + i) * kChunkList + ln];
          s.listed[tc + ln] = w;
          s.sorted[tc + ln] = w;
        }
      }
    }
    const int room = count <= 1024 ? 1024 : count <= 2048 ? 2048 : 4096;
    for (int i = count + tid; i < room; i += kSampleThreads) {
      s.listed[i] = 0;
      s.sorted[i] = 0;
    }
    cut = room == 1024   ? list_prefix<1>(a, want, top, from, total, s)
          : room == 2048 ? list_prefix<2>(a, want, top, from, total, s)
                         : list_prefix<4>(a, want, top, from, total, s);
  }
  if (cut == 0) {
    __syncthreads();
    const int mode = want.k > 0 ? (want.p < 1.0 ? kNotWide : kWideCount)
                     : want.p < 1.0 ? kWideMass
                                    : kWideAll;
    if (mode == kNotWide || !a.bins) {
      sample_row<T>(a, row_i, s);
      return;
    }
    uint64_t* bins = a.bins + (int64_t)blockIdx.x * kWideBins;
    for (int i = tid; i < kWideBins; i += kSampleThreads) bins[i] = 0;
    if (tid == 0) {
      const double part = ceil(want.p * ldexp(total, a.frac));
      WideRow w = {};
      w.mode = (uint32_t)mode;
      w.top = top_key;
      w.goal = mode == kWideCount ? (uint64_t)want.k
               : part < 1.0       ? 1
                                  : (uint64_t)part;
      a.wide[blockIdx.x] = w;
    }
    return;
  }
  // ---- in the row's order
  constexpr int E = kMaxList / kSampleThreads;
  uint64_t m[E], sum = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    const uint64_t w = i < count ? s.listed[i] : 0;
    m[e] = w >= cut ? fixed(weight_of(key_logit((uint32_t)(w >> 32)), top,
                                      want.inv_t),
                            a.frac)
                    : 0;
    sum += m[e];
  }
  uint64_t kept;
  uint64_t part = scan_block(sum, s, &kept);
  uint64_t goal = (uint64_t)(want.u * (double)kept);
  if (goal >= kept) goal = kept - 1;
  if (part <= goal && goal < part + sum) {
    int e = 0;
    while (part + m[e] <= goal) part += m[e++];
    const uint64_t w = s.listed[tid * E + e];
    a.tokens[row_i] = (int64_t)(uint32_t) ~(uint32_t)w;
    a.logprobs[row_i] = (float)(
        log(weight_of(key_logit((uint32_t)(w >> 32)), top, want.inv_t)) -
        log(ldexp((double)kept, -a.frac)));
  }
}

// ---- wide prefixes ----------------------------------------------------------
// A prefix beyond the lists (a nucleus of tens of thousands) is found in two
// more launches over the row, by workgroups of 16 chunks.  The first adds up
// the masses (or counts) of the logits in 2048 bins of (M - x) / T, 1/64 wide;
// integers, so that their order is nothing.  The second finds the bin in which
// the goal lies, adds up each chunk's mass above it, and lists the bin's own
// logits; the row's last workgroup sorts these, finds the last one kept, the
// chunk where u times the kept mass lies, and the token in it.
__device__ __forceinline__ int wide_bin(float x, float top, double c) {
  const double d = (double)top - (double)x;
  return d > 0.0 ? (int)fmin(d * c, (double)(kWideBins - 1)) : 0;
}

template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_bins_kernel(
    SampleParams a) {
  const int wg = (a.chunks + kWideChunks - 1) / kWideChunks;
  const int r = (int)(blockIdx.x / (unsigned)wg);
  const WideRow wide = a.wide[r];
  if (wide.mode != kWideMass && wide.mode != kWideCount) return;
  __shared__ uint64_t bins[kWideBins];
  const int tid = threadIdx.x;
  for (int i = tid; i < kWideBins; i += kSampleThreads) bins[i] = 0;
  __syncthreads();
  const int64_t row_i = a.row0 + r;
  const Wanted want = wanted(a, row_i);
  const float top = key_logit(wide.top);
  const int chunk =
      (int)(blockIdx.x % (unsigned)wg) * kWideChunks + tid / kWave;
  if (chunk < a.chunks) {
    typedef ChunkShape<T> S;
    float x[S::N];
    read_chunk<T>(a.x + row_i * a.ld, chunk * kChunk, a.cols, x);
    const double c = 64.0 * want.inv_t;
#pragma unroll
    for (int e = 0; e < S::N; ++e) {
      // What lies in the last bin has no weight to speak of: 2^-46 and less.
      const int bin = wide_bin(x[e], top, c);
      if (bin == kWideBins - 1) continue;
      atomicAdd((unsigned long long*)&bins[bin],
                wide.mode == kWideCount
                    ? 1ull
                    : (unsigned long long)fixed(
                          weight_of(x[e], top, want.inv_t), a.frac));
    }
  }
  __syncthreads();
  unsigned long long* all =
      (unsigned long long*)(a.bins + (int64_t)r * kWideBins);
  for (int i = tid; i < kWideBins; i += kSampleThreads)
    if (bins[i]) atomicAdd(all + i, (unsigned long long)bins[i]);
}

// Sorts the first `count` of s.sorted (the others of a power of two become 0)
// and finds how many of them, from the largest, it takes to reach `goal`
// (in masses, or in words); 0 if they do not.
template <int E>
__device__ int pivots_kept(const SampleParams& a, const Wanted& want,
                           const WideRow& wide, uint64_t goal, SampleLds& s) {
  const int tid = threadIdx.x;
  sort_words<E>(s.sorted);
  const float top = key_logit(wide.top);
  uint64_t m[E], sum = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint64_t w = s.sorted[tid * E + e];
    m[e] = 0;
    if (w)
      m[e] = wide.mode == kWideCount
                 ? 1
                 : fixed(weight_of(key_logit((uint32_t)(w >> 32)), top,
                                   want.inv_t),
                         a.frac);
    sum += m[e];
  }
  uint64_t all;
  uint64_t before = scan_block(sum, s, &all);
  if (tid == 0) s.found[0] = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint64_t next = before + m[e];
    if (before < goal && goal <= next) s.found[0] = (uint64_t)(tid * E + e + 1);
    before = next;
  }
  __syncthreads();
  const int n = (int)s.found[0];
  __syncthreads();
  return n;
}

template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_wide_kernel(
    SampleParams a) {
  const int wg = (a.chunks + kWideChunks - 1) / kWideChunks;
  const int r = (int)(blockIdx.x / (unsigned)wg);
  const WideRow wide = a.wide[r];
  if (wide.mode == kNotWide) return;
  __shared__ SampleLds s;
  __shared__ int flag;
  const int tid = threadIdx.x, ln = lane();
  const int64_t row_i = a.row0 + r;
  const char* row = a.x + row_i * a.ld;
  const Wanted want = wanted(a, row_i);
  const float top = key_logit(wide.top);
  const double c = 64.0 * want.inv_t;
  typedef ChunkShape<T> S;
  // ---- the bin of the goal
  int pivot = kWideBins;  // all above it
  uint64_t above = 0;
  if (wide.mode != kWideAll) {
    constexpr int B = kWideBins / kSampleThreads;
    const uint64_t* bins = a.bins + (int64_t)r * kWideBins;
    uint64_t b[B], sum = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      b[i] = bins[tid * B + i];
      sum += b[i];
    }
    uint64_t all;
    uint64_t before = scan_block(sum, s, &all);
    if (tid == 0) s.found[0] = kWideBins;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (before < wide.goal && wide.goal <= before + b[i]) {
        s.found[0] = (uint64_t)(tid * B + i);
        s.found[1] = before;
      }
      before += b[i];
    }
    __syncthreads();
    pivot = (int)s.found[0];
    above = s.found[1];
    __syncthreads();
  }
  // (a goal beyond the bins: the row is done over)
  const bool lost = wide.mode != kWideAll && pivot == kWideBins;
  const int chunk =
      (int)(blockIdx.x % (unsigned)wg) * kWideChunks + tid / kWave;
  uint64_t* const pivots = a.pivots + (int64_t)r * kMaxList;
  if (chunk < a.chunks && !lost) {
    float x[S::N];
    read_chunk<T>(row, chunk * kChunk, a.cols, x);
    uint64_t sum = 0;
    int mine = 0;
#pragma unroll
    for (int e = 0; e < S::N; ++e) {
      const int bin = wide_bin(x[e], top, c);
      if (bin < pivot) {
        const double w = weight_of(x[e], top, want.inv_t);
        if (w >= want.min_w) sum += fixed(w, a.frac);
      }
      mine += bin == pivot && pivot < kWideBins;
    }
    if (ballot(mine > 0)) {
      const int incl = wave_scan_incl(mine);
      unsigned to = 0;
      if (ln == kWave - 1) to = atomicAdd(&a.wide[r].pivots, (unsigned)incl);
      to = (unsigned)__builtin_amdgcn_readlane((int)to, kWave - 1);
      to += (unsigned)(incl - mine);
#pragma unroll
      for (int e = 0; e < S::N; ++e) {
        if (wide_bin(x[e], top, c) != pivot) continue;
        const uint32_t i = (uint32_t)(chunk * kChunk + S::at(e));
        // (past the row's end there is -infinity, which is in the last bin)
        if (to < kMaxList)
          st_agent(pivots + to,
                   (uint64_t)logit_key(x[e]) << 32 | (uint32_t)~i);
        ++to;
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += shfl64(sum, ln ^ o);
    if (ln == 0) st_agent(a.chunk_mass + (int64_t)r * a.chunks + chunk, sum);
  }
  if (!last_to_finish(a.ticket + r, wg, a.epoch, &flag)) return;
  // ---- the row's last workgroup
  const unsigned count = ld_agent(&a.wide[r].pivots);
  uint64_t cut = 0;
  bool done = !lost;
  if (wide.mode != kWideAll && done) {
    done = count <= kMaxList && pivot < kWideBins - 1;
    if (done) {
      const int room = count <= 1024 ? 1024 : count <= 2048 ? 2048 : 4096;
      for (int i = tid; i < room; i += kSampleThreads)
        s.sorted[i] = i < (int)count ? ld_agent(pivots + i) : 0;
      const uint64_t goal = wide.goal - above;
      const int kept =
          room == 1024   ? pivots_kept<1>(a, want, wide, goal, s)
          : room == 2048 ? pivots_kept<2>(a, want, wide, goal, s)
                         : pivots_kept<4>(a, want, wide, goal, s);
      done = kept > 0;
      if (done) cut = s.sorted[kept - 1];
    }
  }
  if (!done) {
    __syncthreads();
    sample_row<T>(a, row_i, s);
    return;
  }
  // Masses of the chunks, in the other half of LDS.
  for (int i = tid; i < kMaxChunks; i += kSampleThreads)
    s.listed[i] = i < a.chunks
                      ? ld_agent(a.chunk_mass + (int64_t)r * a.chunks + i)
                      : 0;
  __syncthreads();
  if (cut) {
    for (int i = tid; i < (int)count; i += kSampleThreads) {
      const uint64_t w = s.sorted[i];
      if (w < cut) continue;
      const double x =
          weight_of(key_logit((uint32_t)(w >> 32)), top, want.inv_t);
      if (x >= want.min_w)
        atomicAdd((unsigned long long*)
                      &s.listed[(uint32_t) ~(uint32_t)w / kChunk],
                  (unsigned long long)fixed(x, a.frac));
    }
    __syncthreads();
  }
  const uint64_t mass = s.listed[tid];
  uint64_t total;
  const uint64_t before = scan_block(mass, s, &total);
  uint64_t goal = (uint64_t)(want.u * (double)total);
  if (goal >= total) goal = total - 1;
  if (before <= goal && goal < before + mass) {
    s.found[0] = (uint64_t)tid;
    s.found[1] = before;
  }
  __syncthreads();
  if (tid >= kWave) return;
  // Lane l takes logits 16 l .. of the chunk.
  uint64_t part = s.found[1];
  const int64_t i0 = (int64_t)s.found[0] * kChunk + ln * 16;
  uint64_t m[16], sum = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float y[kSampleVec];
    read_logits<T>(row, i0 + j * kSampleVec, a.cols, y);
#pragma unroll
    for (int e = 0; e < kSampleVec; ++e) {
      const int64_t i = i0 + j * kSampleVec + e;
      const uint64_t word =
          (uint64_t)logit_key(y[e]) << 32 | (uint32_t) ~(uint32_t)i;
      const double w = weight_of(y[e], top, want.inv_t);
      // (-infinity past the end has no weight)
      m[j * kSampleVec + e] =
          word >= cut && w >= want.min_w ? fixed(w, a.frac) : 0;
      sum += m[j * kSampleVec + e];
    }
  }
  part += wave_scan64(sum) - sum;
  if (part <= goal && goal < part + sum) {
    int at = 0;
    bool past = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      part += m[e];
      if (!past) at = e;
      past = past || part > goal;
    }
    a.tokens[row_i] = i0 + at;
    a.logprobs[row_i] =
        (float)(log(weight_of(read_logit<T>(row, i0 + at), top, want.inv_t)) -
                log(ldexp((double)total, -a.frac)));
  }
}

// Rows too long for lists.
template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_row_kernel(
    SampleParams a) {
  __shared__ SampleLds s;
  sample_row<T>(a, (int64_t)blockIdx.x, s);
}

}  // namespace ltk
