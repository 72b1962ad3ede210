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
};

// What a row asks for.
struct Wanted {
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
  uint64_t mass[kSampleBins];
  uint32_t count[kSampleBins];
  uint64_t tile_mass[kMaxTiles];
  int32_t tile_ties[kMaxTiles];
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

template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_row_kernel(
    SampleParams a) {
  __shared__ SampleLds s;
  sample_row<T>(a, (int64_t)blockIdx.x, s);
}

}  // namespace ltk
