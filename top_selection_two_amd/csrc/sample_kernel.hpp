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
// that exact arithmetic gives: weights are taken in 64 bits (4.4 cycles a vector
// instruction, 2.9 in 32 bits) and, where some are kept and others not, added as
// integers, in units of 2^-S of the largest, S = 62 - ceil(log2 cols) and at
// most 51: 2^-45 for 131072 logits.  Sums of a whole row, which one pass finds
// from chunks that do not know the row's largest, are 64-bit floating point, of
// terms of one sign in a fixed order: some 40 roundings and 2^-50.6 for the
// weights, less than 2^-46 in all.
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
  double unit;   // 2^S
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
  uint32_t* wide_list;   // how many, and which rows they are, in any order
  uint64_t* bins;        // [kWideBins]
  uint64_t* chunk_mass;  // [chunk]
  uint64_t* pivots;      // [kMaxList]
};

// What a wide prefix has to reach.
enum { kWideMass, kWideCount, kWideAll, kWideRow };
struct WideRow {
  uint32_t mode;
  uint32_t top;     // the largest logit's key
  uint64_t goal;    // mass or count
  uint32_t pivots;  // listed so far
  uint32_t spare;
  // Rows' counters lie apart: atomics on one line of memory queue up (32 rows
  // of 200000: 25 us for sample_wide_kernel with four rows a line, 21 so).
  uint32_t apart[26];
};
constexpr int kWideBins = 2048;
constexpr double kWidePerBit = 44.0;  // bins of a factor of 2: 2^-46 in all
constexpr int kWideThreads = 512;
constexpr int kWideChunks = kWideThreads / kWave;  // of a workgroup

constexpr int kChunk = 1024;     // logits of a wave
constexpr int kChunkList = 64;   // listed of them at most
constexpr int kMaxChunks = 1024; // of a row with lists
constexpr int kMaxList = 4096;   // of a row
constexpr uint32_t kKeyNone = 0x007fffffu;  // of -infinity

// What a row asks for.
struct Wanted {
  __device__ bool all() const { return k == 0 && p >= 1.0 && min_w <= 0.0; }
  // Does the sum of the row's weights matter?
  __device__ bool sums() const { return k == 0 && (p < 1.0 || min_w <= 0.0); }

  double inv_t;   // log2 e / temperature
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
  r.inv_t = 1.44269504088896340736 / (double)t;
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

// 2^y for y <= 0: 2^n 2^f with |f| <= 1/2, and 2^f = 1 + f g(f) with g the
// polynomial that meets (2^f - 1) / f at the ten zeros of a Chebyshev
// polynomial: 6e-16 of 2^f are left, and 2^0 is 1.
__device__ __forceinline__ double exp2_neg(double y) {
  // Below 2^-1100 nothing is left; a NaN (0 times infinity) is nothing too.
  y = fmax(y, -1100.0);
  const double n = rint(y), f = y - n;
  double s = 7.07097786650813825e-09;
  s = fma(s, f, 1.02059054137655955e-07);
  s = fma(s, f, 1.32154516332214336e-06);
  s = fma(s, f, 1.52526729248507372e-05);
  s = fma(s, f, 1.54035304247765285e-04);
  s = fma(s, f, 1.33335582007945925e-03);
  s = fma(s, f, 9.61812910761866528e-03);
  s = fma(s, f, 5.55041086646516704e-02);
  s = fma(s, f, 2.40226506959100750e-01);
  s = fma(s, f, 6.93147180559946174e-01);
  s = fma(s, f, 1.0);
  return ldexp(s, (int)n);
}

// ln r, 2^-126 <= r <= 1 (the instruction takes no smaller float32), for
// float32: y from the instruction, which is some 2^-20 off, and the series of
// ln (r / e^y) as far as it takes.
__device__ __forceinline__ double ln_of(double r) {
  double y = (double)__builtin_amdgcn_logf((float)r);
  y = y < 0.0 ? y : 0.0;
  const double d = r / exp2_neg(y) - 1.0;
  return fma(y, 0.693147180559945309417, d - 0.5 * d * d);
}

// Weight of a logit next to the row's largest, `top`; inv_t is log2 e / T.
__device__ __forceinline__ double weight_of(float x, float top, double inv_t) {
  // (next to an infinite one: itself 1, and the others -infinity times inv_t)
  if (top == INFINITY) return x == top ? 1.0 : 0.0;
  return exp2_neg(((double)x - (double)top) * inv_t);
}
// A weight in units of 2^-S, S <= 51: the sum with 2^52 is rounded to a whole
// number, which its low bits are.
__device__ __forceinline__ uint64_t fixed(double w, const SampleParams& a) {
  const double v = fma(w, a.unit, 0x1p52);
  return (uint64_t)__double_as_longlong(v) & 0xfffffffffffffull;
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int from) {
  const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)v, from, kWave);
  const uint32_t hi = (uint32_t)__shfl((int)(uint32_t)(v >> 32), from, kWave);
  return ((uint64_t)hi << 32) | lo;
}
// A 64-bit value moved between lanes; 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t move64(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  return ((uint64_t)hi << 32) | lo;
}
// Inclusive prefix sums over a wave, as wave_scan_incl.
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
  v += move64<0x111, 0xf>(v);
  v += move64<0x112, 0xf>(v);
  v += move64<0x114, 0xf>(v);
  v += move64<0x118, 0xf>(v);
  v += move64<0x142, 0xa>(v);
  v += move64<0x143, 0xc>(v);
  return v;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double move_double(double v) {
  return __longlong_as_double(
      (long long)move64<CTRL, ROWS>((uint64_t)__double_as_longlong(v)));
}
__device__ __forceinline__ double wave_scan_double(double v) {
  v += move_double<0x111, 0xf>(v);
  v += move_double<0x112, 0xf>(v);
  v += move_double<0x114, 0xf>(v);
  v += move_double<0x118, 0xf>(v);
  v += move_double<0x142, 0xa>(v);
  v += move_double<0x143, 0xc>(v);
  return v;
}
// A lane's 64-bit value in all.
__device__ __forceinline__ uint64_t lane64(uint64_t v, int from) {
  const uint32_t lo =
      (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, from);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), from);
  return ((uint64_t)hi << 32) | lo;
}

// LDS of a row.
// What scans of a workgroup need.
struct ScanLds {
  uint64_t sums[kSampleWaves];
  uint64_t found[4];
};
struct SampleLds : ScanLds {
  union {
    struct {  // passes over the row
      uint64_t mass[kSampleBins];  // or counts
      uint64_t tile_mass[kMaxTiles];
      int32_t tile_ties[kMaxTiles];
    };
    struct {  // words of a list
      uint64_t words[kMaxList];
      uint64_t some[2][kMaxList];  // those of one bin, in turn
      uint64_t bin_mass[kSampleBins];
      uint32_t bin_count[kSampleBins];
      uint64_t chunk_mass[kMaxChunks];
    };
  };
  uint32_t gathered;
};

// What a workgroup's waves have, in turn: every wave reads all 16 (one a lane)
// and folds them by moves between lanes, which is less code, and quicker, than
// a loop over them.
template <int WAVES = kSampleWaves>
__device__ __forceinline__ uint64_t wave_item(const uint64_t* x) {
  return lane() < WAVES ? x[lane()] : 0;
}

// Exclusive prefix of v over the workgroup's threads, and the total.
template <int WAVES = kSampleWaves>
__device__ __forceinline__ uint64_t scan_block(uint64_t v, ScanLds& s,
                                               uint64_t* total) {
  const int wave = uni((int)threadIdx.x / kWave);
  const uint64_t incl = wave_scan64(v);
  __syncthreads();  // the last call's sums have been read
  if (lane() == kWave - 1) s.sums[wave] = incl;
  __syncthreads();
  const uint64_t all = wave_scan64(wave_item<WAVES>(s.sums));
  *total = lane64(all, WAVES - 1);
  return (wave ? lane64(all, wave - 1) : 0) + incl - v;
}
__device__ __forceinline__ double scan_block(double v, ScanLds& s,
                                             double* total) {
  const int wave = uni((int)threadIdx.x / kWave);
  const double incl = wave_scan_double(v);
  __syncthreads();
  if (lane() == kWave - 1)
    s.sums[wave] = (uint64_t)__double_as_longlong(incl);
  __syncthreads();
  const double all =
      wave_scan_double(__longlong_as_double((long long)wave_item(s.sums)));
  auto of = [&](int w) {
    return __longlong_as_double(
        (long long)lane64((uint64_t)__double_as_longlong(all), w));
  };
  *total = of(kSampleWaves - 1);
  return (wave ? of(wave - 1) : 0.0) + (incl - v);
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t w = shfl64(v, lane() ^ o);
    v = w > v ? w : v;
  }
  return v;
}
__device__ __forceinline__ uint64_t max_block(uint64_t v, ScanLds& s) {
  v = wave_max64(v);
  __syncthreads();
  if (lane() == 0) s.sums[threadIdx.x / kWave] = v;
  __syncthreads();
  return wave_max64(wave_item(s.sums));
}
// The largest of two numbers each.
__device__ __forceinline__ void max_block(uint32_t* x, uint32_t* y,
                                          ScanLds& s) {
  const int a = wave_max(unbias(*x)), b = wave_max(unbias(*y));
  __syncthreads();
  if (lane() == 0)
    s.sums[threadIdx.x / kWave] = (uint64_t)bias(a) << 32 | bias(b);
  __syncthreads();
  const uint64_t v = wave_item(s.sums);
  *x = bias(wave_max(unbias((uint32_t)(v >> 32))));
  *y = bias(wave_max(unbias((uint32_t)v)));
}
// The first thread where `a` holds; where it does in none, the last where `b`
// does.
__device__ __forceinline__ int first_or_last(bool a, bool b, ScanLds& s) {
  const int wave = (int)threadIdx.x / kWave;
  const uint64_t x = ballot(a), y = ballot(b);
  // the larger is the one: 2^16 - thread for the first, thread + 1 for the last
  const uint32_t i =
      x ? 0x10000u - (uint32_t)(wave * kWave + __builtin_ctzll(x)) : 0u;
  const uint32_t j =
      y ? (uint32_t)(wave * kWave + 64 - __builtin_clzll(y)) : 0u;
  uint32_t p = i, q = j;
  max_block(&p, &q, s);
  return p ? (int)(0x10000u - p) : (int)q - 1;
}

// A prefix of the order: all logits with a key above `key`, and the first
// `ties` (by index) of those at it.
struct Prefix {
  uint32_t key;
  int64_t ties;
  uint64_t above;  // count or mass of those above the key
};

// The shortest prefix within `in` whose count or mass reaches `goal`, by digits
// of the key from the top: 11, 11 and 10 bits.
template <int T>
__device__ __forceinline__ Prefix find_prefix(const SampleParams& a,
                                              const char* row, float top,
                                              double inv_t, bool by_mass,
                                              const Prefix& in, uint64_t goal,
                                              SampleLds& s) {
  Prefix out = {0, 0, 0};
  const int tid = threadIdx.x;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    const int high = shift + bits;  // bits above: the prefix found so far
    auto inside = [&](uint32_t k) {
      return high == 32 || k >> high == out.key >> high;
    };
    for (int i = tid; i < kSampleBins; i += kSampleThreads) {
      s.mass[i] = 0;
    }
    __syncthreads();
    for (int64_t i = (int64_t)tid * kSampleVec; i < a.cols; i += kSampleTile) {
      float x[kSampleVec];
      read_logits<T>(row, i, a.cols, x);
#pragma unroll
      for (int e = 0; e < kSampleVec; ++e) {
        const uint32_t k = logit_key(x[e]);
        if (i + e < a.cols && inside(k) && !(by_mass && k <= in.key))
          atomicAdd(
              (unsigned long long*)&s.mass[k >> shift & ((1u << bits) - 1)],
              by_mass
                  ? (unsigned long long)fixed(weight_of(x[e], top, inv_t), a)
                  : 1ull);
        __builtin_amdgcn_sched_barrier(0);  // one at a time: fewer registers
      }
    }
    // of the ties at the bound of `in` only its own count
    if (by_mass && tid == 0 && in.ties > 0 && inside(in.key))
      atomicAdd((unsigned long long*)
                    &s.mass[in.key >> shift & ((1u << bits) - 1)],
                (uint64_t)in.ties *
                    fixed(weight_of(key_logit(in.key), top, inv_t), a));
    __syncthreads();
    // Thread i takes bins 2 i and 2 i + 1 counted from the top.
    const int b = kSampleBins - 1 - 2 * tid;
    const uint64_t c0 = s.mass[b], c1 = s.mass[b - 1];
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
  if (by_mass) one = fixed(weight_of(key_logit(out.key), top, inv_t), a);
  out.ties = (int64_t)((goal - out.above + one - 1) / one);
  return out;
}

// A row by as many passes over it as it takes, in one workgroup.
template <int T>
__device__ __forceinline__ void sample_row(const SampleParams& a, int64_t row_i,
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
#pragma unroll 1
  for (int step = want.k > 0 ? 0 : 1; step < (want.p < 1.0 ? 2 : 1); ++step) {
    uint64_t goal = (uint64_t)want.k;
    if (step == 1) {
      uint64_t mine = 0, all = 0;
      for (int64_t i = (int64_t)tid * kSampleVec; i < a.cols;
           i += kSampleTile) {
        float x[kSampleVec];
        read_logits<T>(row, i, a.cols, x);
#pragma unroll
        for (int e = 0; e < kSampleVec; ++e) {
          if (logit_key(x[e]) > in.key)
            mine += fixed(weight_of(x[e], top, want.inv_t), a);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      scan_block(mine, s, &all);
      all += (uint64_t)in.ties *
             fixed(weight_of(key_logit(in.key), top, want.inv_t), a);
      const double part = ceil(want.p * (double)all);
      goal = part < 1.0 ? 1 : (uint64_t)part;
      goal = goal < all ? goal : all;
    }
    in = find_prefix<T>(a, row, top, want.inv_t, step == 1, in, goal, s);
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
        if (w >= want.min_w) m[e] = fixed(w, a);
      }
      sum += m[e];
      __builtin_amdgcn_sched_barrier(0);
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
        (float)ln_of(weight_of(read_logit<T>(row, i), top, want.inv_t) /
                     ((double)total / a.unit));
  }
}

// ---- lists ------------------------------------------------------------------
// Few of a row's logits decide it as a rule, and one pass over the row finds
// them: every wave reads a chunk of 1024 and leaves
//   the largest, and the sum of the weights next to that (if the row asks);
//   a bound, and the logits from the bound on, at most 64, in the row's order.
// The bound is the rank-th largest of what the 64 lanes have as their largest,
// so that the list has some more than `rank`, whatever the numbers are like.
// (The least of the maxima of 8 or 16 groups of lanes is found in 12 steps
// instead of the sort's 63, 34 us against 39 for 256 rows of 131072, but varies
// so much that its largest over the chunks leaves lists too short for a top-k
// of 500.)
// Above the largest bound of a row's chunks nothing is missing in its lists:
// a prefix of the order that ends above it is found there, among at most 4096
// words.
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

// Arithmetic bounds it, about 650 vector instructions a chunk (three quarters of
// them in 64 bits, for the weights), where bytes would take a third of the time:
// 256 rows of 131072 in bfloat16, 67 MB, 38 us (1.8 TB/s); 64 rows of 100003 in
// float32 14 us (1.8 TB/s).  Rows that ask for no sum are spared it.
template <int T>
__global__ __launch_bounds__(kBlock) void sample_chunk_kernel(SampleParams a) {
  typedef ChunkShape<T> S;
  constexpr int VEC = S::VEC, LOADS = S::LOADS, N = S::N;
  const int wg = (a.chunks + kWaves - 1) / kWaves;
  const int r = (int)(blockIdx.x / (unsigned)wg);
  const int chunk =
      uni((int)(blockIdx.x % (unsigned)wg) * kWaves + (int)threadIdx.x / kWave);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.wide_list[0] = 0;
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
  if (want.sums()) {
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < N; ++e) sum += weight_of(x[e], m, want.inv_t);
    sum = wave_scan_double(sum);
    if (ln == kWave - 1) a.chunk_sum[at] = sum;
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
  // The lane's listed logits as bits; each load's lie before the next load's.
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) bits |= (k[e] >= from ? 1u : 0u) << e;
  uint64_t* list = a.lists + at * kChunkList;
  int before = 0;
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    uint32_t left = bits >> (j * VEC) & ((1u << VEC) - 1);
    const int c = __popc(left);
    const int incl = wave_scan_incl(c);
    int to = before + incl - c;
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
    while (ballot(left != 0)) {  // two or three times as a rule
      if (left) {
        const int e = __builtin_ctz(left);
        left &= left - 1;
        uint32_t key = k[j * VEC];
#pragma unroll
        for (int i = 1; i < VEC; ++i) key = e == i ? k[j * VEC + i] : key;
        const uint32_t i = (uint32_t)(first + (j * kWave + ln) * VEC + e);
        list[to++] = (uint64_t)key << 32 | (uint32_t)~i;
      }
    }
  }
}

// The bin of a logit: factors of 2 from the largest weight, kWidePerBit bins
// to one.
__device__ __forceinline__ int wide_bin(float x, float top, double c) {
  const double d = (double)top - (double)x;
  return d > 0.0 ? (int)fmin(d * c, (double)(kWideBins - 1)) : 0;
}

// Words are a logit's key, and its index the other way round: the order is
// that of larger words first.

// The shortest prefix of the words, in their order, that reaches `goal` (> 0)
// words or units of mass: its last word, its words and its mass.  Word 0: all
// of them do not.
struct Cut {
  uint64_t word, mass;
  uint64_t all;  // mass of all the words
  int count;
};

// `n` words in s.words; `bin_of` puts them in bins, in their order.  A bin with
// more than 64 words is parted again, by the first bits in which they differ.
template <class MassOf, class BinOf>
__device__ __forceinline__ Cut find_cut(int n, bool by_mass, uint64_t goal,
                                        MassOf mass_of, BinOf bin_of,
                                        SampleLds& s) {
  const int tid = threadIdx.x;
  uint64_t cb = 0, mb = 0;  // words and mass before the ones in question
  Cut out = {0, 0, 0, 0};
  int shift = -1;  // of the words, which are the bins then
  const uint64_t* from = s.words;
  auto bin = [&](uint64_t w) {
    return shift < 0 ? bin_of(w)
                     : kSampleBins - 1 -
                           (int)((w >> shift) & (uint64_t)(kSampleBins - 1));
  };
  for (int level = 0;; ++level) {
    for (int i = tid; i < kSampleBins; i += kSampleThreads) {
      s.bin_mass[i] = 0;
      s.bin_count[i] = 0;
    }
    if (tid == 0) {
      s.found[0] = kSampleBins;
      s.gathered = 0;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < n; i += kSampleThreads) {
      const uint64_t w = from[i];
      if (w == 0) continue;
      const int b = bin(w);
      atomicAdd((unsigned long long*)&s.bin_mass[b],
                (unsigned long long)mass_of(w));
      atomicAdd(&s.bin_count[b], 1u);
    }
    __syncthreads();
    // A thread has two bins.
    uint32_t c[2], ct = 0;
    uint64_t m[2], mt = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = s.bin_count[2 * tid + i];
      m[i] = s.bin_mass[2 * tid + i];
      ct += c[i];
      mt += m[i];
    }
    uint64_t all, counts;
    uint64_t m0 = mb + scan_block(mt, s, &all);
    uint64_t c0 = cb + scan_block((uint64_t)ct, s, &counts);
    if (shift < 0) out.all = all;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t at = by_mass ? m0 : c0;
      if (at < goal && goal <= at + (by_mass ? m[i] : c[i])) {
        s.found[0] = (uint64_t)(2 * tid + i);
        s.found[1] = c0;
        s.found[2] = m0;
      }
      c0 += c[i];
      m0 += m[i];
    }
    __syncthreads();
    const int pivot = (int)s.found[0];
    if (pivot == kSampleBins) return out;
    cb = s.found[1];
    mb = s.found[2];
    const uint32_t count = s.bin_count[pivot];
    // The bin's words, in any order.
    uint64_t* const to = s.some[level & 1];
#pragma unroll 1
    for (int i = tid; i < n; i += kSampleThreads) {
      const uint64_t w = from[i];
      if (w != 0 && bin(w) == pivot) to[atomicAdd(&s.gathered, 1u)] = w;
    }
    n = (int)count;
    from = to;
    __syncthreads();
    if (n <= kWave) break;
    // The first bit in which the words differ (some do).
    const uint64_t first = from[0];
    uint64_t differ = 0;
    for (int i = tid; i < n; i += kSampleThreads) differ |= from[i] ^ first;
    // (the largest has its highest bit)
    differ = max_block(differ, s);
    const int high = 63 - __builtin_clzll(differ);
    shift = high > 10 ? high - 10 : 0;
  }
  // One wave: what lies before each word, word by word.
  if (tid < kWave) {
    if (tid == 0) s.found[0] = 0;
    const uint64_t w = tid < n ? from[tid] : 0;
    const uint64_t m = w ? mass_of(w) : 0;
    uint64_t c = cb + 1, before = mb;
    for (int i = 0; i < n; ++i) {
      const uint64_t wi = lane64(w, i), mi = lane64(m, i);
      if (wi > w) {
        ++c;
        before += mi;
      }
    }
    if (w && (by_mass ? before < goal && goal <= before + m : c == goal)) {
      s.found[0] = w;
      s.found[1] = c;
      s.found[2] = before + m;
    }
  }
  __syncthreads();
  out.word = s.found[0];
  out.mass = s.found[2];
  out.count = (int)s.found[1];
  __syncthreads();
  return out;
}

// The chunk where `goal` lies in the masses of the row's chunks (one a
// thread): in every thread, with the mass before it.
__device__ __forceinline__ int find_chunk(uint64_t mass, double u, SampleLds& s,
                          uint64_t* before, uint64_t* goal, uint64_t* total) {
  const uint64_t b = scan_block(mass, s, total);
  *goal = (uint64_t)(u * (double)*total);
  if (*goal >= *total) *goal = *total - 1;
  if (b <= *goal && *goal < b + mass) {
    s.found[0] = (uint64_t)threadIdx.x;
    s.found[1] = b;
  }
  __syncthreads();
  *before = s.found[1];
  return (int)s.found[0];
}

// The prefix of a row whose `n` words from which on nothing is missing are in
// s.words: its last word (1 for all of them), or 0 if they do not reach its
// end.  `whole`: the row has no others; `rare`: some of them are below min_p;
// `total`: the sum of the row's weights, where it is needed.
template <class MassOf, class BinOf>
__device__ __forceinline__ uint64_t list_cut(const SampleParams& a, const Wanted& want, int n,
                             double total, bool whole, bool rare,
                             MassOf mass_of, BinOf bin_of, SampleLds& s) {
  uint64_t word = 1;
  bool beyond = !whole;
  uint64_t part = 0;  // the mass of the first k
#pragma unroll 1
  for (int step = want.k > 0 ? 0 : 1; step < (want.p < 1.0 ? 2 : 1); ++step) {
    uint64_t goal = (uint64_t)want.k;
    if (step == 1) {
      if (want.k > 0 && beyond) return 0;
      const double of = want.k > 0 ? (double)part : total * a.unit;
      const double least = ceil(want.p * of);
      goal = least < 1.0 ? 1 : (uint64_t)least;
      if (want.k > 0 && goal > part) goal = part;
    }
    const Cut c = find_cut(n, step == 1, goal, mass_of, bin_of, s);
    if (step == 0) part = c.word ? c.mass : c.all;
    if (c.word) {
      word = c.word;
      beyond = false;
    }
  }
  // A prefix that goes on does not matter where min_p ends before.
  return beyond && !rare ? 0 : word;
}

// Rows: from their chunks, or over again.  A workgroup a row, of 1024 threads
// with the words in LDS, all of it latency: one row of 32000 takes 14.5 us, 256
// of 131072 together 21.
template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_finish_kernel(
    SampleParams a) {
  __shared__ SampleLds s;
  const int tid = threadIdx.x, wave = uni(tid / kWave), ln = lane();
  const int64_t row_i = a.row0 + blockIdx.x;
  const char* row = a.x + row_i * a.ld;
  const int64_t base = (int64_t)blockIdx.x * a.chunks;
  const bool in = tid < a.chunks;
  // (what a row does not ask for is not written, and not used)
  const uint32_t chunk_top = in ? a.chunk_max[base + tid] : 0;
  const uint32_t chunk_from = in ? a.chunk_from[base + tid] : 0;
  const double chunk_sum = in ? a.chunk_sum[base + tid] : 0.0;
  const int n = in ? (int)a.chunk_n[base + tid] : 0;
  const Wanted want = wanted(a, row_i);
  uint32_t top_key = chunk_top, from = chunk_from;
  max_block(&top_key, &from, s);
  const float top = key_logit(top_key);
  if (top_key == kKeyNone) {
    if (tid == 0) {
      a.tokens[row_i] = -1;
      a.logprobs[row_i] = -INFINITY;
    }
    return;
  }
  double mass = 0.0;
  if (in && want.sums() && !want.greedy)
    mass = chunk_sum * weight_of(key_logit(chunk_top), top, want.inv_t);
  double total;
  const double before_mass = scan_block(mass, s, &total);
  if (want.greedy || want.all()) {
    // ---- the first chunk with the largest logit, or past the goal; where
    // rounding leaves none past it, the last one that has weight
    const double goal = want.u * total;
    const int chunk = first_or_last(
        want.greedy ? chunk_top == top_key
                    : mass > 0.0 && before_mass + mass > goal,
        mass > 0.0, s);
    // A logit a thread.
    if (tid == chunk)
      s.found[0] = (uint64_t)__double_as_longlong(before_mass);
    const int64_t i = (int64_t)chunk * kChunk + tid;
    const float x = i < a.cols ? read_logit<T>(row, i) : -INFINITY;
    double w = weight_of(x, top, want.inv_t);
    if (want.greedy) w = x == top ? 1.0 : 0.0;
    double all;
    double upto = w + scan_block(w, s, &all);
    upto += __longlong_as_double((long long)s.found[0]);
    const int who =
        first_or_last(w > 0.0 && (want.greedy || upto > goal), w > 0.0, s);
    if (tid != who) return;
    a.tokens[row_i] = i;
    // Any weight may be drawn here, down to 2^-1074 of the largest: its
    // logarithm is the logit's difference, and `total` is 1 at least.
    const double y = x == top ? 0.0 : ((double)x - (double)top) * want.inv_t;
    a.logprobs[row_i] =
        want.greedy ? 0.0f
                    : (float)fma(y, 0.693147180559945309417, ln_of(1.0 / total));
    return;
  }
  uint64_t listed;
  const int to = (int)scan_block((uint64_t)n, s, &listed);
  const int count = (int)listed;
  // ---- lists: their words, four a thread
  auto mass_of = [&](uint64_t w) {
    return fixed(weight_of(key_logit((uint32_t)(w >> 32)), top, want.inv_t), a);
  };
  const bool whole = from <= kKeyNone + 1;  // all that has weight is listed
  auto bin_of = [&](uint64_t w) {
    return wide_bin(key_logit((uint32_t)(w >> 32)), top,
                    kWidePerBit * want.inv_t);
  };
  uint64_t cut = 0;
  if (count <= kMaxList && count > 0) {
    // Chunks are dealt to the waves; eight lists of each are on their way
    // together.  Words below the bound are dropped: others are missing there.
    s.bin_count[tid] = (uint32_t)to << 7 | (uint32_t)n;
    __syncthreads();
    bool some_low = false;
    constexpr int U = 8;
    for (int c0 = wave; c0 < a.chunks; c0 += U * kSampleWaves) {
      uint64_t w[U];
      uint32_t at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * kSampleWaves;
        at[u] = c < a.chunks ? s.bin_count[c] : 0;
        w[u] = ln < (int)(at[u] & 127)
                   ? a.lists[(base + c) * kChunkList + ln]
                   : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (ln >= (int)(at[u] & 127)) continue;
        if ((uint32_t)(w[u] >> 32) < from) w[u] = 0;
        s.words[(at[u] >> 7) + ln] = w[u];
      }
    }
    __syncthreads();
    if (want.min_w > 0.0) {
#pragma unroll 1
      for (int i = tid; i < count; i += kSampleThreads) {
        const uint64_t w = s.words[i];
        if (w && weight_of(key_logit((uint32_t)(w >> 32)), top, want.inv_t) <
                     want.min_w)
          some_low = true;
      }
    }
    const bool rare = __syncthreads_or(some_low) != 0;
    cut = list_cut(a, want, count, total, whole, rare, mass_of, bin_of, s);
  }
  if (cut == 0) {
    // (a prefix of a wide one has two goals: by passes over the row)
    const int mode = want.k > 0 ? (want.p < 1.0 ? kWideRow : kWideCount)
                     : want.p < 1.0 ? kWideMass
                                    : kWideAll;
    uint64_t* bins = a.bins + (int64_t)blockIdx.x * kWideBins;
    for (int i = tid; i < kWideBins; i += kSampleThreads) bins[i] = 0;
    if (tid == 0) {
      const double part = ceil(want.p * (total * a.unit));
      WideRow w = {};
      w.mode = (uint32_t)mode;
      w.top = top_key;
      w.goal = mode == kWideCount ? (uint64_t)want.k
               : part < 1.0       ? 1
                                  : (uint64_t)part;
      a.wide[blockIdx.x] = w;
      a.wide_list[1 + atomicAdd(a.wide_list, 1u)] = blockIdx.x;
    }
    return;
  }
  // ---- in the row's order: the chunk, then its list
  s.chunk_mass[tid] = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < count; i += kSampleThreads) {
    const uint64_t w = s.words[i];
    if (w < cut) continue;
    const double x =
        weight_of(key_logit((uint32_t)(w >> 32)), top, want.inv_t);
    if (x >= want.min_w)
      atomicAdd((unsigned long long*)
                    &s.chunk_mass[(uint32_t) ~(uint32_t)w / kChunk],
                (unsigned long long)fixed(x, a));
  }
  __syncthreads();
  uint64_t before, goal, kept;
  const int chunk =
      find_chunk(s.chunk_mass[tid], want.u, s, &before, &goal, &kept);
  if (wave != chunk / kWave) return;
  const int nc = __builtin_amdgcn_readlane(n, chunk % kWave);
  const uint64_t w =
      ln < nc ? a.lists[(base + chunk) * kChunkList + ln] : 0;
  const double x =
      w ? weight_of(key_logit((uint32_t)(w >> 32)), top, want.inv_t) : 0.0;
  const uint64_t m = w >= cut && (uint32_t)(w >> 32) >= from && x >= want.min_w
                         ? fixed(x, a)
                         : 0;
  before += wave_scan64(m) - m;
  if (before <= goal && goal < before + m) {
    a.tokens[row_i] = (int64_t)(uint32_t) ~(uint32_t)w;
    a.logprobs[row_i] = (float)ln_of(x / ((double)kept / a.unit));
  }
}

// ---- wide prefixes ----------------------------------------------------------
// A prefix beyond the lists (a nucleus of tens of thousands) is found in three
// more launches, two of them over the row by workgroups of 8 chunks.  The first
// adds up the masses (or counts) of the logits in 2048 bins of log2 of their
// weight; integers, so that their order is nothing.  The second finds the bin
// in which the goal lies, adds up each chunk's mass above it, and lists the
// bin's own logits; the third ends the row (finish_wide).  32 rows of 200000 in
// float16, all wide: 19, 21 and 17 us (a weight a logit twice more, and atomics;
// a workgroup a row at the end); with no wide row the three take 1.4 us each.
template <int T>
__global__ __launch_bounds__(kWideThreads) void sample_bins_kernel(
    SampleParams a) {
  const int wg = (a.chunks + kWideChunks - 1) / kWideChunks;
  const int tasks = (int)a.wide_list[0] * wg;
  __shared__ uint64_t bins[kWideBins];
  const int tid = threadIdx.x;
  for (int task = (int)blockIdx.x; task < tasks; task += (int)gridDim.x) {
    const int r = (int)a.wide_list[1 + task / wg];
    const WideRow wide = a.wide[r];
    if (wide.mode != kWideMass && wide.mode != kWideCount) continue;
    const int64_t row_i = a.row0 + r;
    const Wanted want = wanted(a, row_i);
    const float top = key_logit(wide.top);
    const int chunk = task % wg * kWideChunks + tid / kWave;
    typedef ChunkShape<T> S;
    float x[S::N];  // on its way while the bins are cleared
    if (chunk < a.chunks)
      read_chunk<T>(a.x + row_i * a.ld, chunk * kChunk, a.cols, x);
    for (int i = tid; i < kWideBins; i += kWideThreads) bins[i] = 0;
    __syncthreads();
    if (chunk < a.chunks) {
      const double c = kWidePerBit * want.inv_t;
#pragma unroll
      for (int e = 0; e < S::N; ++e) {
        // What lies in the last bin has no weight to speak of: 2^-46 and less.
        const int bin = wide_bin(x[e], top, c);
        if (bin == kWideBins - 1) continue;
        atomicAdd((unsigned long long*)&bins[bin],
                  wide.mode == kWideCount
                      ? 1ull
                      : (unsigned long long)fixed(
                            weight_of(x[e], top, want.inv_t), a));
      }
    }
    __syncthreads();
    unsigned long long* all =
        (unsigned long long*)(a.bins + (int64_t)r * kWideBins);
    for (int i = tid; i < kWideBins; i += kWideThreads)
      if (bins[i]) atomicAdd(all + i, (unsigned long long)bins[i]);
    __syncthreads();
  }
}

// The bin of a wide row's goal: kWideBins if the goal is beyond the bins, or
// if there is none (all of them count).
struct Pivot {
  int bin;
  uint64_t above;  // mass or count
};
template <int THREADS>
__device__ __forceinline__ Pivot find_pivot(const SampleParams& a, int r,
                                            const WideRow& wide, ScanLds& s) {
  Pivot out = {kWideBins, 0};
  if (wide.mode == kWideAll) return out;
  const int tid = threadIdx.x;
  constexpr int B = kWideBins / THREADS;
  const uint64_t* bins = a.bins + (int64_t)r * kWideBins;
  uint64_t b[B], sum = 0;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    b[i] = bins[tid * B + i];
    sum += b[i];
  }
  uint64_t all;
  uint64_t before = scan_block<THREADS / kWave>(sum, s, &all);
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
  out.bin = (int)s.found[0];
  out.above = s.found[1];
  return out;
}

template <int T>
__global__ __launch_bounds__(kWideThreads) void sample_wide_kernel(
    SampleParams a) {
  __shared__ ScanLds s;
  const int wg = (a.chunks + kWideChunks - 1) / kWideChunks;
  const int tasks = (int)a.wide_list[0] * wg;
  const int tid = threadIdx.x, ln = lane();
  typedef ChunkShape<T> S;
  for (int task = (int)blockIdx.x; task < tasks; task += (int)gridDim.x) {
    const int r = (int)a.wide_list[1 + task / wg];
    const WideRow wide = a.wide[r];
    if (wide.mode == kWideRow) continue;
    const int64_t row_i = a.row0 + r;
    const Wanted want = wanted(a, row_i);
    const float top = key_logit(wide.top);
    const double c = kWidePerBit * want.inv_t;
    const int chunk = task % wg * kWideChunks + tid / kWave;
    float x[S::N];  // on its way while the pivot is looked for
    if (chunk < a.chunks)
      read_chunk<T>(a.x + row_i * a.ld, chunk * kChunk, a.cols, x);
    const int pivot = find_pivot<kWideThreads>(a, r, wide, s).bin;
    __syncthreads();
    if (pivot == kWideBins && wide.mode != kWideAll) continue;
    if (chunk >= a.chunks) continue;
    uint64_t sum = 0;
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < S::N; ++e) {
      const int bin = wide_bin(x[e], top, c);
      if (bin < pivot) {
        const double w = weight_of(x[e], top, want.inv_t);
        if (w >= want.min_w) sum += fixed(w, a);
      }
      // (past the row's end there is -infinity, which is in the last bin)
      bits |= (bin == pivot ? 1u : 0u) << e;
    }
    sum = wave_scan64(sum);
    if (ln == kWave - 1) a.chunk_mass[(int64_t)r * a.chunks + chunk] = sum;
    const int mine = __popc(bits);
    if (ballot(mine > 0) == 0) continue;
    const int incl = wave_scan_incl(mine);
    unsigned to = 0;
    if (ln == kWave - 1) to = atomicAdd(&a.wide[r].pivots, (unsigned)incl);
    to = (unsigned)__builtin_amdgcn_readlane((int)to, kWave - 1);
    to += (unsigned)(incl - mine);
    uint64_t* const pivots = a.pivots + (int64_t)r * kMaxList;
#pragma unroll
    for (int e = 0; e < S::N; ++e) {
      if (!(bits >> e & 1)) continue;
      const uint32_t i = (uint32_t)(chunk * kChunk + S::at(e));
      if (to < kMaxList)
        pivots[to] = (uint64_t)logit_key(x[e]) << 32 | (uint32_t)~i;
      ++to;
    }
  }
}

// A wide row's end: the last of the bin's logits that is kept, the chunk where
// u times the kept mass lies, and the token in it.  False: the row is done over.
template <int T>
__device__ __forceinline__ bool finish_wide(const SampleParams& a, int r,
                                            SampleLds& s) {
  const int tid = threadIdx.x;
  const WideRow wide = a.wide[r];
  if (wide.mode == kWideRow) return false;
  const int64_t row_i = a.row0 + r;
  const Wanted want = wanted(a, row_i);
  const float top = key_logit(wide.top);
  const double c = kWidePerBit * want.inv_t;
  const Pivot pivot = find_pivot<kSampleThreads>(a, r, wide, s);
  uint64_t mass =
      tid < a.chunks ? a.chunk_mass[(int64_t)r * a.chunks + tid] : 0;
  uint64_t cut = 0;
  auto word_weight = [&](uint64_t w) {
    return weight_of(key_logit((uint32_t)(w >> 32)), top, want.inv_t);
  };
  if (wide.mode != kWideAll) {
    const int count = (int)wide.pivots;
    if (pivot.bin == kWideBins || wide.pivots > (uint32_t)kMaxList)
      return false;
    const uint64_t* const pivots = a.pivots + (int64_t)r * kMaxList;
    for (int i = tid; i < count; i += kSampleThreads) s.words[i] = pivots[i];
    __syncthreads();
    auto mass_of = [&](uint64_t w) { return fixed(word_weight(w), a); };
    auto bin_of = [&](uint64_t w) {  // the bin in 2048 parts
      const float x = key_logit((uint32_t)(w >> 32));
      const double d = ((double)top - (double)x) * c - pivot.bin;
      return d > 0.0 ? (int)fmin(d * kSampleBins, kSampleBins - 1.0) : 0;
    };
    cut = find_cut(count, wide.mode != kWideCount, wide.goal - pivot.above,
                   mass_of, bin_of, s)
              .word;
    if (cut == 0) return false;
    // Masses of the bin's words in their chunks.
    s.chunk_mass[tid] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < count; i += kSampleThreads) {
      const uint64_t w = s.words[i];
      if (w < cut) continue;
      const double x = word_weight(w);
      if (x >= want.min_w)
        atomicAdd((unsigned long long*)
                      &s.chunk_mass[(uint32_t) ~(uint32_t)w / kChunk],
                  (unsigned long long)fixed(x, a));
    }
    __syncthreads();
    mass += s.chunk_mass[tid];
  }
  uint64_t before, goal, total;
  const int chunk = find_chunk(mass, want.u, s, &before, &goal, &total);
  // A logit a thread.  (-infinity past the end has no weight.)
  const int64_t i = (int64_t)chunk * kChunk + tid;
  const float x = i < a.cols ? read_logit<T>(a.x + row_i * a.ld, i) : -INFINITY;
  const uint64_t word = (uint64_t)logit_key(x) << 32 | (uint32_t) ~(uint32_t)i;
  const double w = weight_of(x, top, want.inv_t);
  const uint64_t m = word >= cut && w >= want.min_w ? fixed(w, a) : 0;
  uint64_t all;
  before += scan_block(m, s, &all);
  if (before <= goal && goal < before + m) {
    a.tokens[row_i] = i;
    a.logprobs[row_i] = (float)ln_of(w / ((double)total / a.unit));
  }
  return true;
}

template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_last_kernel(
    SampleParams a) {
  __shared__ SampleLds s;
  const int rows = (int)a.wide_list[0];
  for (int i = (int)blockIdx.x; i < rows; i += (int)gridDim.x) {
    const int r = (int)a.wide_list[1 + i];
    const bool done = finish_wide<T>(a, r, s);
    __syncthreads();
    if (!done && threadIdx.x == 0) a.wide[r].mode = kWideRow;
  }
  __syncthreads();
  // (apart from the others, which need other registers)
  for (int i = (int)blockIdx.x; i < rows; i += (int)gridDim.x) {
    const int r = (int)a.wide_list[1 + i];
    if (a.wide[r].mode != kWideRow) continue;
    sample_row<T>(a, a.row0 + r, s);
    __syncthreads();
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
