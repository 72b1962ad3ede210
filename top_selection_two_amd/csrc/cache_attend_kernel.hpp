// Attention of one new token over a paged cache.
//
// For query j of head h and slot t: x = scale k_scale (q . K_t).  One pass
// over the slots keeps a running maximum m, l = sum exp(x - m) and
// o = sum exp(x - m) V_t; out = v_scale o / l, lse = m + ln l.  Exponentials
// are taken to base 2 (scale is multiplied by log2 e on the host).
//
// The kernel reads every K and V row once and should run at the rate of that
// read.  Work: the slots of a row (a sequence, `hs` of its cache heads and up
// to 16 queries of each) are cut into tiles of 32 slots, a step of one wave for
// each head; the tiles of all rows are dealt out evenly to as many workgroups
// as the chip holds at once, whatever the mix of lengths.  A row that one
// workgroup has alone is finished there; of the others each leaves its
// (m, l, o), and the row's last workgroup to finish joins them.
//
// hs is 1 where a head's slots lie together.  Where slots lie outside heads,
// a head's rows are short pieces far apart, and a workgroup that reads one
// head alone keeps to few of the memory's channels: there the waves of a
// workgroup take kHeadRun heads of the same slots.
//
// Measured (MI355X; a large read reaches 7.2 TB/s): 48 sequences of 4096
// slots, 8 heads of 4 queries of 128 elements, bfloat16, 0.81 GB: 133 us
// (6.0 TB/s), 147 us with the weights, 134 us in float16; 32 sequences of 8192
// slots in pages of 256: 162 us (6.6 TB/s), 163 us in float16; a document of
// 131072 slots, 4 heads of 8 queries: 51 us, of which the rows' stream is 40
// (6.7 TB/s) and joining 64 shares a row 7.  Matrix instructions are busy 8 %
// of the time over bfloat16 rows, 15 % over 8-bit ones, 36 % over float16.
#pragma once

#include <type_traits>

#include "cache_common.hpp"

namespace ltk {

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kTileSlots = 32;  // of one wave
constexpr int kHeadRun = 4;
constexpr int kLdsBytes = 160 * 1024;  // of a compute unit

// What attend_kernel leaves to attend_join_kernel of a row: the workgroups
// that share it, or one of these.
constexpr int kRowDone = -1;    // nothing
constexpr int kRowJoined = -2;  // its weights

struct AttendParams {
  CacheParams c;
  LedgerParams w;
  const char* q;
  int64_t qb, qh;       // bytes
  int32_t group;        // query heads of a cache head
  int32_t gtiles;       // ceil(group / 16)
  int32_t hs;           // cache heads of a row: 1 or kHeadRun
  float scale2;         // scale * log2 e
  const float* k_scale; // NULL: 1
  const float* v_scale;
  // With a ledger: scores of split rows, [row][tile] (see score_at), and the
  // tiles that fit in LDS.
  float* scores;
  int2* shares;         // of each row, unless `direct` (see Shares)
  int32_t row_tiles;    // tiles of a row at full length
  int32_t held_tiles;
  bool direct;          // a row's last workgroup joins it and adds up its
                        // weights; otherwise attend_join_kernel does
  int32_t cols;         // columns of a share's result
  int32_t q_type;
  float* part;          // [grid][2][share_floats]: sums, maxima, weights' sums
  int32_t part_rows;    // queries of a row, at most 16
  int32_t min_tiles;    // least share of a row
  int32_t row_cost;     // what a row costs besides its tiles, in tiles
  int32_t lds_rows;     // part_rows, to a multiple of 4
  uint64_t* ticket;     // one per row
  uint32_t epoch;
  void* out;
  float* lse;
};

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Eight elements of a matrix instruction's operand, as dwords.
struct Frag {
  int d[4];
};

template <int QT>
__device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
  if constexpr (QT == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
        0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(
        __builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
        0);
}

// 16 x 16 x 4: lane 16 q + n takes row (or column) n, contraction index q.
__device__ __forceinline__ f32x4 mma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Two floats rounded to a 16-bit type.
template <int QT>
__device__ __forceinline__ int pack2(float a, float b) {
  if constexpr (QT == kBf16)
    return __builtin_bit_cast(int, bf16x2{(__bf16)a, (__bf16)b});
  else
    return __builtin_bit_cast(int, f16x2{(_Float16)a, (_Float16)b});
}

// Two of the four e4m3 values of a dword in the operand's type (exact: both
// 16-bit types hold every e4m3 value).
template <int QT, bool HI>
__device__ __forceinline__ int widen2(int v) {
  if constexpr (QT == kBf16)
    return __builtin_bit_cast(
        int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, HI));
  else
    return __builtin_bit_cast(
        int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, HI));
}

// A weight (>= 0 or NaN) as the sum of three bfloat16 numbers, the upper
// halves of p; 2^-22 of it is left.  Each but the last is the largest number
// below what is left to hold, so that none is negative and none is 0 unless
// the weight is: their products with an infinity of V add up to it.  (Rounded
// parts are some instructions less, 150.6 us against 151.3 for 48 ragged
// sequences, 111.6 against 112.2 for 8-bit rows, and give NaN there.)
__device__ __forceinline__ void split3(float w, unsigned (&p)[3]) {
  const unsigned u = __float_as_uint(w);
  const unsigned least = u < 0x10000u ? u : 0x10000u;
  p[0] = __builtin_elementwise_sub_sat(u, 1u);
  const float r = w - __uint_as_float(p[0] & 0xffff0000u);
  p[1] = __builtin_elementwise_sub_sat(__float_as_uint(r), 1u);
  p[1] = p[1] > least ? p[1] : least;
  const float s = fmaxf(r - __uint_as_float(p[1] & 0xffff0000u), 0.0f);
  p[2] = __float_as_uint(s) + 0x8000u;
  p[2] = p[2] > least ? p[2] : least;
}

__device__ __forceinline__ float exp2_fast(float x) {
  return __builtin_amdgcn_exp2f(x);
}

__device__ __forceinline__ float quad_max(float v) {  // over lanes l % 16
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

typedef int v2i __attribute__((ext_vector_type(2)));

// K and V rows are read once a call: non-temporal.
template <class T>
__device__ __forceinline__ T ld_once(const char* p) {
  return __builtin_nontemporal_load((const T*)p);
}

// Coherent at device level (sc1), as st_agent and ld_agent, four floats at a
// time and free to be in flight together; `at` in bytes.
__device__ __forceinline__ f32x4 ld_agent4(__amdgpu_buffer_rsrc_t r, int at) {
  return __builtin_bit_cast(
      f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 16));
}
__device__ __forceinline__ float ld_agent1(__amdgpu_buffer_rsrc_t r, int at) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 16));
}
__device__ __forceinline__ void st_agent1(__amdgpu_buffer_rsrc_t r, int at,
                                          float x) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, at, 0, 16);
}
__device__ __forceinline__ void st_agent4(__amdgpu_buffer_rsrc_t r, int at,
                                          f32x4 x) {
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, at,
                                         0, 16);
}

// Scores of a tile: `rows` queries of 32 slots, in groups of four slots.
// The groups of a query are rotated among themselves by exclusive or, so that
// the 16 queries that write a group each do not meet in one bank of LDS.
__device__ __forceinline__ int score_at(int query, int group4) {
  return query * kTileSlots + ((group4 ^ (query & 7)) * 4);
}

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// weights[0 .. 4) += a, as far as they lie below the length.
__device__ __forceinline__ void add_weights(float* w, int32_t left,
                                            f32x4 a) {
  if (left >= 4) {
    *(f32x4u*)w = *(const f32x4u*)w + a;
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < left) w[e] += a[e];
  }
}

// One wave's tile: 32 slots of a row against up to 16 queries.  With lane
// l = 16 q + n, the 16 x 16 x 32 matrix instruction takes row (or column) n,
// contraction indices 8 q .. 8 q + 7 of its operands, and leaves column n,
// rows 4 q .. 4 q + 3 of the result.
//
//  * Scores: slots are rows, queries columns.  Contraction indices may be
//    any elements of the row as long as K and q agree, so a lane reads 16
//    consecutive bytes: bytes 64 c + 16 q of slot 16 tt + n.
//  * Result: lane (q, n) holds query n's scores of slots 16 tt + 4 q + i.
//    These are exactly the contraction indices 8 q + (4 tt + i) that the lane
//    supplies as row n of the weights in the second product, when lane q of
//    the V operand supplies the same slots.  Weights never leave the lane.
//  * V operand: a lane reads VE consecutive elements (n VE ..) of its 8
//    slots and transposes the 8 x VE block in registers; instruction e takes
//    element e, so its column n is the row's element n VE + e.  (float16 rows
//    need no transposition: a 16 x 16 x 4 float32 instruction takes one slot
//    of each lane group, with the weights in the lanes that hold them.)
//
// QT: query type, CT: cache type, NC: 32-element chunks of a row, PG16: pages
// of a multiple of 16 slots, so that each half of a tile lies in one page.
template <int QT, int CT, int NC, bool PG16>
struct Attend {
  // Rows of more than 128 elements need more than 256 registers a lane: one
  // wave to a SIMD instead of two, with twice the bytes in flight each.
  static constexpr int WAVES = NC > 4 ? 4 : 8;
  static constexpr int THREADS = WAVES * kWave;
  static constexpr int ES = CT == kE4m3 ? 1 : 2;
  static constexpr int KL = CT == kE4m3 ? (NC + 1) / 2 : NC;  // K loads a half
  static constexpr int VE = NC == 2 ? 4 : 8;
  static constexpr int VD = VE * ES / 4;             // dwords of a V load
  static constexpr int NB = (NC * 32 + 16 * VE - 1) / (16 * VE);
  static constexpr int COLS = NB * 16 * VE;
  // The first chunk that a row of this class can leave short.
  static constexpr int SHORT = NC == 2 ? 0 : NC == 3 ? 2 : NC == 4 ? 3
                               : NC == 6 ? 4 : 6;
  static constexpr int last_chunk(int load) {
    return (load * 64 + 63) / ES / 32;
  }
  static constexpr int QL = CT == kE4m3 ? 2 * KL : NC;  // q fragments

  struct Ids {
    int32_t id[PG16 ? 2 : 10];  // K halves; without PG16 then the 8 V slots
    int32_t place[PG16 ? 2 : 10];
  };

  // Static LDS; besides it [WAVES][lds_rows][COLS] floats in which the waves
  // (and a row's shares) are joined, at least JOIN of them, and the scores.
  static constexpr int JOIN = 6 * THREADS;
  struct Lds {
    float m[WAVES][16];
    float l[WAVES][16];
    float lse2[WAVES * 16];
    int32_t scan[2][WAVES];
    int32_t base;
    int32_t b;
    int32_t flag;
  };
  // A workgroup alone on a unit has room for the scores of a tile (with 256
  // bytes for the allocation's steps).
  static constexpr bool kScoresFit =
      (int)sizeof(Lds) + 256 + 4 * (WAVES * 16 * COLS) +
          4 * (kHeadRun * 16 * kTileSlots) <=
      kLdsBytes;
  static_assert(kScoresFit && JOIN <= WAVES * 16 * COLS);
};

// Pages of tile `t`'s slots.  Slots past the length repeat the last one;
// an entry that names no page gives -1.
template <class A, bool PG16>
__device__ __forceinline__ typename A::Ids find_tile(const CacheParams& c,
                                                     const int32_t* table,
                                                     int32_t t, int32_t len,
                                                     int q, int n) {
  typename A::Ids r;
  if constexpr (PG16) {
#pragma unroll
    for (int tt = 0; tt < 2; ++tt) {
      int32_t s = t * kTileSlots + tt * 16;
      s = s < len ? s : 0;
      const int32_t p = uni(quotient(c.page, s));
      r.place[tt] = s - p * c.page.d;
      r.id[tt] = ld_const(table + p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      int32_t s = t * kTileSlots + (i < 2 ? i * 16 + n
                                          : (i - 2) / 4 * 16 + q * 4 +
                                                (i - 2) % 4);
      s = s < len ? s : len - 1;
      const int32_t p = quotient(c.page, s);
      r.place[i] = s - p * c.page.d;
      r.id[i] = table[p];
    }
  }
  return r;
}

template <int QT, int CT, int NC, bool PG16, int HS>
__global__ __launch_bounds__((Attend<QT, CT, NC, PG16>::THREADS),
                             (Attend<QT, CT, NC, PG16>::WAVES / 4)) void
attend_kernel(AttendParams p) {
  typedef Attend<QT, CT, NC, PG16> A;
  constexpr int kAttWaves = A::WAVES, kAttThreads = A::THREADS;
  constexpr int ES = A::ES, KL = A::KL, VE = A::VE, VD = A::VD, NB = A::NB;
  constexpr int COLS = A::COLS, QL = A::QL;
  __shared__ typename A::Lds lds;
  const CacheParams& c = p.c;
  const int tid = threadIdx.x, wave = uni(tid / kWave), ln = tid % kWave;
  const int q = ln / 16, n = ln % 16;
  const int hg = c.heads / HS * p.gtiles;  // rows of a sequence
  // Waves: head hsub of the row's, every ts-th tile from tsub on.
  constexpr int ts = kAttWaves / HS;
  const int hsub = wave % HS, tsub = wave / HS;

  // ---- this workgroup's run of units -------------------------------------
  const int32_t top_len = c.pages > 0 ? c.cap : 0;
  auto len_of = [&](int b) { return clamp_len(c.lens[b], top_len); };
  // Length of a sequence that is the same in every lane.
  auto len_uni = [&](int b) {
    return clamp_len(ld_const(c.lens + b), top_len);
  };
  // Two ways of dealing.  Shares: a row of n tiles is cut into ceil(n / per)
  // equal shares, one to a workgroup, as long as there are no more shares than
  // workgroups.  A workgroup then has one row, and few rows are split: joining
  // one costs as much as many tiles.  Runs: with more rows, every workgroup
  // takes `per` consecutive tiles of whatever rows; what a row costs besides
  // its tiles (loading the queries, joining the waves) counts as row_cost
  // tiles before its first.
  int32_t u0 = 0, u1 = 0, per = 1, base = 0, share = -1, cuts = 1;
  int32_t cost = p.row_cost;
  int b = 0;
  const int32_t grid = (int32_t)gridDim.x, wg = (int32_t)blockIdx.x;
  auto tiles_of = [&](int32_t len) {  // an empty row has an output too
    return len > 0 ? (len + kTileSlots - 1) / kTileSlots : 1;
  };
  auto cuts_of = [&](int32_t tiles) { return (tiles + per - 1) / per; };
  // Share `i` of a sequence.  (None is empty: the shares before the last hold
  // at most (cuts - 1) per < n tiles.)
  auto take_share = [&](int32_t i, int32_t tiles) {
    cuts = cuts_of(tiles);
    const int32_t hi = i / cuts;
    share = i % cuts;
    const int32_t each = (tiles + cuts - 1) / cuts, r0 = hi * tiles;
    const int32_t end = (share + 1) * each < tiles ? (share + 1) * each : tiles;
    base = 0;
    cost = 0;
    u0 = r0 + share * each;
    u1 = r0 + end;
  };
  auto deal = [&](int32_t all) {
    per = (all + grid - 1) / grid;
    if (per < p.min_tiles) per = p.min_tiles;
  };
  if (c.batch == 1) {
    const int32_t tiles = tiles_of(len_uni(0)), all = (tiles + cost) * hg;
    deal(all);
    if (cuts_of(tiles) * hg <= grid) {
      if (wg >= cuts_of(tiles) * hg) return;
      take_share(wg, tiles);
    } else {
      u0 = wg * per;
      u1 = u0 + per < all ? u0 + per : all;
      if (u0 >= u1) return;
    }
  } else {
    // Thread i takes sequences [i * each, (i + 1) * each).
    const int each = (c.batch + kAttThreads - 1) / kAttThreads;
    int32_t mine = 0;
    for (int i = tid * each; i < (tid + 1) * each && i < c.batch; ++i)
      mine += (tiles_of(len_of(i)) + cost) * hg;
    const int32_t incl = wave_scan_incl(mine);
    if (ln == kWave - 1) lds.scan[0][wave] = incl;
    __syncthreads();
    int32_t before = incl - mine, all = 0;
    for (int i = 0; i < kAttWaves; ++i) {
      if (i < wave) before += lds.scan[0][i];
      all += lds.scan[0][i];
    }
    all = uni(all);
    deal(all);
    int32_t mine_s = 0;
    for (int i = tid * each; i < (tid + 1) * each && i < c.batch; ++i)
      mine_s += cuts_of(tiles_of(len_of(i))) * hg;
    const int32_t incl_s = wave_scan_incl(mine_s);
    if (ln == kWave - 1) lds.scan[1][wave] = incl_s;
    __syncthreads();
    int32_t before_s = incl_s - mine_s, all_s = 0;
    for (int i = 0; i < kAttWaves; ++i) {
      if (i < wave) before_s += lds.scan[1][i];
      all_s += lds.scan[1][i];
    }
    all_s = uni(all_s);
    const bool shares = all_s <= grid;
    const int32_t at = shares ? wg : wg * per;
    if (at >= (shares ? all_s : all)) return;
    int32_t f = shares ? before_s : before;
    if (at >= f && at < f + (shares ? mine_s : mine)) {
      int i = tid * each;
      for (;; ++i) {
        const int32_t tiles = tiles_of(len_of(i));
        const int32_t n = (shares ? cuts_of(tiles) : tiles + cost) * hg;
        if (f + n > at) break;
        f += n;
      }
      lds.b = i;
      lds.base = f;
    }
    __syncthreads();
    b = uni(lds.b);
    base = uni(lds.base);
    if (shares) {
      take_share(at - base, tiles_of(len_uni(b)));
    } else {
      u0 = at;
      u1 = u0 + per < all ? u0 + per : all;
    }
  }

  int32_t len = len_uni(b);
  int32_t row_tiles = tiles_of(len);
  int32_t u = u0;

  // Scores of the tiles that this workgroup holds in LDS; `held` of them.
  // Those of a row that it has alone become weights as soon as the row's sum
  // is known.  Those of a row that others share go to memory, at the end of
  // the run (or when LDS is full): a few per cent of writes strewn among the
  // reads cost the stream more than ten times their bytes (48 sequences of
  // 4096 slots, 8 heads of 4 queries: 165 us with each tile's scores written
  // at once, 129 us with none).
  extern __shared__ float4 dynamic_lds[];
  float* const join = (float*)dynamic_lds;
  const int join_floats = max(kAttWaves * p.lds_rows * COLS, A::JOIN);
  float* const held_scores = join + join_floats;
  const int head_floats = p.part_rows * kTileSlots;
  const int tile_floats = HS * head_floats;  // scores of a tile
  int32_t held = 0;
  // A share of a row that is not finished: its row, length, workgroups, and
  // the tiles [from, from + count) at `at` in LDS.
  struct Share {
    int32_t b, hi, len, first, last;
    int32_t from, count, at;
    bool open;
  };
  Share pend = {};
  auto row_scores = [&](const Share& r) {
    return p.scores + ((int64_t)r.b * hg + r.hi) * p.row_tiles * tile_floats;
  };
  auto flush = [&](Share& r) {
    if (r.count > 0) {
      const int bytes = r.count * tile_floats * 4;
      const __amdgpu_buffer_rsrc_t to = __builtin_amdgcn_make_buffer_rsrc(
          uni_ptr(row_scores(r) + (int64_t)r.from * tile_floats), (short)0,
          bytes, 0x00020000);
      const f32x4* from = (const f32x4*)(held_scores + r.at * tile_floats);
      for (int i = tid; i < bytes / 16; i += kAttThreads)
        st_agent4(to, i * 16, from[i]);
    }
    r.from += r.count;
    r.count = 0;
  };
  // weights += sum over queries of exp2(x - lse2), for a row whose lse2 is in
  // LDS; scores of the share's tiles from LDS, the others from memory.
  auto finish_weights = [&](const Share& r, int queries) {
    const int h0 = r.hi / p.gtiles * HS;
    const __amdgpu_buffer_rsrc_t mem = __builtin_amdgcn_make_buffer_rsrc(
        uni_ptr(row_scores(r)), (short)0, tiles_of(r.len) * tile_floats * 4,
        0x00020000);
    for (int s = 0; s < HS; ++s) {
      float* w = p.w.w + r.b * p.w.wb + (h0 + s) * p.w.wh;
      for (int32_t i = tid; i * 4 < r.len; i += kAttThreads) {
        const int32_t t = i / 8;
        const bool here = t >= r.from && t < r.from + r.count;
        const int32_t at =
            (here ? t - r.from + r.at : t) * tile_floats + s * head_floats;
        f32x4 a = {0, 0, 0, 0};
        for (int g0 = 0; g0 < queries; g0 += 4) {
          f32x4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int g = g0 + k < queries ? g0 + k : g0;
            const int o = at + score_at(g, i % 8);
            x[k] = here ? *(const f32x4*)(held_scores + o)
                        : ld_agent4(mem, o * 4);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (g0 + k >= queries) continue;
            const float z = lds.lse2[s * 16 + g0 + k];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              a[e] += x[k][e] == -INFINITY ? 0.0f : exp2_fast(x[k][e] - z);
          }
        }
        add_weights(w + i * 4, r.len - i * 4, a);
      }
    }
  };

  while (u < u1) {
    // ---- a row's share ------------------------------------------------------
    while (u >= base + (row_tiles + cost) * hg) {
      base += (row_tiles + cost) * hg;
      ++b;
      len = len_uni(b);
      row_tiles = tiles_of(len);
    }
    const int hi = uni((u - base) / (row_tiles + cost));
    // The row's tiles count as [r0, r1), after its cost.
    const int32_t r0 = base + hi * (row_tiles + cost) + cost;
    const int32_t r1 = r0 + row_tiles;
    const int32_t s0 = u > r0 ? u : r0, s1 = r1 < u1 ? r1 : u1;
    if (s0 >= s1) break;  // the run ends before the row's first tile
    const int h0 = hi / p.gtiles * HS, g0 = hi % p.gtiles * 16;
    const int h = h0 + hsub;
    const int queries = p.group - g0 < 16 ? p.group - g0 : 16;
    const int32_t* table = c.table + b * c.table_stride;
    const int32_t tiles = (len + kTileSlots - 1) / kTileSlots;
    const char* kh = c.k + h * c.ks.head;
    const char* vh = c.v + h * c.vs.head;
    Share cur = {b, hi, len, share < 0 ? r0 / per : wg - share,
                 share < 0 ? (r1 - 1) / per : wg - share + cuts - 1,
                 s0 - r0, 0, held, true};
    const float scale = p.scale2 * (p.k_scale ? ld_const(p.k_scale + h) : 1.0f);

    float m = -INFINITY, l = 0.0f;
    f32x4 o[NB * VE];
#pragma unroll
    for (int i = 0; i < NB * VE; ++i) o[i] = f32x4{0, 0, 0, 0};

    // Query fragments: those of 8-bit rows pair up to match 16-byte loads.
    // Columns past the row's queries repeat the last and are not used.
    Frag qf[QL];
    {
      const char* from = p.q + b * p.qb +
                         (h * p.group + g0 + min(n, queries - 1)) * p.qh;
#pragma unroll
      for (int f = 0; f < QL; ++f) {
        const int d = CT == kE4m3 ? f / 2 * 64 + q * 16 + f % 2 * 8
                                  : f * 32 + q * 8;
        const v4i x = *(const v4i*)(from + (d < c.dim ? d * 2 : 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[f].d[e] = x[e];
      }
    }

    for (int32_t ta = s0 - r0, te; ta < s1 - r0; ta = te) {
      // ---- tiles [ta, te) of the row: all of the share, or what LDS holds
      te = s1 - r0;
      float* tile_scores = nullptr;
      if (p.scores) {
        if (held == p.held_tiles) {
          __syncthreads();
          flush(pend);
          flush(cur);
          drain_memory_ops();  // finish_weights may read them back
          __syncthreads();
          held = 0;
          cur.at = 0;
        }
        if (te - ta > p.held_tiles - held) te = ta + p.held_tiles - held;
        tile_scores =
            held_scores + (held + tsub) * tile_floats + hsub * head_floats;
        held += te - ta;
        cur.count += te - ta;
      }
      int32_t t = ta + tsub;
      const int32_t t1 = te < tiles ? te : tiles;
      if (t >= t1) continue;

      v4i kr[2][KL];
      int vr[NB][8][VD];
      auto load_k = [&](const typename A::Ids& id) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          const int32_t pg = page_ok(id.id[tt], c.pages) ? id.id[tt] : 0;
          const char* row =
              PG16 ? kh + (int64_t)pg * c.ks.page +
                         (int64_t)id.place[tt] * c.ks.slot +
                         (uint32_t)(n * (int32_t)c.ks.slot)
                   : kh + (int64_t)pg * c.ks.page +
                         (int64_t)id.place[tt] * c.ks.slot;
#pragma unroll
          for (int k = 0; k < KL; ++k) {
            const int at = k * 64 + q * 16;
            const bool in = A::last_chunk(k) < A::SHORT || at < c.row_bytes;
            kr[tt][k] = ld_once<v4i>(row + (in ? at : 0));
          }
        }
      };
      auto load_v = [&](const typename A::Ids& id) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = PG16 ? j / 4 : j + 2;
          const int32_t pg = page_ok(id.id[at], c.pages) ? id.id[at] : 0;
          const char* row =
              PG16 ? vh + (int64_t)pg * c.vs.page +
                         (int64_t)id.place[at] * c.vs.slot +
                         (uint32_t)((q * 4 + j % 4) * (int32_t)c.vs.slot)
                   : vh + (int64_t)pg * c.vs.page +
                         (int64_t)id.place[at] * c.vs.slot;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            // Columns past the row repeat its first; they are never stored.
            const int col = (nb * 16 + n) * VE * ES;
            const char* src = row + (col < c.row_bytes ? col : 0);
            if constexpr (VD == 4) {
              const v4i x = ld_once<v4i>(src);
#pragma unroll
              for (int e = 0; e < 4; ++e) vr[nb][j][e] = x[e];
            } else if constexpr (VD == 2) {
              const v2i x = ld_once<v2i>(src);
              vr[nb][j][0] = x[0];
              vr[nb][j][1] = x[1];
            } else {
              vr[nb][j][0] = ld_once<int>(src);
            }
          }
        }
      };

      typename A::Ids cur = find_tile<A, PG16>(c, table, t, len, q, n);
      load_k(cur);
      load_v(cur);
      typename A::Ids next =
          find_tile<A, PG16>(c, table, t + ts, len, q, n);
      // Elements past the row's end are 0 in K and in q (here, where the
      // first tile is on its way).
#pragma unroll
      for (int f = 0; f < QL; ++f) {
        const int d = CT == kE4m3 ? f / 2 * 64 + q * 16 + f % 2 * 8
                                  : f * 32 + q * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[f].d[e] = d < c.dim ? qf[f].d[e] : 0;
      }

      auto step = [&](auto more) {
        // Scores of 2 x 16 slots.
        f32x4 s[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          s[tt] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KL; ++k) {
            v4i x = kr[tt][k];
            if (A::last_chunk(k) >= A::SHORT) {
              const bool in = k * 64 + q * 16 < c.row_bytes;
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = in ? x[e] : 0;
            }
            if constexpr (CT == kE4m3) {
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const Frag a = {{widen2<QT, false>(x[2 * f]),
                                 widen2<QT, true>(x[2 * f]),
                                 widen2<QT, false>(x[2 * f + 1]),
                                 widen2<QT, true>(x[2 * f + 1])}};
                s[tt] = mma<QT>(a, qf[2 * k + f], s[tt]);
              }
            } else {
              s[tt] = mma<QT>(Frag{{x[0], x[1], x[2], x[3]}}, qf[k], s[tt]);
            }
          }
        }
        // The next tile's K goes on its way, then the page numbers of the
        // tile after it: the wait for these, next time, leaves the V loads
        // behind them in flight.
        typename A::Ids after;
        sched_fence();
        if constexpr (decltype(more)::value) {
          load_k(next);
          after = find_tile<A, PG16>(c, table, t + 2 * ts, len, q, n);
        }
        sched_fence();
        // Slots that count.
        bool ok[8];
        bool all = (t + 1) * kTileSlots <= len;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int32_t slot = t * kTileSlots + j / 4 * 16 + q * 4 + j % 4;
          const bool good =
              page_ok(cur.id[PG16 ? j / 4 : j + 2], c.pages);
          ok[j] = slot < len && good;
          all = all && good;
        }
        if (PG16 ? !all : ballot(!all) != 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < VD; ++e)
                vr[nb][j][e] = ok[j] ? vr[nb][j][e] : 0;
        }
        float x[8];
        float hi_x = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = ok[j] ? s[j / 4][j % 4] * scale : -INFINITY;
          hi_x = fmaxf(hi_x, x[j]);
        }
        if (tile_scores) {
          if (n < queries) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
              *(f32x4*)(tile_scores + score_at(n, tt * 4 + q)) =
                  f32x4{x[4 * tt], x[4 * tt + 1], x[4 * tt + 2],
                        x[4 * tt + 3]};
          }
          tile_scores += ts * tile_floats;
        }
        // The reference m of a query only moves when a score passes it by
        // 2^8: until then exp2(x - m) stays below 2^8 and nothing has to be
        // rescaled (a running maximum settles after a few tiles anyway).
        if (ballot(hi_x > m + 8.0f) != 0) {
          const float mn = fmaxf(m, quad_max(hi_x));
          const float f = mn == m ? 1.0f : exp2_fast(m - mn);
          m = mn;
          l *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float fi = __shfl(f, q * 4 + i, kWave);
#pragma unroll
            for (int e = 0; e < NB * VE; ++e) o[e][i] *= fi;
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = exp2_fast(x[j] - ref);
#pragma unroll
        for (int j = 0; j < 8; j += 2) l += w[j] + w[j + 1];
        if constexpr (CT == kF16) {
          // Product in float32: a weight counts however small it is, where the
          // rows of the larger ones are zero, and below 2^-14 float16 has not
          // the bits, below 2^-25 not the range.  Instruction j of a column
          // block contracts over the j-th slot of the four lane groups.
          // Against 16-bit operands these are eight times the matrix cycles:
          // 133 us against 132 for 48 sequences of up to 8000 slots, 8 heads
          // of 4 queries of 128 elements, 11.0 against 9.4 for 211 slots.
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int e = 0; e < VE; e += 2) {
                const f16x2 y = __builtin_bit_cast(f16x2, vr[nb][j][e / 2]);
                f32x4* acc = &o[nb * VE + e];
                acc[0] = mma4(w[j], (float)y[0], acc[0]);
                acc[1] = mma4(w[j], (float)y[1], acc[1]);
              }
        } else {
          // Weights enter the product as three bfloat16 numbers each (see
          // split3), which has the range of float32: out is rounded once, at
          // the end.  (bfloat16 holds e4m3 rows exactly.)
          Frag part[3];
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            unsigned a[3], b[3];
            split3(w[j], a);
            split3(w[j + 1], b);
#pragma unroll
            for (int i = 0; i < 3; ++i)
              part[i].d[j / 2] =
                  (int)__builtin_amdgcn_perm(b[i], a[i], 0x07060302u);
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            int y[8][VE / 2];  // 8 slots of VE elements
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if constexpr (CT == kE4m3) {
#pragma unroll
                for (int e = 0; e < VD; ++e) {
                  y[j][2 * e] = widen2<kBf16, false>(vr[nb][j][e]);
                  y[j][2 * e + 1] = widen2<kBf16, true>(vr[nb][j][e]);
                }
              } else {
#pragma unroll
                for (int e = 0; e < VD; ++e) y[j][e] = vr[nb][j][e];
              }
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              // element e of the 8 slots: low or high halves, in pairs
              const unsigned sel = e % 2 ? 0x07060302u : 0x05040100u;
              Frag v;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                v.d[j] = (int)__builtin_amdgcn_perm((unsigned)y[2 * j + 1][e / 2],
                                                    (unsigned)y[2 * j][e / 2],
                                                    sel);
              f32x4& acc = o[nb * VE + e];
#pragma unroll
              for (int i = 0; i < 3; ++i) acc = mma<kBf16>(part[i], v, acc);
            }
          }
        }
        sched_fence();
        if constexpr (decltype(more)::value) {
          load_v(next);
          cur = next;
          next = after;
          sched_fence();
        }
      };
      for (; t + ts < t1; t += ts) step(std::true_type());
      step(std::false_type());
    }
    l = quad_sum(l);

    // ---- the workgroup's waves joined ---------------------------------------
    const bool whole = s0 == r0 && s1 == r1;
    // Bytes of a share's result, and where this one lies: a workgroup can
    // have a row's end and, last, another's beginning.
    const int32_t part_rows = HS * p.part_rows;
    const int32_t part_size = share_floats(part_rows, COLS) * 4;
    const int32_t part = (wg * 2 + (s0 == r0)) * part_size;
    const int32_t at_m = part_rows * COLS * 4, at_l = at_m + part_rows * 4;
    const __amdgpu_buffer_rsrc_t parts = __builtin_amdgcn_make_buffer_rsrc(
        p.part, (short)0, grid * 2 * part_size, 0x00020000);
    // Four columns of query g of head s of a row: out, and with the first of
    // them lse.
    auto store = [&](const Share& r, int s, int g, int col, float top,
                     float sum, f32x4 x) {
      const int h = r.hi / p.gtiles * HS + s;
      const int64_t row = ((int64_t)r.b * c.heads + h) * p.group +
                          r.hi % p.gtiles * 16 + g;
      if (col == 0) {
        const float z = sum == 0.0f ? -INFINITY : top + log2f(sum);
        lds.lse2[s * 16 + g] = z;
        p.lse[row] = z * kLn2;
      }
      if (col >= c.dim) return;
      const float f = (p.v_scale ? p.v_scale[h] : 1.0f) / sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = sum == 0.0f ? 0.0f : x[e] * f;
      *(int2*)((char*)p.out + (row * c.dim + col) * 2) =
          make_int2(pack2<QT>(x[0], x[1]), pack2<QT>(x[2], x[3]));
    };
    auto weight = [](float m, float top) {
      return m == top ? 1.0f : exp2_fast(m - top);
    };
    if (q == 0) {
      lds.m[wave][n] = m;
      lds.l[wave][n] = l;
    }
    if (q * 4 < queries) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < VE; e += 4) {
            f32x4 x;
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = o[nb * VE + e + k][i];
            *(f32x4*)&join[(wave * p.lds_rows + q * 4 + i) * COLS +
                           (nb * 16 + n) * VE + e] = x;
          }
    }
    __syncthreads();
    for (int at = tid; at < HS * queries * (COLS / 4); at += kAttThreads) {
      const int col = at % (COLS / 4) * 4, sg = at / (COLS / 4);
      const int s = HS > 1 ? sg / queries : 0, g = sg - s * queries;
      float top = -INFINITY, sum = 0.0f;
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < ts; ++i)
        top = fmaxf(top, lds.m[i * HS + s][g]);
#pragma unroll
      for (int i = 0; i < ts; ++i) {
        const int w = i * HS + s;
        const float f = weight(lds.m[w][g], top);
        sum += lds.l[w][g] * f;
        x += *(const f32x4*)&join[(w * p.lds_rows + g) * COLS + col] * f;
      }
      if (whole) {
        store(cur, s, g, col, top, sum, x);
      } else {
        const int row = s * p.part_rows + g;
        if (col == 0) {
          st_agent1(parts, part + at_m + row * 4, top);
          st_agent1(parts, part + at_l + row * 4, sum);
        }
        st_agent4(parts, part + (row * COLS + col) * 4, x);
      }
    }
    __syncthreads();

    if (p.scores) {
      const bool added = whole && p.gtiles == 1;
      if (!p.direct && s0 == r0 && tid == 0)
        p.shares[(int64_t)b * hg + hi] =
            added   ? make_int2(kRowDone, 0)
            : whole ? make_int2(kRowJoined, 0)
                    : make_int2(cur.first, cur.last);
      if (added) {
        finish_weights(cur, queries);
        held -= cur.count;
        __syncthreads();
      }
      // (The rows of a head with more than 16 queries share its weights, and
      // leave them to the second kernel.)
      if (whole && !added) {
        flush(cur);
        held = cur.at;
        __syncthreads();
      }
    }
    // Nothing left to this workgroup but, perhaps, the next row's cost.
    const bool at_end = s1 == u1 || r1 + cost >= u1;
    if (!whole && p.scores && !at_end) pend = cur;

    // ---- shares of split rows joined, by the last workgroup of each ----------
    if (p.scores && at_end) {
      flush(pend);
      if (!whole) flush(cur);
    }
    if (p.scores && !p.direct) {
      u = s1;
      continue;
    }
    for (int which = 0; which < 2; ++which) {
      Share& r = which ? cur : pend;
      if (which ? whole || (p.scores && !at_end) : !at_end || !pend.open)
        continue;
      const int32_t first = r.first, last = r.last;
      if (!last_to_finish(p.ticket + (int64_t)r.b * hg + r.hi,
                          last - first + 1, p.epoch, &lds.flag))
        continue;
      const int g0 = r.hi % p.gtiles * 16;
      const int queries = p.group - g0 < 16 ? p.group - g0 : 16;
      auto part_of = [&](int32_t w) {
        return (w * 2 + (w == first)) * part_size;
      };
      // Four columns a thread, VP times over; with threads to spare, the
      // shares are split over `subs` of them.
      constexpr int VP = NC > 4 ? 4 : 1;
      constexpr int J = NC > 4 ? 4 : 8;  // shares whose loads are in flight
      const int vecs = HS * queries * (COLS / 4);
      const int subs =
          min(vecs < kAttThreads ? kAttThreads / vecs : 1, last - first + 1);
      const int sub = subs > 1 ? tid / vecs : 0;
      for (int at0 = subs > 1 ? tid % vecs : tid; at0 < vecs;
           at0 += VP * kAttThreads) {
      float top[VP], sum[VP];
      f32x4 x[VP];
#pragma unroll
      for (int v = 0; v < VP; ++v) {
        top[v] = -INFINITY;
        sum[v] = 0.0f;
        x[v] = f32x4{0, 0, 0, 0};
      }
      if (sub < subs) {
        for (int32_t w = first + sub; w <= last; w += J * subs) {
          f32x4 d[VP][J];
          float mw[VP][J], lw[VP][J];
#pragma unroll
          for (int v = 0; v < VP; ++v) {
            const int at = at0 + v * kAttThreads;
            const int sg = at / (COLS / 4), col = at % (COLS / 4) * 4;
            const int s = HS > 1 ? sg / queries : 0;
            const int row = s * p.part_rows + sg - s * queries;
#pragma unroll
            for (int j = 0; j < J; ++j) {
              // past the last: beyond the buffer, which reads nothing
              const int32_t wj = w + j * subs;
              const int32_t pj =
                  wj <= last && at < vecs ? part_of(wj) : 0x40000000;
              d[v][j] = ld_agent4(parts, pj + (row * COLS + col) * 4);
              mw[v][j] = ld_agent1(parts, pj + at_m + row * 4);
              lw[v][j] = ld_agent1(parts, pj + at_l + row * 4);
            }
          }
#pragma unroll
          for (int v = 0; v < VP; ++v) {
            float next = top[v];
#pragma unroll
            for (int j = 0; j < J; ++j)
              if (w + j * subs <= last) next = fmaxf(next, mw[v][j]);
            const float f0 = weight(top[v], next);
            top[v] = next;
            sum[v] *= f0;
            x[v] *= f0;
#pragma unroll
            for (int j = 0; j < J; ++j) {
              const float f =
                  w + j * subs <= last ? weight(mw[v][j], next) : 0.0f;
              sum[v] += lw[v][j] * f;
              x[v] += d[v][j] * f;
            }
          }
        }
      }
      if (subs > 1) {  // then a thread has v = 0 alone
        f32x4* xs = (f32x4*)join;
        float2* ts = (float2*)(join + 4 * kAttThreads);
        if (sub < subs) {
          xs[sub * vecs + at0] = x[0];
          ts[sub * vecs + at0] = make_float2(top[0], sum[0]);
        }
        __syncthreads();
        if (sub == 0) {
          float next = top[0];
          for (int i = 1; i < subs; ++i)
            next = fmaxf(next, ts[i * vecs + at0].x);
          const float f0 = weight(top[0], next);
          sum[0] *= f0;
          x[0] *= f0;
          for (int i = 1; i < subs; ++i) {
            const float2 z = ts[i * vecs + at0];
            const float f = weight(z.x, next);
            sum[0] += z.y * f;
            x[0] += xs[i * vecs + at0] * f;
          }
          top[0] = next;
        }
      }
#pragma unroll
      for (int v = 0; v < VP; ++v) {
        const int at = at0 + v * kAttThreads, sg = at / (COLS / 4);
        const int s = HS > 1 ? sg / queries : 0;
        if (sub == 0 && at < vecs)
          store(r, s, sg - s * queries, at % (COLS / 4) * 4, top[v], sum[v],
                x[v]);
      }
      }
      __syncthreads();
      if (p.scores) finish_weights(r, queries);
      __syncthreads();
    }
    u = s1;
  }
}

// What a launch of the kernel needs.
struct AttendNeeds {
  int cols;  // columns of a partial result
  int threads;
  int lds;   // bytes of static LDS
  int join;  // floats of dynamic LDS at least
};

// The kernel for a row length, page size and order of heads.  The type pairs
// are translation units of their own (cache_attend.hip).
template <int Q, int C>
const void* attend_fn_dim(int dim, bool pg16, bool heads, AttendNeeds* n);

}  // namespace ltk
