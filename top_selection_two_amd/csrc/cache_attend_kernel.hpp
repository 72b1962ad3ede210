// Attention of one new token over a paged cache.
//
// For query j of head h and slot t: x = scale k_scale (q . K_t).  One pass
// over the slots keeps a running maximum m, l = sum exp(x - m) and
// o = sum exp(x - m) V_t; out = v_scale o / l, lse = m + ln l.  Exponentials
// are taken to base 2 (scale is multiplied by log2 e on the host).
//
// The kernel reads every K and V row once and should run at the rate of that
// read.  Work: the slots of a row (a sequence, a cache head and up to 16 of
// its queries) are cut into units of kUnit slots; the units of all rows, in
// order, are dealt out in equal runs to as many workgroups as the chip holds
// at once, so that sequences of any mix of lengths load it evenly.  A row that
// lies within one run is finished there; of the others each run leaves its
// (m, l, o), and the row's last workgroup to finish joins them.
#pragma once

#include <type_traits>

#include "cache_common.hpp"

namespace ltk {

struct AttendParams {
  CacheParams c;
  LedgerParams w;
  const char* q;
  int64_t qb, qh;       // bytes
  int32_t group;        // query heads of a cache head
  int32_t gtiles;       // rows of a cache head: ceil(group / 16)
  float scale2;         // scale * log2 e
  const float* k_scale; // NULL: 1
  const float* v_scale;
  float* scores;        // [batch][q heads][score_ld], with a ledger
  int64_t score_ld;     // cap rounded up to a tile
  float* part;          // [grid][2][part_rows * columns + 2 * part_rows]
  int32_t part_rows;    // queries of a row, at most 16
  uint64_t* ticket;     // one per row
  uint32_t epoch;
  void* out;
  float* lse;
};

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kAttWaves = 8;
constexpr int kAttThreads = kAttWaves * kWave;
constexpr int kTileSlots = 32;                       // of one wave
constexpr int kUnit = kTileSlots * kAttWaves;        // of a workgroup

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

// Two floats rounded to the operand's type, and back.
template <int QT>
__device__ __forceinline__ int pack2(float a, float b) {
  if constexpr (QT == kBf16)
    return __builtin_bit_cast(int, bf16x2{(__bf16)a, (__bf16)b});
  else
    return __builtin_bit_cast(int, f16x2{(_Float16)a, (_Float16)b});
}
template <int QT>
__device__ __forceinline__ void unpack2(int v, float* a, float* b) {
  if constexpr (QT == kBf16) {
    *a = __int_as_float(v << 16);
    *b = __int_as_float(v & (int)0xffff0000);
  } else {
    const f16x2 h = __builtin_bit_cast(f16x2, v);
    *a = (float)h[0];
    *b = (float)h[1];
  }
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
//    element e, so its column n is the row's element n VE + e.
//
// QT: query type, CT: cache type, NC: 32-element chunks of a row, PG16: pages
// of a multiple of 16 slots, so that each half of a tile lies in one page.
template <int QT, int CT, int NC, bool PG16>
struct Attend {
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

  struct Lds {
    float o[kAttWaves][4][COLS];
    float m[kAttWaves][16];
    float l[kAttWaves][16];
    float top[16], sum[16];
    int32_t scan[kAttWaves];
    int32_t base;
    int32_t b;
    int32_t flag;
  };
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
      r.id[tt] = table[p];
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

template <int QT, int CT, int NC, bool PG16>
__global__ __launch_bounds__(kAttThreads, 2) void attend_kernel(
    AttendParams p) {
  typedef Attend<QT, CT, NC, PG16> A;
  constexpr int ES = A::ES, KL = A::KL, VE = A::VE, VD = A::VD, NB = A::NB;
  constexpr int COLS = A::COLS, QL = A::QL;
  __shared__ typename A::Lds lds;
  const CacheParams& c = p.c;
  const int tid = threadIdx.x, wave = uni(tid / kWave), ln = tid % kWave;
  const int q = ln / 16, n = ln % 16;
  const int hg = c.heads * p.gtiles;  // rows of a sequence

  // ---- this workgroup's run of units -------------------------------------
  // Units of a sequence, at least one a row: an empty row has an output too.
  const int32_t top_len = c.pages > 0 ? c.cap : 0;
  auto len_of = [&](int b) { return clamp_len(c.lens[b], top_len); };
  auto units_of = [&](int b) {
    const int32_t len = len_of(b);
    return (len > 0 ? (len + kUnit - 1) / kUnit : 1) * hg;
  };
  int32_t u0, u1, per, base;
  int b;
  {
    // Thread i takes sequences [i * each, (i + 1) * each).
    const int each = (c.batch + kAttThreads - 1) / kAttThreads;
    int32_t mine = 0;
    for (int i = tid * each; i < (tid + 1) * each && i < c.batch; ++i)
      mine += units_of(i);
    const int32_t incl = wave_scan_incl(mine);
    if (ln == kWave - 1) lds.scan[wave] = incl;
    __syncthreads();
    int32_t before = incl - mine, all = 0;
    for (int i = 0; i < kAttWaves; ++i) {
      if (i < wave) before += lds.scan[i];
      all += lds.scan[i];
    }
    all = uni(all);
    per = (all + (int32_t)gridDim.x - 1) / (int32_t)gridDim.x;
    u0 = (int32_t)blockIdx.x * per;
    u1 = u0 + per < all ? u0 + per : all;
    if (u0 >= all) return;
    if (u0 >= before && u0 < before + mine) {
      int i = tid * each;
      for (int32_t un; before + (un = units_of(i)) <= u0; ++i) before += un;
      lds.b = i;
      lds.base = before;
    }
    __syncthreads();
    b = uni(lds.b);
    base = uni(lds.base);
  }

  int32_t len = len_of(b);
  int32_t row_units = units_of(b) / hg;
  int32_t u = u0;
  while (u < u1) {
    // ---- a row's share of the run ------------------------------------------
    while (u >= base + row_units * hg) {
      base += row_units * hg;
      ++b;
      len = len_of(b);
      row_units = units_of(b) / hg;
    }
    const int hi = uni((u - base) / row_units);
    const int h = hi / p.gtiles, g0 = hi % p.gtiles * 16;
    const int32_t r0 = base + hi * row_units, r1 = r0 + row_units;
    const int32_t s1 = r1 < u1 ? r1 : u1;
    const int queries = p.group - g0 < 16 ? p.group - g0 : 16;
    const int64_t qrow = (int64_t)b * c.heads * p.group + h * p.group + g0;
    const int32_t* table = c.table + b * c.table_stride;
    const int32_t tiles = (len + kTileSlots - 1) / kTileSlots;
    int32_t t = (u - r0) * kAttWaves + wave;
    int32_t t1 = (s1 - r0) * kAttWaves;
    if (t1 > tiles) t1 = tiles;
    const char* kh = c.k + h * c.ks.head;
    const char* vh = c.v + h * c.vs.head;
    float* scores =
        p.scores ? p.scores + (qrow + n) * p.score_ld : nullptr;
    const float scale = p.scale2 * (p.k_scale ? p.k_scale[h] : 1.0f);

    float m = -INFINITY, l = 0.0f;
    f32x4 o[NB * VE];
#pragma unroll
    for (int i = 0; i < NB * VE; ++i) o[i] = f32x4{0, 0, 0, 0};

    if (t < t1) {
      // Query fragments: those of 8-bit rows pair up to match 16-byte loads.
      Frag qf[QL];
#pragma unroll
      for (int f = 0; f < QL; ++f) {
        const int d = CT == kE4m3 ? f / 2 * 64 + q * 16 + f % 2 * 8
                                  : f * 32 + q * 8;
        v4i x = {0, 0, 0, 0};
        if (n < queries && d < c.dim)
          x = *(const v4i*)(p.q + b * p.qb + (h * p.group + g0 + n) * p.qh +
                            d * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[f].d[e] = x[e];
      }

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
            kr[tt][k] = *(const v4i*)(row + (in ? at : 0));
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
              const v4i x = *(const v4i*)src;
#pragma unroll
              for (int e = 0; e < 4; ++e) vr[nb][j][e] = x[e];
            } else if constexpr (VD == 2) {
              const int2 x = *(const int2*)src;
              vr[nb][j][0] = x.x;
              vr[nb][j][1] = x.y;
            } else {
              vr[nb][j][0] = *(const int*)src;
            }
          }
        }
      };

      typename A::Ids cur = find_tile<A, PG16>(c, table, t, len, q, n);
      load_k(cur);
      load_v(cur);
      typename A::Ids next =
          find_tile<A, PG16>(c, table, t + kAttWaves, len, q, n);

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
          after = find_tile<A, PG16>(c, table, t + 2 * kAttWaves, len, q, n);
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
        if (scores && n < queries) {
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) {
            uint64_t* dst = (uint64_t*)(scores + t * kTileSlots + tt * 16 +
                                        q * 4);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              st_agent(dst + e,
                       (uint64_t)__float_as_uint(x[4 * tt + 2 * e]) |
                           (uint64_t)__float_as_uint(x[4 * tt + 2 * e + 1])
                               << 32);
          }
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
        // A weight enters the product as two numbers of the operand's type,
        // its rounding and what that lost (2^-17 relative left in bfloat16):
        // out is then rounded once, at the end, as if the weights had stayed
        // in float32.
        Frag hi, lo;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float e0 = exp2_fast(x[j] - ref), e1 = exp2_fast(x[j + 1] - ref);
          l += e0 + e1;
          hi.d[j / 2] = pack2<QT>(e0, e1);
          float a0, a1;
          unpack2<QT>(hi.d[j / 2], &a0, &a1);
          lo.d[j / 2] = pack2<QT>(e0 - a0, e1 - a1);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          int w[8][VE / 2];  // 8 slots of VE elements
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if constexpr (CT == kE4m3) {
#pragma unroll
              for (int e = 0; e < VD; ++e) {
                w[j][2 * e] = widen2<QT, false>(vr[nb][j][e]);
                w[j][2 * e + 1] = widen2<QT, true>(vr[nb][j][e]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < VD; ++e) w[j][e] = vr[nb][j][e];
            }
          }
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            // element e of the 8 slots: low or high halves, in pairs
            const unsigned sel = e % 2 ? 0x07060302u : 0x05040100u;
            Frag v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v.d[j] = (int)__builtin_amdgcn_perm((unsigned)w[2 * j + 1][e / 2],
                                                  (unsigned)w[2 * j][e / 2],
                                                  sel);
            f32x4& acc = o[nb * VE + e];
            acc = mma<QT>(hi, v, acc);
            acc = mma<QT>(lo, v, acc);
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
      for (; t + kAttWaves < t1; t += kAttWaves) step(std::true_type());
      step(std::false_type());
      l = quad_sum(l);
    }

    // ---- the workgroup's waves joined ---------------------------------------
    const bool whole = u == r0 && s1 == r1;
    const int32_t first = r0 / per, last = (r1 - 1) / per;
    const int64_t part_size = (int64_t)p.part_rows * (COLS + 2);
    float* part = p.part + ((int64_t)blockIdx.x * 2 + (u == r0)) * part_size;
    if (q == 0) {
      lds.m[wave][n] = m;
      lds.l[wave][n] = l;
    }
    __syncthreads();
    if (tid < 16) {
      float top = -INFINITY, sum = 0.0f;
      for (int w = 0; w < kAttWaves; ++w) top = fmaxf(top, lds.m[w][tid]);
      for (int w = 0; w < kAttWaves; ++w) {
        const float f =
            lds.m[w][tid] == top ? 1.0f : exp2_fast(lds.m[w][tid] - top);
        lds.m[w][tid] = f;
        sum += lds.l[w][tid] * f;
      }
      lds.top[tid] = top;
      lds.sum[tid] = sum;
      if (tid < queries) {
        if (whole) {
          p.lse[qrow + tid] =
              sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        } else {
          st_agent(part + p.part_rows * COLS + tid, top);
          st_agent(part + p.part_rows * (COLS + 1) + tid, sum);
        }
      }
    }
    const float vs = p.v_scale ? p.v_scale[h] : 1.0f;
    auto store = [&](int g, int col, float x) {
      const int64_t at = (qrow + g) * c.dim + col;
      if constexpr (QT == kBf16)
        ((__bf16*)p.out)[at] = (__bf16)x;
      else
        ((_Float16*)p.out)[at] = (_Float16)x;
    };
    for (int g4 = 0; g4 < queries; g4 += 4) {
      if (q == g4 / 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
              f32x4 x;
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = o[nb * VE + e + k][i];
              *(f32x4*)&lds.o[wave][i][(nb * 16 + n) * VE + e] = x;
            }
      }
      __syncthreads();
      for (int at = tid; at < 4 * COLS; at += kAttThreads) {
        const int i = at / COLS, col = at % COLS, g = g4 + i;
        if (g >= queries || col >= c.dim) continue;
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttWaves; ++w) x += lds.o[w][i][col] * lds.m[w][g];
        if (whole)
          store(g, col, lds.sum[g] == 0.0f ? 0.0f : x * vs / lds.sum[g]);
        else
          st_agent(part + g * COLS + col, x);
      }
      __syncthreads();
    }

    // ---- the row's runs joined, by the last of them --------------------------
    if (!whole &&
        last_to_finish(p.ticket + (int64_t)b * hg + hi, last - first + 1,
                       p.epoch, &lds.flag)) {
      auto part_of = [&](int32_t w) {
        return p.part + ((int64_t)w * 2 + (w == first)) * part_size;
      };
      const int g = tid / 32;  // 16 queries by 32 threads
      float top = -INFINITY, sum = 0.0f;
      if (g < queries) {
        for (int32_t w = first + tid % 32; w <= last; w += 32)
          top = fmaxf(top, ld_agent(part_of(w) + p.part_rows * COLS + g));
#pragma unroll
        for (int k = 16; k > 0; k >>= 1)
          top = fmaxf(top, __shfl_xor(top, k, kWave));
        for (int32_t w = first + tid % 32; w <= last; w += 32) {
          const float* pm = part_of(w) + p.part_rows * COLS + g;
          const float mw = ld_agent(pm);
          sum += ld_agent(pm + p.part_rows) *
                 (mw == top ? 1.0f : exp2_fast(mw - top));
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor(sum, k, kWave);
        if (tid % 32 == 0) {
          lds.top[g] = top;
          lds.sum[g] = sum;
          p.lse[qrow + g] =
              sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
      }
      __syncthreads();
      for (int at = tid; at < queries * COLS; at += kAttThreads) {
        const int gg = at / COLS, col = at % COLS;
        if (col >= c.dim) continue;
        const float tg = lds.top[gg];
        float x = 0.0f;
#pragma unroll 8
        for (int32_t w = first; w <= last; ++w) {
          const float* pw = part_of(w);
          const float mw = ld_agent(pw + p.part_rows * COLS + gg);
          x += ld_agent(pw + gg * COLS + col) *
               (mw == tg ? 1.0f : exp2_fast(mw - tg));
        }
        store(gg, col, lds.sum[gg] == 0.0f ? 0.0f : x * vs / lds.sum[gg]);
      }
    }
    u = s1;
  }
}

// weights[t] += sum over the head's queries of exp(x - lse).  One workgroup
// per chunk of kBlock slots of a sequence and head, round robin.
__global__ __launch_bounds__(kBlock) void attend_weights_kernel(
    AttendParams p) {
  const CacheParams& c = p.c;
  const int32_t chunks = (c.cap + kBlock - 1) / kBlock;
  const int64_t all = (int64_t)c.batch * c.heads * chunks;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int row = (int)(i / chunks);  // sequence and head
    const int b = row / c.heads, h = row % c.heads;
    const int32_t len = clamp_len(c.lens[b], c.pages > 0 ? c.cap : 0);
    const int32_t t = (int32_t)(i % chunks) * kBlock + threadIdx.x;
    if (t >= len) continue;
    const int64_t first = (int64_t)row * p.group;
    float a = 0.0f;
    for (int g = 0; g < p.group; ++g) {
      const float lse2 = p.lse[first + g] * (1.0f / kLn2);
      const float x = p.scores[(first + g) * p.score_ld + t];
      a += x == -INFINITY ? 0.0f : exp2_fast(x - lse2);
    }
    p.w.w[b * p.w.wb + h * p.w.wh + t] += a;
  }
}

}  // namespace ltk
