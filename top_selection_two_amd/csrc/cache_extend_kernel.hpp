// New tokens' heads enter a paged cache: queries and keys normed and rotated,
// keys and values rounded to the cache's type.
//
// A row (one head of one token) of `dim` elements x becomes, for q and k,
// y = x (mean x^2 + eps)^-1/2 g and then pairs (a, b) of y turned by the angle
// position * freqs[j]: (a cos - b sin, b cos + a sin).  All of it is computed
// in 64 bits (4.4 cycles an instruction, 2.9 in 32 bits) and rounded at the
// end, through float32 where the type has 16 or 8 bits: a cache's 4-bit row,
// where a unit in the last place of a float32 can move an element by half its
// value, does not depend on how the sums were ordered.
//
// Bytes bound long calls: x is read once and y written once, a lane has 16 bytes
// of a row (extend_kernel, below).  12 prompts of 100 to 4001 tokens, 32 + 8 + 8
// heads of 128, bfloat16, 0.60 GB: 139 us (4.3 TB/s; a large copy reaches 5.2);
// into 4 bits, 6 prompts of 700 to 2048 tokens, 16 + 4 + 4 heads, 90 MB: 40 us
// (2.3 TB/s; the vector unit is busy half of the time with norms, turns and
// codes).  Few tokens are dealt out row by row: a token of 64 sequences takes
// 6 us, four dependent reads (starts, length, table, rows) and a launch; among
// other calls 10.9, which the host needs.
#pragma once

#include "cache_common.hpp"

namespace ltk {

struct ExtendParams {
  CacheParams c;
  BlockParams s;
  LedgerParams w;     // w.w NULL: none
  const char* q;      // NULL: none
  const char* k;
  const char* v;
  char* q_out;
  int64_t qt, qh, kt, kh, vt, vh, ot, oh;  // bytes
  const int32_t* starts;
  const int32_t* seen;  // NULL: the lengths
  const void* q_norm;   // NULL: none
  const void* k_norm;
  const float* freqs;   // NULL: none
  const float* k_scale; // NULL: 1
  const float* v_scale;
  int32_t* out_lens;
  int32_t tokens, q_heads;
  int32_t norm_type;
  int32_t half;         // pairs that turn
  bool interleaved;
  bool rest;            // queries of no sequence go to q_out as they are
  double eps, inv_dim;
  int32_t splits;       // waves of a token
};

typedef int v2i_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr int kUnit = 8;  // elements of a lane

// Two numbers rounded to float32 and then to a 16-bit type.  (Left to itself
// the compiler rounds once, by ten instructions more an element.)
template <int T>
__device__ __forceinline__ int round_pair(double a, double b) {
  float x = (float)a, y = (float)b;
  pin(x);
  pin(y);
  if constexpr (T == kBf16)
    return __builtin_bit_cast(int, bf16x2_t{(__bf16)x, (__bf16)y});
  else
    return __builtin_bit_cast(int, f16x2_t{(_Float16)x, (_Float16)y});
}

// The value of a lane that a data-parallel move names.
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xf,
                                             0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xf,
                                             0xf, false);
  return __hiloint2double(hi, lo);
}
constexpr int kDppXor1 = 0xb1;        // within quads
constexpr int kDppXor2 = 0x4e;
constexpr int kDppHalfMirror = 0x141; // 7 - i of 8
constexpr int kDppMirror = 0x140;     // 15 - i of 16
// Sum over runs of LPH lanes, the same in all of them: after each step the
// lanes that have been joined agree, so that a mirror is as good as a shift.
template <int LPH>
__device__ __forceinline__ double run_sum(double v) {
  v += dpp64<kDppXor1>(v);
  v += dpp64<kDppXor2>(v);
  v += dpp64<kDppHalfMirror>(v);
  if constexpr (LPH > 8) v += dpp64<kDppMirror>(v);
  if constexpr (LPH > 16) v += __shfl_xor(v, 16, kWave);
  return v;
}

// To e4m3's range (NaN stays).
__device__ __forceinline__ float within_e4m3(double x) {
  const float f = (float)x;
  return f != f ? f : fminf(fmaxf(f, -448.0f), 448.0f);
}

// Scale byte of a block whose largest magnitude is `top`: 2^(byte - 127) is
// the least power of two s with top < 7 s, so that no element is further from
// what it becomes than half a step.  With top = m 2^E, 1 <= m < 2: s =
// 2^(E - 2) if m < 1.75, twice that otherwise.
__device__ __forceinline__ int block_byte(double top) {
  const int hi = __double2hiint(top);
  if (hi >= 0x7ff00000) return 255;  // an infinity or NaN
  const int e =
      (hi >> 20) - 1023 - 2 + ((hi & 0xfffff) >= 0xc0000) + 127;
  return e < 0 ? 0 : e > 254 ? 254 : e;
}

// A magnitude of at most 7 or so, and its sign, in float32: the bits that do
// not fit leave their trace in the last one, so that rounding again to fewer
// bits is as rounding once.  Below 2^-126 what comes out is tiny, whatever it
// is.
__device__ __forceinline__ float sticky_float(double y) {
  const int hi = __double2hiint(y), lo = __double2loint(y);
  int t = (hi & 0x7fffffff) - ((1023 - 127) << 20);
  t = t > 0 ? t : 0;
  t = t < 0x0fdfffff ? t : 0x0fdfffff;  // float32's largest exponent
  unsigned m = __builtin_amdgcn_alignbit((unsigned)t, (unsigned)lo, 29);
  const unsigned rest = (unsigned)lo & 0x1fffffffu;
  m |= rest < 1u ? rest : 1u;
  return __uint_as_float(m | ((unsigned)hi & 0x80000000u));
}

// The 4-bit codes of x / 2^(byte - 127): the nearest of 0 .5 1 1.5 2 3 4 6, of
// two the even code, and 6 beyond.
__device__ __forceinline__ unsigned codes_of(const double* x, int byte) {
  unsigned code = 0;
  const int by = 127 - byte;
#define LTK_PAIR(i)                                                     \
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(                      \
      code, sticky_float(ldexp(x[2 * i], by)),                          \
      sticky_float(ldexp(x[2 * i + 1], by)), 1.0f, i)
  LTK_PAIR(0);
  LTK_PAIR(1);
  LTK_PAIR(2);
  LTK_PAIR(3);
#undef LTK_PAIR
  return code;
}

// cos and sin of position * freq.  The turns are taken modulo 1 in 64 bits
// from 1 / (2 pi) in two parts, so that far positions keep their angle.
__device__ __forceinline__ void angle(int64_t position, float freq,
                                      double* cos_, double* sin_) {
  constexpr double kInv = 0x1.45f306dc9c883p-3;     // 1 / (2 pi)
  constexpr double kInvLow = -0x1.6b01ec5417056p-57;  // and what is left
  const double a = (double)position * (double)freq;
  const double t = a * kInv;
  const double low = fma(a, kInv, -t) + a * kInvLow;
  const double r = (t - rint(t)) + low;
  sincospi(2.0 * r, sin_, cos_);
}

// 1 / sqrt(a) for a normal a > 0: the instruction's approximation and two of
// Newton's steps, each of which doubles its bits.
__device__ __forceinline__ double inv_sqrt(double a) {
  double y = __builtin_amdgcn_rsq(a);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double e = fma(-a * y, y, 1.0);
    y = fma(0.5 * y, e, y);
  }
  return y;
}

// Four consecutive numbers of a row, in one of two types.
typedef int v2i4_t __attribute__((ext_vector_type(2), aligned(4)));
typedef int v2i2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef int v4i4_t __attribute__((ext_vector_type(4), aligned(4)));
template <int T>
__device__ __forceinline__ void widen4(const v2i_t& v, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int d = v[i];
    if constexpr (T == kBf16) {
      x[2 * i] = __int_as_float(d << 16);
      x[2 * i + 1] = __int_as_float(d & 0xffff0000);
    } else {
      const f16x2_t h = __builtin_bit_cast(f16x2_t, d);
      x[2 * i] = (float)h[0];
      x[2 * i + 1] = (float)h[1];
    }
  }
}
// Weights e .. e + 3 of a norm, of the rows' type or float32.
template <int QT>
__device__ __forceinline__ void norm4(const void* g, int type, int e,
                                      float* w) {
  if (type == kF32) {
    const v4i4_t a = *(const v4i4_t*)((const float*)g + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __int_as_float(a[i]);
  } else {
    const v2i2_t a = *(const v2i2_t*)((const uint16_t*)g + e);
    widen4<QT>(v2i_t{a[0], a[1]}, w);
  }
}

// A wave takes a token's rows, or with few tokens a part of them: 64 / LPH
// rows at a time, LPH lanes a row, all of one kind (q, k or v).  A lane has 8
// elements of a row, in two runs of 4: where halves of the row turn against
// one another, a run of each half, so that it turns its elements by itself.
// Its runs lie at the same place in every row, so that it has the sines and
// cosines that it needs, found by all lanes of the wave once a token, and its
// norm's weights in registers; nothing is shared with other waves.  (Keys for
// 4-bit rows, whose blocks are consecutive, are turned with another lane's.)
template <int QT, int CT, int LPH>
__global__ __launch_bounds__(kBlock, 4) void extend_kernel(ExtendParams p) {
  const CacheParams& c = p.c;
  constexpr int kRows = kWave / LPH;
  __shared__ double2 turn_lds[kWaves][kMaxDim / 2];
  const int tid = threadIdx.x, wave = uni(tid / kWave), ln = tid % kWave;
  const int32_t top_len = c.pages > 0 ? c.cap : 0;
  auto bound = [&](int32_t s) { return s < 0 ? 0 : s > p.tokens ? p.tokens : s; };
  // Lengths after the call, kBlock sequences a workgroup.
  const int64_t mine = (int64_t)blockIdx.x * kBlock + tid;
  if (mine < c.batch) {
    const int32_t len = clamp_len(c.lens[mine], top_len);
    const int32_t s0 = bound(p.starts[mine]), s1 = bound(p.starts[mine + 1]);
    const int64_t next = (int64_t)len + (s1 > s0 ? s1 - s0 : 0);
    p.out_lens[mine] = next > top_len ? top_len : (int32_t)next;
  }
  // (tasks count in 32 bits)
  const unsigned task = (unsigned)blockIdx.x * kWaves + (unsigned)wave;
  const int32_t token =
      uni((int32_t)(p.splits > 1 ? task / (unsigned)p.splits : task));
  const int part = uni((int)(task - (unsigned)token * (unsigned)p.splits));
  if (token >= p.tokens) return;

  const int ul = ln % LPH, sub = ln / LPH;
  const bool in = ul * kUnit < c.dim;
  const bool turns = ul < p.half / 4;
  const bool halves = turns && !p.interleaved;
  // First elements of the lane's runs, in a row whose halves turn.
  const int run0 = halves ? 4 * ul : kUnit * ul;
  const int run1 = halves ? p.half + 4 * ul : kUnit * ul + 4;
  auto by_halves = [](int kind) {
    return kind == 0 || (kind == 1 && CT != kE2m1);
  };
  const int gq = (p.q_heads + kRows - 1) / kRows;
  const int gk = (c.heads + kRows - 1) / kRows;
  const int groups = gq + 2 * gk;
  // Rows of a group: of q (0), k (1) or v (2); none past the last head.  The
  // first head is the same in every lane, whose own is `sub` beyond it: only
  // that part of an address differs from lane to lane.
  auto kind_of = [&](int g) { return g < gq ? 0 : g < gq + gk ? 1 : 2; };
  auto first_of = [&](int g, int kind) {
    return (kind == 0 ? g : kind == 1 ? g - gq : g - gq - gk) * kRows;
  };
  const int64_t q_lane = sub * p.qh, k_lane = sub * p.kh, v_lane = sub * p.vh;
  const int64_t o_lane = sub * p.oh;
  const int64_t ck_lane = sub * c.ks.head, cv_lane = sub * c.vs.head;
  struct Raw {
    v2i_t a, b;
  };
  const char* const q_tok = p.q + token * p.qt;
  const char* const k_tok = p.k + token * p.kt;
  const char* const v_tok = p.v + token * p.vt;
  auto load = [&](int g) {
    Raw r = {{0, 0}, {0, 0}};
    if (g >= groups) return r;
    const int kind = kind_of(g), h0 = first_of(g, kind);
    const char* from;
    bool have;
    if (kind == 0) {
      from = q_tok + h0 * p.qh + q_lane;
      have = in && h0 + sub < p.q_heads;
    } else if (kind == 1) {
      from = k_tok + h0 * p.kh + k_lane;
      have = in && h0 + sub < p.c.heads;
    } else {
      from = v_tok + h0 * p.vh + v_lane;
      have = in && h0 + sub < p.c.heads;
    }
    if (have) {
      const bool split = by_halves(kind);
      r.a = *(const v2i_t*)(from + (split ? run0 : kUnit * ul) * 2);
      r.b = *(const v2i_t*)(from + (split ? run1 : kUnit * ul + 4) * 2);
    }
    return r;
  };
  Raw next = load(part);

  if (p.rest) {  // queries of no sequence, a row at a time
    const int32_t lo = c.batch > 0 ? bound(ld_const(p.starts)) : 0;
    const int32_t hi = c.batch > 0 ? bound(ld_const(p.starts + c.batch)) : 0;
    if (token < lo || token >= hi) {
      // (The launch's parameters are read again: kept for here they would cost
      // the loop below registers: prompts into 4 bits 9 us more.)
      typedef const __attribute__((address_space(4))) ExtendParams Again;
      uintptr_t again = (uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
      int32_t at = token, h = part;
      asm volatile("" : "+s"(again), "+s"(at), "+s"(h));
      Again& a = *(Again*)again;
      if (ln * 16 < a.c.dim * 2)
#pragma unroll 1
        for (; h < a.q_heads; h += a.splits)
          *(v4i*)(a.q_out + at * a.ot + h * a.oh + ln * 16) =
              *(const v4i*)(a.q + at * a.qt + h * a.qh + ln * 16);
      return;
    }
  }

  // ---- the token's sequence: the last whose start is not beyond it
  int32_t b = 0;
  for (int32_t j = 0; j < c.batch; j += kWave)
    b += popc(ballot(j + ln < c.batch &&
                     bound(p.starts[min(j + ln, c.batch - 1) + 1]) <= token));
  b = uni(b);
  const int32_t first = b < c.batch ? bound(ld_const(p.starts + b)) : 0;
  if (b >= c.batch || first > token) return;
  const int32_t nth = token - first;
  const int32_t len = clamp_len(ld_const(c.lens + b), top_len);
  const int64_t position =
      (int64_t)(p.seen ? ld_const(p.seen + b) : len) + nth;
  const int64_t slot = (int64_t)len + nth;
  int32_t place = 0, page = -1;
  if (slot < top_len)
    page = find_page(c, c.table + b * c.table_stride, (int32_t)slot, &place);
  page = uni(page);
  place = uni(place);
  // ---- its angles: a lane's four are 4 ul .. 4 ul + 3 in either pairing
  double cs[4], sn[4];
  double2* const turn = turn_lds[wave];
  if (p.half > 0) {
    for (int i = ln; i < p.half; i += kWave) {
      double x, y;
      angle(position, p.freqs[i], &x, &y);
      turn[i] = make_double2(x, y);
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double2 z = turns ? turn[4 * ul + e] : make_double2(1.0, 0.0);
      cs[e] = z.x;
      sn[e] = z.y;
    }
  }
  // ---- its rows
  const bool wide_norm = p.norm_type == kF32;
  int kind = -1;
  float w[kUnit];  // norm weights of the lane's elements
  for (int g = part; g < groups; g += p.splits) {
    const Raw raw = next;
    next = load(g + p.splits);
    const int was = kind;
    kind = kind_of(g);
    const bool split = by_halves(kind);
    const int h0 = first_of(g, kind), h = h0 + sub;
    const bool have = in && h < (kind == 0 ? p.q_heads : c.heads);
    const void* norm = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
    if (norm && kind != was) {
      norm4<QT>(norm, p.norm_type, !in ? 0 : split ? run0 : kUnit * ul, w);
      norm4<QT>(norm, p.norm_type, !in ? 0 : split ? run1 : kUnit * ul + 4,
                w + 4);
    }
    float f[kUnit];
    widen4<QT>(raw.a, f);
    widen4<QT>(raw.b, f + 4);
    double x[kUnit];
    double inv = 1.0;
#pragma unroll
    for (int e = 0; e < kUnit; ++e) x[e] = (double)f[e];
    if (norm) {
      double ss = 0.0;
#pragma unroll
      for (int e = 0; e < kUnit; ++e) ss = fma(x[e], x[e], ss);
      const double ms = run_sum<LPH>(ss) * p.inv_dim + p.eps;
      // (of zeros with eps = 0: infinity, and NaN as 0 times it)
      inv = ms > 0.0 ? inv_sqrt(ms) : INFINITY;
      if (!(ms < INFINITY)) inv = ms == INFINITY ? 0.0 : ms;
      // A product of two float16 numbers is exact in float32 (one of bfloat16
      // numbers is not: it can leave its range); the division by the row's size
      // comes after the turn.
      if (QT == kBf16 || wide_norm) {
#pragma unroll
        for (int e = 0; e < kUnit; ++e) x[e] *= (double)w[e];
      } else {
#pragma unroll
        for (int e = 0; e < kUnit; ++e) x[e] = (double)(f[e] * w[e]);
      }
    }
    if (p.half > 0 && kind != 2) {
      if (p.interleaved) {
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double a = x[2 * e], d = x[2 * e + 1];
            x[2 * e] = fma(-d, sn[e], a * cs[e]);
            x[2 * e + 1] = fma(a, sn[e], d * cs[e]);
          }
        }
      } else if (split) {
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double a = x[e], d = x[4 + e];
            x[e] = fma(-d, sn[e], a * cs[e]);
            x[4 + e] = fma(a, sn[e], d * cs[e]);
          }
        }
      } else {
        // Units of 8 in a row: turned with the unit of the other half.
        const int step = p.half / kUnit;
        const bool turned = ul < 2 * step, low = ul < step;
        const int other = turned ? (low ? ul + step : ul - step) : ul;
#pragma unroll
        for (int e = 0; e < kUnit; ++e) {
          const double z = __shfl(x[e], ln - ul + other, kWave);
          const double2 t = turned ? turn[(low ? ul : other) * kUnit + e]
                                   : make_double2(1.0, 0.0);
          const double y = fma(z, low ? -t.y : t.y, x[e] * t.x);
          x[e] = turned ? y : x[e];
        }
      }
    }
    if (norm) {
#pragma unroll
      for (int e = 0; e < kUnit; ++e) x[e] *= inv;
    }
    // ---- out
    if (kind == 0) {
      if (have) {
        char* to = p.q_out + token * p.ot + h0 * p.oh + o_lane;
        *(v2i_t*)(to + run0 * 2) =
            v2i_t{round_pair<QT>(x[0], x[1]), round_pair<QT>(x[2], x[3])};
        *(v2i_t*)(to + run1 * 2) =
            v2i_t{round_pair<QT>(x[4], x[5]), round_pair<QT>(x[6], x[7])};
      }
      continue;
    }
    const bool is_v = kind == 2;
    const float* scale = is_v ? p.v_scale : p.k_scale;
    if (scale) {
      const double s = have ? (double)scale[h] : 1.0;
#pragma unroll
      for (int e = 0; e < kUnit; ++e) x[e] /= s;
    }
    if (p.w.w && !is_v && have && ul == 0 && slot < top_len) {
      p.w.w[b * p.w.wb + h * p.w.wh + slot] = 0.0f;
      p.w.pos[b * p.w.pb + h * p.w.ph + slot] = (int32_t)position;
    }
    if (page < 0) continue;
    char* dst = const_cast<char*>(
        is_v ? c.v + row_offset(c.vs, page, h0, place) + cv_lane
             : c.k + row_offset(c.ks, page, h0, place) + ck_lane);
    if constexpr (CT == kE2m1) {
      double top = 0.0;
      bool odd = false;  // a NaN: max would drop it
#pragma unroll
      for (int e = 0; e < kUnit; ++e) {
        odd = odd || x[e] != x[e];
        top = fmax(top, fabs(x[e]));
      }
      if (odd) top = INFINITY;
      top = fmax(top, dpp64<kDppXor1>(top));
      top = fmax(top, dpp64<kDppXor2>(top));
      const int byte = block_byte(top);
      const unsigned code = codes_of(x, byte);
      if (!have) continue;
      *(unsigned*)(dst + ul * 4) = byte < 255 ? code : 0;
      if (ul % 4 == 0) {
        char* blocks = const_cast<char*>(
            is_v ? p.s.v + row_offset(p.s.vs, page, h, place)
                 : p.s.k + row_offset(p.s.ks, page, h, place));
        blocks[ul / 4] = (char)byte;
      }
    } else {
      if (!have) continue;
      const int e0 = split ? run0 : kUnit * ul;
      const int e1 = split ? run1 : kUnit * ul + 4;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const double* y = x + 4 * i;
        const int e = i ? e1 : e0;
        if constexpr (CT == kE4m3) {
          const int d = __builtin_amdgcn_cvt_pk_fp8_f32(
              within_e4m3(y[0]), within_e4m3(y[1]), 0, false);
          *(int*)(dst + e) = __builtin_amdgcn_cvt_pk_fp8_f32(
              within_e4m3(y[2]), within_e4m3(y[3]), d, true);
        } else {
          *(v2i_t*)(dst + e * 2) =
              v2i_t{round_pair<CT>(y[0], y[1]), round_pair<CT>(y[2], y[3])};
        }
      }
    }
  }
}

}  // namespace ltk
