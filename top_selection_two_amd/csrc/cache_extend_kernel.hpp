// New tokens' heads enter a paged cache: queries and keys normed and rotated,
// keys and values rounded to the cache's type.
//
// A row (one head of one token) of `dim` elements x becomes, for q and k,
// y = x (mean x^2 + eps)^-1/2 g and then pairs (a, b) of y turned by the angle
// position * freqs[j]: (a cos - b sin, b cos + a sin).  All of it is computed
// in 64 bits and rounded once: vector instructions in 64 bits run at the rate
// of those in 32, and a cache's 4-bit row, where a unit in the last place of a
// float32 can move an element by half its value, does not depend on how the
// sums were ordered.
#pragma once

#include "cache_common.hpp"

namespace ltk {

struct ExtendParams {
  CacheParams c;
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
  double eps, dim;
  int32_t splits;       // workgroups of a token
};

typedef int v2i_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr int kUnit = 8;  // elements of a lane: 16 bytes of the input

template <int T>
__device__ __forceinline__ void widen_pair(int v, double* x) {
  if constexpr (T == kBf16) {
    x[0] = (double)__int_as_float(v << 16);
    x[1] = (double)__int_as_float(v & 0xffff0000);
  } else {
    const f16x2_t h = __builtin_bit_cast(f16x2_t, v);
    x[0] = (double)(float)h[0];
    x[1] = (double)(float)h[1];
  }
}
template <int T>
__device__ __forceinline__ void widen_unit(const v4i& v, double (&x)[kUnit]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) widen_pair<T>(v[i], x + 2 * i);
}

// Two numbers rounded to a 16-bit type.
template <int T>
__device__ __forceinline__ int round_pair(double a, double b) {
  if constexpr (T == kBf16)
    return __builtin_bit_cast(int, bf16x2_t{(__bf16)(float)a, (__bf16)(float)b});
  else
    return __builtin_bit_cast(int,
                              f16x2_t{(_Float16)(float)a, (_Float16)(float)b});
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

// The 4-bit code of x / 2^(byte - 127): the nearest of 0 .5 1 1.5 2 3 4 6,
// the even code where two are.
__device__ __forceinline__ unsigned code_of(double x, int byte) {
  const double y = ldexp(x, 127 - byte);
  const double a = fabs(y);
  const int mag = (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) +
                  (a > 2.5) + (a >= 3.5) + (a > 5.0);
  return (unsigned)mag | ((unsigned)__double2hiint(x) >> 31) << 3;
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

// One workgroup takes a token's rows (or with few tokens a part of them),
// LPH lanes a row and a unit of 8 elements a lane.
template <int QT, int CT, int LPH>
__global__ __launch_bounds__(kBlock) void extend_kernel(ExtendParams p) {
  const CacheParams& c = p.c;
  __shared__ double cs[kMaxDim / 2], sn[kMaxDim / 2];
  __shared__ int counts[kWaves];
  const int tid = threadIdx.x;
  const int32_t top_len = c.pages > 0 ? c.cap : 0;
  auto start = [&](int32_t j) {
    const int32_t s = ld_const(p.starts + j);
    return s < 0 ? 0 : s > p.tokens ? p.tokens : s;
  };
  // Lengths after the call, kBlock sequences a workgroup.
  const int64_t mine = (int64_t)blockIdx.x * kBlock + tid;
  if (mine < c.batch) {
    const int32_t len = clamp_len(c.lens[mine], top_len);
    const int32_t s0 = start((int32_t)mine), s1 = start((int32_t)mine + 1);
    const int64_t next = (int64_t)len + (s1 > s0 ? s1 - s0 : 0);
    p.out_lens[mine] = next > top_len ? top_len : (int32_t)next;
  }
  const int32_t token = (int32_t)(blockIdx.x / (unsigned)p.splits);
  const int part = (int)(blockIdx.x % (unsigned)p.splits);
  if (token >= p.tokens) return;
  // Its sequence: the last whose start is not beyond it.
  int n = 0;
  for (int32_t j = tid; j < c.batch; j += kBlock)
    n += popc(ballot(start(j + 1) <= token)) * (tid % kWave == 0);
  if (tid % kWave == 0) counts[tid / kWave] = n;
  __syncthreads();
  int32_t b = 0;
  for (int i = 0; i < kWaves; ++i) b += counts[i];
  b = uni(b);
  if (b >= c.batch || start(b) > token) return;
  const int32_t nth = token - start(b);
  const int32_t len = clamp_len(ld_const(c.lens + b), top_len);
  const int64_t position =
      (int64_t)(p.seen ? ld_const(p.seen + b) : len) + nth;
  const int64_t slot = (int64_t)len + nth;
  int32_t place = 0, page = -1;
  if (slot < top_len)
    page = find_page(c, c.table + b * c.table_stride, (int32_t)slot, &place);
  if (p.half > 0) {
    for (int i = tid; i < p.half; i += kBlock)
      angle(position, p.freqs[i], &cs[i], &sn[i]);
    __syncthreads();
  }
  const int ul = tid % LPH;
  const int units = c.dim / kUnit;
  const bool in = ul < units;
  const int rows = p.q_heads + 2 * c.heads;
  constexpr int kRows = kBlock / LPH;
  for (int r0 = part * kRows; r0 < rows; r0 += p.splits * kRows) {
    const int row = r0 + tid / LPH;
    const bool have = in && row < rows;
    const bool is_q = row < p.q_heads;
    const bool is_v = row >= p.q_heads + c.heads;
    const int h = is_q ? row : row - p.q_heads - (is_v ? c.heads : 0);
    v4i raw = {0, 0, 0, 0};
    if (have)
      raw = *(const v4i*)((is_q   ? p.q + token * p.qt + h * p.qh
                           : is_v ? p.v + token * p.vt + h * p.vh
                                  : p.k + token * p.kt + h * p.kh) +
                          ul * 16);
    double x[kUnit];
    widen_unit<QT>(raw, x);
    // ---- norm
    const void* g = is_q ? p.q_norm : is_v ? nullptr : p.k_norm;
    double inv = 1.0;
    auto weight = [&](int e) {
      return p.norm_type == kF32 ? (double)((const float*)g)[e]
             : p.norm_type == kBf16
                 ? (double)__int_as_float((int)((const uint16_t*)g)[e] << 16)
                 : (double)(float)((const _Float16*)g)[e];
    };
    if (p.q_norm || p.k_norm) {
      double ss = 0.0;
#pragma unroll
      for (int e = 0; e < kUnit; ++e) ss = fma(x[e], x[e], ss);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor(ss, o, kWave);
      if (g && have) {
        inv = 1.0 / sqrt(ss / p.dim + p.eps);
#pragma unroll
        for (int e = 0; e < kUnit; ++e) x[e] *= inv * weight(ul * kUnit + e);
      }
    }
    // ---- rotation
    if (p.half > 0) {
      if (p.interleaved) {
        if (!is_v && have && ul * kUnit < 2 * p.half) {
#pragma unroll
          for (int e = 0; e < kUnit; e += 2) {
            const int j = (ul * kUnit + e) / 2;
            const double a = x[e], d = x[e + 1];
            x[e] = a * cs[j] - d * sn[j];
            x[e + 1] = d * cs[j] + a * sn[j];
          }
        }
      } else {
        // The other half's unit of the row, from its lane.
        const int step = p.half / kUnit;
        const bool first = ul < step;
        const bool turns = ul < 2 * step;
        const int other = turns ? (first ? ul + step : ul - step) : ul;
        const int from = tid % kWave - ul + other;
        v4i far;
#pragma unroll
        for (int i = 0; i < 4; ++i) far[i] = __shfl(raw[i], from, kWave);
        if (!is_v && have && turns) {
          double z[kUnit];
          widen_unit<QT>(far, z);
#pragma unroll
          for (int e = 0; e < kUnit; ++e) {
            const int j = (first ? ul : other) * kUnit + e;
            if (g) z[e] *= inv * weight(other * kUnit + e);
            x[e] = first ? x[e] * cs[j] - z[e] * sn[j]
                         : x[e] * cs[j] + z[e] * sn[j];
          }
        }
      }
    }
    // ---- out
    if (is_q && have)
      *(v4i*)(p.q_out + token * p.ot + h * p.oh + ul * 16) =
          v4i{round_pair<QT>(x[0], x[1]), round_pair<QT>(x[2], x[3]),
              round_pair<QT>(x[4], x[5]), round_pair<QT>(x[6], x[7])};
    const float* scale = is_v ? p.v_scale : p.k_scale;
    if (scale && !is_q && have) {
      const double s = (double)scale[h];
#pragma unroll
      for (int e = 0; e < kUnit; ++e) x[e] /= s;
    }
    int byte = 0;
    if constexpr (CT == kE2m1) {
      double top = 0.0;
      bool odd = false;  // a NaN: max would drop it
#pragma unroll
      for (int e = 0; e < kUnit; ++e) {
        odd = odd || x[e] != x[e];
        top = fmax(top, fabs(x[e]));
      }
      if (odd) top = INFINITY;
      top = fmax(top, __shfl_xor(top, 1, kWave));
      top = fmax(top, __shfl_xor(top, 2, kWave));
      byte = block_byte(top);
    }
    if (is_q || !have) continue;
    if (p.w.w && !is_v && ul == 0 && slot < top_len) {
      p.w.w[b * p.w.wb + h * p.w.wh + slot] = 0.0f;
      p.w.pos[b * p.w.pb + h * p.w.ph + slot] = (int32_t)position;
    }
    if (page < 0) continue;
    char* dst = const_cast<char*>(
        is_v ? c.v + row_offset(c.vs, page, h, place)
             : c.k + row_offset(c.ks, page, h, place));
    if constexpr (CT == kE2m1) {
      unsigned code = 0;
      if (byte < 255) {
#pragma unroll
        for (int e = 0; e < kUnit; ++e) code |= code_of(x[e], byte) << (4 * e);
      }
      *(unsigned*)(dst + ul * 4) = code;
      if (ul % 4 == 0) {
        char* blocks = const_cast<char*>(
            is_v ? c.vb + row_offset(c.vbs, page, h, place)
                 : c.kb + row_offset(c.kbs, page, h, place));
        blocks[ul / 4] = (char)byte;
      }
    } else if constexpr (CT == kE4m3) {
      v2i_t d;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(within_e4m3(x[4 * i]),
                                                within_e4m3(x[4 * i + 1]), 0,
                                                false);
        d[i] = __builtin_amdgcn_cvt_pk_fp8_f32(within_e4m3(x[4 * i + 2]),
                                               within_e4m3(x[4 * i + 3]), w,
                                               true);
      }
      *(v2i_t*)(dst + ul * 8) = d;
    } else {
      *(v4i*)(dst + ul * 16) =
          v4i{round_pair<CT>(x[0], x[1]), round_pair<CT>(x[2], x[3]),
              round_pair<CT>(x[4], x[5]), round_pair<CT>(x[6], x[7])};
    }
  }
}

}  // namespace ltk
