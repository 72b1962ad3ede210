// Attention of one new token over a paged cache.
//
// For query head j of head h and slot t: x = scale k_scale (q . K_t).  One
// pass over the slots keeps the running maximum m, l = sum exp(x - m) and
// o = sum exp(x - m) V_t, rescaling l and o by exp(m_old - m_new) whenever m
// grows; out = v_scale o / l, lse = m + ln l.  Exponentials are taken to base
// 2 (scale is multiplied by log2 e on the host).
#pragma once

#include "cache_common.hpp"

namespace ltk {

struct AttendParams {
  CacheParams c;
  LedgerParams w;
  const char* q;
  int64_t qb, qh;       // bytes
  int32_t group;        // query heads of a cache head
  float scale2;         // scale * log2 e
  const float* k_scale; // NULL: 1
  const float* v_scale;
  float* scores;        // [batch][q heads][cap], with a ledger
  void* out;
  float* lse;
};

constexpr float kLn2 = 0.693147180559945309f;

// Element i of a row as float32.
template <int T>
__device__ __forceinline__ float element(const char* row, int i) {
  if constexpr (T == kBf16) {
    return __uint_as_float((uint32_t)((const uint16_t*)row)[i] << 16);
  } else if constexpr (T == kF16) {
    return (float)((const _Float16*)row)[i];
  } else {
    return __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t*)row)[i], 0);
  }
}

template <int QT>
__device__ __forceinline__ void store_element(void* p, int64_t i, float x) {
  if constexpr (QT == kBf16)
    ((__bf16*)p)[i] = (__bf16)x;
  else
    ((_Float16*)p)[i] = (_Float16)x;
}

template <int QT, int CT>
__global__ __launch_bounds__(kBlock) void attend_kernel(AttendParams p) {
  constexpr int R = 4;  // elements of a row per lane, up to 256
  const CacheParams& c = p.c;
  __shared__ float part[kWaves][2 + R * kWave];
  const int qheads = c.heads * p.group;
  const int b = blockIdx.x / qheads, j = blockIdx.x % qheads;
  const int h = j / p.group;
  const int wave = threadIdx.x / kWave, ln = threadIdx.x % kWave;
  const int32_t len = clamp_len(c.lens[b], c.cap);
  const int32_t* table = c.table + b * c.table_stride;
  const float scale = p.scale2 * (p.k_scale ? p.k_scale[h] : 1.0f);
  const char* qrow = p.q + b * p.qb + j * p.qh;
  float* scores = p.scores ? p.scores + (int64_t)blockIdx.x * c.cap : nullptr;
  float q[R], o[R] = {};
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int d = ln + i * kWave;
    q[i] = d < c.dim ? element<QT>(qrow, d) : 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int32_t t = wave; t < len; t += kWaves) {
    int32_t place;
    const int32_t id = find_page(c, table, t, &place);
    float x = -INFINITY;
    if (id >= 0) {
      const char* row = c.k + row_offset(c.ks, id, h, place);
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int d = ln + i * kWave;
        if (d < c.dim) s += q[i] * element<CT>(row, d);
      }
      x = scale * wave_fold(s, [](float a, float e) { return a + e; });
    }
    if (scores && ln == 0) scores[t] = x;
    if (id < 0) continue;
    const float mn = fmaxf(m, x);
    const float f = m == mn ? 1.0f : exp2f(m - mn);
    const float e = x == -INFINITY ? 0.0f : exp2f(x - mn);
    const char* row = c.v + row_offset(c.vs, id, h, place);
    m = mn;
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int d = ln + i * kWave;
      if (d < c.dim) o[i] = o[i] * f + e * element<CT>(row, d);
    }
  }
  if (ln == 0) {
    part[wave][0] = m;
    part[wave][1] = l;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) part[wave][2 + ln + i * kWave] = o[i];
  __syncthreads();
  const int d = threadIdx.x;
  float top = -INFINITY, sum = 0.0f, acc = 0.0f;
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, part[w][0]);
  for (int w = 0; w < kWaves; ++w) {
    const float f = part[w][0] == top ? 1.0f : exp2f(part[w][0] - top);
    sum += part[w][1] * f;
    acc += part[w][2 + d] * f;
  }
  const bool none = sum == 0.0f;  // no slot, or none with a finite score
  if (d < c.dim) {
    const float vs = p.v_scale ? p.v_scale[h] : 1.0f;
    store_element<QT>(p.out, (int64_t)blockIdx.x * c.dim + d,
                      none ? 0.0f : acc * vs / sum);
  }
  if (d == 0)
    p.lse[blockIdx.x] = none ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// weights[t] += sum over the head's queries of exp(x - lse).
__global__ __launch_bounds__(kBlock) void attend_weights_kernel(
    AttendParams p) {
  const CacheParams& c = p.c;
  const int row = blockIdx.y;  // sequence and head
  const int b = row / c.heads, h = row % c.heads;
  const int32_t len = clamp_len(c.lens[b], c.cap);
  const int32_t t = blockIdx.x * kBlock + threadIdx.x;
  if (t >= len) return;
  const int64_t first = (int64_t)row * p.group;
  float a = 0.0f;
  for (int g = 0; g < p.group; ++g) {
    const float lse2 = p.lse[first + g] * (1.0f / kLn2);
    const float x = p.scores[(first + g) * c.cap + t];
    a += x == -INFINITY ? 0.0f : exp2f(x - lse2);
  }
  p.w.w[b * p.w.wb + h * p.w.wh + t] += a;
}

}  // namespace ltk
