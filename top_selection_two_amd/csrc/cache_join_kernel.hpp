// The second launch of an attention call: rows of many scores.
#pragma once

#include "cache_attend_kernel.hpp"

namespace ltk {

// What attend_kernel left: for the rows that several workgroups share, lse and
// out from the shares' results, and weights[t] += sum over the head's queries
// of exp(x - lse).  A workgroup for every kWeightSlots slots of a sequence and
// head, four slots a thread; the columns of out are dealt to the row's first
// kJoiners workgroups, so that a row of many shares is joined by many.
constexpr int kWeightSlots = 4 * kBlock;
constexpr int kJoiners = 16;

__global__ __launch_bounds__(kBlock) void attend_join_kernel(AttendParams p) {
  const CacheParams& c = p.c;
  __shared__ float lds_top[16], lds_sum[16], lds_lse2[16];
  __shared__ f32x4 lds_x[kBlock];
  const int tid = threadIdx.x;
  const int32_t i = blockIdx.x * kBlock + tid, t = i / 8;
  const int head_floats = p.part_rows * kTileSlots;
  const int part_rows = p.hs * p.part_rows;
  const int64_t part_size = share_floats(part_rows, p.cols);
  const int vecs_of_row = p.cols / 4;
  for (int row = blockIdx.y; row < c.batch * c.heads; row += gridDim.y) {
    const int b = row / c.heads, h = row % c.heads, hsub = h % p.hs;
    const int32_t len =
        clamp_len(ld_const(c.lens + b), c.pages > 0 ? c.cap : 0);
    const int workers = min((int)gridDim.x, kJoiners), wg = (int)blockIdx.x;
    if (wg >= workers && wg * kWeightSlots >= len) continue;
    // The rows of its head's queries.
    const int64_t row0 = ((int64_t)b * (c.heads / p.hs) + h / p.hs) * p.gtiles;
    f32x4 a = {0, 0, 0, 0};
    bool any = false;
    for (int gt = 0; gt < p.gtiles; ++gt) {
      const int* at = (const int*)(p.shares + row0 + gt);
      const int2 sh = make_int2(ld_const(at), ld_const(at + 1));
      if (sh.x == kRowDone) continue;
      any = true;
      const int queries = p.group - gt * 16 < 16 ? p.group - gt * 16 : 16;
      const int64_t qrow = (int64_t)row * p.group + gt * 16;
      auto part_of = [&](int w) {
        return p.part + ((int64_t)w * 2 + (w == sh.x)) * part_size;
      };
      const int64_t at_m = (int64_t)part_rows * p.cols + hsub * p.part_rows;
      __syncthreads();  // the last round's LDS is free
      if (sh.x == kRowJoined) {
        if (tid < queries) lds_lse2[tid] = p.lse[qrow + tid] * (1.0f / kLn2);
      } else {
        const int g = tid / 16;  // 16 threads a query
        float top = -INFINITY, sum = 0.0f;
        if (g < queries) {
          for (int w = sh.x + tid % 16; w <= sh.y; w += 16) {
            const float* m = part_of(w) + at_m + g;
            const float next = fmaxf(top, m[0]);
            sum = sum * (top == next ? 1.0f : exp2_fast(top - next)) +
                  m[part_rows] *
                      (m[0] == next ? 1.0f : exp2_fast(m[0] - next));
            top = next;
          }
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          const float t2 = __shfl_xor(top, o, kWave);
          const float s2 = __shfl_xor(sum, o, kWave);
          const float next = fmaxf(top, t2);
          sum = sum * (top == next ? 1.0f : exp2_fast(top - next)) +
                s2 * (t2 == next ? 1.0f : exp2_fast(t2 - next));
          top = next;
        }
        if (g < queries && tid % 16 == 0) {
          const float z = sum == 0.0f ? -INFINITY : top + log2f(sum);
          lds_top[g] = top;
          lds_sum[g] = sum;
          lds_lse2[g] = z;
          if (blockIdx.x == 0) p.lse[qrow + g] = z * kLn2;
        }
      }
      __syncthreads();
      if (i * 4 < len) {
        const float* x0 = p.scores + (((row0 + gt) * p.row_tiles + t) * p.hs +
                                      hsub) * head_floats;
        for (int g0 = 0; g0 < queries; g0 += 4) {
          f32x4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = *(const f32x4*)(
                x0 + score_at(g0 + k < queries ? g0 + k : g0, i % 8));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (g0 + k >= queries) continue;
            const float z = lds_lse2[g0 + k];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              a[e] += x[k][e] == -INFINITY ? 0.0f : exp2_fast(x[k][e] - z);
          }
        }
      }
      if (sh.x == kRowJoined) continue;
      // This workgroup's columns [v0, v1), four each; the shares are split
      // over `subs` threads.
      const int vecs = queries * vecs_of_row;
      const int each = (vecs + workers - 1) / workers;
      const int v0 = wg < workers ? wg * each : vecs;
      const int v1 = v0 + each < vecs ? v0 + each : vecs;
      for (int va = v0; va < v1; va += kBlock) {
        const int nv = v1 - va < kBlock ? v1 - va : kBlock;
        const int subs = min(kBlock / nv, sh.y - sh.x + 1);
        const int sub = tid / nv, v = va + tid % nv;
        const int g = v / vecs_of_row, col = v % vecs_of_row * 4;
        f32x4 x = {0, 0, 0, 0};
        if (sub < subs) {
          const float top = lds_top[g];
#pragma unroll 4
          for (int w = sh.x + sub; w <= sh.y; w += subs) {
            const float* pw = part_of(w);
            const float m = pw[at_m + g];
            x += *(const f32x4*)(pw + (int64_t)(hsub * p.part_rows + g) *
                                          p.cols + col) *
                 (m == top ? 1.0f : exp2_fast(m - top));
          }
        }
        __syncthreads();
        lds_x[tid] = x;
        __syncthreads();
        if (sub != 0) continue;
        for (int k = 1; k < subs; ++k) x += lds_x[k * nv + tid];
        if (col >= c.dim) continue;
        const float sum = lds_sum[g];
        const float f = (p.v_scale ? p.v_scale[h] : 1.0f) / sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = sum == 0.0f ? 0.0f : x[e] * f;
        int2* out = (int2*)((char*)p.out + ((qrow + g) * c.dim + col) * 2);
        *out = p.q_type == kBf16 ? make_int2(pack2<kBf16>(x[0], x[1]),
                                             pack2<kBf16>(x[2], x[3]))
                                 : make_int2(pack2<kF16>(x[0], x[1]),
                                             pack2<kF16>(x[2], x[3]));
      }
    }
    if (any && i * 4 < len)
      add_weights(p.w.w + b * p.w.wb + h * p.w.wh + i * 4, len - i * 4, a);
  }
}

}  // namespace ltk
