// Host side of sampling (sample_logits of include/libtopk.h).
#include <hip/hip_runtime.h>

#include "libtopk.h"
#include "sample_kernel.hpp"

namespace {

using namespace ltk;

static_assert(kLogBf16 == LIBTOPK_BF16 && kLogF16 == LIBTOPK_F16 &&
                  kLogF32 == LIBTOPK_F32 &&
                  kMaxCols == LIBTOPK_MAX_LOGITS,
              "the kernels' constants are the header's");

bool misaligned(const void* p, uintptr_t a) { return (uintptr_t)p & (a - 1); }

bool meets(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

int ceil_log2(int32_t n) {
  int s = 0;
  while (((int64_t)1 << s) < n) ++s;
  return s;
}

}  // namespace

extern "C" int sample_logits(const void* logits, int32_t dtype, int64_t rows,
                             int64_t cols, int64_t ld,
                             const libtopk_sampling_t* how, const float* u,
                             int64_t* tokens, float* logprobs,
                             libtopk_stream_t stream) {
  if (!how || (dtype != LIBTOPK_BF16 && dtype != LIBTOPK_F16 &&
               dtype != LIBTOPK_F32))
    return LIBTOPK_ERR_INVALID;
  const int64_t size = dtype == LIBTOPK_F32 ? 4 : 2;
  if (rows < 0 || rows >= LIBTOPK_MAX_SAMPLE_ROWS || cols < 1 ||
      cols > LIBTOPK_MAX_LOGITS || ld < cols || ld > ((int64_t)1 << 36))
    return LIBTOPK_ERR_INVALID;
  const void* settings[4] = {how->temperature, how->top_k, how->top_p,
                             how->min_p};
  for (const void* p : settings)
    if (misaligned(p, 4)) return LIBTOPK_ERR_INVALID;
  if (rows == 0) return LIBTOPK_OK;
  if (!logits || !u || !tokens || !logprobs || misaligned(logits, size) ||
      misaligned(u, 4) || misaligned(tokens, 8) || misaligned(logprobs, 4))
    return LIBTOPK_ERR_INVALID;
  const int64_t span = ((rows - 1) * ld + cols) * size;
  const void* outs[2] = {tokens, logprobs};
  const int64_t out_bytes[2] = {rows * 8, rows * 4};
  for (int i = 0; i < 2; ++i) {
    if (meets(outs[i], out_bytes[i], logits, span) ||
        meets(outs[i], out_bytes[i], u, rows * 4))
      return LIBTOPK_ERR_INVALID;
    for (const void* p : settings)
      if (p && meets(outs[i], out_bytes[i], p, rows * 4))
        return LIBTOPK_ERR_INVALID;
  }
  if (meets(tokens, rows * 8, logprobs, rows * 4)) return LIBTOPK_ERR_INVALID;
  SampleParams p = {};
  p.x = (const char*)logits;
  p.ld = ld * size;
  p.cols = (int32_t)cols;
  p.frac = 62 - ceil_log2((int32_t)cols);
  p.temperature = how->temperature;
  p.top_k = how->top_k;
  p.top_p = how->top_p;
  p.min_p = how->min_p;
  p.temperature_all = how->temperature_all;
  p.top_k_all = how->top_k_all;
  p.top_p_all = how->top_p_all;
  p.min_p_all = how->min_p_all;
  p.u = u;
  p.tokens = tokens;
  p.logprobs = logprobs;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return LIBTOPK_ERR_HIP;
  }
  const void* fn = dtype == LIBTOPK_F32 ? (const void*)&sample_row_kernel<kLogF32>
                   : dtype == LIBTOPK_BF16
                       ? (const void*)&sample_row_kernel<kLogBf16>
                       : (const void*)&sample_row_kernel<kLogF16>;
  void* args[] = {&p};
  if (hipLaunchKernel(fn, dim3((unsigned)rows), dim3(kSampleThreads), args, 0,
                      (hipStream_t)stream) != hipSuccess) {
    (void)hipGetLastError();
    return LIBTOPK_ERR_HIP;
  }
  return LIBTOPK_OK;
}
