// Host side of sampling (sample_logits of include/libtopk.h).
#include <hip/hip_runtime.h>

#include "libtopk.h"
#include "sample_kernel.hpp"
#include "workspace.hpp"

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

constexpr int64_t kSampleWork = (int64_t)1 << 26;

struct Kernels {
  const void *row, *chunk, *finish, *bins, *wide, *last;
};
template <int T>
Kernels kernels_of() {
  return {(const void*)&sample_row_kernel<T>,
          (const void*)&sample_chunk_kernel<T>,
          (const void*)&sample_finish_kernel<T>,
          (const void*)&sample_bins_kernel<T>,
          (const void*)&sample_wide_kernel<T>,
          (const void*)&sample_last_kernel<T>};
}
Kernels kernels(int32_t dtype) {
  return dtype == LIBTOPK_F32    ? kernels_of<kLogF32>()
         : dtype == LIBTOPK_BF16 ? kernels_of<kLogBf16>()
                                 : kernels_of<kLogF16>();
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
  const int frac = 62 - ceil_log2((int32_t)cols);
  p.unit = (double)((uint64_t)1 << (frac < 51 ? frac : 51));
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
  int rc = current_device(&dev);
  if (rc != LIBTOPK_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  const Kernels fn = kernels(dtype);
  const int64_t chunks = (cols + kChunk - 1) / kChunk;
  if (chunks > kMaxChunks)
    return launch(fn.row, dim3((unsigned)rows), kSampleThreads, p, st);
  p.chunks = (int32_t)chunks;
  // Some 3000 words a row at most.
  const int64_t rank = kMaxList * 5 / 8 / chunks;
  p.rank = (int32_t)(rank < 2 ? 2 : rank > 32 ? 32 : rank);
  // Batches of rows share the workspace, which stays below 64 MB.
  const int64_t per = chunks * (8 + 3 * 4 + 8 + 8 * kChunkList) +
                      8 * (kWideBins + kMaxList) + (int64_t)sizeof(WideRow) + 4;
  int64_t batch = kSampleWork / per;
  if (batch > rows) batch = rows;
  Work work;
  rc = get_work(dev, st, (size_t)(batch * per + 4), 1, &work);
  if (rc != LIBTOPK_OK) return rc;
  const int64_t n = batch * chunks;
  p.lists = (uint64_t*)work.base;
  p.chunk_sum = (double*)(p.lists + n * kChunkList);
  p.chunk_mass = (uint64_t*)(p.chunk_sum + n);
  p.bins = p.chunk_mass + n;
  p.pivots = p.bins + batch * kWideBins;
  p.wide = (WideRow*)(p.pivots + batch * kMaxList);
  p.chunk_max = (uint32_t*)(p.wide + batch);
  p.chunk_from = p.chunk_max + n;
  p.chunk_n = p.chunk_from + n;
  p.wide_list = p.chunk_n + n;
  // Without settings there are no prefixes, and none that goes beyond lists.
  const bool wide =
      (how->top_p || how->top_p_all < 1.0f || how->top_k ||
       how->top_k_all > 0 || how->min_p || how->min_p_all > 0.0f);
  const int64_t parts = (chunks + kWideChunks - 1) / kWideChunks;
  int units = 0;
  rc = units_of(dev, &units);
  if (rc != LIBTOPK_OK) return rc;
  for (int64_t r = 0; r < rows && rc == LIBTOPK_OK; r += batch) {
    const int64_t m = rows - r < batch ? rows - r : batch;
    p.row0 = r;
    rc = launch(fn.chunk, dim3((unsigned)(m * ((chunks + kWaves - 1) / kWaves))),
                kBlock, p, st);
    if (rc == LIBTOPK_OK)
      rc = launch(fn.finish, dim3((unsigned)m), kSampleThreads, p, st);
    // The parts of whatever rows are wide, two workgroups a unit.
    const int64_t most = 2 * (int64_t)units;
    const unsigned grid = (unsigned)(m * parts < most ? m * parts : most);
    if (rc == LIBTOPK_OK && wide)
      rc = launch(fn.bins, dim3(grid), kWideThreads, p, st);
    if (rc == LIBTOPK_OK && wide)
      rc = launch(fn.wide, dim3(grid), kWideThreads, p, st);
    if (rc == LIBTOPK_OK && wide)
      rc = launch(fn.last, dim3((unsigned)(m < units ? m : units)),
                  kSampleThreads, p, st);
  }
  return rc;
}
