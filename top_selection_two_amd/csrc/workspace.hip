// Workspaces of calls (workspace.hpp).
#include "workspace.hpp"

#include <cstdio>
#include <cstdlib>
#include <map>
#include <new>
#include <utility>
#include <vector>

namespace ltk {

// ---- workspace --------------------------------------------------------------
// Areas that a (device, stream) has used are kept until cache_release(): a
// captured graph may hold their addresses.  Growth at least doubles, so all
// of them together stay below twice the largest.
namespace {
struct Buffer {
  char* base = nullptr;
  size_t bytes = 0;
  std::vector<void*> old;
};

// A call holds its area from here to its last launch: the launches of a call
// hand results to one another in the area, and another thread's on the same
// stream must not come between them.
struct Area {
  std::mutex mu;
  Buffer work;     // partial results, scores, lists: any contents
  Buffer tickets;  // completion tickets and nothing else (see Tagged)
  uint32_t epoch = 0;
};

std::mutex g_mu;
std::map<std::pair<int, void*>, Area> g_areas;
std::map<int, int> g_cus;             // device -> compute units
std::map<const void*, int> g_fit;     // kernel -> workgroups of a unit
}  // namespace

void debug_hip(const char* what, hipError_t e) {
  static const bool on = getenv("LIBTOPK_DEBUG") != nullptr;
  if (on) fprintf(stderr, "libtopk: %s: %s\n", what, hipGetErrorString(e));
}

int current_device(int* dev) {
  if (hipGetDevice(dev) != hipSuccess) {
    (void)hipGetLastError();
    return LIBTOPK_ERR_HIP;
  }
  return LIBTOPK_OK;
}

static __global__ void fill_words(uint64_t* p, int64_t n, uint64_t seed) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  // seed 0: clear; otherwise a SplitMix64-style mix of seed and index
  uint64_t z = seed + 0x9e3779b97f4a7c15ull * (uint64_t)(i + 1);
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  p[i] = seed ? (z ^ (z >> 31)) | 1ull : 0ull;
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return LIBTOPK_OK;
  debug_hip(what, e);
  return LIBTOPK_ERR_HIP;
}

int fill(uint64_t* p, size_t words, uint64_t seed, hipStream_t s) {
  hipLaunchKernelGGL(fill_words, dim3((unsigned)((words + 255) / 256)),
                     dim3(256), 0, s, p, (int64_t)words, seed);
  return launched("fill_words");
}

// Caller holds the area.
static int grow(Buffer* b, size_t bytes, hipStream_t stream, bool clear) {
  if (b->bytes >= bytes) return LIBTOPK_OK;
  if (getenv("LIBTOPK_TEST_FAIL_ALLOC")) return LIBTOPK_ERR_NOMEM;
  hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(stream, &st) != hipSuccess) {
    (void)hipGetLastError();
    return LIBTOPK_ERR_HIP;
  }
  if (st != hipStreamCaptureStatusNone) return LIBTOPK_ERR_NOMEM;
  size_t want = 2 * b->bytes > bytes ? 2 * b->bytes : bytes;
  if (want < ((size_t)1 << 16)) want = (size_t)1 << 16;
  b->old.reserve(b->old.size() + 1);
  void* p = nullptr;
  hipError_t e = hipMalloc(&p, want);
  if (e != hipSuccess && want > bytes) {
    (void)hipGetLastError();
    want = bytes;
    e = hipMalloc(&p, want);
  }
  if (e != hipSuccess) {
    debug_hip("hipMalloc(cache workspace)", e);
    (void)hipGetLastError();
    return LIBTOPK_ERR_NOMEM;
  }
  if (clear) {
    const int rc = fill((uint64_t*)p, want / 8, 0, stream);
    if (rc != LIBTOPK_OK) {
      (void)hipFree(p);
      return rc;
    }
  }
  if (b->base) b->old.push_back(b->base);
  b->base = (char*)p;
  b->bytes = want;
  return LIBTOPK_OK;
}

int get_work(int dev, hipStream_t stream, size_t bytes, size_t tickets,
             Work* out) {
  try {
    Area* a;
    {
      std::lock_guard<std::mutex> lock(g_mu);
      a = &g_areas[std::make_pair(dev, (void*)stream)];  // stays where it is
    }
    out->hold = std::unique_lock<std::mutex>(a->mu);
    int rc = grow(&a->work, bytes, stream, false);
    if (rc == LIBTOPK_OK) rc = grow(&a->tickets, tickets * 8, stream, true);
    if (rc != LIBTOPK_OK) return rc;
    if (++a->epoch == 0) ++a->epoch;
    out->base = a->work.base;
    out->tickets = (uint64_t*)a->tickets.base;
    out->ticket_words = a->tickets.bytes / 8;
    out->epoch = a->epoch;
    return LIBTOPK_OK;
  } catch (const std::bad_alloc&) {
    return LIBTOPK_ERR_NOMEM;
  } catch (...) {
    return LIBTOPK_ERR_HIP;
  }
}

// Compute units of a device.
int units_of(int dev, int* out) {
  try {
    std::lock_guard<std::mutex> lock(g_mu);
    int& cus = g_cus[dev];
    if (cus < 1 &&
        (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount,
                               dev) != hipSuccess ||
         cus < 1)) {
      (void)hipGetLastError();
      cus = 256;
    }
    *out = cus;
    return LIBTOPK_OK;
  } catch (...) {
    return LIBTOPK_ERR_NOMEM;
  }
}

// Workgroups of `fn` that a compute unit holds at once.
int resident(const void* fn, int threads, int* out) {
  try {
    std::lock_guard<std::mutex> lock(g_mu);
    int& fit = g_fit[fn];
    if (fit < 1 &&
        (hipOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, threads, 0) !=
             hipSuccess ||
         fit < 1)) {
      (void)hipGetLastError();
      fit = 1;
    }
    *out = fit;
    return LIBTOPK_OK;
  } catch (...) {
    return LIBTOPK_ERR_NOMEM;
  }
}

}  // namespace ltk

extern "C" {

using namespace ltk;

void cache_release(void) {
  std::lock_guard<std::mutex> lock(g_mu);
  int prev = -1;
  (void)hipGetDevice(&prev);
  for (auto& kv : g_areas) {
    if (hipSetDevice(kv.first.first) != hipSuccess) continue;
    (void)hipDeviceSynchronize();
    for (Buffer* b : {&kv.second.work, &kv.second.tickets}) {
      for (void* o : b->old) (void)hipFree(o);
      if (b->base) (void)hipFree(b->base);
    }
  }
  g_areas.clear();
  if (prev >= 0) (void)hipSetDevice(prev);
  (void)hipGetLastError();
}

int cache_debug_scramble(libtopk_stream_t stream, uint64_t seed) {
  int dev = 0;
  int rc = current_device(&dev);
  if (rc != LIBTOPK_OK) return rc;
  Work work;
  rc = get_work(dev, (hipStream_t)stream, 1, 1, &work);
  if (rc != LIBTOPK_OK) return rc;
  return fill(work.tickets, work.ticket_words, seed | 1u, (hipStream_t)stream);
}

}  // extern "C"
