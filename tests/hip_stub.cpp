// A host without a GPU, for tests of what the C entry points of a call do on
// the host: the HIP calls that libtopk.so makes, answered here (a symbol of
// the program comes before the library's), with a log of the launches.
//
// usage: hip_stub <test>; prints what the test looks at.
#include <hip/hip_runtime_api.h>

#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <unistd.h>

#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "libtopk.h"

struct Launch {
  int thread, call;
  dim3 grid, block;
  size_t lds;
};
static std::mutex log_mu;
static std::vector<Launch> launches;
static thread_local int this_thread = 0, this_call = 0;
static int pause_us = 0, fit = 1;
static uintptr_t next_address = (uintptr_t)1 << 40;

extern "C" {
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipGetDeviceCount(int* n) { return *n = 1, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "stub"; }
hipError_t hipFree(void*) { return hipSuccess; }
hipError_t hipMalloc(void** p, size_t n) {
  std::lock_guard<std::mutex> lock(log_mu);
  *p = (void*)next_address;
  next_address += (n + 4095) / 4096 * 4096;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  return *v = 256, hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  return *s = hipStreamCaptureStatusNone, hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*,
                                                        int, size_t) {
  return *n = fit, hipSuccess;
}
// What kernel<<<grid, block, lds, stream>>>(...) becomes.
struct Config {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
};
static thread_local Config config;
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds,
                                      hipStream_t s) {
  config = {grid, block, lds, s};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds,
                                     hipStream_t* s) {
  *grid = config.grid;
  *block = config.block;
  *lds = config.lds;
  *s = config.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**,
                           size_t lds, hipStream_t) {
  {
    std::lock_guard<std::mutex> lock(log_mu);
    launches.push_back({this_thread, this_call, grid, block, lds});
  }
  if (pause_us) usleep(pause_us);
  return hipSuccess;
}
}

// Addresses that are never dereferenced.
static char* const kFake = (char*)0x10000000;
template <class T>
static T* fake(int i) {
  return (T*)(kFake + (size_t)i * 0x40000000);
}

static libtopk_cache_t cache_of(int batch, int heads, int width, int dim) {
  libtopk_cache_t c = {};
  c.k = fake<char>(0);
  c.v = fake<char>(64);
  c.k_slot_stride = c.v_slot_stride = dim;
  c.k_head_stride = c.v_head_stride = 16 * dim;
  c.k_page_stride = c.v_page_stride = (int64_t)heads * 16 * dim;
  c.pages = (int64_t)batch * width;
  c.table_stride = width;
  c.table = fake<int32_t>(128);
  c.lens = fake<int32_t>(129);
  c.batch = batch;
  c.table_width = width;
  c.heads = heads;
  c.page = 16;
  c.dim = dim;
  c.dtype = LIBTOPK_BF16;
  return c;
}

static libtopk_ledger_t ledger_of(int i, int heads, int slots) {
  libtopk_ledger_t l = {};
  l.weights = fake<float>(i);
  l.positions = fake<int32_t>(i + 16);
  l.weights_head_stride = l.positions_head_stride = slots;
  l.weights_batch_stride = l.positions_batch_stride = (int64_t)heads * slots;
  l.slots = slots;
  return l;
}

static int attend(const libtopk_cache_t& c, int group,
                  const libtopk_ledger_t* l, libtopk_stream_t s) {
  return cache_attend(&c, fake<char>(130), LIBTOPK_BF16, c.heads * group,
                      (int64_t)c.heads * group * c.dim, c.dim, 1.0f, nullptr,
                      nullptr, l, fake<char>(132), fake<float>(134), s);
}

static int evict(const libtopk_cache_t& c, const libtopk_ledger_t& l,
                 int keep, libtopk_stream_t s) {
  const libtopk_ledger_t after = ledger_of(200, c.heads, keep);
  return cache_evict(&c, fake<int32_t>(136), &l, keep, 0, 0, &after,
                     fake<int32_t>(137), s);
}

static int append(const libtopk_cache_t& c, const libtopk_ledger_t& l,
                  libtopk_stream_t s) {
  return cache_append(&c, fake<char>(140), fake<char>(142),
                      (int64_t)c.heads * c.dim, c.dim, 64, fake<int32_t>(136),
                      &l, 0, 0, fake<int32_t>(137), fake<int32_t>(138), s);
}

// Threads that each make calls on one stream, `call(thread)`: are a call's
// launches next to one another?
template <class F>
static int threads_test(int threads, F call) {
  pause_us = 300;
  std::vector<std::thread> t;
  int failed = 0;
  for (int i = 0; i < threads; ++i)
    t.emplace_back([&, i] {
      this_thread = i;
      for (this_call = 0; this_call < 12; ++this_call) {
        if (call(i) == LIBTOPK_OK) continue;
        std::lock_guard<std::mutex> lock(log_mu);
        ++failed;
      }
    });
  for (std::thread& x : t) x.join();
  int torn = 0, most = 0, run = 0;
  std::vector<std::string> seen;
  for (size_t i = 0; i < launches.size(); ++i) {
    const Launch &a = launches[i];
    const bool same = i > 0 && launches[i - 1].thread == a.thread &&
                      launches[i - 1].call == a.call;
    run = same ? run + 1 : 1;
    most = run > most ? run : most;
    if (same) continue;
    const std::string id =
        std::to_string(a.thread) + "." + std::to_string(a.call);
    for (const std::string& x : seen) torn += x == id;
    seen.push_back(id);
  }
  printf("failed %d torn %d calls %zu most %d\n", failed, torn, seen.size(),
         most);
  return 0;
}

static int cache_threads_test() {
  const libtopk_cache_t c = cache_of(2, 4, 256, 64);  // 4096 slots a head
  const libtopk_cache_t wide = cache_of(1, 2, 2048, 64);  // 32768
  const libtopk_ledger_t l = ledger_of(160, 4, 4096);
  const libtopk_ledger_t wl = ledger_of(160, 2, 32768);
  return threads_test(3, [&](int i) {
    return i == 0   ? evict(c, l, 512, nullptr)
           : i == 1 ? evict(wide, wl, 512, nullptr)
                    : attend(c, 16, &l, nullptr);
  });
}

static int selection_threads_test() {
  const int32_t* in = fake<int32_t>(0);
  return threads_test(4, [&](int i) {
    if (i == 0)
      return topk_i32(in, 1 << 20, 1000, fake<int32_t>(64), nullptr);
    if (i == 1)  // a longer input each time: the segments' scratch grows
      return topk_segmented_i32(in, (int64_t)(this_call + 1) << 21,
                                fake<int64_t>(65), 100, 20, fake<int32_t>(66),
                                nullptr, nullptr);
    if (i == 2)
      return topk_segmented_i32(in, 1 << 20, fake<int64_t>(65), 100, 20,
                                fake<int32_t>(67), nullptr, nullptr);
    return histogram_i32(in, 1 << 20, 0, 0, 256, fake<int64_t>(68), nullptr);
  });
}

// Batches of many rows: status and launches of each call, and the most
// threads along an axis of a launch.
static int many_rows_test(int batch, int heads, int width) {
  const libtopk_cache_t c = cache_of(batch, heads, width, 16);
  libtopk_ledger_t l = ledger_of(160, heads, width * 16);
  // (arrays of so many rows span more than the fake addresses are apart)
  l.weights = (float*)((uintptr_t)1 << 50);
  l.positions = (int32_t*)((uintptr_t)1 << 51);
  libtopk_cache_t big = c;
  big.k = (void*)((uintptr_t)1 << 52);
  big.v = (void*)((uintptr_t)1 << 53);
  big.table = (int32_t*)((uintptr_t)1 << 54);
  for (int i = 0; i < 2; ++i) {
    launches.clear();
    int rc;
    if (i == 0) {
      rc = cache_append(&big, (char*)((uintptr_t)1 << 55),
                        (char*)((uintptr_t)1 << 56), (int64_t)heads * 16, 16,
                        4, fake<int32_t>(136), &l, 0, 0, fake<int32_t>(138),
                        (int32_t*)((uintptr_t)1 << 57), nullptr);
    } else {
      libtopk_ledger_t after = ledger_of(160, heads, 4);
      after.weights = (float*)((uintptr_t)1 << 55);
      after.positions = (int32_t*)((uintptr_t)1 << 56);
      rc = cache_evict(&big, fake<int32_t>(136), &l, 4, 0, 0, &after,
                       fake<int32_t>(138), nullptr);
    }
    uint64_t threads = 0;
    for (const Launch& x : launches) {
      const uint64_t t = (uint64_t)x.grid.x * x.block.x;
      threads = t > threads ? t : threads;
    }
    const char* name = i ? "evict" : "append";
    printf("%s %d %s_launches %zu %s_wide %d\n", name, rc, name,
           launches.size(), name, threads >> 32 != 0);
  }
  return 0;
}

// LDS that attention with weights asks for, when the device says that `per_cu`
// workgroups fit a compute unit.
static int lds_test(int dim, bool slots_first, int per_cu) {
  fit = per_cu;
  libtopk_cache_t c = cache_of(8, 4, 1024, dim);
  if (slots_first) {
    c.k_head_stride = c.v_head_stride = dim;
    c.k_slot_stride = c.v_slot_stride = 4 * dim;
  }
  const libtopk_ledger_t l = ledger_of(160, 4, 16384);
  const int rc = attend(c, 16, &l, nullptr);
  const Launch* a = &launches[0];  // the one that takes LDS at the launch
  for (const Launch& x : launches)
    if (x.lds > a->lds) a = &x;
  printf("rc %d lds %zu threads %u groups %u\n", rc, a->lds, a->block.x,
         a->grid.x);
  return 0;
}

int main(int n, char** a) {
  const std::string what = n > 1 ? a[1] : "";
  if (what == "threads") return cache_threads_test();
  if (what == "selection_threads") return selection_threads_test();
  if (what == "rows" && n > 4)
    return many_rows_test(atoi(a[2]), atoi(a[3]), atoi(a[4]));
  if (what == "lds" && n > 4)
    return lds_test(atoi(a[2]), atoi(a[3]) != 0, atoi(a[4]));
  return 2;
}
