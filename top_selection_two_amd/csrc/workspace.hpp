// Workspaces of the calls that keep some, one for each device and stream, and
// what else a call asks about its device (workspace.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "libtopk.h"

namespace ltk {

// Workspace of a call on a stream: `bytes` of any contents, `tickets` words,
// and the call's epoch (never 0, which cleared words carry).
struct Work {
  char* base;
  uint64_t* tickets;
  size_t ticket_words;  // all there are
  uint32_t epoch;
  std::unique_lock<std::mutex> hold;  // of the area, while this lives
};

int get_work(int dev, hipStream_t stream, size_t bytes, size_t tickets,
             Work* out);
int current_device(int* dev);
// Compute units of a device.
int units_of(int dev, int* out);
// Workgroups of `fn` that a compute unit holds at once.
int resident(const void* fn, int threads, int* out);
// Clears words (seed 0), or fills them with pseudo-random ones.
int fill(uint64_t* p, size_t words, uint64_t seed, hipStream_t s);
// Status after a launch by <<< >>>.
int launched(const char* what);
void debug_hip(const char* what, hipError_t e);

template <class P>
int launch(const void* fn, dim3 grid, int threads, P params, hipStream_t s,
           size_t lds = 0) {
  void* args[] = {&params};
  const hipError_t e = hipLaunchKernel(fn, grid, dim3(threads), args, lds, s);
  if (e != hipSuccess) {
    debug_hip("kernel launch", e);
    (void)hipGetLastError();
    return LIBTOPK_ERR_HIP;
  }
  return LIBTOPK_OK;
}

}  // namespace ltk
