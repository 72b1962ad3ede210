// The attention kernels of one pair of query type (LTK_Q) and cache type
// (LTK_C), given on the command line: built once for each pair, side by side.
#include <hip/hip_runtime.h>

#include "cache_attend_kernel.hpp"

namespace ltk {

template <int Q, int C, int NC>
const void* attend_fn_nc(bool pg16, bool heads, AttendNeeds* needs) {
  typedef Attend<Q, C, NC, true> A;
  *needs = {A::COLS, A::THREADS, (int)sizeof(typename A::Lds), A::JOIN};
  if (heads)
    return pg16 ? (const void*)&attend_kernel<Q, C, NC, true, kHeadRun>
                : (const void*)&attend_kernel<Q, C, NC, false, kHeadRun>;
  return pg16 ? (const void*)&attend_kernel<Q, C, NC, true, 1>
              : (const void*)&attend_kernel<Q, C, NC, false, 1>;
}
template <int Q, int C>
const void* attend_fn_dim(int dim, bool pg16, bool heads, AttendNeeds* n) {
  return dim <= 64    ? attend_fn_nc<Q, C, 2>(pg16, heads, n)
         : dim <= 96  ? attend_fn_nc<Q, C, 3>(pg16, heads, n)
         : dim <= 128 ? attend_fn_nc<Q, C, 4>(pg16, heads, n)
         : dim <= 192 ? attend_fn_nc<Q, C, 6>(pg16, heads, n)
                      : attend_fn_nc<Q, C, 8>(pg16, heads, n);
}

template const void* attend_fn_dim<LTK_Q, LTK_C>(int, bool, bool,
                                                 AttendNeeds*);

}  // namespace ltk
