// What the kernels on a paged key-value cache share: the cache as they see
// it, 16-byte moves, and reductions over a wave and a workgroup.
#pragma once

#include "cache_layout.hpp"
#include "wave.hpp"

namespace ltk {

// Element types, as in include/libtopk.h.
constexpr int kBf16 = 0, kF16 = 1, kE4m3 = 2, kF32 = 3, kE2m1 = 4;
constexpr int kMaxDim = 256;
constexpr int kBlockElems = 32;  // of a 4-bit row that share a scale

struct CacheParams {
  const char* k;
  const char* v;
  RowStrides ks, vs;  // bytes
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int64_t pages;
  Divisor page;
  int32_t batch, heads, dim;
  int32_t cap;        // slots that the table (and the ledger) can name
  int32_t row_bytes;  // dim elements
};

// Scales of 4-bit rows: a byte for each 32 elements (bytes throughout).  Apart
// from the rest, so that calls without them do not carry them.
struct BlockParams {
  const char* k;
  const char* v;
  RowStrides ks, vs;
  int32_t n;  // of a row
};

struct LedgerParams {
  float* w;
  int32_t* pos;
  int64_t wb, wh, pb, ph;  // elements
};

// Load, through the scalar cache, of a value that no kernel in flight writes
// (tables, lengths, scales), from an address that is the same in every lane.
// Scalar loads have a counter of their own: waiting for one leaves the vector
// loads before and after it in flight.
template <class T>
__device__ __forceinline__ T ld_const(const T* p) {
  typedef const __attribute__((address_space(4))) T ConstT;
  return *(ConstT*)(uintptr_t)p;
}

// Page of slot t of a sequence whose table row is `table` (-1: none), and the
// slot's place within the page.
__device__ __forceinline__ int32_t find_page(const CacheParams& c,
                                             const int32_t* table, int32_t t,
                                             int32_t* place) {
  const int32_t p = quotient(c.page, t);
  *place = t - p * c.page.d;
  const int32_t id = table[p];
  return page_ok(id, c.pages) ? id : -1;
}

template <class T, class Op>
__device__ __forceinline__ T wave_fold(T v, Op op) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = op(v, __shfl_xor(v, o, kWave));
  return v;
}

}  // namespace ltk
