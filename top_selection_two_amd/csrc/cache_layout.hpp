// Where the rows of a paged cache lie, and the order in which its slots are
// retained: plain integer arithmetic, the same on host and device (constexpr
// functions are both), so that it is tested on the CPU.
#pragma once

#include <stdint.h>

namespace ltk {

// n / d for 0 <= n < 2^31 by one multiplication.  With 2^(s-1) < d <= 2^s and
// m = ceil(2^(31+s) / d) <= 2^31 * 2, the excess e = m d - 2^(31+s) is below
// d <= 2^s, so n m / 2^(31+s) exceeds n / d by n e / (d 2^(31+s)) < 1 / d:
// too little to pass the next integer.
struct Divisor {
  uint64_t m;
  int32_t shift;
  int32_t d;
};

constexpr Divisor make_divisor(int32_t d) {
  int s = 0;
  while (((int64_t)1 << s) < d) ++s;
  const uint64_t p = (uint64_t)1 << (31 + s);
  return Divisor{(p + (uint64_t)d - 1) / (uint64_t)d, 31 + s, d};
}

constexpr int32_t quotient(const Divisor& v, int32_t n) {
  return (int32_t)(((uint64_t)(uint32_t)n * v.m) >> v.shift);
}

// Slots in use: the given length within what the table (and the ledger) hold.
constexpr int32_t clamp_len(int32_t len, int32_t cap) {
  return len < 0 ? 0 : len > cap ? cap : len;
}

// Does a table entry name a page?
constexpr bool page_ok(int32_t id, int64_t pages) {
  return id >= 0 && (int64_t)id < pages;
}

// Byte strides of one of the cache's two arrays.
struct RowStrides {
  int64_t page, head, slot;
};

constexpr int64_t row_offset(const RowStrides& s, int32_t id, int32_t head,
                             int32_t place) {
  return (int64_t)id * s.page + (int64_t)head * s.head +
         (int64_t)place * s.slot;
}

// Floats of a share's result of an attention row: `cols` sums, a maximum and a
// weight's sum for each of `rows` queries, in whole 16-byte units, in which
// the next share's result is read too.
constexpr int32_t share_floats(int32_t rows, int32_t cols) {
  return (rows * (cols + 2) + 3) / 4 * 4;
}

// The largest key: protected slots.
constexpr int32_t kKeySafe = 0x7fffffff;

// Key of a slot: larger is kept before.  `bits` are the weight's float32 bits;
// flipping all but the sign of a negative number's bits makes integer order
// the order of the numbers.  The window's lower end is taken in 64 bits, since
// seen - recent can pass the least int32.
constexpr int32_t rank_key(int32_t bits, int32_t position, int32_t seen,
                           int32_t sinks, int32_t recent) {
  const bool safe =
      position < sinks || (int64_t)position >= (int64_t)seen - recent;
  return safe ? kKeySafe : bits ^ ((bits >> 31) & 0x7fffffff);
}

// Key and slot as one number that orders slots totally: larger is kept
// before, the earlier slot first among equal keys.
constexpr uint64_t rank_word(int32_t key, int32_t slot) {
  return ((uint64_t)((uint32_t)key ^ 0x80000000u) << 32) |
         (uint32_t)~(uint32_t)slot;
}

}  // namespace ltk
