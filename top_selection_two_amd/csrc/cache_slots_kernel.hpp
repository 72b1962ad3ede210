// Append to and eviction from a paged cache by accumulated attention weight.
//
// Slots are retained in the order of (key, earlier slot first): the key is
// the weight's float32 bits mapped to integer order, protected slots carry
// the largest key (rank_key, rank_word).  Append replaces the last slot in
// that order, eviction keeps the first `keep`.
#pragma once

#include <type_traits>

#include "cache_common.hpp"

namespace ltk {

typedef float f32x4s __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x4s __attribute__((ext_vector_type(4), aligned(4)));

struct SlotsParams {
  CacheParams c;
  LedgerParams w;
  const int32_t* seen;
  int32_t sinks, recent;
  // append
  const char* k_new;
  const char* v_new;
  int64_t nb, nh;  // bytes
  int32_t limit;
  int32_t* out_slots;
  // evict
  int32_t keep;
  LedgerParams after;
  int32_t* pairs;     // [rows][2][pair_cap]: holes, then movers
  int32_t* moves;     // [rows]: pairs of the row
  int32_t pair_cap;
  Divisor row_units;  // 16-byte units of a row
  uint32_t* hist;     // [rows][3][kBins], long rows
  int4* counts;       // [rows][chunks], long rows
  int2* state;        // [rows][4]: cut and want before each digit, long rows
  int32_t chunks;
  int32_t* out_lens;
};
struct Slots4Params : SlotsParams {
  BlockParams s;
};

__device__ __forceinline__ uint64_t min64(uint64_t a, uint64_t b) {
  return a < b ? a : b;
}

// A row (sequence and head) of the ledger as the kernels read it.
struct LedgerRow {
  int b, h;
  int32_t len, seen;
  const float* w;
  const int32_t* pos;
};

__device__ __forceinline__ LedgerRow ledger_row(const SlotsParams& p,
                                                int row) {
  LedgerRow r;
  r.b = row / p.c.heads;
  r.h = row % p.c.heads;
  r.len = clamp_len(ld_const(p.c.lens + r.b), p.c.cap);
  r.seen = ld_const(p.seen + r.b);
  r.w = p.w.w + r.b * p.w.wb + r.h * p.w.wh;
  r.pos = p.w.pos + r.b * p.w.pb + r.h * p.w.ph;
  return r;
}

// ---- append ------------------------------------------------------------------
// One workgroup per sequence and head.  A full row is read once, four slots a
// thread at a time, for the least (key, slot) word; the reads of a row of some
// thousand slots are all in flight together.
__global__ __launch_bounds__(kBlock) void append_kernel(SlotsParams p) {
  const CacheParams& c = p.c;
  const int row = blockIdx.x;
  const LedgerRow r = ledger_row(p, row);
  const int32_t len = r.len;
  // The new row's bytes, loaded ahead of the search.
  const int units = c.row_bytes / 16;
  const int tid = threadIdx.x;
  const bool is_k = tid < units, mover = tid < 2 * units;
  const int off = (is_k ? tid : tid - units) * 16;
  v4i bytes = {0, 0, 0, 0};
  if (mover)
    bytes = *(const v4i*)((is_k ? p.k_new : p.v_new) + r.b * p.nb +
                          r.h * p.nh + off);
  __shared__ uint64_t low[kWaves];
  int32_t slot;
  if (len < p.limit) {
    slot = len < c.cap ? len : -1;
  } else {
    uint64_t last = ~0ull;
    const int32_t whole = len & ~3;
    constexpr int J = 4;
    for (int32_t t0 = tid * 4; t0 < whole; t0 += J * 4 * kBlock) {
      f32x4s w[J];
      i32x4s at[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int32_t t = t0 + j * 4 * kBlock;
        const int32_t in = t < whole ? t : t0;  // a repeat changes nothing
        w[j] = *(const f32x4s*)(r.w + in);
        at[j] = *(const i32x4s*)(r.pos + in);
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int32_t t = t0 + j * 4 * kBlock;
        const int32_t in = t < whole ? t : t0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          last = min64(last, rank_word(rank_key(__float_as_int(w[j][e]),
                                                at[j][e], r.seen, p.sinks,
                                                p.recent),
                                       in + e));
      }
    }
    const int32_t t = whole + tid;
    if (t < len)
      last = min64(last, rank_word(rank_key(__float_as_int(r.w[t]), r.pos[t],
                                            r.seen, p.sinks, p.recent),
                                   t));
    last = wave_fold(last, min64);
    if (tid % kWave == 0) low[tid / kWave] = last;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) last = min64(last, low[i]);
    slot = (int32_t)~(uint32_t)last;
  }
  if (tid == 0) {
    p.out_slots[row] = slot;
    if (r.h == 0) p.out_lens[r.b] = len < p.limit && slot >= 0 ? len + 1 : len;
    if (slot >= 0) {
      const_cast<float*>(r.w)[slot] = 0.0f;
      const_cast<int32_t*>(r.pos)[slot] = r.seen;
    }
  }
  if (slot < 0) return;
  int32_t place;
  const int32_t id =
      find_page(c, c.table + r.b * c.table_stride, slot, &place);
  if (id < 0) return;
  if (mover) {
    const char* dst = is_k ? c.k + row_offset(c.ks, id, r.h, place)
                           : c.v + row_offset(c.vs, id, r.h, place);
    *(v4i*)(const_cast<char*>(dst) + off) = bytes;
  }
}

// ---- eviction ----------------------------------------------------------------
// The key of the last kept slot is found digit by digit (11, 11 and 10 bits)
// from histograms of the keys; ties at it are kept in slot order.  Holes
// (slots below `keep` that are not kept) and movers (kept slots at or beyond
// it) are listed in slot order by counting, and a second kernel moves the
// rows, which is most of the bytes.
//
// Rows of up to kShortSlots slots are selected by one workgroup that holds
// their keys in registers.  Longer rows are cut into chunks of kChunkSlots,
// a workgroup each, and the digits, the ties and the lists become launches.
constexpr int kEvThreads = 1024;
constexpr int kEvWaves = kEvThreads / kWave;
constexpr int kBins = 2048;
constexpr int kShortSlots = 16 * kEvThreads;
constexpr int kChunkKeys = 4;
constexpr int kChunkSlots = kChunkKeys * kEvThreads;

struct Digit {
  int shift, bits;
};
__device__ __forceinline__ Digit digit(int pass) {
  return pass == 0 ? Digit{21, 11} : pass == 1 ? Digit{10, 11} : Digit{0, 10};
}

// Sum of the counts v (the same in a wave's lanes) of the waves before this
// one, and of all.  `lds` is the caller's for this one call.
__device__ __forceinline__ int wave_offset(int v, int* lds, int* total) {
  if (lane() == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kEvWaves; ++i) {
    const int x = lds[i];
    if (i < (int)threadIdx.x / kWave) before += x;
    all += x;
  }
  *total = uni(all);
  return uni(before);
}

// Exclusive prefix sum of v over the workgroup, and the total.
__device__ __forceinline__ int block_scan(int v, int* lds, int* total) {
  const int incl = wave_scan_incl(v);
  __syncthreads();
  if (threadIdx.x % kWave == kWave - 1) lds[threadIdx.x / kWave] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kEvWaves; ++i) {
    const int x = lds[i];
    if (i < (int)threadIdx.x / kWave) before += x;
    all += x;
  }
  *total = all;
  return before + incl - v;
}

// The bin that holds the `want`-th largest key of a histogram, and how many
// keys lie in the bins above it.  Thread i takes bins 2 i and 2 i + 1 counted
// from the top.
struct Found {
  int bin, above;
};
__device__ __forceinline__ Found find_bin(const uint32_t* hist, int want,
                                          int* lds, Found* out) {
  const int b = kBins - 1 - 2 * (int)threadIdx.x;
  const int c0 = (int)hist[b], c1 = (int)hist[b - 1];
  int total;
  const int before = block_scan(c0 + c1, lds, &total);
  if (before < want && want <= before + c0) *out = Found{b, before};
  if (before + c0 < want && want <= before + c0 + c1)
    *out = Found{b - 1, before + c0};
  __syncthreads();
  return *out;
}

// Keys of KPT slots a thread: wave w holds slots first + (w KPT + j) 64 + lane,
// so that slot order is wave, j, lane.
template <int KPT>
__device__ __forceinline__ int32_t key_slot(int32_t first, int j) {
  return first + ((int)threadIdx.x / kWave * KPT + j) * kWave +
         (int)threadIdx.x % kWave;
}

template <int KPT>
__device__ __forceinline__ void load_keys(const SlotsParams& p,
                                          const LedgerRow& r, int32_t first,
                                          uint32_t (&u)[KPT], float (&w)[KPT],
                                          int32_t (&at)[KPT]) {
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int32_t t = key_slot<KPT>(first, j);
    const int32_t in = t < r.len ? t : 0;
    w[j] = r.w[in];
    at[j] = r.pos[in];
  }
#pragma unroll
  for (int j = 0; j < KPT; ++j)
    u[j] = bias(rank_key(__float_as_int(w[j]), at[j], r.seen, p.sinks,
                         p.recent));
}

template <int KPT>
__device__ __forceinline__ void load_keys(const SlotsParams& p,
                                          const LedgerRow& r, int32_t first,
                                          uint32_t (&u)[KPT]) {
  float w[KPT];
  int32_t at[KPT];
  load_keys<KPT>(p, r, first, u, w, at);
}

// Adds the digits of the keys that begin with `prefix` (all bits above the
// digit) to a histogram in LDS.  A wave whose keys all fall into one bin
// (protected slots, equal weights) adds once: its lanes would queue there.
template <int KPT>
__device__ __forceinline__ void count_digits(const uint32_t (&u)[KPT],
                                             int32_t first, int32_t len,
                                             uint32_t prefix, Digit d,
                                             uint32_t* hist) {
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int32_t t = key_slot<KPT>(first, j);
    const uint32_t head = d.shift + d.bits == 32
                              ? 0u
                              : u[j] >> (d.shift + d.bits) <<
                                    (d.shift + d.bits);
    const bool in = t < len && head == prefix;
    const uint32_t bin = (u[j] >> d.shift) & ((1u << d.bits) - 1u);
    const uint64_t all = ballot(in);
    if (all == 0) continue;
    const uint32_t bin0 = (uint32_t)__builtin_amdgcn_readlane(
        (int)bin, __builtin_ctzll(all));
    if (ballot(in && bin == bin0) == all) {
      if (lane() == 0) atomicAdd(&hist[bin0], (uint32_t)popc(all));
    } else if (in) {
      atomicAdd(&hist[bin], 1u);
    }
  }
}

__device__ __forceinline__ void clear_bins(uint32_t* hist) {
  for (int i = threadIdx.x; i < kBins; i += kEvThreads) hist[i] = 0u;
}

// Lists a chunk's holes and movers and writes what stays in place; before the
// chunk lie `ties` slots with key = cut, `holes` holes and `movers` movers.
// `need` ties are kept in all.  Returns (in every thread) holes and movers
// up to and with this chunk.
template <int KPT>
__device__ __forceinline__ int2 list_chunk(const SlotsParams& p,
                                           const LedgerRow& r, int row,
                                           int32_t first,
                                           const uint32_t (&u)[KPT],
                                           const float (&w)[KPT],
                                           const int32_t (&at)[KPT],
                                           uint32_t cut, int need, int ties,
                                           int holes, int movers,
                                           int (*lds)[kEvWaves]) {
  static_assert(KPT * kEvThreads < 1 << 16, "two counts in a word");
  const int keep = p.keep;
  int n_tie = 0;
#pragma unroll
  for (int j = 0; j < KPT; ++j)
    n_tie += popc(ballot(key_slot<KPT>(first, j) < r.len && u[j] == cut));
  int total;
  int tie = ties + wave_offset(n_tie, lds[0], &total);
  uint64_t hole_m[KPT], move_m[KPT];
  int n = 0;  // holes, and 2^16 times movers
  float* w2 = p.after.w + r.b * p.after.wb + r.h * p.after.wh;
  int32_t* pos2 = p.after.pos + r.b * p.after.pb + r.h * p.after.ph;
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int32_t t = key_slot<KPT>(first, j);
    const bool in = t < r.len;
    const uint64_t eq = ballot(in && u[j] == cut);
    const bool kept = in && (u[j] > cut || (u[j] == cut &&
                                            tie + lanes_below(eq) < need));
    tie += popc(eq);
    hole_m[j] = ballot(in && t < keep && !kept);
    move_m[j] = ballot(kept && t >= keep);
    n += popc(hole_m[j]) + (popc(move_m[j]) << 16);
    if (kept && t < keep) {
      w2[t] = w[j];
      pos2[t] = at[j];
    }
  }
  const int before = wave_offset(n, lds[1], &total);
  int ih = holes + (before & 0xffff), im = movers + (before >> 16);
  int32_t* list = p.pairs + (int64_t)row * 2 * p.pair_cap;
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int32_t t = key_slot<KPT>(first, j);
    const int a = ih + lanes_below(hole_m[j]), b = im + lanes_below(move_m[j]);
    if (hole_m[j] >> lane() & 1 && a < p.pair_cap) list[a] = t;
    if (move_m[j] >> lane() & 1 && b < p.pair_cap) list[p.pair_cap + b] = t;
    ih += popc(hole_m[j]);
    im += popc(move_m[j]);
  }
  return make_int2(holes + (total & 0xffff), movers + (total >> 16));
}

// Rows that are short enough to stay as they are: copied, and padded.
__device__ __forceinline__ void copy_row(const SlotsParams& p,
                                         const LedgerRow& r, int from,
                                         int step) {
  float* w2 = p.after.w + r.b * p.after.wb + r.h * p.after.wh;
  int32_t* pos2 = p.after.pos + r.b * p.after.pb + r.h * p.after.ph;
  for (int32_t t = from; t < p.keep; t += step) {
    w2[t] = t < r.len ? r.w[t] : 0.0f;
    pos2[t] = t < r.len ? r.pos[t] : -1;
  }
}

template <int KPT>
__global__ __launch_bounds__(kEvThreads) void evict_short_kernel(
    SlotsParams p) {
  __shared__ uint32_t hist[kBins];
  __shared__ int lds[kEvWaves], sums[2][kEvWaves];
  __shared__ Found found;
  const int row = blockIdx.x, keep = p.keep;
  const LedgerRow r = ledger_row(p, row);
  if (threadIdx.x == 0) {
    if (r.h == 0) p.out_lens[r.b] = r.len < keep ? r.len : keep;
    if (p.moves && r.len <= keep) p.moves[row] = 0;
  }
  if (r.len <= keep) {
    copy_row(p, r, threadIdx.x, kEvThreads);
    return;
  }
  uint32_t u[KPT];
  float w[KPT];
  int32_t at[KPT];
  load_keys<KPT>(p, r, 0, u, w, at);
  uint32_t cut = 0;
  int want = keep;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const Digit d = digit(pass);
    clear_bins(hist);
    __syncthreads();
    count_digits<KPT>(u, 0, r.len, cut, d, hist);
    __syncthreads();
    const Found f = find_bin(hist, want, lds, &found);
    cut |= (uint32_t)f.bin << d.shift;
    want -= f.above;
  }
  const int2 n =
      list_chunk<KPT>(p, r, row, 0, u, w, at, cut, want, 0, 0, 0, sums);
  if (threadIdx.x == 0) p.moves[row] = n.y;
}

// ---- long rows ---------------------------------------------------------------
// hist[row][i] collects digit i of all chunks.  state[row][i] holds the cut's
// bits above digit i and the rank looked for below them; the launch after a
// digit's finds it from the histogram, in every workgroup, and the first chunk
// writes it down for the launch after that.
__device__ __forceinline__ void next_state(const SlotsParams& p, int row,
                                           int chunk, int done, int* lds,
                                           Found* found, uint32_t* cut,
                                           int* want) {
  int2 z = make_int2(0, p.keep);
  if (done > 0) {
    if (done > 1) z = p.state[(int64_t)row * 4 + done - 1];
    const Found f = find_bin(p.hist + ((int64_t)row * 3 + done - 1) * kBins,
                             z.y, lds, found);
    z.x |= (int)((uint32_t)f.bin << digit(done - 1).shift);
    z.y -= f.above;
    if (chunk == 0 && threadIdx.x == 0) p.state[(int64_t)row * 4 + done] = z;
  }
  *cut = (uint32_t)z.x;
  *want = z.y;
}

__global__ __launch_bounds__(kEvThreads) void evict_digit_kernel(
    SlotsParams p, int pass) {
  __shared__ uint32_t hist[kBins];
  __shared__ int lds[kEvWaves];
  __shared__ Found found;
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int32_t first = chunk * kChunkSlots;
  const LedgerRow r = ledger_row(p, row);
  if (r.len <= p.keep || first >= r.len) return;
  uint32_t u[kChunkKeys];
  load_keys<kChunkKeys>(p, r, first, u);
  clear_bins(hist);
  uint32_t cut;
  int want;
  next_state(p, row, chunk, pass, lds, &found, &cut, &want);
  __syncthreads();
  count_digits<kChunkKeys>(u, first, r.len, cut, digit(pass), hist);
  __syncthreads();
  uint32_t* all = p.hist + ((int64_t)row * 3 + pass) * kBins;
  for (int i = threadIdx.x; i < kBins; i += kEvThreads)
    if (hist[i]) atomicAdd(all + i, hist[i]);
}

// Of each chunk: slots with key above the cut and at it, below `keep` (x, y)
// and from it on (z, w).
__global__ __launch_bounds__(kEvThreads) void evict_count_kernel(
    SlotsParams p) {
  __shared__ int lds[kEvWaves];
  __shared__ Found found;
  __shared__ int sums[4];
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int32_t first = chunk * kChunkSlots;
  const LedgerRow r = ledger_row(p, row);
  if (r.len <= p.keep || first >= r.len) return;
  uint32_t u[kChunkKeys];
  load_keys<kChunkKeys>(p, r, first, u);
  if (threadIdx.x < 4) sums[threadIdx.x] = 0;
  uint32_t cut;
  int want;
  next_state(p, row, chunk, 3, lds, &found, &cut, &want);
  int n[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < kChunkKeys; ++j) {
    const int32_t t = key_slot<kChunkKeys>(first, j);
    const bool in = t < r.len, low = t < p.keep;
    n[0] += popc(ballot(in && low && u[j] > cut));
    n[1] += popc(ballot(in && low && u[j] == cut));
    n[2] += popc(ballot(in && !low && u[j] > cut));
    n[3] += popc(ballot(in && !low && u[j] == cut));
  }
  if (lane() == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n[i]) atomicAdd(&sums[i], n[i]);
  __syncthreads();
  if (threadIdx.x == 0)
    p.counts[(int64_t)row * p.chunks + chunk] =
        make_int4(sums[0], sums[1], sums[2], sums[3]);
}

__global__ __launch_bounds__(kEvThreads) void evict_list_kernel(
    SlotsParams p) {
  __shared__ int sums[2][kEvWaves];
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int32_t first = chunk * kChunkSlots;
  const LedgerRow r = ledger_row(p, row);
  if (chunk == 0 && r.h == 0 && threadIdx.x == 0)
    p.out_lens[r.b] = r.len < p.keep ? r.len : p.keep;
  if (r.len <= p.keep) {
    if (chunk == 0 && threadIdx.x == 0) p.moves[row] = 0;
    copy_row(p, r, chunk * kEvThreads + threadIdx.x, p.chunks * kEvThreads);
    return;
  }
  if (first >= r.len) return;
  uint32_t u[kChunkKeys];
  float w[kChunkKeys];
  int32_t at[kChunkKeys];
  load_keys<kChunkKeys>(p, r, first, u, w, at);
  const int2 z = p.state[(int64_t)row * 4 + 3];
  const uint32_t cut = (uint32_t)z.x;
  const int want = z.y;
  // Ties, kept slots below `keep` and kept slots from it on, before this
  // chunk (every wave for itself, a chunk a lane): of a chunk's ties those are
  // kept that come before the want-th.
  const int4* counts = p.counts + (int64_t)row * p.chunks;
  int ties = 0, low = 0, high = 0;
  for (int i0 = 0; i0 < chunk; i0 += kWave) {
    const int i = i0 + lane();
    const int4 n = i < chunk ? counts[i] : make_int4(0, 0, 0, 0);
    const int incl = wave_scan_incl(n.y + n.w);
    const int before = ties + incl - n.y - n.w;
    const int left = max(want - before, 0), left2 = max(want - before - n.y, 0);
    low += __builtin_amdgcn_readlane(wave_scan_incl(n.x + min(n.y, left)), 63);
    high +=
        __builtin_amdgcn_readlane(wave_scan_incl(n.z + min(n.w, left2)), 63);
    ties += __builtin_amdgcn_readlane(incl, 63);
  }
  const int below = first < p.keep ? first : p.keep;
  const int2 n = list_chunk<kChunkKeys>(p, r, row, first, u, w, at, cut, want,
                                        ties, below - low, high, sums);
  if (r.len - first <= kChunkSlots && threadIdx.x == 0) p.moves[row] = n.y;
}

// ---- moves -------------------------------------------------------------------
// Pair i of a row: slot movers[i] goes to slot holes[i].  A thread moves 16
// bytes of a pair's K row and of its V row; the first thread of a pair takes
// its weight and position along.  One pair a thread and as many workgroups as
// it takes: the chain pair -> pages -> bytes is hidden by other waves, and two
// or four pairs a thread were slower (16 prompts of up to 8192 slots cut to
// 2048, slots outside heads: 33 us against 35 and 41), as were separate
// threads for K and V, which find the same pages twice (46 us).
template <bool BLOCKS>
__global__ __launch_bounds__(kBlock) void evict_move_kernel(
    std::conditional_t<BLOCKS, Slots4Params, SlotsParams> p) {
  const CacheParams& c = p.c;
  const int32_t i = blockIdx.x * kBlock + threadIdx.x;
  const int32_t pair = quotient(p.row_units, i);
  const int32_t off = (i - pair * p.row_units.d) * 16;
  for (int row = blockIdx.y; row < c.batch * c.heads; row += gridDim.y) {
    if (pair >= ld_const(p.moves + row)) continue;
    const int b = row / c.heads, h = row % c.heads;
    const int32_t* table = c.table + b * c.table_stride;
    const int32_t* holes = p.pairs + (int64_t)row * 2 * p.pair_cap;
    const int32_t to = holes[pair], from = holes[p.pair_cap + pair];
    if (off == 0) {
      p.after.w[b * p.after.wb + h * p.after.wh + to] =
          p.w.w[b * p.w.wb + h * p.w.wh + from];
      p.after.pos[b * p.after.pb + h * p.after.ph + to] =
          p.w.pos[b * p.w.pb + h * p.w.ph + from];
    }
    int32_t zt, zf;
    const int32_t it = find_page(c, table, to, &zt);
    const int32_t jf = find_page(c, table, from, &zf);
    if (it < 0 || jf < 0) continue;
    const v4i x = __builtin_nontemporal_load(
        (const v4i*)(c.k + row_offset(c.ks, jf, h, zf) + off));
    const v4i y = __builtin_nontemporal_load(
        (const v4i*)(c.v + row_offset(c.vs, jf, h, zf) + off));
    // The scales of 4-bit rows go along, by the thread of a row's first unit.
    // (16 prompts of up to 8192 slots cut to 2048, 8 heads of 128: 31 us in 4
    // bits, 36 with slots outside heads; 44 and 43 in bfloat16.)
    if constexpr (BLOCKS) {
      if (off == 0) {
        const BlockParams& s = p.s;
        const char* kf = s.k + row_offset(s.ks, jf, h, zf);
        const char* vf = s.v + row_offset(s.vs, jf, h, zf);
        char* kt = const_cast<char*>(s.k + row_offset(s.ks, it, h, zt));
        char* vt = const_cast<char*>(s.v + row_offset(s.vs, it, h, zt));
        for (int e = 0; e < s.n; ++e) {
          const char a = kf[e], b = vf[e];
          kt[e] = a;
          vt[e] = b;
        }
      }
    }
    __builtin_nontemporal_store(
        x, (v4i*)const_cast<char*>(c.k + row_offset(c.ks, it, h, zt) + off));
    __builtin_nontemporal_store(
        y, (v4i*)const_cast<char*>(c.v + row_offset(c.vs, it, h, zt) + off));
  }
}

}  // namespace ltk
