// Append to and eviction from a paged cache by accumulated attention weight.
//
// Slots are retained in the order of (key, earlier slot first): the key is
// the weight's float32 bits mapped to integer order, protected slots carry
// the largest key (rank_key, rank_word).  Append replaces the last slot in
// that order, eviction keeps the first `keep`.
#pragma once

#include "cache_common.hpp"

namespace ltk {

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
  int32_t pair_cap;
  int32_t* out_lens;
};

__device__ __forceinline__ uint64_t min64(uint64_t a, uint64_t b) {
  return a < b ? a : b;
}

// Key of slot t of a ledger row.
__device__ __forceinline__ int32_t slot_key(const float* w, const int32_t* pos,
                                            int32_t t, int32_t seen,
                                            int32_t sinks, int32_t recent) {
  return rank_key(__float_as_int(w[t]), pos[t], seen, sinks, recent);
}

// One workgroup per sequence and head.
__global__ __launch_bounds__(kBlock) void append_kernel(SlotsParams p) {
  const CacheParams& c = p.c;
  const int row = blockIdx.x;
  const int b = row / c.heads, h = row % c.heads;
  const int32_t len = clamp_len(c.lens[b], c.cap);
  const int32_t seen = p.seen[b];
  float* w = p.w.w + b * p.w.wb + h * p.w.wh;
  int32_t* pos = p.w.pos + b * p.w.pb + h * p.w.ph;
  __shared__ uint64_t low[kWaves];
  int32_t slot;
  if (len < p.limit) {
    slot = len < c.cap ? len : -1;
  } else {
    uint64_t last = ~0ull;
    for (int32_t t = threadIdx.x; t < len; t += kBlock)
      last = min64(last, rank_word(slot_key(w, pos, t, seen, p.sinks,
                                            p.recent), t));
    last = wave_fold(last, min64);
    if (threadIdx.x % kWave == 0) low[threadIdx.x / kWave] = last;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) last = min64(last, low[i]);
    slot = (int32_t)~(uint32_t)last;
  }
  if (threadIdx.x == 0) {
    p.out_slots[row] = slot;
    if (h == 0) p.out_lens[b] = len < p.limit && slot >= 0 ? len + 1 : len;
    if (slot >= 0) {
      w[slot] = 0.0f;
      pos[slot] = seen;
    }
  }
  if (slot < 0) return;
  int32_t place;
  const int32_t id =
      find_page(c, c.table + b * c.table_stride, slot, &place);
  if (id < 0) return;
  const int units = c.row_bytes / 16;
  const int u = threadIdx.x;
  if (u < 2 * units) {
    const bool is_k = u < units;
    const int off = (is_k ? u : u - units) * 16;
    const char* src = (is_k ? p.k_new : p.v_new) + b * p.nb + h * p.nh + off;
    const char* dst = is_k ? c.k + row_offset(c.ks, id, h, place)
                           : c.v + row_offset(c.vs, id, h, place);
    *(v4i*)(const_cast<char*>(dst) + off) = *(const v4i*)src;
  }
}

// Sum over the workgroup, in every thread.
__device__ __forceinline__ int block_sum(int v, int* lds) {
  v = wave_fold(v, [](int a, int e) { return a + e; });
  __syncthreads();
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  int s = 0;
  for (int i = 0; i < kWaves; ++i) s += lds[i];
  return s;
}

// Threads below this one for which f is true; *total of the workgroup.
__device__ __forceinline__ int block_rank(bool f, int* lds, int* total) {
  const uint64_t m = ballot(f);
  __syncthreads();
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = popc(m);
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kWaves; ++i) {
    if (i < (int)threadIdx.x / kWave) before += lds[i];
    all += lds[i];
  }
  *total = all;
  return before + lanes_below(m);
}

// One workgroup per sequence and head: the key of the last kept slot by
// bitwise search, the lists of holes and movers by ordered counting, then the
// moves.
__global__ __launch_bounds__(kBlock) void evict_kernel(SlotsParams p) {
  const CacheParams& c = p.c;
  const int row = blockIdx.x;
  const int b = row / c.heads, h = row % c.heads;
  const int32_t len = clamp_len(c.lens[b], c.cap);
  const int32_t seen = p.seen[b], keep = p.keep;
  const float* w = p.w.w + b * p.w.wb + h * p.w.wh;
  const int32_t* pos = p.w.pos + b * p.w.pb + h * p.w.ph;
  float* w2 = p.after.w + b * p.after.wb + h * p.after.wh;
  int32_t* pos2 = p.after.pos + b * p.after.pb + h * p.after.ph;
  if (h == 0 && threadIdx.x == 0) p.out_lens[b] = len < keep ? len : keep;
  for (int32_t t = threadIdx.x; t < keep; t += kBlock) {
    w2[t] = t < len ? w[t] : 0.0f;
    pos2[t] = t < len ? pos[t] : -1;
  }
  if (len <= keep) return;
  __shared__ int lds[kWaves];
  // The largest u with at least `keep` keys >= u (keys biased to unsigned).
  uint32_t cut = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t u = cut | (1u << bit);
    int n = 0;
    for (int32_t t = threadIdx.x; t < len; t += kBlock)
      n += bias(slot_key(w, pos, t, seen, p.sinks, p.recent)) >= u;
    if (block_sum(n, lds) >= keep) cut = u;
  }
  int above = 0;
  for (int32_t t = threadIdx.x; t < len; t += kBlock)
    above += bias(slot_key(w, pos, t, seen, p.sinks, p.recent)) > cut;
  int ties = keep - block_sum(above, lds);  // of the slots with key = cut
  int32_t* holes = p.pairs + (int64_t)row * 2 * p.pair_cap;
  int32_t* movers = holes + p.pair_cap;
  int nh = 0, nm = 0;
  for (int32_t t0 = 0; t0 < len; t0 += kBlock) {
    const int32_t t = t0 + threadIdx.x;
    const bool in = t < len;
    const uint32_t u =
        in ? bias(slot_key(w, pos, t, seen, p.sinks, p.recent)) : 0u;
    int total;
    const int r = block_rank(in && u == cut, lds, &total);
    const bool kept = in && (u > cut || (u == cut && r < ties));
    ties -= total;
    const bool hole = in && t < keep && !kept, mover = kept && t >= keep;
    int i = nh + block_rank(hole, lds, &total);
    if (hole && i < p.pair_cap) holes[i] = t;
    nh += total;
    i = nm + block_rank(mover, lds, &total);
    if (mover && i < p.pair_cap) movers[i] = t;
    nm += total;
  }
  __syncthreads();
  const int32_t* table = c.table + b * c.table_stride;
  const int units = c.row_bytes / 16;
  for (int i = threadIdx.x / kWave; i < nm && i < p.pair_cap; i += kWaves) {
    const int32_t to = holes[i], from = movers[i];
    if (threadIdx.x % kWave == 0) {
      w2[to] = w[from];
      pos2[to] = pos[from];
    }
    int32_t zt, zf;
    const int32_t it = find_page(c, table, to, &zt);
    const int32_t jf = find_page(c, table, from, &zf);
    if (it < 0 || jf < 0) continue;
    const int u = threadIdx.x % kWave;
    if (u < 2 * units) {
      const bool is_k = u < units;
      const int off = (is_k ? u : u - units) * 16;
      const RowStrides& s = is_k ? c.ks : c.vs;
      const char* base = (is_k ? c.k : c.v) + off;
      *(v4i*)const_cast<char*>(base + row_offset(s, it, h, zt)) =
          *(const v4i*)(base + row_offset(s, jf, h, zf));
    }
  }
}

}  // namespace ltk
