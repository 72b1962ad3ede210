// Host side of the operators on a paged key-value cache (cache_attend,
// cache_append, cache_evict of include/libtopk.h): argument checks, workspace
// and launches.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <map>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "libtopk.h"
#include "cache_join_kernel.hpp"
#include "cache_slots_kernel.hpp"

namespace {

using namespace ltk;

static_assert(kBf16 == LIBTOPK_BF16 && kF16 == LIBTOPK_F16 &&
                  kE4m3 == LIBTOPK_E4M3,
              "the kernels' types are the header's");

constexpr int64_t kMaxSlots = (int64_t)1 << 30;
constexpr int64_t kSpan = (int64_t)1 << 60;  // bytes that an array may span

// ---- workspace --------------------------------------------------------------
// Areas that a (device, stream) has used are kept until cache_release(): a
// captured graph may hold their addresses.  Growth at least doubles, so all
// of them together stay below twice the largest.
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

__global__ void fill_words(uint64_t* p, int64_t n, uint64_t seed) {
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
int grow(Buffer* b, size_t bytes, hipStream_t stream, bool clear) {
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

// Workspace of a call on `stream`: `bytes` of any contents, `tickets` words,
// and the call's epoch (never 0, which cleared words carry).
struct Work {
  char* base;
  uint64_t* tickets;
  size_t ticket_words;  // all there are
  uint32_t epoch;
  std::unique_lock<std::mutex> hold;  // of the area, while this lives
};

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

// ---- argument checks --------------------------------------------------------
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Range {
  uintptr_t lo, hi;
  Range(const void* p, int64_t bytes)
      : lo((uintptr_t)p), hi((uintptr_t)p + (uintptr_t)bytes) {}
  bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
};

// Bytes from the first element to the last of an array of sizes n[i] and
// strides s[i] (>= 0) bytes with rows of `row` bytes; -1 if a stride is
// negative or the span too large.
int64_t span(const int64_t* n, const int64_t* s, int dims, int64_t row) {
  int64_t all = row;
  for (int i = 0; i < dims; ++i) {
    if (n[i] < 1) return 0;
    if (s[i] < 0) return -1;
    if (n[i] > 1 && s[i] > (kSpan - all) / (n[i] - 1)) return -1;
    all += (n[i] - 1) * s[i];
  }
  return all;
}

int elem_size(int dtype) { return dtype == LIBTOPK_E4M3 ? 1 : 2; }

// Do the rows of an array (as for span, strides >= 0) lie apart: does each
// axis, from the innermost on, step over all that the ones within it span?
bool apart(const int64_t* n, const int64_t* s, int dims, int64_t row) {
  int64_t all = row;
  bool done[4] = {};
  for (int k = 0; k < dims; ++k) {
    int in = -1;
    for (int i = 0; i < dims; ++i)
      if (!done[i] && (in < 0 || s[i] < s[in])) in = i;
    done[in] = true;
    if (n[in] <= 1) continue;
    if (s[in] < all) return false;
    all += (n[in] - 1) * s[in];
  }
  return true;
}

// Checks a cache and fills in what the kernels take of it; `k` and `v` get
// the arrays' extents.  Rows that are written must not share a byte.
int check_cache(const libtopk_cache_t* c, bool written, CacheParams* p,
                Range* k, Range* v, Range* table, Range* lens) {
  if (!c) return LIBTOPK_ERR_INVALID;
  if (c->dtype != LIBTOPK_BF16 && c->dtype != LIBTOPK_F16 &&
      c->dtype != LIBTOPK_E4M3)
    return LIBTOPK_ERR_INVALID;
  const int es = elem_size(c->dtype);
  if (c->batch < 0 || c->heads < 1 || c->heads > 65535 || c->page < 1 ||
      c->dim < 1 || c->dim > LIBTOPK_MAX_DIM || c->dim * es % 16 != 0 ||
      c->table_width < 1 || c->pages < 0 || c->pages > INT32_MAX)
    return LIBTOPK_ERR_INVALID;
  if ((int64_t)c->table_width * c->page >= kMaxSlots ||
      (int64_t)c->batch * c->heads > INT32_MAX)
    return LIBTOPK_ERR_INVALID;
  if (c->batch > 1 && (c->table_stride < 0 || c->table_stride > kSpan / 4))
    return LIBTOPK_ERR_INVALID;
  const int64_t ks[3] = {c->k_page_stride, c->k_head_stride, c->k_slot_stride};
  const int64_t vs[3] = {c->v_page_stride, c->v_head_stride, c->v_slot_stride};
  const int64_t n[3] = {c->pages, c->heads, c->page};
  int64_t kb[3], vb[3];
  for (int i = 0; i < 3; ++i) {
    if (ks[i] < 0 || ks[i] > kSpan || vs[i] < 0 || vs[i] > kSpan)
      return LIBTOPK_ERR_INVALID;
    kb[i] = ks[i] * es;
    vb[i] = vs[i] * es;
    if (n[i] > 1 && (kb[i] % 16 || vb[i] % 16)) return LIBTOPK_ERR_INVALID;
  }
  const int64_t klen = span(n, kb, 3, c->dim * es);
  const int64_t vlen = span(n, vb, 3, c->dim * es);
  if (klen < 0 || vlen < 0) return LIBTOPK_ERR_INVALID;
  if (written && !(apart(n, kb, 3, c->dim * es) && apart(n, vb, 3, c->dim * es)))
    return LIBTOPK_ERR_INVALID;
  if (c->pages > 0 && (!c->k || !c->v)) return LIBTOPK_ERR_INVALID;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return LIBTOPK_ERR_INVALID;
  if (c->batch > 0 && (!c->table || !c->lens)) return LIBTOPK_ERR_INVALID;
  if (!aligned(c->table, 4) || !aligned(c->lens, 4))
    return LIBTOPK_ERR_INVALID;
  const int64_t tn[1] = {c->batch}, ts[1] = {c->table_stride * 4};
  const int64_t tlen = span(tn, ts, 1, (int64_t)c->table_width * 4);
  if (tlen < 0) return LIBTOPK_ERR_INVALID;
  *k = Range(c->k, klen);
  *v = Range(c->v, vlen);
  *table = Range(c->table, tlen);
  *lens = Range(c->lens, (int64_t)c->batch * 4);
  p->k = (const char*)c->k;
  p->v = (const char*)c->v;
  p->ks = RowStrides{kb[0], kb[1], kb[2]};
  p->vs = RowStrides{vb[0], vb[1], vb[2]};
  p->table = c->table;
  p->table_stride = c->table_stride;
  p->lens = c->lens;
  p->pages = c->pages;
  p->page = make_divisor(c->page);
  p->batch = c->batch;
  p->heads = c->heads;
  p->dim = c->dim;
  p->cap = c->table_width * c->page;
  p->row_bytes = c->dim * es;
  return LIBTOPK_OK;
}

// Checks a ledger; its rows must not share an entry where they are written.
int check_ledger(const libtopk_ledger_t* l, int64_t batch, int64_t heads,
                 bool positions, bool written, LedgerParams* p, Range* w,
                 Range* pos) {
  if (!l || l->slots < 1) return LIBTOPK_ERR_INVALID;
  const int64_t n[2] = {batch, heads};
  const int64_t ws[2] = {l->weights_batch_stride, l->weights_head_stride};
  const int64_t ps[2] = {l->positions_batch_stride, l->positions_head_stride};
  const int64_t* st[2] = {ws, ps};
  const void* base[2] = {l->weights, l->positions};
  Range* out[2] = {w, pos};
  for (int a = 0; a < (positions ? 2 : 1); ++a) {
    if ((batch > 0 && !base[a]) || !aligned(base[a], 4))
      return LIBTOPK_ERR_INVALID;
    int64_t bytes[2];
    for (int i = 0; i < 2; ++i) {
      if (st[a][i] < 0 || st[a][i] > kSpan / 4) return LIBTOPK_ERR_INVALID;
      bytes[i] = st[a][i] * 4;
    }
    if (written) {
      // the inner of the two axes steps over whole rows, the outer over
      // whole runs of them
      const bool head_inner = st[a][1] <= st[a][0] || n[0] <= 1;
      const int in = head_inner ? 1 : 0, ou = 1 - in;
      if (n[in] > 1 && st[a][in] < l->slots) return LIBTOPK_ERR_INVALID;
      if (n[ou] > 1 &&
          st[a][ou] < (n[in] > 1 ? (n[in] - 1) * st[a][in] : 0) + l->slots)
        return LIBTOPK_ERR_INVALID;
    }
    const int64_t len = span(n, bytes, 2, (int64_t)l->slots * 4);
    if (len < 0) return LIBTOPK_ERR_INVALID;
    *out[a] = Range(base[a], len);
  }
  p->w = l->weights;
  p->pos = l->positions;
  p->wb = ws[0];
  p->wh = ws[1];
  p->pb = ps[0];
  p->ph = ps[1];
  return LIBTOPK_OK;
}

const void* attend_fn(int q, int c, int dim, bool pg16, bool heads,
                      AttendNeeds* n) {
  if (q == kBf16)
    return c == kE4m3 ? attend_fn_dim<kBf16, kE4m3>(dim, pg16, heads, n)
                      : attend_fn_dim<kBf16, kBf16>(dim, pg16, heads, n);
  return c == kE4m3 ? attend_fn_dim<kF16, kE4m3>(dim, pg16, heads, n)
                    : attend_fn_dim<kF16, kF16>(dim, pg16, heads, n);
}

constexpr int kMaxRuns = 1024;  // workgroups of an attention call
// Rows of at most this many scores are joined and get their weights from
// their last workgroup, longer ones from a second launch.  (211 slots of 8
// heads of 4 queries: 9.5 us in one launch, 11.2 in two; 16 sequences of 5000
// slots, one head of 16 queries: 37 us in one launch, 29 in two.)
constexpr int kDirectScores = 32768;
// Least share of a row, in tiles (see the dealing in attend_kernel): below
// it, joining costs more than the tiles that others take over (about 6 us
// against 0.6 us a tile of 128 elements).
constexpr int kMinTiles = 24;
static_assert(kBins % 2 == 0 && kBins == 2 * kEvThreads,
              "a thread searches two bins");

// Can this many workgroups be launched along an axis?  (Fewer than 2^32
// threads can.)
bool launchable(int64_t groups, int threads) {
  return groups <= (int64_t)(UINT32_MAX / (uint32_t)threads);
}

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

}  // namespace

extern "C" {

int cache_attend(const libtopk_cache_t* cache, const void* q, int32_t q_dtype,
                 int32_t q_heads, int64_t q_batch_stride,
                 int64_t q_head_stride, float scale, const float* k_scale,
                 const float* v_scale, const libtopk_ledger_t* ledger,
                 void* out, float* lse, libtopk_stream_t stream) {
  AttendParams p = {};
  const Range none(nullptr, 0);
  Range k = none, v = none, table = none, lens = none, w = none, pos = none;
  int rc = check_cache(cache, false, &p.c, &k, &v, &table, &lens);
  if (rc != LIBTOPK_OK) return rc;
  if (q_dtype != LIBTOPK_BF16 && q_dtype != LIBTOPK_F16)
    return LIBTOPK_ERR_INVALID;
  if (cache->dtype != LIBTOPK_E4M3 && cache->dtype != q_dtype)
    return LIBTOPK_ERR_INVALID;
  if (q_heads < 1 || q_heads % cache->heads != 0) return LIBTOPK_ERR_INVALID;
  const int64_t rows = (int64_t)cache->batch * q_heads;
  if (rows > INT32_MAX) return LIBTOPK_ERR_INVALID;
  if (q_batch_stride < 0 || q_head_stride < 0 || q_batch_stride > kSpan ||
      q_head_stride > kSpan || (cache->batch > 1 && q_batch_stride % 8) ||
      (q_heads > 1 && q_head_stride % 8))
    return LIBTOPK_ERR_INVALID;
  if (ledger) {
    rc = check_ledger(ledger, cache->batch, cache->heads, false, true, &p.w,
                      &w, &pos);
    if (rc != LIBTOPK_OK) return rc;
    if (ledger->slots < p.c.cap) p.c.cap = ledger->slots;
  }
  if (cache->batch == 0) return LIBTOPK_OK;
  if (!q || !out || !lse || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return LIBTOPK_ERR_INVALID;
  const int64_t qn[2] = {cache->batch, q_heads};
  const int64_t qs[2] = {q_batch_stride * 2, q_head_stride * 2};
  const int64_t qlen = span(qn, qs, 2, (int64_t)cache->dim * 2);
  if (qlen < 0) return LIBTOPK_ERR_INVALID;
  const Range outs[3] = {Range(out, rows * cache->dim * 2),
                         Range(lse, rows * 4), w};
  const Range ins[7] = {Range(q, qlen), k, v, table, lens,
                        Range(k_scale, k_scale ? cache->heads * 4 : 0),
                        Range(v_scale, v_scale ? cache->heads * 4 : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : ins)
      if (outs[i].meets(r)) return LIBTOPK_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (outs[i].meets(outs[j])) return LIBTOPK_ERR_INVALID;
  }
  p.q = (const char*)q;
  p.qb = qs[0];
  p.qh = qs[1];
  p.group = q_heads / cache->heads;
  p.scale2 = scale * 1.44269504088896341f;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.out = out;
  p.lse = lse;
  p.gtiles = (p.group + 15) / 16;
  int dev = 0;
  rc = current_device(&dev);
  if (rc != LIBTOPK_OK) return rc;
  hipStream_t s = (hipStream_t)stream;
  // Halves of a tile that lie in one page each get their addresses from
  // scalar registers (and 16 rows must lie within 2^31 bytes).
  const bool pg16 = cache->page % 16 == 0 && p.c.ks.slot < (1 << 27) &&
                    p.c.vs.slot < (1 << 27);
  int dev_units = 0;
  rc = units_of(dev, &dev_units);
  if (rc != LIBTOPK_OK) return rc;
  // Heads side by side within a slot, and work enough (at full lengths) that
  // a workgroup's waves need not share one head's tiles: several heads a
  // workgroup (48 ragged sequences of 8 heads: 132 us against 151 with one
  // head a workgroup and 135 with eight).
  const int64_t tiles = ((int64_t)p.c.cap + kTileSlots - 1) / kTileSlots;
  const bool heads =
      p.c.ks.head < p.c.ks.slot && p.c.vs.head < p.c.vs.slot &&
      cache->heads % kHeadRun == 0 &&
      (int64_t)cache->batch * cache->heads * p.gtiles * tiles >=
          (int64_t)dev_units * 2 * kMinTiles;
  p.hs = heads ? kHeadRun : 1;
  AttendNeeds needs;
  const void* fn =
      attend_fn(q_dtype, cache->dtype, cache->dim, pg16, heads, &needs);
  int fit = 0;
  rc = resident(fn, needs.threads, &fit);
  if (rc != LIBTOPK_OK) return rc;
  p.part_rows = p.group < 16 ? p.group : 16;
  p.lds_rows = (p.part_rows + 3) / 4 * 4;
  const int waves = needs.threads / kWave;
  int join = waves * p.lds_rows * needs.cols;
  if (join < needs.join) join = needs.join;
  size_t lds = (size_t)join * 4;
  const size_t tile_bytes = (size_t)kTileSlots * p.hs * p.part_rows * 4;
  // Workgroups that share a unit share its LDS: with a ledger each needs room
  // for the scores of a tile (one alone has it, see kScoresFit).
  const int64_t fixed = needs.lds + 256 + (int64_t)lds;
  while (ledger && fit > 1 &&
         kLdsBytes / fit < fixed + (int64_t)tile_bytes)
    --fit;
  const int64_t slots = (int64_t)fit * dev_units < kMaxRuns
                            ? (int64_t)fit * dev_units
                            : kMaxRuns;
  // A share that is dealt out costs about as much, besides its tiles, as
  // 128 KiB of them (loading the queries, joining the waves), a split row
  // some twice that.
  p.row_cost = 2048 / p.c.row_bytes;
  p.min_tiles = 2 * p.row_cost < kMinTiles ? 2 * p.row_cost : kMinTiles;
  p.row_cost = p.row_cost / p.hs > 1 ? p.row_cost / p.hs : 1;
  p.min_tiles = p.min_tiles / p.hs > 1 ? p.min_tiles / p.hs : 1;
  // Tiles of all rows must count in 31 bits.
  const int64_t att_rows =
      (int64_t)cache->batch * (cache->heads / p.hs) * p.gtiles;
  if (att_rows > INT32_MAX / (tiles + p.row_cost + kMinTiles))
    return LIBTOPK_ERR_INVALID;
  int64_t grid = att_rows * tiles;
  if (grid > slots) grid = slots;
  const size_t part_bytes = round_up(
      (size_t)grid * 2 * share_floats(p.hs * p.part_rows, needs.cols) * 4, 256);
  size_t score_bytes = 0, share_bytes = 0;
  if (ledger) {
    p.row_tiles = (int32_t)tiles;
    p.direct = p.gtiles == 1 && (int64_t)p.c.cap * p.group * p.hs <= kDirectScores;
    score_bytes = (size_t)(att_rows * tiles) * tile_bytes;
    if (!p.direct) share_bytes = round_up((size_t)att_rows * 8, 256);
    // What LDS is left when `fit` workgroups share a unit holds scores, but
    // no more than the longest run.
    int64_t run = (att_rows * (tiles + p.row_cost) + grid - 1) / grid;
    if (run < p.min_tiles) run = p.min_tiles;
    int64_t room = (kLdsBytes / fit - fixed) / (int64_t)tile_bytes;
    if (room > run) room = run;
    p.held_tiles = (int32_t)room;
    lds += (size_t)room * tile_bytes;
  }
  Work work;
  rc = get_work(dev, s, part_bytes + score_bytes + share_bytes,
                (size_t)att_rows, &work);
  if (rc != LIBTOPK_OK) return rc;
  p.part = (float*)work.base;
  if (ledger) p.scores = (float*)(work.base + part_bytes);
  if (share_bytes)
    p.shares = (int2*)(work.base + part_bytes + score_bytes);
  p.cols = needs.cols;
  p.q_type = q_dtype;
  p.ticket = work.tickets;
  p.epoch = work.epoch;
  rc = launch(fn, dim3((unsigned)grid), needs.threads, p, s, lds);
  if (rc != LIBTOPK_OK || !ledger || p.direct) return rc;
  const int64_t wrows = (int64_t)cache->batch * cache->heads;
  // Few rows: workgroups enough to share out the joining, too.
  int64_t chunks = (p.c.cap + kWeightSlots - 1) / kWeightSlots;
  const int64_t joiners = 1024 / wrows < kJoiners ? 1024 / wrows : kJoiners;
  if (chunks < joiners) chunks = joiners;
  return launch((const void*)&attend_join_kernel,
                dim3((unsigned)chunks,
                     (unsigned)(wrows < 65535 ? wrows : 65535)),
                kBlock, p, s);
}

int cache_append(const libtopk_cache_t* cache, const void* k_new,
                 const void* v_new, int64_t new_batch_stride,
                 int64_t new_head_stride, int32_t limit, const int32_t* seen,
                 const libtopk_ledger_t* ledger, int32_t sinks, int32_t recent,
                 int32_t* out_lens, int32_t* out_slots,
                 libtopk_stream_t stream) {
  SlotsParams p = {};
  const Range none(nullptr, 0);
  Range k = none, v = none, table = none, lens = none, w = none, pos = none;
  int rc = check_cache(cache, true, &p.c, &k, &v, &table, &lens);
  if (rc != LIBTOPK_OK) return rc;
  rc = check_ledger(ledger, cache->batch, cache->heads, true, true, &p.w, &w,
                    &pos);
  if (rc != LIBTOPK_OK) return rc;
  if (limit < 1 || sinks < 0 || recent < 0) return LIBTOPK_ERR_INVALID;
  const int es = elem_size(cache->dtype);
  if (new_batch_stride < 0 || new_head_stride < 0 ||
      new_batch_stride > kSpan || new_head_stride > kSpan ||
      (cache->batch > 1 && new_batch_stride * es % 16) ||
      (cache->heads > 1 && new_head_stride * es % 16))
    return LIBTOPK_ERR_INVALID;
  if (cache->batch == 0) return LIBTOPK_OK;
  if (!k_new || !v_new || !seen || !out_lens || !out_slots ||
      !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(seen, 4) ||
      !aligned(out_lens, 4) || !aligned(out_slots, 4))
    return LIBTOPK_ERR_INVALID;
  if (ledger->slots < p.c.cap) p.c.cap = ledger->slots;
  const int64_t nn[2] = {cache->batch, cache->heads};
  const int64_t ns[2] = {new_batch_stride * es, new_head_stride * es};
  const int64_t nlen = span(nn, ns, 2, (int64_t)cache->dim * es);
  if (nlen < 0) return LIBTOPK_ERR_INVALID;
  const int64_t rows = (int64_t)cache->batch * cache->heads;
  if (!launchable(rows, kBlock)) return LIBTOPK_ERR_INVALID;
  const Range outs[6] = {Range(out_lens, (int64_t)cache->batch * 4),
                         Range(out_slots, rows * 4), w, pos, k, v};
  const Range ins[5] = {Range(k_new, nlen), Range(v_new, nlen), table, lens,
                        Range(seen, (int64_t)cache->batch * 4)};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : ins)
      if (outs[i].meets(r)) return LIBTOPK_ERR_INVALID;
    // k and v may interleave (one array of pages that holds both)
    for (int j = 0; j < i; ++j)
      if (!(i == 5 && j == 4) && outs[i].meets(outs[j]))
        return LIBTOPK_ERR_INVALID;
  }
  p.seen = seen;
  p.sinks = sinks;
  p.recent = recent;
  p.k_new = (const char*)k_new;
  p.v_new = (const char*)v_new;
  p.nb = ns[0];
  p.nh = ns[1];
  p.limit = limit;
  p.out_lens = out_lens;
  p.out_slots = out_slots;
  int dev = 0;
  rc = current_device(&dev);
  if (rc != LIBTOPK_OK) return rc;
  return launch((const void*)&append_kernel, dim3((unsigned)rows), kBlock, p,
                (hipStream_t)stream);
}

int cache_evict(const libtopk_cache_t* cache, const int32_t* seen,
                const libtopk_ledger_t* ledger, int32_t keep, int32_t sinks,
                int32_t recent, const libtopk_ledger_t* after,
                int32_t* out_lens, libtopk_stream_t stream) {
  SlotsParams p = {};
  const Range none(nullptr, 0);
  Range k = none, v = none, table = none, lens = none, w = none, pos = none;
  Range w2 = none, pos2 = none;
  int rc = check_cache(cache, true, &p.c, &k, &v, &table, &lens);
  if (rc != LIBTOPK_OK) return rc;
  rc = check_ledger(ledger, cache->batch, cache->heads, true, false, &p.w, &w,
                    &pos);
  if (rc != LIBTOPK_OK) return rc;
  if (keep < 1 || sinks < 0 || recent < 0 || !after || after->slots < keep)
    return LIBTOPK_ERR_INVALID;
  libtopk_ledger_t used = *after;
  used.slots = keep;
  rc = check_ledger(&used, cache->batch, cache->heads, true, true, &p.after,
                    &w2, &pos2);
  if (rc != LIBTOPK_OK) return rc;
  if (cache->batch == 0) return LIBTOPK_OK;
  if (!seen || !out_lens || !aligned(seen, 4) || !aligned(out_lens, 4))
    return LIBTOPK_ERR_INVALID;
  if (ledger->slots < p.c.cap) p.c.cap = ledger->slots;
  const int64_t rows = (int64_t)cache->batch * cache->heads;
  const Range outs[5] = {Range(out_lens, (int64_t)cache->batch * 4), w2, pos2,
                         k, v};
  const Range ins[5] = {w, pos, table, lens,
                        Range(seen, (int64_t)cache->batch * 4)};
  for (int i = 0; i < 5; ++i) {
    for (const Range& r : ins)
      if (outs[i].meets(r)) return LIBTOPK_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (!(i == 4 && j == 3) && outs[i].meets(outs[j]))
        return LIBTOPK_ERR_INVALID;
  }
  p.seen = seen;
  p.sinks = sinks;
  p.recent = recent;
  p.keep = keep;
  p.out_lens = out_lens;
  // Moves of a row: at most the kept slots, and at most the slots beyond.
  p.pair_cap = p.c.cap > keep ? (p.c.cap - keep < keep ? p.c.cap - keep : keep)
                              : 0;
  const bool is_long = p.pair_cap > 0 && p.c.cap > kShortSlots;
  p.chunks = is_long ? (p.c.cap + kChunkSlots - 1) / kChunkSlots : 1;
  if (!launchable(rows * p.chunks, kEvThreads)) return LIBTOPK_ERR_INVALID;
  p.row_units = make_divisor(p.c.row_bytes / 16);
  if ((int64_t)p.pair_cap * p.row_units.d > INT32_MAX - kBlock)
    return LIBTOPK_ERR_INVALID;
  int dev = 0;
  rc = current_device(&dev);
  if (rc != LIBTOPK_OK) return rc;
  hipStream_t s = (hipStream_t)stream;
  if (p.pair_cap == 0) {  // every row is short enough as it is
    return launch((const void*)&evict_short_kernel<1>, dim3((unsigned)rows),
                  kEvThreads, p, s);
  }
  const size_t pair_bytes = round_up((size_t)rows * p.pair_cap * 8, 256);
  const size_t move_bytes = round_up((size_t)rows * 4, 256);
  const size_t hist_words = is_long ? (size_t)rows * 3 * kBins / 2 : 0;
  const size_t count_bytes = is_long ? (size_t)rows * p.chunks * 16 : 0;
  const size_t state_bytes = is_long ? (size_t)rows * 32 : 0;
  Work work;
  rc = get_work(dev, s, pair_bytes + move_bytes + hist_words * 8 + count_bytes +
                       state_bytes,
                1, &work);
  if (rc != LIBTOPK_OK) return rc;
  char* at = work.base;
  p.pairs = (int32_t*)at;
  p.moves = (int32_t*)(at += pair_bytes);
  p.hist = (uint32_t*)(at += move_bytes);
  p.counts = (int4*)(at += hist_words * 8);
  p.state = (int2*)(at += count_bytes);
  const unsigned wide = (unsigned)(rows * p.chunks);
  if (is_long) {
    rc = fill((uint64_t*)p.hist, hist_words, 0, s);
    for (int pass = 0; pass < 3 && rc == LIBTOPK_OK; ++pass) {
      hipLaunchKernelGGL(evict_digit_kernel, dim3(wide), dim3(kEvThreads), 0,
                         s, p, pass);
      rc = launched("evict_digit_kernel");
    }
    if (rc == LIBTOPK_OK)
      rc = launch((const void*)&evict_count_kernel, dim3(wide), kEvThreads, p,
                  s);
    if (rc == LIBTOPK_OK)
      rc = launch((const void*)&evict_list_kernel, dim3(wide), kEvThreads, p,
                  s);
  } else {
    const int keys = (p.c.cap + kEvThreads - 1) / kEvThreads;
    const void* fn = keys <= 2   ? (const void*)&evict_short_kernel<2>
                     : keys <= 4 ? (const void*)&evict_short_kernel<4>
                     : keys <= 8 ? (const void*)&evict_short_kernel<8>
                                 : (const void*)&evict_short_kernel<16>;
    rc = launch(fn, dim3(wide), kEvThreads, p, s);
  }
  if (rc != LIBTOPK_OK) return rc;
  const int64_t units = (int64_t)p.pair_cap * p.row_units.d;
  return launch((const void*)&evict_move_kernel,
                dim3((unsigned)((units + kBlock - 1) / kBlock),
                     (unsigned)(rows < 65535 ? rows : 65535)),
                kBlock, p, s);
}

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
