// Host side of the operators on a paged key-value cache (cache_attend,
// cache_append, cache_evict, cache_extend of include/libtopk.h): argument checks
// and launches.
#include <hip/hip_runtime.h>

#include "libtopk.h"
#include "workspace.hpp"
#include "cache_extend_kernel.hpp"
#include "cache_join_kernel.hpp"
#include "cache_slots_kernel.hpp"

namespace {

using namespace ltk;

static_assert(kBf16 == LIBTOPK_BF16 && kF16 == LIBTOPK_F16 &&
                  kE4m3 == LIBTOPK_E4M3 && kF32 == LIBTOPK_F32 &&
                  kE2m1 == LIBTOPK_E2M1 &&
                  kBlockElems == LIBTOPK_BLOCK_ELEMS &&
                  kMaxDim == LIBTOPK_MAX_DIM,
              "the kernels' types are the header's");

constexpr int64_t kMaxSlots = (int64_t)1 << 30;
constexpr int64_t kSpan = (int64_t)1 << 60;  // bytes that an array may span

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

// Bytes of what a cache's strides count: an element, or a pair of 4-bit ones.
int unit_size(int dtype) {
  return dtype == LIBTOPK_E4M3 || dtype == LIBTOPK_E2M1 ? 1 : 2;
}
int64_t row_size(int dtype, int64_t dim) {
  return dtype == LIBTOPK_E2M1 ? dim / 2 : dim * unit_size(dtype);
}

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

// Extents of a cache's arrays.
struct CacheRanges {
  Range k{nullptr, 0}, v{nullptr, 0}, table{nullptr, 0}, lens{nullptr, 0};
  Range kb{nullptr, 0}, vb{nullptr, 0};  // scales of 4-bit rows
};

// One of the cache's arrays of rows (or of their scales): strides in units of
// `unit` bytes, rows of `row` bytes; fills in the strides in bytes and the
// extent.  Rows that are written must not share a byte.
bool check_rows(const void* p, const int64_t (&n)[3], const int64_t (&stride)[3],
                int64_t unit, int64_t row, int64_t align, bool written,
                RowStrides* out, Range* extent) {
  int64_t b[3];
  for (int i = 0; i < 3; ++i) {
    if (stride[i] < 0 || stride[i] > kSpan) return false;
    b[i] = stride[i] * unit;
    if (n[i] > 1 && b[i] % align) return false;
  }
  const int64_t len = span(n, b, 3, row);
  if (len < 0 || (written && !apart(n, b, 3, row))) return false;
  if ((n[0] > 0 && !p) || !aligned(p, (uintptr_t)align)) return false;
  *out = RowStrides{b[0], b[1], b[2]};
  *extent = Range(p, len);
  return true;
}

// Checks a cache and fills in what the kernels take of it, and the extents of
// its arrays.
int check_cache(const libtopk_cache_t* c, bool written, CacheParams* p,
                BlockParams* blocks,
                CacheRanges* r) {
  if (!c) return LIBTOPK_ERR_INVALID;
  const bool e2m1 = c->dtype == LIBTOPK_E2M1;
  if (c->dtype != LIBTOPK_BF16 && c->dtype != LIBTOPK_F16 &&
      c->dtype != LIBTOPK_E4M3 && !e2m1)
    return LIBTOPK_ERR_INVALID;
  if (c->batch < 0 || c->heads < 1 || c->heads > 65535 || c->page < 1 ||
      c->dim < 1 || c->dim > LIBTOPK_MAX_DIM ||
      (e2m1 && c->dim % kBlockElems != 0) ||
      row_size(c->dtype, c->dim) % 16 != 0 || c->table_width < 1 ||
      c->pages < 0 || c->pages > INT32_MAX)
    return LIBTOPK_ERR_INVALID;
  if ((int64_t)c->table_width * c->page >= kMaxSlots ||
      (int64_t)c->batch * c->heads > INT32_MAX)
    return LIBTOPK_ERR_INVALID;
  if (c->batch > 1 && (c->table_stride < 0 || c->table_stride > kSpan / 4))
    return LIBTOPK_ERR_INVALID;
  const int64_t n[3] = {c->pages, c->heads, c->page};
  const int64_t ks[3] = {c->k_page_stride, c->k_head_stride, c->k_slot_stride};
  const int64_t vs[3] = {c->v_page_stride, c->v_head_stride, c->v_slot_stride};
  const int64_t unit = unit_size(c->dtype), row = row_size(c->dtype, c->dim);
  if (!check_rows(c->k, n, ks, unit, row, 16, written, &p->ks, &r->k) ||
      !check_rows(c->v, n, vs, unit, row, 16, written, &p->vs, &r->v))
    return LIBTOPK_ERR_INVALID;
  if (e2m1) {  // older callers' structs end before these
    const int64_t kbs[3] = {c->k_block_page_stride, c->k_block_head_stride,
                            c->k_block_slot_stride};
    const int64_t vbs[3] = {c->v_block_page_stride, c->v_block_head_stride,
                            c->v_block_slot_stride};
    blocks->n = c->dim / kBlockElems;
    if (!check_rows(c->k_blocks, n, kbs, 1, blocks->n, 1, written, &blocks->ks,
                    &r->kb) ||
        !check_rows(c->v_blocks, n, vbs, 1, blocks->n, 1, written, &blocks->vs,
                    &r->vb))
      return LIBTOPK_ERR_INVALID;
    blocks->k = (const char*)c->k_blocks;
    blocks->v = (const char*)c->v_blocks;
  }
  if (c->batch > 0 && (!c->table || !c->lens)) return LIBTOPK_ERR_INVALID;
  if (!aligned(c->table, 4) || !aligned(c->lens, 4))
    return LIBTOPK_ERR_INVALID;
  const int64_t tn[1] = {c->batch}, ts[1] = {c->table_stride * 4};
  const int64_t tlen = span(tn, ts, 1, (int64_t)c->table_width * 4);
  if (tlen < 0) return LIBTOPK_ERR_INVALID;
  r->table = Range(c->table, tlen);
  r->lens = Range(c->lens, (int64_t)c->batch * 4);
  p->k = (const char*)c->k;
  p->v = (const char*)c->v;
  p->table = c->table;
  p->table_stride = c->table_stride;
  p->lens = c->lens;
  p->pages = c->pages;
  p->page = make_divisor(c->page);
  p->batch = c->batch;
  p->heads = c->heads;
  p->dim = c->dim;
  p->cap = c->table_width * c->page;
  p->row_bytes = (int32_t)row;
  return LIBTOPK_OK;
}

// An array of a cache's rows, or of their scales: strides and rows in bytes.
struct Rows {
  const char* at;
  RowStrides s;
  int64_t row;
};

// Do two arrays of rows, each with its own apart, share a byte, the second `d`
// bytes behind the first?  Taken axis by axis from the outermost on, which has
// to be the same axis and stride in both (arrays that interleave any other way
// count as shared): of its slices only a few, next to one another, can meet.
bool shared(const int64_t (&n)[3], const Rows& a, const Rows& b, int64_t d,
            unsigned done) {
  const int64_t sa[3] = {a.s.page, a.s.head, a.s.slot};
  const int64_t sb[3] = {b.s.page, b.s.head, b.s.slot};
  int64_t la = a.row, lb = b.row;
  int ia = -1, ib = -1;
  for (int i = 0; i < 3; ++i) {
    if (done >> i & 1 || n[i] < 2) continue;
    la += (n[i] - 1) * sa[i];
    lb += (n[i] - 1) * sb[i];
    if (ia < 0 || sa[i] > sa[ia]) ia = i;
    if (ib < 0 || sb[i] > sb[ib]) ib = i;
  }
  if (d >= la || d + lb <= 0) return false;
  if (ia < 0 || ia != ib || sa[ia] != sb[ia]) return true;
  // Slice i + k of b against slice i of a: d + k s behind it.
  const int64_t s = sa[ia], most = n[ia] - 1;
  la -= most * s;
  lb -= most * s;
  int64_t k = -(d + lb) / s - 1, last = (la - d) / s + 1;
  if (k < -most) k = -most;
  if (last > most) last = most;
  for (; k <= last; ++k)
    if (shared(n, a, b, d + k * s, done | 1u << ia)) return true;
  return false;
}

// Are the arrays that a call writes to arrays of their own?  They may
// interleave.  With `twins` k and v, and so their scales, may be one array.
bool distinct(const CacheParams& c, const BlockParams& s, bool e2m1,
              bool twins) {
  const int64_t n[3] = {c.pages, c.heads, c.page.d};
  if (c.pages < 1) return true;
  const Rows x[4] = {{c.k, c.ks, c.row_bytes},
                     {c.v, c.vs, c.row_bytes},
                     {s.k, s.ks, s.n},
                     {s.v, s.vs, s.n}};
  auto same = [&](const Rows& a, const Rows& b) {
    return a.at == b.at && (n[0] < 2 || a.s.page == b.s.page) &&
           (n[1] < 2 || a.s.head == b.s.head) &&
           (n[2] < 2 || a.s.slot == b.s.slot);
  };
  twins = twins && same(x[0], x[1]) && (!e2m1 || same(x[2], x[3]));
  for (int i = 1; i < (e2m1 ? 4 : 2); ++i)
    for (int j = 0; j < i; ++j)
      if (!(twins && i == j + 1 && j != 1) &&
          shared(n, x[j], x[i], (int64_t)((uintptr_t)x[i].at -
                                          (uintptr_t)x[j].at), 0))
        return false;
  return true;
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
  if (c == kE2m1)
    return q == kBf16 ? attend_fn_dim<kBf16, kE2m1>(dim, pg16, heads, n)
                      : attend_fn_dim<kF16, kE2m1>(dim, pg16, heads, n);
  if (q == kBf16)
    return c == kE4m3 ? attend_fn_dim<kBf16, kE4m3>(dim, pg16, heads, n)
                      : attend_fn_dim<kBf16, kBf16>(dim, pg16, heads, n);
  return c == kE4m3 ? attend_fn_dim<kF16, kE4m3>(dim, pg16, heads, n)
                    : attend_fn_dim<kF16, kF16>(dim, pg16, heads, n);
}

template <int Q, int C>
const void* extend_fn_dim(int dim, int* lanes) {
  *lanes = dim <= 64 ? 8 : dim <= 128 ? 16 : 32;
  return dim <= 64    ? (const void*)&extend_kernel<Q, C, 8>
         : dim <= 128 ? (const void*)&extend_kernel<Q, C, 16>
                      : (const void*)&extend_kernel<Q, C, 32>;
}
// Lanes of a row, and the kernel, for inputs of type q and a cache of type c
// (q's own or a narrower one).
const void* extend_fn(int q, int c, int dim, int* lanes) {
  if (q == kBf16)
    return c == kE2m1   ? extend_fn_dim<kBf16, kE2m1>(dim, lanes)
           : c == kE4m3 ? extend_fn_dim<kBf16, kE4m3>(dim, lanes)
                        : extend_fn_dim<kBf16, kBf16>(dim, lanes);
  return c == kE2m1   ? extend_fn_dim<kF16, kE2m1>(dim, lanes)
         : c == kE4m3 ? extend_fn_dim<kF16, kE4m3>(dim, lanes)
                      : extend_fn_dim<kF16, kF16>(dim, lanes);
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
  Attend4Params p = {};
  CacheRanges at;
  Range w(nullptr, 0), pos(nullptr, 0);
  int rc = check_cache(cache, false, &p.c, &p.s, &at);
  if (rc != LIBTOPK_OK) return rc;
  if (q_dtype != LIBTOPK_BF16 && q_dtype != LIBTOPK_F16)
    return LIBTOPK_ERR_INVALID;
  if (cache->dtype != LIBTOPK_E4M3 && cache->dtype != LIBTOPK_E2M1 &&
      cache->dtype != q_dtype)
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
  const Range ins[9] = {Range(q, qlen), at.k, at.v, at.table, at.lens,
                        Range(k_scale, k_scale ? cache->heads * 4 : 0),
                        Range(v_scale, v_scale ? cache->heads * 4 : 0),
                        at.kb, at.vb};
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
  if (cache->dtype == kE2m1) {
    // 4-bit rows cost their widening rather than their bytes, so a share's
    // cost in tiles stops growing with shorter rows, and halves of a row are
    // worth joining sooner.  (7 sequences of up to 1777 slots, 12 heads of 64
    // elements: 19.1 us as for rows of their bytes, 16.9 us so; 48 of up to
    // 8000 slots, 8 heads of 128: 80 us at 32, 88 at 16, 84 at 64.  These two
    // are what it was measured by: 32 is the best of the powers of two there.)
    if (p.row_cost > 32) p.row_cost = 32;
    p.min_tiles = kMinTiles / 2;
  }
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
  const dim3 blocks((unsigned)grid);
  const AttendParams& base = p;
  rc = cache->dtype == LIBTOPK_E2M1
           ? launch(fn, blocks, needs.threads, p, s, lds)
           : launch(fn, blocks, needs.threads, base, s, lds);
  if (rc != LIBTOPK_OK || !ledger || p.direct) return rc;
  const int64_t wrows = (int64_t)cache->batch * cache->heads;
  // Few rows: workgroups enough to share out the joining, too.
  int64_t chunks = (p.c.cap + kWeightSlots - 1) / kWeightSlots;
  const int64_t joiners = 1024 / wrows < kJoiners ? 1024 / wrows : kJoiners;
  if (chunks < joiners) chunks = joiners;
  return launch((const void*)&attend_join_kernel,
                dim3((unsigned)chunks,
                     (unsigned)(wrows < 65535 ? wrows : 65535)),
                kBlock, base, s);
}

int cache_append(const libtopk_cache_t* cache, const void* k_new,
                 const void* v_new, int64_t new_batch_stride,
                 int64_t new_head_stride, int32_t limit, const int32_t* seen,
                 const libtopk_ledger_t* ledger, int32_t sinks, int32_t recent,
                 int32_t* out_lens, int32_t* out_slots,
                 libtopk_stream_t stream) {
  SlotsParams p = {};
  BlockParams none = {};
  CacheRanges at;
  Range w(nullptr, 0), pos(nullptr, 0);
  int rc = check_cache(cache, true, &p.c, &none, &at);
  if (rc != LIBTOPK_OK) return rc;
  if (cache->dtype == LIBTOPK_E2M1) return LIBTOPK_ERR_INVALID;
  rc = check_ledger(ledger, cache->batch, cache->heads, true, true, &p.w, &w,
                    &pos);
  if (rc != LIBTOPK_OK) return rc;
  if (limit < 1 || sinks < 0 || recent < 0) return LIBTOPK_ERR_INVALID;
  const int es = unit_size(cache->dtype);
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
                         Range(out_slots, rows * 4), w, pos, at.k, at.v};
  const Range ins[5] = {Range(k_new, nlen), Range(v_new, nlen), at.table,
                        at.lens, Range(seen, (int64_t)cache->batch * 4)};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : ins)
      if (outs[i].meets(r)) return LIBTOPK_ERR_INVALID;
    // k and v may interleave (one array of pages that holds both)
    for (int j = 0; j < i; ++j)
      if (!(i == 5 && j == 4) && outs[i].meets(outs[j]))
        return LIBTOPK_ERR_INVALID;
  }
  if (!distinct(p.c, none, false, k_new == v_new)) return LIBTOPK_ERR_INVALID;
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
  Slots4Params all = {};
  SlotsParams& p = all;
  CacheRanges at;
  Range w(nullptr, 0), pos(nullptr, 0), w2(nullptr, 0), pos2(nullptr, 0);
  int rc = check_cache(cache, true, &p.c, &all.s, &at);
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
  const Range outs[7] = {Range(out_lens, (int64_t)cache->batch * 4), w2, pos2,
                         at.k, at.v, at.kb, at.vb};
  const Range ins[5] = {w, pos, at.table, at.lens,
                        Range(seen, (int64_t)cache->batch * 4)};
  for (int i = 0; i < 7; ++i) {
    for (const Range& r : ins)
      if (outs[i].meets(r)) return LIBTOPK_ERR_INVALID;
    // the cache's own arrays may interleave
    for (int j = 0; j < (i < 3 ? i : 3); ++j)
      if (outs[i].meets(outs[j])) return LIBTOPK_ERR_INVALID;
  }
  if (!distinct(p.c, all.s, cache->dtype == LIBTOPK_E2M1, true))
    return LIBTOPK_ERR_INVALID;
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
  char* area = work.base;
  p.pairs = (int32_t*)area;
  p.moves = (int32_t*)(area += pair_bytes);
  p.hist = (uint32_t*)(area += move_bytes);
  p.counts = (int4*)(area += hist_words * 8);
  p.state = (int2*)(area += count_bytes);
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
  const dim3 grid((unsigned)((units + kBlock - 1) / kBlock),
                  (unsigned)(rows < 65535 ? rows : 65535));
  return cache->dtype == LIBTOPK_E2M1
             ? launch((const void*)&evict_move_kernel<true>, grid, kBlock, all,
                      s)
             : launch((const void*)&evict_move_kernel<false>, grid, kBlock, p,
                      s);
}

int cache_extend(const libtopk_cache_t* cache, const libtopk_tokens_t* tokens,
                 const libtopk_ledger_t* ledger, int32_t* out_lens,
                 libtopk_stream_t stream) {
  ExtendParams p = {};
  CacheRanges at;
  Range w(nullptr, 0), pos(nullptr, 0);
  int rc = check_cache(cache, true, &p.c, &p.s, &at);
  if (rc != LIBTOPK_OK) return rc;
  if (ledger) {
    rc = check_ledger(ledger, cache->batch, cache->heads, true, true, &p.w, &w,
                      &pos);
    if (rc != LIBTOPK_OK) return rc;
    if (ledger->slots < p.c.cap) p.c.cap = ledger->slots;
  }
  if (!tokens) return LIBTOPK_ERR_INVALID;
  const libtopk_tokens_t& t = *tokens;
  if ((t.dtype != LIBTOPK_BF16 && t.dtype != LIBTOPK_F16) ||
      (cache->dtype != t.dtype && cache->dtype != LIBTOPK_E4M3 &&
       cache->dtype != LIBTOPK_E2M1))
    return LIBTOPK_ERR_INVALID;
  const int32_t dim = cache->dim, q_heads = t.q ? t.q_heads : 0;
  if (t.tokens < 0 || (t.q && t.q_heads < 1) || dim % kUnit != 0 ||
      t.rot < 0 || t.rot > dim || t.rot % 16 != 0)
    return LIBTOPK_ERR_INVALID;
  if ((t.q_norm || t.k_norm) &&
      ((t.norm_dtype != LIBTOPK_F32 && t.norm_dtype != t.dtype) ||
       !(t.eps >= 0.0f)))
    return LIBTOPK_ERR_INVALID;
  const int norm_bytes = t.norm_dtype == LIBTOPK_F32 ? 4 : 2;
  if (!aligned(t.q_norm, (uintptr_t)norm_bytes) ||
      !aligned(t.k_norm, (uintptr_t)norm_bytes) || !aligned(t.freqs, 4) ||
      !aligned(t.k_scale, 4) || !aligned(t.v_scale, 4) ||
      !aligned(t.starts, 4) || !aligned(t.seen, 4) || !aligned(out_lens, 4) ||
      (t.rot > 0 && !t.freqs))
    return LIBTOPK_ERR_INVALID;
  // Rows of the new tokens' arrays: [tokens][heads][dim].
  auto extent = [&](const void* x, int64_t heads, int64_t ts, int64_t hs,
                    bool written, int64_t (&bytes)[2], Range* r) {
    if (ts < 0 || hs < 0 || ts > kSpan || hs > kSpan ||
        (t.tokens > 1 && ts % 8) || (heads > 1 && hs % 8))
      return false;
    const int64_t n[2] = {t.tokens, heads};
    bytes[0] = ts * 2;
    bytes[1] = hs * 2;
    const int64_t len = span(n, bytes, 2, (int64_t)dim * 2);
    if (len < 0 || (len > 0 && !x) || !aligned(x, 16)) return false;
    if (written && len > 0 && !apart(n, bytes, 2, (int64_t)dim * 2))
      return false;
    *r = Range(x, len);
    return true;
  };
  Range q(nullptr, 0), k(nullptr, 0), v(nullptr, 0), out(nullptr, 0);
  int64_t qs[2] = {0, 0}, ks[2], vs[2], os[2] = {0, 0};
  if (!extent(t.k, cache->heads, t.k_token_stride, t.k_head_stride, false, ks,
              &k) ||
      !extent(t.v, cache->heads, t.v_token_stride, t.v_head_stride, false, vs,
              &v) ||
      (t.q &&
       (!extent(t.q, q_heads, t.q_token_stride, t.q_head_stride, false, qs,
                &q) ||
        !extent(t.q_out, q_heads, t.q_out_token_stride, t.q_out_head_stride,
                true, os, &out))))
    return LIBTOPK_ERR_INVALID;
  const bool rest = t.q && t.rest != 0;
  if (cache->batch == 0 && !(rest && t.tokens > 0)) return LIBTOPK_OK;
  if (cache->batch > 0 && (!t.starts || !out_lens)) return LIBTOPK_ERR_INVALID;
  // Queries may be turned where they are, also between the keys and values
  // of one array: with the same stride from token to token, a token's rows of
  // the two lie apart within it.
  const bool same = t.q && t.q == t.q_out && qs[0] == os[0] && qs[1] == os[1];
  auto beside = [&](const void* x, int64_t heads, const int64_t (&s)[2]) {
    if (!same || s[0] != os[0] || t.tokens < 1) return false;
    const int64_t mine = (q_heads - 1) * os[1] + (int64_t)dim * 2;
    const int64_t its = (heads - 1) * s[1] + (int64_t)dim * 2;
    if (t.tokens == 1 || s[0] < 1) return false;
    const uintptr_t a = (uintptr_t)t.q_out, b = (uintptr_t)x;
    const int64_t d = b >= a ? (int64_t)((b - a) % (uintptr_t)s[0])
                             : (s[0] - (int64_t)((a - b) % (uintptr_t)s[0])) %
                                   s[0];
    return d >= mine && d + its <= s[0];
  };
  const bool beside_k = beside(t.k, cache->heads, ks);
  const bool beside_v = beside(t.v, cache->heads, vs);
  const int64_t batch = cache->batch;
  const Range outs[8] = {Range(out_lens, batch * 4), out, w, pos, at.k, at.v,
                         at.kb, at.vb};
  const Range ins[12] = {
      q, k, v, at.table, at.lens,
      Range(t.starts, t.starts ? (batch + 1) * 4 : 0),
      Range(t.seen, t.seen ? batch * 4 : 0),
      Range(t.q_norm, t.q_norm ? (int64_t)dim * norm_bytes : 0),
      Range(t.k_norm, t.k_norm ? (int64_t)dim * norm_bytes : 0),
      Range(t.freqs, t.freqs ? (int64_t)t.rot / 2 * 4 : 0),
      Range(t.k_scale, t.k_scale ? (int64_t)cache->heads * 4 : 0),
      Range(t.v_scale, t.v_scale ? (int64_t)cache->heads * 4 : 0)};
  for (int i = 0; i < 8; ++i) {
    for (int j = 0; j < 12; ++j)
      if (!(i == 1 && ((same && j == 0) || (beside_k && j == 1) ||
                       (beside_v && j == 2))) &&
          outs[i].meets(ins[j]))
        return LIBTOPK_ERR_INVALID;
    // the cache's own arrays may interleave
    for (int j = 0; j < (i < 4 ? i : 4); ++j)
      if (outs[i].meets(outs[j])) return LIBTOPK_ERR_INVALID;
  }
  if (!distinct(p.c, p.s, cache->dtype == LIBTOPK_E2M1, false))
    return LIBTOPK_ERR_INVALID;
  p.q = (const char*)t.q;
  p.k = (const char*)t.k;
  p.v = (const char*)t.v;
  p.q_out = (char*)t.q_out;
  p.qt = qs[0];
  p.qh = qs[1];
  p.kt = ks[0];
  p.kh = ks[1];
  p.vt = vs[0];
  p.vh = vs[1];
  p.ot = os[0];
  p.oh = os[1];
  p.starts = t.starts;
  p.seen = t.seen;
  p.q_norm = t.q ? t.q_norm : nullptr;
  p.k_norm = t.k_norm;
  p.freqs = t.freqs;
  p.k_scale = t.k_scale;
  p.v_scale = t.v_scale;
  p.out_lens = out_lens;
  p.tokens = t.tokens;
  p.q_heads = q_heads;
  p.norm_type = t.norm_dtype;
  p.half = t.rot / 2;
  p.interleaved = t.interleaved != 0;
  p.rest = rest;
  p.eps = t.eps;
  p.inv_dim = 1.0 / dim;
  int dev = 0;
  rc = current_device(&dev);
  if (rc != LIBTOPK_OK) return rc;
  int lanes = 0;
  const void* fn = extend_fn(t.dtype, cache->dtype, dim, &lanes);
  const int64_t each = kWave / lanes;  // rows at a time
  const int64_t groups = (q_heads + each - 1) / each +
                         2 * ((cache->heads + each - 1) / each);
  int units = 0;
  rc = units_of(dev, &units);
  if (rc != LIBTOPK_OK) return rc;
  // Few tokens are dealt out row by row, to 16 waves a unit.
  int64_t splits = 1;
  if (t.tokens > 0) {
    splits = ((int64_t)units * 16 + t.tokens - 1) / t.tokens;
    if (splits > groups) splits = groups;
  }
  p.splits = (int32_t)splits;
  int64_t grid = ((int64_t)t.tokens * splits + kWaves - 1) / kWaves;
  const int64_t least = (batch + kBlock - 1) / kBlock;
  if (grid < least) grid = least;
  if (!launchable(grid, kBlock)) return LIBTOPK_ERR_INVALID;
  return launch(fn, dim3((unsigned)grid), kBlock, p, (hipStream_t)stream);
}

}  // extern "C"
