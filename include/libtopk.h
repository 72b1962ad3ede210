/*
 * libtopk — two-stage parallel reduction and Top-K selection over int32
 * arrays on AMD Instinct MI355X (gfx950).  C ABI, no C++ or PyTorch types.
 *
 * Sources (the pages the method is taken from):
 *   [TopK]   "CUDA并行优化实战：从TopK问题剖析共享内存与规约算法设计"
 *            (CUDA optimisation in practice: shared memory and reduction
 *            design through the TopK problem)
 *   [Reduce] "CUDA归约优化完全指南：从入门到精通"
 *            (A complete guide to CUDA reduction optimisation)
 *
 * Common conventions
 * ------------------
 *  - `in`, `out` and `out_i64` are DEVICE pointers on the calling thread's
 *    current HIP device.  They are owned by the caller; the library never
 *    frees or retains them.  `in` must be 4-byte aligned (16-byte alignment
 *    takes the fastest path; otherwise up to three leading elements are
 *    peeled).  `in` and the output must not overlap.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Both calls are
 *    asynchronous and stream-ordered: they return once the work is enqueued
 *    and never synchronise the host.  The result is valid once the stream
 *    reaches the call; `in` must stay alive and unmodified until then.
 *  - Arguments are validated before anything is enqueued; on any error
 *    nothing is launched and the output is untouched.  Launch and
 *    allocation failures are reported as LIBTOPK_ERR_HIP / _NOMEM; a fault
 *    inside a kernel surfaces at the caller's next synchronisation.
 *  - The library owns a small scratch area per (device, stream), about
 *    1.6 MiB: per-block candidates (1.5 MiB, int32 and key-value), partial
 *    results, histogram counters and tickets; the first topk_i32 call with
 *    k > LIBTOPK_MAX_K on the pair adds a 16 MiB candidate buffer (and
 *    64 KiB for sample lists).  It is
 *    allocated by the
 *    first call on that pair (so do that first call before capturing the
 *    stream into a HIP graph), kept for reuse, and freed by
 *    libtopk_release() or at process exit.  No per-call clearing is
 *    enqueued: the words that the workgroups of one launch count into
 *    (completion tickets, histogram counters) carry that launch's epoch,
 *    so no result depends on what an earlier call, finished or not, left
 *    in the scratch.
 *  - Calls on different streams may run concurrently.  Thread-safe: a call's
 *    launches follow one another on its stream, also when other host threads
 *    call on it.
 *  - No C++ exception crosses this interface.  The library prints nothing
 *    unless LIBTOPK_DEBUG is set in the environment (then HIP failures are
 *    described on stderr).
 */
#ifndef LIBTOPK_H
#define LIBTOPK_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Layout-compatible with HIP's hipStream_t (a pointer to struct
 * ihipStream_t); callers may pass a hipStream_t directly. */
struct ihipStream_t;
typedef struct ihipStream_t *libtopk_stream_t;

/* Status codes returned by every entry point. */
enum {
    LIBTOPK_OK = 0,
    LIBTOPK_ERR_INVALID = 1,     /* bad pointer, size, k or op            */
    LIBTOPK_ERR_UNSUPPORTED = 2, /* k above the call's supported maximum  */
    LIBTOPK_ERR_NOMEM = 3,       /* scratch allocation failed             */
    LIBTOPK_ERR_HIP = 4          /* no device, or a HIP call / launch failed */
};

/* Reduction operators for reduce_i32. */
enum { LIBTOPK_SUM = 0, LIBTOPK_MAX = 1, LIBTOPK_MIN = 2 };

/* Largest k of every top-k entry point (the register-list path). */
#define LIBTOPK_MAX_K 128

/* Largest k of topk_i32, which takes k above LIBTOPK_MAX_K through radix
 * selection. */
#define LIBTOPK_MAX_K_SELECT 16384

/* Most bins of histogram_i32. */
#define LIBTOPK_MAX_BINS 4096

/*
 * topk_i32 — the k largest values of in[0..n), written to out[0..k) in
 * descending order, duplicates kept with their multiplicity.
 *
 * Operation: [TopK] §1 (find the 20 largest of 1e8 values) and §2 (the
 * two-stage design: §2.1 each thread keeps a descending local top-k list
 * over a grid-stride share of the input, and the block merges the lists;
 * §2.2 a second, single-block stage merges the per-block candidates; the
 * result must be identical to the CPU's).  For k <= LIBTOPK_MAX_K both
 * stages run in one launch: the last workgroup to finish stage 1 performs
 * stage 2.  Larger k, up to LIBTOPK_MAX_K_SELECT, goes through radix
 * selection ("GPU基数排序优化：10亿级数据处理与性能调优" §3.2–3.3: 8-bit digit
 * histograms kept per warp in shared memory): four digit passes find the
 * k-th largest value, a gather pass collects the values above it, and one
 * workgroup sorts the k results.  Once a digit leaves fewer than 2^22
 * candidates they are copied aside and the remaining passes read only
 * them.  From n = 2^18 on (when n is large enough for k), a sample first
 * fixes a threshold and a filter pass copies the values above it aside;
 * when that copy is small (the usual case) one workgroup selects the
 * top-k from it, the digit passes return at once, and the input is read
 * once.  Six stream-ordered launches, eight on sampled inputs.
 *
 *   in   device, int32[n], read once (k <= LIBTOPK_MAX_K)
 *   n    number of elements, 1 <= n <= 2^32
 *   k    1 <= k <= min(n, LIBTOPK_MAX_K_SELECT)
 *   out  device, int32[k], written in full
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, n out of
 * range, k < 1 or k > n; LIBTOPK_ERR_UNSUPPORTED for
 * k > LIBTOPK_MAX_K_SELECT.
 */
int topk_i32(const int32_t *in, int64_t n, int32_t k, int32_t *out,
             libtopk_stream_t stream);

/* Bytes of the fixed device array behind topk_i32_noalloc (528 KiB). */
#define LIBTOPK_NOALLOC_SCRATCH_BYTES 540672

/*
 * topk_i32_noalloc — topk_i32 for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, and harnesses
 * that forbid hipMalloc.  Same operation, arguments, output and errors as
 * topk_i32 for k <= LIBTOPK_MAX_K (one launch), but the call never
 * allocates: no hipMalloc, hipFree or allocating library routine.  Its
 * scratch (stage-1 candidates, block maxima and completion tickets) is a
 * fixed array of LIBTOPK_NOALLOC_SCRATCH_BYTES in the library's device
 * memory, one per device, held until the process ends; it is sized for
 * every k <= LIBTOPK_MAX_K and every n <= 2^32.  The first call on a device
 * looks up the array's address and clears its tickets with a small kernel
 * on `stream` (no allocation).
 *
 * Every call on one device shares that device's array, which keeps the
 * last call's contents: calls that overlap on one device (different
 * streams, or different host threads) race and give wrong results; order
 * them on one stream or otherwise.
 *
 *   in, n, out, stream   as for topk_i32
 *   k    1 <= k <= min(n, LIBTOPK_MAX_K)
 *
 * Errors: as topk_i32; k > LIBTOPK_MAX_K returns LIBTOPK_ERR_UNSUPPORTED
 * (radix selection needs megabytes of candidate space, not in the array).
 */
int topk_i32_noalloc(const int32_t *in, int64_t n, int32_t k, int32_t *out,
                     libtopk_stream_t stream);

/*
 * reduce_i32 — fold in[0..n) with one operator into a single int64.
 *
 * Operation: [Reduce] "Basic concepts" (a reduction combines every element
 * through one binary operation into one result; the worked example sums
 * [1..8] to 36) and the "complete multi-level reduction" driver (a first
 * pass leaves one partial per block, a further pass combines them).  Here
 * exactly two stages run in one launch: per-block partials, then the last
 * workgroup to finish combines them.
 *
 *   in       device, int32[n] (may be NULL when n == 0)
 *   n        0 <= n <= 2^32
 *   op       LIBTOPK_SUM: exact int64 sum (cannot overflow for n <= 2^32);
 *            LIBTOPK_MAX / LIBTOPK_MIN: the extreme value, sign-extended.
 *            n == 0 yields the identity: 0, INT32_MIN or INT32_MAX.
 *   out_i64  device, int64[1]
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, n out of
 * range or an unknown op.
 */
int reduce_i32(const int32_t *in, int64_t n, int32_t op, int64_t *out_i64,
               libtopk_stream_t stream);

/*
 * topk_kv_i32 / topk_kv_f32 — the k largest elements of in[0..n) with their
 * positions: out_values[i] and out_indices[i] for i < k, ordered by value,
 * descending, and among equal values by position, ascending (the earlier
 * element first), so the result is unique.
 *
 * Operation: [TopK] §6 (the reduction keeps a candidate list of items
 * ordered by their score) with [TopK] §2's two stages, and "GPU基数排序优化：
 * 10亿级数据处理与性能调优" §8 (key-value pairs carried together; float keys
 * through a bit transform).  Float order: the order-preserving map of the
 * bits to unsigned integers (negative: all bits flipped; otherwise the sign
 * bit set): numerical order on numbers, -0 below +0, positive NaNs above
 * +infinity, negative NaNs below -infinity.  One launch, as topk_i32.
 *
 *   in           device, int32[n] or float32[n], read once
 *   n            1 <= n < 2^32 (positions must fit 32 bits)
 *   k            1 <= k <= min(n, LIBTOPK_MAX_K)
 *   out_values   device, int32[k] / float32[k] (the input's own bits)
 *   out_indices  device, int64[k], positions in [0, n)
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer (out_indices
 * 8-byte aligned), n out of range, k < 1 or k > n, or overlapping buffers;
 * LIBTOPK_ERR_UNSUPPORTED for k > LIBTOPK_MAX_K.
 */
int topk_kv_i32(const int32_t *in, int64_t n, int32_t k, int32_t *out_values,
                int64_t *out_indices, libtopk_stream_t stream);
int topk_kv_f32(const float *in, int64_t n, int32_t k, float *out_values,
                int64_t *out_indices, libtopk_stream_t stream);

/*
 * reduce_stats_i32 — count, sum, max, min and sum of squares of in[0..n),
 * all from one read of the data.
 *
 * Operation: [TopK] §6 (the two-stage reduction also serves large-scale
 * statistics such as the mean and the variance) and [Reduce] "Basic
 * concepts" (each statistic is a fold through one binary operator).  Mean
 * and population variance follow from the result: sum / count and
 * (count * sumsq - sum^2) / count^2.  Two stages in one launch, as
 * reduce_i32.
 *
 *   in       device, int32[n] (may be NULL when n == 0)
 *   n        0 <= n <= 2^32
 *   out      device, int64[6], written in full:
 *              out[0]  count = n
 *              out[1]  exact sum (int64; cannot overflow for n <= 2^32)
 *              out[2]  max, sign-extended (INT32_MIN when n == 0)
 *              out[3]  min, sign-extended (INT32_MAX when n == 0)
 *              out[4]  sum of squares, low 64 bits  } one unsigned 128-bit
 *              out[5]  sum of squares, high 64 bits } integer, exact
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer (out must be
 * 8-byte aligned), n out of range, or overlapping in and out.
 */
int reduce_stats_i32(const int32_t *in, int64_t n, int64_t *out,
                     libtopk_stream_t stream);

/*
 * topk_batched_i32 — the top-k of every row of a row-major int32 matrix:
 * out[r * k + i], i < k, is the i-th largest value of row r, which is
 * in[r * ld .. r * ld + cols); each row's k values in descending order,
 * duplicates kept.
 *
 * Operation: [TopK] §6 (the two-stage pattern as a building block, e.g.
 * candidate selection per user in a recommender) with [TopK] §2's two
 * stages per row.  Long rows get several workgroups each and the last of a
 * row's workgroups merges its candidates; rows of up to 4096 elements are
 * handled one wave per row.
 *
 *   in    device, int32, rows of `cols` elements `ld` elements apart;
 *         elements between cols and ld of a row are never read
 *   rows  0 <= rows (0: nothing is enqueued and LIBTOPK_OK is returned
 *         once cols, ld and k are valid; in and out may then be NULL)
 *   cols  1 <= cols <= 2^32
 *   ld    row stride in elements, ld >= cols (any value: rows need not be
 *         16-byte aligned)
 *   k     1 <= k <= min(cols, LIBTOPK_MAX_K)
 *   out   device, int32[rows * k], written in full
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, rows < 0,
 * cols or ld out of range, k < 1 or k > cols, an input span beyond 2^60
 * elements, or overlapping input and output; LIBTOPK_ERR_UNSUPPORTED for
 * k > LIBTOPK_MAX_K.
 */
int topk_batched_i32(const int32_t *in, int64_t rows, int64_t cols,
                     int64_t ld, int32_t k, int32_t *out,
                     libtopk_stream_t stream);

/*
 * topk_merge_i32 — merge several top-k results: the k largest values of the
 * union of m lists, written to out[0..k) in descending order.
 *
 * Operation: [TopK] §6 (several TopK results merged again) and §2.2 (the
 * second stage merges per-block top-k lists into the final one).  Only the
 * first min(len, k) entries of a list are read, plus what the merge needs
 * to bound the result.  Typical inputs: the outputs of topk_i32 on shards
 * of one array (the merge of the shards' top-k lists is the top-k of the
 * whole), or the rows written by topk_batched_i32.
 *
 *   lists  device, int32[m * len], list j at lists + j * len; every list
 *          MUST be in descending order (as the top-k calls write them).
 *          The library does not check this; on a list out of order the
 *          result is unspecified (nothing is read outside lists[]).
 *   m      1 <= m <= 2^20 lists
 *   len    entries per list, len >= 1
 *   k      1 <= k <= min(m * len, LIBTOPK_MAX_K)
 *   out    device, int32[k], written in full
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, m or len
 * out of range, k < 1 or k > m * len, or overlapping lists and out;
 * LIBTOPK_ERR_UNSUPPORTED for k > LIBTOPK_MAX_K.
 */
int topk_merge_i32(const int32_t *lists, int64_t m, int32_t len, int32_t k,
                   int32_t *out, libtopk_stream_t stream);

/*
 * topk_segmented_i32 — the top-k of every segment of one array, segments
 * of any lengths given by offsets: segment s is
 * in[offsets[s] .. offsets[s + 1]), and out[s * k + i], i < min(k, len_s),
 * is its i-th largest value (descending, duplicates kept).  A segment
 * shorter than k (empty included) fills the rest of its k slots with
 * INT32_MIN; counts[s] = min(k, len_s) tells that padding from real
 * INT32_MIN values.
 *
 * Operation: [TopK] §6 (the two-stage pattern as a building block, e.g.
 * candidate selection per user, whose candidate lists differ in length;
 * several TopK results merged again) with [TopK] §2's two stages per
 * segment.  Two launches on `stream`: one wave per segment finishes
 * segments of up to 4096 elements in registers and plans the rest on the
 * device; persistent workgroups then stream the longer segments (a
 * segment above 2^16 elements in up to 1024 parts, whose candidates the
 * last part to finish merges).
 *
 *   in       device, int32[n] (may be NULL when n == 0)
 *   n        elements of in, 0 <= n <= 2^32
 *   offsets  device, int64[nseg + 1], 8-byte aligned; the caller promises
 *            0 <= offsets[0] <= offsets[1] <= ... <= offsets[nseg] <= n.
 *            The library does not check this (the offsets live on the
 *            device); with offsets that break it the results are
 *            unspecified, but nothing outside in[0..n), out and counts is
 *            read or written.
 *   nseg     0 <= nseg < 2^31 (0: nothing is enqueued, LIBTOPK_OK once k
 *            is valid; the pointers may then be NULL)
 *   k        1 <= k <= LIBTOPK_MAX_K
 *   out      device, int32[nseg * k], written in full
 *   counts   device, int32[nseg], or NULL when not wanted
 *
 * Scratch: besides the per-stream area, about 0.6 KiB per 1,000 elements
 * of n (lists and the parts' candidates), allocated on the first call with
 * a larger n on the stream (which then synchronises the stream once).
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, n or nseg
 * out of range, k < 1, or overlapping buffers; LIBTOPK_ERR_UNSUPPORTED for
 * k > LIBTOPK_MAX_K.
 */
int topk_segmented_i32(const int32_t *in, int64_t n, const int64_t *offsets,
                       int64_t nseg, int32_t k, int32_t *out, int32_t *counts,
                       libtopk_stream_t stream);

/*
 * histogram_i32 — counts of the values of in[0..n) in nbins equal bins:
 * out[b] = the number of elements v with
 *     lo + b * 2^shift <= v <= lo + (b + 1) * 2^shift - 1
 * (bounds taken in exact integer arithmetic); values outside all bins are
 * not counted.
 *
 * Operation: [TopK] §6 (histogram computation as a use of the two-stage
 * reduction) and "GPU基数排序优化：10亿级数据处理与性能调优" §3.3 (one
 * shared-memory histogram per warp, merged at the end, rather than global
 * atomics per element).  One launch: per-wave histograms in LDS, per-block
 * totals added into device counters, and the last workgroup to finish
 * writes the result and clears the counters.
 *
 *   in     device, int32[n] (may be NULL when n == 0)
 *   n      0 <= n <= 2^32
 *   lo     the first bin's lowest value (any int32)
 *   shift  bin width 2^shift, 0 <= shift <= 31
 *   nbins  1 <= nbins <= LIBTOPK_MAX_BINS
 *   out    device, int64[nbins], 8-byte aligned, written in full
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, n, shift
 * or nbins out of range, or overlapping in and out.
 */
int histogram_i32(const int32_t *in, int64_t n, int32_t lo, int32_t shift,
                  int32_t nbins, int64_t *out, libtopk_stream_t stream);

/* ---------------------------------------------------------------------------
 * Operators on a paged key-value cache of a decoder: attention of one new
 * token, append, eviction by accumulated attention weight, and extension by
 * new tokens.
 *
 * The cache holds K and V rows of `dim` elements in pages of `page` slots.
 * Sequence b's slot t (0 <= t < lens[b]) of head h is the row at
 *
 *     k + table[b * table_stride + t / page] * k_page_stride
 *       + h * k_head_stride + (t % page) * k_slot_stride      (elements)
 *
 * and likewise in v, so both orders within a page (heads outside slots, or
 * slots outside heads) and any padding are strides.  `lens` and `table` are
 * read on the device: no call needs a length on the host.
 *
 *  - A length is read as if clamped to [0, table_width * page] (and to the
 *    slots of the ledger, where a call takes one).
 *  - A table entry outside [0, pages) names no page.  Attention leaves its
 *    slots out (score -infinity, weight unchanged), append and evict neither
 *    read nor write rows there.  Nothing outside the given arrays is ever
 *    read or written.
 *  - Pages that append, evict or extend write to must belong to one sequence
 *    alone; attention may share them.  For these calls each axis of k, and of v,
 *    steps over all that the axes within it span (no stride of 0), and no two
 *    of k, v and their scales share a byte.  They may interleave: from the
 *    outermost axis to the one within which they lie side by side, both then
 *    have the same axis and stride.  (In evict, and in append with one array
 *    of new rows, k and v may be one array.)
 *
 * Workspace: per (device, stream), grown on demand by doubling; an area is
 * kept until cache_release() (or process exit) once it has been used, so a
 * captured graph that uses it stays valid.  Under stream capture nothing is
 * allocated: a call that needs a larger area then returns LIBTOPK_ERR_NOMEM,
 * so make one call of the same sizes on the stream before capturing it.  A
 * captured graph uses the workspace of the stream that it was captured on:
 * its replays must not overlap with calls on that stream, nor with replays of
 * other graphs that were captured on it.
 * ------------------------------------------------------------------------ */

/* Element types of queries and cache rows. */
enum {
    LIBTOPK_BF16 = 0,
    LIBTOPK_F16 = 1,
    LIBTOPK_E4M3 = 2, /* 8-bit float, 4 exponent bits, no infinity; cache only */
    LIBTOPK_F32 = 3,  /* logits and norm weights only */
    LIBTOPK_E2M1 = 4  /* 4-bit float (0 .5 1 1.5 2 3 4 6 and their negatives),
                         cache only: two to a byte, the even element in the low
                         half, and a scale 2^(byte - 127) for each
                         LIBTOPK_BLOCK_ELEMS of a row (255: NaN) */
};

/* Elements of a 4-bit row that share a scale. */
#define LIBTOPK_BLOCK_ELEMS 32

/* Largest row length of a cache. */
#define LIBTOPK_MAX_DIM 256

typedef struct libtopk_cache {
    void *k; /* device, 16-byte aligned */
    void *v;
    int64_t k_page_stride, k_head_stride, k_slot_stride; /* elements; each a */
    int64_t v_page_stride, v_head_stride, v_slot_stride; /* multiple of 16 B */
    int64_t pages;        /* pages of k and of v, 0 <= pages < 2^31       */
    int64_t table_stride; /* entries between two sequences' table rows    */
    const int32_t *table; /* device, int32[batch][table_width]            */
    const int32_t *lens;  /* device, int32[batch]: slots in use           */
    int32_t batch;        /* 0 <= batch                                   */
    int32_t table_width;  /* 1 <= table_width; table_width * page < 2^30  */
    int32_t heads;        /* 1 <= heads <= 65535                          */
    int32_t page;         /* slots of a page, 1 <= page                   */
    int32_t dim;          /* 1 <= dim <= LIBTOPK_MAX_DIM, rows of a whole
                             number of 16-byte units                      */
    int32_t dtype;        /* LIBTOPK_BF16, _F16, _E4M3 or _E2M1           */
    /* With LIBTOPK_E2M1 alone (otherwise not read, so that they may be left
     * out of an older caller's struct): strides of k and v count bytes, dim is
     * a multiple of 32, and the scales of slot t's row are the dim / 32 bytes
     * at k_blocks + table[..] * k_block_page_stride + h * k_block_head_stride
     * + (t % page) * k_block_slot_stride, at any alignment; likewise v's. */
    void *k_blocks; /* device */
    void *v_blocks;
    int64_t k_block_page_stride, k_block_head_stride, k_block_slot_stride;
    int64_t v_block_page_stride, v_block_head_stride, v_block_slot_stride;
} libtopk_cache_t;

/* What is kept for every slot besides its rows: the attention weight that it
 * has drawn, and its token's position.  Entry t of sequence b, head h is
 * weights[b * weights_batch_stride + h * weights_head_stride + t]. */
typedef struct libtopk_ledger {
    float *weights;     /* device */
    int32_t *positions; /* device */
    int64_t weights_batch_stride, weights_head_stride;
    int64_t positions_batch_stride, positions_head_stride;
    int32_t slots; /* entries of a row, >= 1 */
} libtopk_ledger_t;

/*
 * cache_attend -- attention of one new token a sequence over its slots.
 * q_heads / heads consecutive query heads share a head of the cache (query
 * head j reads head j / (q_heads / heads)).  With x[j][t] = scale *
 * k_scale[h] * (q[b][j] . K[b][h][t]) over the slots t of sequence b:
 *
 *     lse[b][j] = ln sum_t exp x[j][t]
 *     out[b][j] = v_scale[h] * sum_t exp(x[j][t] - lse[b][j]) V[b][h][t]
 *     weights[b][h][t] += sum_{j of h} exp(x[j][t] - lse[b][j])
 *
 * A sequence with no slot gets out = 0 and lse = -infinity.  Scores, weights,
 * sums and the running output are float32 (the weights that multiply bfloat16,
 * 8-bit and 4-bit rows to 2^-22); only out is rounded, once.  Elements of 4-bit
 * rows below 2^-126 may count as 0.  Results do not depend on the order in which
 * workgroups run.
 *
 * Every weight counts that float32 can hold next to the largest (scores down
 * to 87 below it); an infinite V element under one makes its column infinite
 * (NaN with one of the other sign, or a NaN).  Before the division by their
 * sum weights reach up to 2^8, so that V elements beyond 2^119 / len can
 * overflow.  A sequence has one query token; the weights that a prompt's
 * slots have drawn come from a call a token, or from the caller's own
 * attention over the prompt.
 *
 *   q        device, q_dtype (LIBTOPK_BF16 or LIBTOPK_F16; the cache's own,
 *            or either over an LIBTOPK_E4M3 or LIBTOPK_E2M1 cache), 16-byte
 *            aligned, element strides q_batch_stride and q_head_stride
 *            (multiples of 8)
 *   q_heads  a positive multiple of cache->heads
 *   k_scale, v_scale   device, float32[heads], or NULL for 1
 *   ledger   NULL, or where the weights are accumulated (positions unused)
 *   out      device, q_dtype[batch][q_heads][dim], contiguous, 16-byte
 *            aligned
 *   lse      device, float32[batch][q_heads], contiguous
 *
 * Workspace: partial results of at most 1024 workgroups, and with a ledger
 * one float32 a query head and slot of the table's width (rounded up to 32):
 * 4.3 GB for 256 sequences of 32 query heads and a table of 131072 slots.
 * One launch, or two with a ledger and long rows (more than 32768 scores a
 * row) or more than 16 queries a head.  Lengths being on the device, a row
 * counts as long as the table (or the ledger) lets it be: a table no wider
 * than needed is faster, here and in cache_evict.
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, a size,
 * stride or type outside the above, outputs that overlap an input, or more
 * than 2^31 tiles of 32 slots over all sequences, heads and 16-query groups;
 * LIBTOPK_ERR_NOMEM if the workspace cannot grow.
 */
int cache_attend(const libtopk_cache_t *cache, const void *q, int32_t q_dtype,
                 int32_t q_heads, int64_t q_batch_stride,
                 int64_t q_head_stride, float scale, const float *k_scale,
                 const float *v_scale, const libtopk_ledger_t *ledger,
                 void *out, float *lse, libtopk_stream_t stream);

/*
 * cache_append -- the new token's rows enter the cache.  For sequence b and
 * head h, slot s = lens[b] while lens[b] < limit; afterwards the slot that is
 * last in the order of retention among the lens[b] in use:
 *
 *     t comes before u when key(t) > key(u), or key(t) = key(u) and t < u;
 *     key(t) = the largest int32 for a protected slot (its position below
 *     `sinks`, or at least seen[b] - recent), otherwise weights[b][h][t] in
 *     the order-preserving map of float32 bits to int32 (numerical order;
 *     NaN beyond the infinity of its sign).
 *
 * The rows of slot s become k_new[b][h] and v_new[b][h], its weight 0 and its
 * position seen[b].  out_slots[b][h] = s, and out_lens[b] = lens[b] + 1 if
 * lens[b] < limit, otherwise lens[b].  Where slot s would lie beyond the table
 * or the ledger, nothing is written, out_slots is -1 and the length stays.
 * A replaced slot whose table entry names no page loses weight and position
 * as any other; only its rows are written nowhere.
 *
 *   cache    of a type other than LIBTOPK_E2M1 (rows enter a 4-bit cache by
 *            cache_extend)
 *   k_new, v_new   device, the cache's type, 16-byte aligned, element strides
 *                  new_batch_stride and new_head_stride (multiples of 16 B)
 *   limit    >= 1 slots
 *   seen     device, int32[batch]: tokens before this one (its position)
 *   ledger   weights and positions, both updated in place
 *   sinks, recent   >= 0
 *   out_lens   device, int32[batch]; may not be cache->lens
 *   out_slots  device, int32[batch][heads]
 *
 * Errors: as cache_attend, and LIBTOPK_ERR_INVALID for 2^24 rows (batch *
 * heads) or more.
 */
int cache_append(const libtopk_cache_t *cache, const void *k_new,
                 const void *v_new, int64_t new_batch_stride,
                 int64_t new_head_stride, int32_t limit, const int32_t *seen,
                 const libtopk_ledger_t *ledger, int32_t sinks, int32_t recent,
                 int32_t *out_lens, int32_t *out_slots,
                 libtopk_stream_t stream);

/*
 * cache_evict -- cut every sequence back to its `keep` first slots in the
 * order of retention (see cache_append), each head for itself.  The kept slots
 * below `keep` stay where they are; the i-th kept slot at or beyond `keep`
 * (ascending) moves, rows, weight and position, to the i-th slot below `keep`
 * that is not kept (ascending).  Sequences of at most `keep` slots do not
 * change.
 *
 * weights and positions of `after` get the `keep` entries of every row
 * (entries past the new length: 0 and -1); out_lens[b] = min(lens[b], keep).
 * `ledger` is only read.  Two launches, seven when the table (or the ledger)
 * can name more than 16384 slots, one when it can name no more than `keep`.
 *
 *   keep     1 <= keep <= after->slots
 *   after    device arrays that overlap neither the ledger nor each other
 *   out_lens device, int32[batch]; may not be cache->lens
 *
 * Errors: as cache_attend, and LIBTOPK_ERR_INVALID for 2^22 rows (batch *
 * heads) or more, where rows in the seven launches count once for every 4096
 * slots that the table (or the ledger) can name.
 */
int cache_evict(const libtopk_cache_t *cache, const int32_t *seen,
                const libtopk_ledger_t *ledger, int32_t keep, int32_t sinks,
                int32_t recent, const libtopk_ledger_t *after,
                int32_t *out_lens, libtopk_stream_t stream);

/*
 * cache_extend -- the heads of new tokens enter the cache, several tokens a
 * sequence.  Token i of the tokens [starts[b], starts[b + 1]) is sequence b's
 * at slot t = lens[b] + i - starts[b] and position s = seen[b] + i -
 * starts[b].  Its rows x of k (and q, where given) become
 *
 *     y = x * (mean of x^2 + eps)^(-1/2) * k_norm      (or q_norm; if given)
 *
 * and then each of the rot / 2 pairs (y[c], y[d]) of its first rot elements
 *
 *     (y[c] cos a - y[d] sin a, y[d] cos a + y[c] sin a),  a = s * freqs[j]
 *
 * with (c, d) = (j, j + rot / 2), or (2 j, 2 j + 1) if `interleaved`.  Rows of
 * k and v are divided by k_scale[h], v_scale[h] (as cache_attend multiplies)
 * and stored in the cache's type; q goes to q_out in its own.  All of it is
 * computed in 64 bits and rounded at the end, through float32 where the type
 * has 16 or 8 bits.  Numbers beyond an LIBTOPK_E4M3 cache's range become its
 * largest.  In an LIBTOPK_E2M1 cache a block of 32 elements, the largest of
 * magnitude m, gets the scale s = 2^(byte - 127), the least (of 0 <= byte <=
 * 254) with m < 7 s, and each element the nearest 4-bit number to x / s, of
 * two the even code; a block with an infinity or NaN gets 255.
 *
 * With a ledger, weight and position of the new slots become 0 and s.
 * out_lens[b] is the length with the new slots.  Where a slot would lie beyond
 * the table or the ledger, nothing is written for it (q_out is) and the length
 * stops there; where the table names no page, no row is written.  Tokens that
 * belong to no sequence (before starts[0] and from starts[batch] on) are left
 * alone, in q_out too unless `rest` is set.
 *
 *   starts   device, int32[batch + 1], non-decreasing within [0, tokens]: the
 *            caller's promise; otherwise which rows are written is
 *            unspecified (none outside the arrays)
 *   out_lens device, int32[batch]; may not be cache->lens
 *
 * One launch, no workspace.  Errors: LIBTOPK_ERR_INVALID for a NULL or
 * misaligned pointer, a size, stride or type outside the above, an output that
 * overlaps an input or another output (k and v may interleave; q_out may be
 * q), or more than 2^24 workgroups (a token each, or with few tokens several).
 */
typedef struct libtopk_tokens {
    const void *q;       /* device, dtype[tokens][q_heads][dim]; NULL: none */
    const void *k, *v;   /* device, dtype[tokens][heads][dim]               */
    void *q_out;         /* device, as q; with q's strides it may be q      */
    /* elements, multiples of 8; all of these arrays 16-byte aligned */
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t q_out_token_stride, q_out_head_stride;
    const int32_t *starts;
    const int32_t *seen;  /* device, int32[batch]; NULL: the lengths         */
    const void *q_norm;   /* device, norm_dtype[dim], or NULL                */
    const void *k_norm;
    const float *freqs;   /* device, float32[rot / 2]                        */
    const float *k_scale; /* device, float32[heads], or NULL for 1           */
    const float *v_scale;
    int32_t tokens, q_heads;
    int32_t dtype;        /* LIBTOPK_BF16 or LIBTOPK_F16; the cache's type is
                             this, LIBTOPK_E4M3 or LIBTOPK_E2M1              */
    int32_t norm_dtype;   /* dtype or LIBTOPK_F32                            */
    int32_t rot;          /* 0 <= rot <= dim, a multiple of 16               */
    int32_t interleaved;
    float eps;            /* >= 0                                            */
    int32_t rest;         /* q_out's rows of tokens that belong to no sequence:
                             0 left alone, 1 their rows of q as they are     */
} libtopk_tokens_t;

int cache_extend(const libtopk_cache_t *cache, const libtopk_tokens_t *tokens,
                 const libtopk_ledger_t *ledger, int32_t *out_lens,
                 libtopk_stream_t stream);

/* Free the workspaces of the cache_* calls and sample_logits after
 * synchronising their devices.  Must not race with other calls, nor precede the replay of a graph
 * that captured one. */
void cache_release(void);

/* Test hook, as libtopk_debug_scramble: overwrite the completion tickets of
 * the cache_* calls and sample_logits on `stream` with pseudo-random
 * words. */
int cache_debug_scramble(libtopk_stream_t stream, uint64_t seed);

/* ---------------------------------------------------------------------------
 * sample_logits -- a token for each row of logits.
 *
 * With x the row's logits (NaN counts as -infinity, -0 as 0), M the largest,
 * w_i = exp((x_i - M) / temperature), and the order "larger logit first, of
 * equal ones the lower index first":
 *
 *   1. the first top_k logits are kept (all, if top_k < 1);
 *   2. of these the shortest prefix, of one at least, whose weights sum to
 *      top_p times the sum of all of these (all, unless top_p < 1);
 *   3. of these those with w_i >= min_p (min_p above 1 counts as 1; all, if
 *      min_p is not above 0);
 *   4. token = the lowest index i of a kept logit where the sum of the kept
 *      weights up to and with i exceeds u times the sum of all kept weights.
 *
 * logprob = ln(w_token / sum of the kept weights), what the token was drawn
 * with.  A temperature that is not above 0 takes the first of the largest
 * logits, with logprob 0.  A row without a logit above -infinity gets token -1
 * and logprob -infinity; where M is +infinity the logits that equal it have
 * weight 1 and the others none.  u is read as within [0, 1) (NaN as 0): at its
 * upper end the last kept token that has weight is taken.
 *
 * Weights are computed in 64 bits.  The kept ones are added as integers in
 * units of 2^-min(51, 62 - ceil(log2 cols)) of the largest (2^-45 for 131072
 * logits), to the nearest of which each is rounded, so that one below half a
 * unit is never drawn.  Sums of all weights of a row of at most 2^20 logits are
 * added in 64-bit floating point instead, to 2^-46 of them: those that a row
 * without top_k, top_p and min_p is drawn by, which draws weights down to 2^-1074
 * of the largest, and what top_p without top_k is taken of.  Results do not
 * depend on the order in which workgroups run.
 *
 *   logits   device, dtype[rows][cols] (LIBTOPK_F32, _BF16 or _F16), rows ld
 *            elements apart, ld >= cols, at any alignment of the type
 *   rows     0 <= rows < LIBTOPK_MAX_SAMPLE_ROWS
 *   cols     1 <= cols <= LIBTOPK_MAX_LOGITS
 *   how      each setting from a device array of a number a row, or, where
 *            that is NULL, the one number given for all rows
 *   u        device, float32[rows], uniform random numbers
 *   tokens   device, int64[rows]
 *   logprobs device, float32[rows]
 *
 * Workspace: that of the cache_* calls on the stream (the same rules, for a
 * capture too), about 50 KiB a row and 540 bytes for every 1024 logits, and at
 * most 64 MiB: more rows go in batches.  Two launches a batch, five with any of
 * top_k, top_p and min_p; rows of more than 2^20 logits take one launch, no
 * workspace, and a workgroup a row.
 *
 * Errors: LIBTOPK_ERR_INVALID for a NULL or misaligned pointer, a size or type
 * outside the above, or an output that overlaps an input or the other output;
 * LIBTOPK_ERR_NOMEM if the workspace cannot grow.
 */
#define LIBTOPK_MAX_LOGITS (1 << 24)
#define LIBTOPK_MAX_SAMPLE_ROWS (1 << 22)

typedef struct libtopk_sampling {
    const float *temperature; /* device, float32[rows], or NULL */
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
    float temperature_all;
    int32_t top_k_all;
    float top_p_all;
    float min_p_all;
} libtopk_sampling_t;

int sample_logits(const void *logits, int32_t dtype, int64_t rows,
                  int64_t cols, int64_t ld, const libtopk_sampling_t *how,
                  const float *u, int64_t *tokens, float *logprobs,
                  libtopk_stream_t stream);

/* Static, human-readable text for a status code (never NULL). */
const char *libtopk_strerror(int status);

/* LIBTOPK_MAX_K. */
int libtopk_max_k(void);

/*
 * Number of stage-1 workgroups for later calls in this process: 0 restores
 * the automatic choice, otherwise 1..1024.  Results never depend on it (the
 * tests sweep it); it exists for tuning.  Returns LIBTOPK_ERR_INVALID for a
 * value outside 0..1024.
 */
int libtopk_set_grid(int32_t blocks);

/*
 * Workgroups that a topk_i32 call of size n (k <= LIBTOPK_MAX_K) would
 * launch under the current setting (reporting and traffic accounting; no
 * device work).  Returns 0 for n < 1.  With no grid set, the other calls
 * choose their own counts: reductions, statistics and selection for
 * k > LIBTOPK_MAX_K launch at most one workgroup per compute unit,
 * histograms at most two, all of them fewer on small inputs, and key-value
 * calls whose kernel fits only one workgroup per compute unit (k > 64) at
 * most one per unit.
 */
int32_t libtopk_grid_for(int64_t n);

/*
 * Test hook: overwrite, on `stream`, the completion tickets and histogram
 * counters that later calls will use with pseudo-random nonzero words
 * derived from `seed` -- which == 0: those of the scratch of calls on
 * `stream` (allocated first if need be), with the counters and tickets of
 * the segmented top-k once it has run there; which == 1: the tickets of the
 * fixed array of topk_i32_noalloc on the current device.  These words are
 * tagged with each launch's epoch, so no later result may depend on what
 * they held; tests use this to check that.  They index no memory, so any
 * value is safe.  Returns LIBTOPK_ERR_INVALID for another `which`.
 */
int libtopk_debug_scramble(libtopk_stream_t stream, int32_t which,
                           uint64_t seed);

/*
 * Free every cached scratch area after synchronising the devices that own
 * them.  The next call allocates afresh.  Must not race with other calls.
 */
void libtopk_release(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBTOPK_H */
