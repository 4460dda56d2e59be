/*
 * qgkv.h -- C ABI of the paged key-value cache and the attention over it
 * (libqgemv.so, AMD Instinct MI355X, gfx950).
 *
 * The products of qgemv.h make a decode layer's q, k, v and take its attention
 * output; this part holds what lies between: the new tokens' keys and values
 * are appended to pages of a cache, one-token, verify (several drafted tokens)
 * and prompt rows attend to them, and the pages of sequences are shared, cut,
 * freed and moved together -- all on the device, on the caller's stream, with
 * no copy to the host, so that a decode step can be captured in a HIP graph.
 *
 * The cache.  Caller-owned device memory (row-major):
 *   pool    fp16 or bf16 [pages][layers][2][kv_heads][page_size][head_dim],
 *           index 0 of the third axis keys, 1 values; 16-byte aligned
 *   tables  int32 [max_seqs][max_pages]: entry i of a slot is the page of its
 *           tokens [i * page_size, (i + 1) * page_size), -1 where it has none
 *   lens    int32 [max_seqs]: tokens of each slot (0: the slot is empty)
 *   refs    int32 [pages], 16-byte aligned: table entries that name the page
 *           (0: it is free)
 *   info    int32 [4]: [0] QG_KV_* bits, set by calls that found something to
 *           refuse on the device and never cleared by them; [1] pages that the
 *           last refused qgkv_extend was short of; [2] live pages and [3] moved
 *           pages of the last qgkv_compact
 * An empty cache is tables -1 and all else 0.  The layout of one cache serves
 * all layers of a model: extend once per step, append and attend per layer.
 *
 * Rows of a call (qg_kv_batch).  n entries; entry j is the slot seqs[j] (NULL:
 * slot j) with R_j new rows, rows row_start[j] .. row_start[j + 1] - 1 of the
 * call's `rows` rows (NULL: rows / n each).  They are the LAST R_j tokens of the
 * slot, whose length already counts them: row i stands at position
 * p = lens - R_j + i.  Of more than max_rows rows the later ones are left out (not
 * written, no output); the others keep their positions.  seqs and row_start are
 * device memory and may change between replays of a captured call.  A slot index
 * out of range acts as an empty slot.  A row at a position before 0 (an idle slot,
 * length 0) is not written by append and sees nothing in attend: its output is 0.
 *
 * Attention.  With h' = h / (q_heads / kv_heads) and s_t = scale * q_h . k_t,h',
 *   out_h = sum_t exp(s_t) v_t,h' / sum_t exp(s_t)
 * over the tokens t <= p that lie in the window, t > p - window (window 0: all),
 * or among the first `sinks`, t < sinks.  Scores, maxima, sums and outputs are
 * held in fp32; the weights exp(s_t - max) are rounded once to the cache's type
 * to enter the matrix cores beside the values, and the output is rounded once.  The
 * sum is of the unrounded weights.  A weight's rounding is off by 2^-11 of it (bf16 2^-8)
 * or, if that is more, in fp16 by 2^-36 of the row's largest weight; fp16 weights are
 * carried larger by a power of two for that, which the division takes away.
 * Tokens that a row does not see never reach it, whatever they hold (NaN,
 * infinities, memory never written).  A NaN or infinity that it sees makes its
 * output NaN (or infinite where IEEE arithmetic gives that).
 *
 * Determinism.  Every reduction runs in an order that the lengths and row
 * counts of the call fix; no floating-point atomics: same inputs, same bits.
 * The split of a sequence's tokens over workgroups depends on the other
 * sequences of the call, so a row's bits may differ between batches.
 *
 * Ownership, streams, errors: as in qgemv.h.  The handle keeps the pointers of
 * its descriptor (the memory stays the caller's and must outlive it) and owns
 * a workspace, so calls on one handle are ordered by the caller.  Page ids out
 * of [0, pages) in a table are read as page 0 and never written through: no
 * content of tables, lens, seqs or row_start makes a kernel leave the caller's
 * memory.
 */
#ifndef QGKV_H
#define QGKV_H

#include "qgemv.h"
#include "qgstep.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qg_kv* qg_kv_handle;

typedef enum { QG_KV_F16 = 0, QG_KV_BF16 = 1 } qg_kv_type;

/* bits of info[0] */
enum {
  QG_KV_SHORT = 1, /* qgkv_extend: not enough free pages; nothing was changed                  */
  QG_KV_LONG = 2,  /* qgkv_extend: a length past max_pages * page_size; nothing was changed    */
  QG_KV_PAIR = 4   /* qgkv_fork / qgkv_trim: an entry was refused (see there) and skipped       */
};

enum { QG_KV_MAX_SEQS = 1024, QG_KV_MIN_PAGE = 16, QG_KV_MAX_PAGE = 256 };

typedef struct {
  int32_t pages;     /* pages of the pool, 1 .. 2^20                                  */
  int32_t layers;    /* >= 1                                                          */
  int32_t kv_heads;  /* >= 1                                                          */
  int32_t head_dim;  /* 64, 128 or 256                                                */
  int32_t page_size; /* tokens of a page: 16, 32, 64, 128 or 256                      */
  int32_t max_seqs;  /* slots, 1 .. QG_KV_MAX_SEQS                                    */
  int32_t max_pages; /* entries of a slot's table, >= 1; max_pages * page_size <= 2^30 */
  int32_t dtype;     /* qg_kv_type                                                    */
  void* pool;
  int32_t* tables;
  int32_t* lens;
  int32_t* refs;
  int32_t* info;
} qg_kv_desc;

typedef struct {
  int32_t n;                /* entries, 1 .. max_seqs (0 without rows)                         */
  int32_t rows;             /* rows of the call over all entries; 0: the call does nothing     */
  int32_t max_rows;         /* with row_start: at least the largest R_j (an entry's rows past
                               it are left out); ignored without                               */
  const int32_t* seqs;      /* device [n] or NULL                                              */
  const int32_t* row_start; /* device [n + 1], ascending from 0 to rows, or NULL               */
} qg_kv_batch;

/* A 3-d operand [rows][heads][head_dim] of the cache's type: strides in
 * elements, multiples of 8 (that of a single row or head is not used);
 * head_dim is contiguous; 16-byte aligned.  So k and v may be columns of stacked
 * q|k|v rows. */
typedef struct {
  void* ptr;
  int64_t row_stride;
  int64_t head_stride;
} qg_kv_rows;

/* Validate the descriptor, check that the device is gfx950 and allocate the
 * handle's workspace.  Synchronises `stream`.  On failure *out is NULL. */
qg_status qgkv_create(qg_kv_handle* out, const qg_kv_desc* desc, void* stream);

/* Free the handle and its workspace (NULL is accepted). */
qg_status qgkv_destroy(qg_kv_handle h);

/* Make room: lens[s] += n_new[s] for every slot (n_new: device int32
 * [max_seqs]; values below 0 count as 0).  Pages are taken lowest free id
 * first, slots in order.  A partly filled last page that another slot also
 * names is first copied to a fresh page (all layers) -- unless every slot that
 * names it grows in this call, where the lowest of them keeps it.  All or
 * nothing: if pages are short or a table is too small, nothing changes, info
 * says so, and qgkv_append on this handle writes nothing until an extend is
 * granted or the caller has cleared that bit of info[0].  (qgkv_attend computes
 * as ever, from the lengths that stand.) */
qg_status qgkv_extend(qg_kv_handle h, const int32_t* n_new, void* stream);

/* dst[i] becomes a second name of src[i]'s tokens: same pages, refs + 1, no
 * copy (device int32 [n], 1 <= n <= max_seqs).  An entry is refused if an index is
 * out of range, dst is not empty or was named by an earlier entry, or src is
 * also a dst of the call. */
qg_status qgkv_fork(qg_kv_handle h, const int32_t* src, const int32_t* dst, int32_t n, void* stream);

/* Cut slot seqs[i] to its first min(keep[i], lens) tokens (keep NULL or <= 0:
 * free it): pages past them are let go, refs - 1; 1 <= n <= max_seqs.  An entry
 * is refused if its index is out of range or was named by an earlier entry. */
qg_status qgkv_trim(qg_kv_handle h, const int32_t* seqs, const int32_t* keep, int32_t n, void* stream);

/* Move the live pages together: with m live pages, those with id >= m, in
 * ascending order, move into the free ids below m, in ascending order; tables
 * and refs follow. */
qg_status qgkv_compact(qg_kv_handle h, void* stream);

/* Write the rows' keys and values of one layer into their pages: k and v are
 * [rows][kv_heads][head_dim]; a slot takes one entry of the call at most.
 * Writes nothing while a refused qgkv_extend stands (see there): the rows'
 * places are then other tokens'. */
qg_status qgkv_append(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* k, const qg_kv_rows* v,
                      void* stream);

/* The same with rotary positions (qgstep.h): a row's k is rotated to its position on its
 * way into the page, v written as it is, and its q (q_heads heads; 0: none, q and q_out are not
 * looked at) rotated into q_out, [rows][q_heads][head_dim].  q_out may be q (same
 * pointer and strides), and otherwise overlaps neither q nor itself; it never
 * overlaps k or v, but may lie in other columns of the same rows.  q_out of a row at a
 * position before 0 is 0; rows of no entry, or left out by max_rows, keep theirs.  While a
 * refused qgkv_extend stands only q_out is written. */
qg_status qgkv_append_rotary(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* k, const qg_kv_rows* v,
                             const qg_kv_rows* q, const qg_kv_rows* q_out, int32_t q_heads, const qgs_rotary* rotary,
                             void* stream);

/* out = attention of q over the cached tokens of one layer: q and out are
 * [rows][q_heads][head_dim], q_heads a multiple of kv_heads; scale > 0;
 * window >= 0 and sinks >= 0 as above.  out overlaps neither q nor itself
 * (refused where it can be told from pointers and equal strides).  One call takes
 * entries of any row counts, but is made for those near max_rows: long slots with
 * few rows are better attended in a call of their own (one new row in each of 47 slots
 * of 3 to 24,577 tokens beside 512 rows of another: 458 us, in two calls 212). */
qg_status qgkv_attend(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* q, const qg_kv_rows* out,
                      int32_t q_heads, float scale, int32_t window, int32_t sinks, void* stream);

/* qgkv_attend for entries that share tokens: the same outputs, to their roundings, but
 * the tokens that all entries of a group have in common are read once for the group and
 * not once for each.  Entries groups[g] .. groups[g + 1] - 1 are group g (device int32
 * [n_groups + 1], ascending from 0 to n, may change between replays of a captured
 * call; NULL: all entries are one group).  What a group shares is found in the tables: the
 * leading pages that all its entries name alike (those of qgkv_fork), up to the first
 * of their rows, in whole multiples of 64 tokens, 256 at least; entries that see nothing are left
 * aside.
 *   least  bytes of keys and values from which on it is done: of the shared tokens, each counted once for every
 *          entry that reads it, over all groups.  0: always.  Negative: where it was measured to pay, which
 *          goes by the head size, the entries, their rows and the bytes of the shared tokens.  Otherwise
 *          the call is qgkv_attend, bit for bit, but for some 11 us that finding out takes (none where n
 *          slots as long as their tables would hold too little).
 * Calls of very many rows (more than 512 / kv_heads blocks of 128 (row, q head of a kv head) pairs) are
 * qgkv_attend too.  The split of tokens depends on the group, so a row's bits may differ from
 * qgkv_attend's. */
qg_status qgkv_attend_shared(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* q, const qg_kv_rows* out,
                             int32_t q_heads, float scale, int32_t window, int32_t sinks, const int32_t* groups,
                             int32_t n_groups, int64_t least, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QGKV_H */
