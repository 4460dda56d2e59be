/*
 * qgstep.h -- C ABI of what a decode step does with rows between its products
 * (libqgemv.so, AMD Instinct MI355X, gfx950): the norm before a product with the
 * residual's addition, rotary positions, and picking tokens from logits.  (Rotary
 * positions on the way into the paged cache: qgkv_append_rotary in qgkv.h.)
 *
 * Everything runs on the caller's stream and copies nothing to the host; the
 * calls allocate nothing and keep nothing, so they can be captured in HIP graphs,
 * and calls on different streams are independent.  Reductions run in an order that
 * the sizes of the call fix, or add integers: same inputs, same bits, and a row's
 * results do not depend on the call's other rows.  Errors and
 * streams as in qgemv.h; device pointers are of the current device's memory.
 */
#ifndef QGSTEP_H
#define QGSTEP_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QGS_F16 = 0, QGS_BF16 = 1, QGS_F32 = 2 } qgs_type; /* QGS_F32: logits only */
typedef enum { QGS_SAME = 0, QGS_INT8 = 1, QGS_E4M3 = 2 } qgs_codes;

enum { QGS_MAX_NORM = 32768, QGS_MAX_VOCAB = 1 << 20 };

/* Root-mean-square norm of rows of n elements.
 *   h = x + residual, rounded once to the type and stored in residual (NULL: h = x)
 *   y = h * weight / sqrt(mean(h^2) + eps)              (weight NULL: 1)
 * The mean is of the stored h, in fp32 (scaled where squares would overflow or vanish); h / sqrt(..) is fp32's, with
 * the fewer bits of its numbers below 2^-126 there, and y, its product with weight, is rounded once.
 * codes QGS_SAME: out is y, of x's type.  QGS_INT8, QGS_E4M3: for each `group` elements
 * of a row (0: the whole row; 32, 64 or 128, the last may be short) a scale
 * s = max |y| / 127 (int8) or / 448 (e4m3: 4 exponent and 3 mantissa bits, no infinity),
 * fp32, and out holds y / s (of fp32 y, in fp32) rounded to nearest even, held to 127 or 448 (which it passes only where s
 * is too small for fp32's 24 bits); a group of zeros has scale 0 (so has one whose s is below fp32's
 * smallest number), one that holds a NaN or infinity scale NaN, and both have codes 0.
 * Rows may lie at any strides (elements) and need no alignment past their
 * type's; rows of one operand do not overlap.  out may be x (same pointer and
 * stride, QGS_SAME); no other operands share memory. */
typedef struct {
  const void* x;
  void* residual;     /* in and out, or NULL */
  const void* weight; /* [n] or NULL */
  void* out;
  float* scales;      /* [rows][ceil(n / group)], or NULL with QGS_SAME */
  int64_t x_stride, residual_stride, out_stride;
  int32_t rows, n;    /* rows 0: nothing to do; n 1 .. QGS_MAX_NORM */
  int32_t dtype;      /* QGS_F16 or QGS_BF16: x, residual, weight */
  int32_t codes;      /* qgs_codes */
  int32_t group;
  float eps;          /* > 0 */
} qgs_norm;

qg_status qgs_rms_norm(const qgs_norm* d, void* stream);

/* Rotary positions.  The first `dim` elements of a head are dim / 2 pairs: elements
 * j and j + dim / 2 (layout QGS_HALVES) or 2 j and 2 j + 1 (QGS_PAIRS).  At position p
 * pair j = (a, b) becomes
 *   size * (a cos t - b sin t, a sin t + b cos t),   t = 2 pi p turns[j] / 2^64,
 * in fp32, rounded once; elements from dim on are copied.  turns[j] is the pair's
 * frequency in turns per position as a 64-bit binary fraction: p * turns[j] modulo 2^64 is
 * exact for any position, so far positions lose nothing (an angle held in fp32 is
 * off by 2^-24 of itself, 0.06 at position 2^20). */
typedef enum { QGS_HALVES = 0, QGS_PAIRS = 1 } qgs_layout;
typedef struct {
  const uint64_t* turns; /* device [dim / 2], 16-byte aligned */
  int32_t dim;           /* a multiple of 16, up to head_dim */
  int32_t layout;        /* qgs_layout */
  float size;            /* finite */
} qgs_rotary;

/* Rotate x [rows][heads][head_dim] into out (same shape; out may be x with the same
 * strides, and otherwise shares no memory with it): row i stands at positions[i].
 * head_dim is a multiple of 16 up to 1024; strides in elements, multiples of 8;
 * pointers 16-byte aligned. */
typedef struct {
  const void* x;
  void* out;
  const int32_t* positions; /* device [rows] */
  int64_t x_row, x_head, out_row, out_head;
  int32_t rows, heads, head_dim, dtype; /* rows 0: nothing to do */
} qgs_rows;

qg_status qgs_rotate(const qgs_rows* d, const qgs_rotary* rotary, void* stream);

/* Pick a token of each row of logits [rows][vocab].  A row's tokens are ordered by
 * falling logit, equal ones by rising index.  With w_i = exp((l_i - max l) / temperature):
 *   top_k > 0   the first top_k tokens are kept
 *   top_p < 1   of these the fewest first ones whose w sum to top_p of all of theirs (one
 *               at least)
 *   min_p > 0   of these the ones with w_i >= min_p (that is of the largest)
 * and the picked token is the first, by index, up to which the kept tokens' w sum to
 * more than u * (all kept).  temperature <= 0 (or NaN): the first token of the order.  prob: w of the
 * token over the sum of the kept ones.  A NaN logit counts as -inf; tokens of -inf are
 * never picked, and a row of nothing else gives token -1 and prob 0.  (top_k <= 0, top_p
 * >= 1 or NaN, min_p <= 0 or NaN: no such limit.  u is held to [0, 1).)
 *
 * Weights are computed in fp64 and held as multiples of 2^-43 (2^-44 of the largest and 2^-49 of
 * itself is the most that one is off, and tokens below 2^-44 are not picked); their sums are
 * exact, so results depend on nothing but the row. */
typedef struct {
  const void* logits;
  int64_t stride;           /* elements from a row to the next */
  int32_t rows, vocab;      /* rows 0: nothing to do; vocab 1 .. QGS_MAX_VOCAB */
  int32_t dtype;            /* qgs_type */
  const float* u;           /* device [rows] */
  const float* temperature; /* device [rows]; NULL: temperature1 for every row */
  const int32_t* top_k;     /* likewise */
  const float* top_p;
  const float* min_p;
  float temperature1;
  int32_t top_k1;
  float top_p1, min_p1;
  int32_t* tokens;          /* device [rows] */
  float* probs;             /* device [rows] or NULL */
} qgs_sampling;

/* Bytes of the workspace that a call of so many rows and tokens takes. */
qg_status qgs_sample_workspace(int32_t rows, int32_t vocab, size_t* bytes);

/* workspace: device, 16-byte aligned, of at least that size; its contents do not matter
 * before or after the call. */
qg_status qgs_sample(const qgs_sampling* d, void* workspace, size_t bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QGSTEP_H */
