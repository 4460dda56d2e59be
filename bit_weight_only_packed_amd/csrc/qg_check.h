// qg_check.h -- what the entry points check of operands [rows][heads][D]: strides, and
// whether an output shares memory with itself or with another operand.
#pragma once
#include <algorithm>
#include <cstdlib>

#include "qg_error.h"
#include "qg_kv.h"

namespace qg {

// (the stride of one row or head alone is never used, and has been made 0)
inline qg_status check_strides(const char* name, int64_t row, int64_t head) {
  if (row % 8 || head % 8 || row < 0 || head < 0)
    return fail(QG_ERR_INVALID_ARG, "%s: strides %lld, %lld are not multiples of 8 elements", name, (long long)row, (long long)head);
  return QG_OK;
}

// Whether two of the D-element runs that begin at r * row + h * head (r < rows, h < heads)
// and at those places + ofs share elements; with ofs 0 two runs of the same kind.
inline bool runs_meet(int64_t row, int64_t head, int64_t rows, int64_t heads, int64_t D, int64_t ofs) {
  if (ofs == 0 && rows > 1 && row < D) return true;
  for (int64_t dh = 1 - heads; dh < heads; ++dh) {
    if (ofs == 0 && dh == 0) continue;
    const int64_t to = ofs + dh * head;  // less the dr rows that come nearest to it
    const int64_t dr = row > 0 ? std::clamp(to / row, 1 - rows, rows - 1) : 0;
    for (int64_t x = std::max(dr - 1, 1 - rows); x <= std::min(dr + 1, rows - 1); ++x)
      if (std::abs(to - x * row) < D) return true;
  }
  return false;
}

// an output [rows][heads][D] against itself
inline qg_status check_nested(const KvRows& out, int64_t rows, int64_t heads, int64_t D) {
  const int64_t ow = (heads - 1) * out.head + D;  // a row's extent
  const bool nested = (heads == 1 || out.head >= D) && (rows == 1 || out.row >= ow);
  if (!nested && runs_meet(out.row, out.head, rows, heads, D, 0))
    return fail(QG_ERR_INVALID_ARG, "out: strides %lld, %lld: rows or heads overlap", (long long)out.row, (long long)out.head);
  return QG_OK;
}

// out [rows][heads][D] against itself and against q of the same shape.  What is plainly apart
// is not looked into: rows that hold their heads, operands in different memory or in columns of
// one tensor's rows.  (Operands of different strides that share memory are left to the caller.)
inline qg_status check_overlap(const KvRows& q, const KvRows& out, int64_t rows, int64_t heads, int64_t D, const char* what) {
  const int64_t ow = (heads - 1) * out.head + D, qw = (heads - 1) * q.head + D;  // a row's extent
  const qg_status s = check_nested(out, rows, heads, D);
  if (s != QG_OK) return s;
  const int64_t ofs = (int64_t)((intptr_t)out.ptr - (intptr_t)q.ptr) / 2;
  if (ofs >= (rows - 1) * q.row + qw || -ofs >= (rows - 1) * out.row + ow) return QG_OK;
  if (rows > 1 && q.row == out.row && q.row > 0) {
    const int64_t at = (ofs % q.row + q.row) % q.row;
    if (at >= qw && at + ow <= q.row) return QG_OK;
  }
  if (ofs == 0 || ((rows == 1 || q.row == out.row) && (heads == 1 || q.head == out.head) &&
                   runs_meet(q.row, q.head, rows, heads, D, ofs)))
    return fail(QG_ERR_INVALID_ARG, "%s", what);
  return QG_OK;
}

// whether two operands of the same rows and different heads are plainly apart: in different
// memory, or in other columns of the same rows
inline bool apart(const KvRows& a, int64_t a_heads, const KvRows& b, int64_t b_heads, int64_t rows, int64_t D) {
  const int64_t aw = (a_heads - 1) * a.head + D, bw = (b_heads - 1) * b.head + D;
  const int64_t ofs = (int64_t)((intptr_t)b.ptr - (intptr_t)a.ptr) / 2;
  if (ofs >= (rows - 1) * a.row + aw || -ofs >= (rows - 1) * b.row + bw) return true;
  if (rows == 1 || a.row != b.row || a.row <= 0) return false;
  const int64_t at = (ofs % a.row + a.row) % a.row;
  return at >= aw && at + bw <= a.row;
}

}  // namespace qg
