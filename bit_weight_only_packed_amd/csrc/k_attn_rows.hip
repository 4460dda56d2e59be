// k_attn_rows.hip -- launcher of the many-row attention kernel (qg_attn_rows.h).
#include <algorithm>

#include "qg_attn_rows.h"

namespace qg {

namespace {

// Blocks of a launch at most: a launch holds fewer than 2^32 threads.  More than one is for
// ragged calls alone, in which nearly all blocks are those of rows that their entry has not.
constexpr unsigned kRowsLaunch = 1u << 23;
static_assert((uint64_t)kRowsLaunch * 64 * ROWS_WAVES < (uint64_t)1 << 32, "threads of a launch");

template <int D> hipError_t go(AttnArgs a, bool bf16, unsigned blocks, hipStream_t st) {
  const unsigned grid = blocks * (unsigned)a.splits;
  for (unsigned at = 0; at < grid; at += kRowsLaunch) {
    const unsigned part = std::min(grid - at, kRowsLaunch);
    a.first = (int)at;  // (0 where blocks are shared: their grids are small)
    if (bf16) k_attn_rows<D, true><<<part, 64 * ROWS_WAVES, 0, st>>>(a);
    else k_attn_rows<D, false><<<part, 64 * ROWS_WAVES, 0, st>>>(a);
  }
  if (a.splits > 1) {
    const unsigned join = blocks * (unsigned)(ROWS_BLOCK / RJ_ROWS);
    if (bf16) k_attn_rows_join<D, true><<<join, RJ_THREADS, 0, st>>>(a);
    else k_attn_rows_join<D, false><<<join, RJ_THREADS, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

int rows_parts(int D, int cap, int splits1) {
  const int kt = D == 256 ? RowsShape<256>::KT : RowsShape<128>::KT;
  return rw_parts((cap + kt - 1) / kt, splits1);
}

hipError_t launch_attn_rows(const AttnArgs& a, int D, bool bf16, unsigned blocks, hipStream_t st) {
  if (D == 64) return go<64>(a, bf16, blocks, st);
  if (D == 128) return go<128>(a, bf16, blocks, st);
  return go<256>(a, bf16, blocks, st);
}

}  // namespace qg
