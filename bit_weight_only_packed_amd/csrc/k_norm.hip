// k_norm.hip -- launcher of the norm (qg_norm.h).
#include <algorithm>

#include "qg_norm.h"

namespace qg {

namespace {

constexpr int kRowsLaunch = 1 << 21;  // a launch holds fewer than 2^32 threads

template <bool BF, int C> void go(NormArgs a, int codes, unsigned threads, hipStream_t st) {
  const int rows = a.rows;
  for (int at = 0; at < rows; at += kRowsLaunch) {
    const unsigned grid = (unsigned)std::min(rows - at, kRowsLaunch);
    a.first = at;
    if (codes == QGS_SAME) k_rms_norm<BF, C, QGS_SAME><<<grid, threads, 0, st>>>(a);
    else if (codes == QGS_INT8) k_rms_norm<BF, C, QGS_INT8><<<grid, threads, 0, st>>>(a);
    else k_rms_norm<BF, C, QGS_E4M3><<<grid, threads, 0, st>>>(a);
  }
}

template <bool BF> hipError_t by_chunks(const NormArgs& a, int codes, int cus, hipStream_t st) {
  const int chunks = (a.n + 7) / 8;
  const bool few = a.rows <= 2 * cus;
  int C = few ? 1 : 2;
  while (chunks > 1024 * C) C *= 2;
  const unsigned threads = (unsigned)((chunks + C - 1) / C + 63) / 64 * 64;
  if (C == 1) go<BF, 1>(a, codes, threads, st);
  else if (C == 2) go<BF, 2>(a, codes, threads, st);
  else go<BF, 4>(a, codes, threads, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, bool bf16, int codes, int cus, hipStream_t st) {
  return bf16 ? by_chunks<true>(a, codes, cus, st) : by_chunks<false>(a, codes, cus, st);
}

}  // namespace qg
