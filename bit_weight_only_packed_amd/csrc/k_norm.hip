// k_norm.hip -- launcher of the norm (qg_norm.h).
#include <algorithm>

#include "qg_norm.h"

namespace qg {

namespace {

constexpr int kBlocks = 1 << 21;  // of a launch, which holds fewer than 2^32 threads

template <bool BF, int C, bool TEAM> void go(NormArgs a, int codes, int rows_of_block, unsigned threads, hipStream_t st) {
  const int64_t blocks = ((int64_t)a.rows + rows_of_block - 1) / rows_of_block;
  for (int64_t at = 0; at < blocks; at += kBlocks) {
    const unsigned grid = (unsigned)std::min<int64_t>(blocks - at, kBlocks);
    a.first = (int)(at * rows_of_block);
    if (codes == QGS_SAME) k_rms_norm<BF, C, QGS_SAME, TEAM><<<grid, threads, 0, st>>>(a);
    else if (codes == QGS_INT8) k_rms_norm<BF, C, QGS_INT8, TEAM><<<grid, threads, 0, st>>>(a);
    else k_rms_norm<BF, C, QGS_E4M3, TEAM><<<grid, threads, 0, st>>>(a);
  }
}

// Chunks of a thread, by n alone, so that a row's sum runs in the same order in every call.  us, fp16 with
// the residual, one, two and four chunks: 8,191 rows of 5,120 60 / 55 / 57, of 1,280 19 / 19 / 20; 30,000 of 512
// 23 / 24 / 32; one row of 5,120 6.3 each.
template <bool BF> hipError_t by_chunks(NormArgs a, int codes, hipStream_t st) {
  const int chunks = (a.n + 7) / 8;
  const auto threads = [&](int C) { return (unsigned)((chunks + C - 1) / C + 63) / 64 * 64; };
  a.team = 1;
  while (a.team < chunks) a.team *= 2;
  if (a.team <= 32) go<BF, 1, true>(a, codes, NM_TEAMS / a.team, NM_TEAMS, st);
  else if (chunks <= 64) go<BF, 1, false>(a, codes, 1, threads(1), st);
  else if (chunks <= 2 * 1024) go<BF, 2, false>(a, codes, 1, threads(2), st);
  else if (chunks <= 3 * 1024) go<BF, 3, false>(a, codes, 1, threads(3), st);
  else go<BF, 4, false>(a, codes, 1, threads(4), st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, bool bf16, int codes, hipStream_t st) {
  return bf16 ? by_chunks<true>(a, codes, st) : by_chunks<false>(a, codes, st);
}

}  // namespace qg
