// k_attn_share.hip -- launchers of the attention of shared tokens (qg_attn_share.h).
#include "qg_attn_share.h"

namespace qg {

namespace {

template <int D> hipError_t go(const AttnArgs& a, bool bf16, unsigned blocks, hipStream_t st) {
  const unsigned grid = blocks * (unsigned)a.splits;
  if (bf16) k_attn_rows<D, true, RW_PREFIX><<<grid, 64 * ROWS_WAVES, 0, st>>>(a);
  else k_attn_rows<D, false, RW_PREFIX><<<grid, 64 * ROWS_WAVES, 0, st>>>(a);
  if (a.splits > 1) k_share_join<D><<<blocks * (unsigned)(ROWS_BLOCK / RJ_ROWS), RJ_THREADS, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_share_plan(const ShareArgs& a, hipStream_t st) {
  k_share_plan<<<(unsigned)a.b.n, SP_T, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_attn_prefix(const AttnArgs& a, int D, bool bf16, unsigned blocks, hipStream_t st) {
  if (D == 64) return go<64>(a, bf16, blocks, st);
  if (D == 128) return go<128>(a, bf16, blocks, st);
  return go<256>(a, bf16, blocks, st);
}

}  // namespace qg
