// k_attn_rows.hip -- launcher of the many-row attention kernel (qg_attn_rows.h).
#include "qg_attn_rows.h"

namespace qg {

namespace {

template <int D, bool BF> hipError_t go(const AttnArgs& a, unsigned blocks, hipStream_t st) {
  k_attn_rows<D, BF><<<blocks * (unsigned)a.splits, 64 * RowsShape<D>::NW, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_rows(const AttnArgs& a, int D, bool bf16, unsigned blocks, hipStream_t st) {
  if (D == 64) return bf16 ? go<64, true>(a, blocks, st) : go<64, false>(a, blocks, st);
  if (D == 128) return bf16 ? go<128, true>(a, blocks, st) : go<128, false>(a, blocks, st);
  return bf16 ? go<256, true>(a, blocks, st) : go<256, false>(a, blocks, st);
}

}  // namespace qg
