// k_attn_rows.hip -- launcher of the many-row attention kernel (qg_attn_rows.h).
#include "qg_attn_rows.h"

namespace qg {

namespace {

template <int D, bool BF> hipError_t go(const AttnArgs& a, unsigned blocks, hipStream_t st) {
  k_attn_rows<D, BF><<<blocks * (unsigned)a.splits, 64 * RW_NW, RowsShape<D>::lds, st>>>(a);
  return hipGetLastError();
}

template <int D, bool BF> hipError_t allow() {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attn_rows<D, BF>),
                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)RowsShape<D>::lds);
}

}  // namespace

hipError_t launch_attn_rows(const AttnArgs& a, int D, bool bf16, unsigned blocks, hipStream_t st) {
  if (D == 64) return bf16 ? go<64, true>(a, blocks, st) : go<64, false>(a, blocks, st);
  if (D == 128) return bf16 ? go<128, true>(a, blocks, st) : go<128, false>(a, blocks, st);
  return bf16 ? go<256, true>(a, blocks, st) : go<256, false>(a, blocks, st);
}

hipError_t attn_rows_allow_lds() {
  hipError_t e = allow<64, false>();
  if (e == hipSuccess) e = allow<64, true>();
  if (e == hipSuccess) e = allow<128, false>();
  if (e == hipSuccess) e = allow<128, true>();
  if (e == hipSuccess) e = allow<256, false>();
  if (e == hipSuccess) e = allow<256, true>();
  return e;
}

}  // namespace qg
