// k_kv_pages.hip -- launchers of the page operations and of the append (qg_kv_pages.h).
#include <algorithm>

#include "qg_kv_pages.h"

namespace qg {

hipError_t launch_kv_fork(const KvPool& p, const int32_t* src, const int32_t* dst, int n, hipStream_t st) {
  k_kv_fork<<<(unsigned)n, 256, 0, st>>>(p, src, dst, n);
  return hipGetLastError();
}

hipError_t launch_kv_trim(const KvPool& p, const int32_t* seqs, const int32_t* keep, int n, hipStream_t st) {
  k_kv_trim<<<(unsigned)n, 256, 0, st>>>(p, seqs, keep);
  return hipGetLastError();
}

hipError_t launch_kv_extend(const KvPool& p, const int32_t* n_new, int cus, hipStream_t st) {
  k_kv_extend<<<1, KV_PLAN, 0, st>>>(p, n_new);
  const int64_t pieces = (p.page_bytes + KV_PIECE - 1) / KV_PIECE * std::min(p.max_seqs, p.pages);
  k_kv_copy<false><<<(unsigned)std::min<int64_t>(8 * cus, pieces), 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const KvPool& p, int cus, hipStream_t st) {
  k_kv_compact<<<1, KV_PLAN, 0, st>>>(p);
  k_kv_copy<true><<<(unsigned)(8 * cus), 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_kv_append(const KvDev& c, const KvBatchDev& b, const KvRows& k, const KvRows& v, const int32_t* refused,
                            const int32_t* info, int D, hipStream_t st) {
  const int64_t items = (int64_t)b.max_rows * 2 * c.kv_heads;
  const int per = 256 / (D / 8);  // items of a workgroup
  const dim3 grid((unsigned)std::min<int64_t>((items + per - 1) / per, 4096), (unsigned)b.n);
  if (D == 64) k_kv_append<64><<<grid, 256, 0, st>>>(c, b, k, v, refused, info);
  else if (D == 128) k_kv_append<128><<<grid, 256, 0, st>>>(c, b, k, v, refused, info);
  else k_kv_append<256><<<grid, 256, 0, st>>>(c, b, k, v, refused, info);
  return hipGetLastError();
}

}  // namespace qg
