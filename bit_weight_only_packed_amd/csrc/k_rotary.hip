// k_rotary.hip -- launchers of the rotary kernels (qg_rotary.h).
#include <algorithm>

#include "qg_rotary.h"

namespace qg {

namespace {

// Threads that share a row's heads: as few as fill the chip, so that angles serve many
// heads, and at most a head each.
int slots_for(int64_t rows, int units, int heads, int cus) {
  const int64_t want = (int64_t)cus * 1024, have = rows * units;
  const int64_t s = have > 0 ? (want + have - 1) / have : 1;
  return (int)std::min<int64_t>(heads, std::max<int64_t>(s, (heads + 7) / 8));
}

}  // namespace

hipError_t launch_rotate(const RotArgs& args, bool bf16, int cus, hipStream_t st) {
  RotArgs a = args;
  const int units = a.head_dim / 16;
  a.slots = slots_for(a.rows, units, a.heads, cus);
  const int64_t blocks = ((int64_t)a.rows * units * a.slots + 255) / 256;
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, 1 << 20);
  if (bf16) k_rotate<true><<<grid, 256, 0, st>>>(a);
  else k_rotate<false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_append_rotary(const RotAppend& args, int D, bool bf16, int cus, hipStream_t st) {
  RotAppend a = args;
  const int units = D / 16, heads = a.q_heads + 2 * a.c.kv_heads;
  a.slots = slots_for(a.b.rows, units, heads, cus);
  const int64_t blocks = ((int64_t)a.b.max_rows * units * a.slots + 255) / 256;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, 4096), (unsigned)a.b.n);
  const auto go = [&](auto f) { f<<<grid, 256, 0, st>>>(a); };
  if (D == 64) bf16 ? go(k_kv_append_rotary<64, true>) : go(k_kv_append_rotary<64, false>);
  else if (D == 128) bf16 ? go(k_kv_append_rotary<128, true>) : go(k_kv_append_rotary<128, false>);
  else bf16 ? go(k_kv_append_rotary<256, true>) : go(k_kv_append_rotary<256, false>);
  return hipGetLastError();
}

}  // namespace qg
