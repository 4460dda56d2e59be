// k_attn_step.hip -- launcher of the few-row attention kernel (qg_attn_step.h).
#include "qg_attn_step.h"

namespace qg {

namespace {

template <int D, bool BF, int MT> hipError_t go(const AttnArgs& a, bool shared, hipStream_t st) {
  const size_t lds = StepShape<D, MT>::lds + step_list_bytes(a.b.n);
  if (shared) k_attn_step<D, BF, MT, true><<<(unsigned)a.workers, 64 * step_waves(D), lds, st>>>(a);
  else k_attn_step<D, BF, MT, false><<<(unsigned)a.workers, 64 * step_waves(D), lds, st>>>(a);
  return hipGetLastError();
}

template <int D, int MT> hipError_t by_type(const AttnArgs& a, bool bf16, bool shared, hipStream_t st) {
  return bf16 ? go<D, true, MT>(a, shared, st) : go<D, false, MT>(a, shared, st);
}

template <int D> hipError_t by_rows(const AttnArgs& a, bool bf16, int MT, bool shared, hipStream_t st) {
  if constexpr (step_max_rows(D) > 16) {
    if (MT == 2) return by_type<D, 2>(a, bf16, shared, st);
  }
  return by_type<D, 1>(a, bf16, shared, st);
}

template <int D, bool BF, int MT> hipError_t allow() {
  hipError_t e = hipSuccess;
  for (const void* f : {reinterpret_cast<const void*>(&k_attn_step<D, BF, MT, false>),
                        reinterpret_cast<const void*>(&k_attn_step<D, BF, MT, true>)})
    if (e == hipSuccess)
      e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize,
                              (int)(StepShape<D, MT>::lds + step_list_bytes(KV_MAX_SEQS)));
  return e;
}

}  // namespace

hipError_t launch_attn_step(const AttnArgs& a, int D, bool bf16, int MT, bool shared, hipStream_t st) {
  if (D == 64) return by_rows<64>(a, bf16, MT, shared, st);
  if (D == 128) return by_rows<128>(a, bf16, MT, shared, st);
  return by_rows<256>(a, bf16, MT, shared, st);
}

hipError_t attn_step_allow_lds() {
  hipError_t e = hipSuccess;
  const auto both = [&](auto f, auto g) {
    if (e == hipSuccess) e = f();
    if (e == hipSuccess) e = g();
  };
  both(allow<64, false, 1>, allow<64, true, 1>);
  both(allow<64, false, 2>, allow<64, true, 2>);
  both(allow<128, false, 1>, allow<128, true, 1>);
  both(allow<128, false, 2>, allow<128, true, 2>);
  both(allow<256, false, 1>, allow<256, true, 1>);
  return e;
}

}  // namespace qg
