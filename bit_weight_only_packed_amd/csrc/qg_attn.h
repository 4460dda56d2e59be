// qg_attn.h -- what the two attention kernels share: the matrix instructions for
// fp16 and bf16, rounding, and the partial results that meet across workgroups.
//
// Both compute, for a row at position p and the tokens t that it sees,
//   o = sum_t 2^(c s_t - m) v_t / sum_t 2^(c s_t - m),  s_t = q . k_t,
//   c = scale * log2(e), m the running maximum of c s_t,
// in one pass over the tokens: when m grows, what has been summed is multiplied
// by 2^(m_old - m).  Partial results (o, m, l) of disjoint token ranges join as
//   M = max m_i,  o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// A range in which a row sees nothing has m = -inf and contributes 0.
#pragma once
#include "qg_kv.h"

namespace qg {

typedef _Float16 at_h8 __attribute__((ext_vector_type(8)));
typedef __bf16 at_b8 __attribute__((ext_vector_type(8)));
typedef _Float16 at_h2 __attribute__((ext_vector_type(2)));
typedef __bf16 at_b2 __attribute__((ext_vector_type(2)));
typedef float at_f2 __attribute__((ext_vector_type(2)));
typedef float at_f4 __attribute__((ext_vector_type(4)));
typedef float at_f16 __attribute__((ext_vector_type(16)));

template <bool BF> __device__ __forceinline__ at_f4 at_mfma16(kv_u4 a, kv_u4 b, at_f4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(at_b8, a), __builtin_bit_cast(at_b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(at_h8, a), __builtin_bit_cast(at_h8, b), c, 0, 0, 0);
}
template <bool BF> __device__ __forceinline__ at_f16 at_mfma32(kv_u4 a, kv_u4 b, at_f16 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(at_b8, a), __builtin_bit_cast(at_b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(at_h8, a), __builtin_bit_cast(at_h8, b), c, 0, 0, 0);
}

// two fp32 rounded to nearest even, low half first
template <bool BF> __device__ __forceinline__ uint32_t at_pack(float lo, float hi) {
  const at_f2 v = {lo, hi};
  if constexpr (BF) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, at_b2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, at_h2));
}

__device__ __forceinline__ float at_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
// the subtrahend of an exponent: 0 where nothing has been seen (2^(-inf - 0) = 0)
__device__ __forceinline__ float at_safe(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// low (H = 0) or high halves of two words beside each other: (a, b)
template <int H> __device__ __forceinline__ uint32_t at_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, H ? 0x07060302u : 0x05040100u);
}

// Non-finite values.  A weight of 0 does not keep a NaN or infinity out of a sum
// of products, so where a tile holds tokens that some of its rows see and others
// do not, its values are looked at, and where one is not finite the products run
// over the values with 0 in its place, and the rows that do see it (a product of
// indicators) get it added: +inf, -inf, or both for a NaN.
template <bool BF> __device__ __forceinline__ uint32_t at_exp_mask() { return BF ? 0x7F80u : 0x7C00u; }
template <bool BF> __device__ __forceinline__ bool at_odd1(uint32_t h) { return (h & at_exp_mask<BF>()) == at_exp_mask<BF>(); }
template <bool BF> __device__ __forceinline__ bool at_odd(uint32_t w) { return at_odd1<BF>(w) || at_odd1<BF>(w >> 16); }
template <bool BF> __device__ __forceinline__ uint32_t at_one() { return BF ? 0x3F80u : 0x3C00u; }
// one half: finite part, and indicators of +inf-or-NaN and -inf-or-NaN
template <bool BF> __device__ __forceinline__ uint32_t at_fin1(uint32_t h) { return at_odd1<BF>(h) ? 0u : h & 0xFFFFu; }
template <bool BF> __device__ __forceinline__ uint32_t at_ind1(uint32_t h, bool neg) {
  const bool nan = (h & 0x7FFFu) > at_exp_mask<BF>();
  return at_odd1<BF>(h) && (nan || ((h & 0x8000u) != 0) == neg) ? at_one<BF>() : 0u;
}
template <bool BF> __device__ __forceinline__ uint32_t at_fin(uint32_t w) {
  return at_fin1<BF>(w) | at_fin1<BF>(w >> 16) << 16;
}
template <bool BF> __device__ __forceinline__ uint32_t at_ind(uint32_t w, bool neg) {
  return at_ind1<BF>(w, neg) | at_ind1<BF>(w >> 16, neg) << 16;
}
// what a row that sees p values of +inf or NaN and n of -inf or NaN has to add
__device__ __forceinline__ float at_add_odd(float p, float n) {
  const float inf = __builtin_inff();
  return (p > 0.0f ? inf : 0.0f) + (n > 0.0f ? -inf : 0.0f);
}

// Partials go past the per-XCD L2 caches (agent scope), as in qg_common.h.
__device__ __forceinline__ void at_st(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float at_ld(const float* p) {
  return __hip_atomic_load(const_cast<float*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The workgroup's arrival at a counter of n, after its partial: true in the one
// that completes the count (which leaves the counter at zero for the next launch).
__device__ __forceinline__ bool at_last(int* counter, int n, int* flag) {
  __builtin_amdgcn_s_waitcnt(0);  // this thread's stores have completed
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
    if (last) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = last;
  }
  __syncthreads();
  return *flag != 0;
}

// N columns of a finished row: r-th row of a kv head (new token r / G, q head
// r % G of the group), columns c ..  L = 0 is a row that sees nothing (p < 0, output
// 0) or one whose every score is -inf (0 / 0).
template <bool BF, int N>
__device__ __forceinline__ void at_store(const AttnArgs& a, const KvEntry& e, int head, int r, int c, const float* o, float L) {
  const int i = r / a.G;
  const float inv = L != 0.0f ? 1.0f / L : (e.len - e.rows + i < 0 ? 0.0f : __builtin_nanf(""));
  uint16_t* to = const_cast<uint16_t*>(a.out.ptr) + (int64_t)(e.row0 + i) * a.out.row +
                 (int64_t)(head * a.G + r - i * a.G) * a.out.head + c;
  uint32_t w[N / 2];
#pragma unroll
  for (int x = 0; x < N / 2; ++x) w[x] = at_pack<BF>(o[2 * x] * inv, o[2 * x + 1] * inv);
  if constexpr (N == 4) {
    *reinterpret_cast<kv_u2*>(to) = kv_u2{w[0], w[1]};
  } else {
#pragma unroll
    for (int x = 0; x < N / 2; x += 4) *reinterpret_cast<kv_u4*>(to + 2 * x) = kv_u4{w[x], w[x + 1], w[x + 2], w[x + 3]};
  }
}

// Join n partials of rows r0 .. r0 + nrows - 1 of (entry, head) in the order 0, 1,
// ...; slot(k) is the k-th: [ld][D] fp32, then (m, l) of each row.  The loads of
// eight partials are in flight at once.
template <bool BF, int D, class F>
__device__ __forceinline__ void at_join(const AttnArgs& a, const KvEntry& e, int head, int r0, int nrows, int ld, int n, F slot) {
  constexpr int NB = 8;
  for (int it = threadIdx.x; it < nrows * (D / 4); it += blockDim.x) {
    const int r = it / (D / 4), c = (it % (D / 4)) * 4;
    float M = -__builtin_inff(), L = 0.0f, o[4] = {0, 0, 0, 0};
    for (int k0 = 0; k0 < n; k0 += NB) {
      float pm[NB], pl[NB], po[NB][4];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float* s = slot(min(k0 + k, n - 1));
        pm[k] = at_ld(s + (size_t)ld * D + 2 * r);
        pl[k] = at_ld(s + (size_t)ld * D + 2 * r + 1);
#pragma unroll
        for (int x = 0; x < 4; ++x) po[k][x] = at_ld(s + (size_t)r * D + c + x);
      }
      float Mn = M;
#pragma unroll
      for (int k = 0; k < NB; ++k) Mn = fmaxf(Mn, pm[k]);
      const float f0 = at_exp2(M - at_safe(Mn));
      M = Mn;
      L *= f0;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] *= f0;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (k0 + k >= n) break;
        const float f = at_exp2(pm[k] - at_safe(Mn));
        L = __builtin_fmaf(f, pl[k], L);
#pragma unroll
        for (int x = 0; x < 4; ++x) o[x] = __builtin_fmaf(f, po[k][x], o[x]);
      }
    }
    at_store<BF, 4>(a, e, head, r0 + r, c, o, L);
  }
}

// The tokens that rows at positions p0 .. p1 see between them, as tiles of TK:
// the tiles of the sinks, then those of the window up to p1.  n tiles; tile j
// of them covers tokens TK * at(j) ...
template <int TK> struct TileRange {
  int ns, skip, n;
  __device__ __forceinline__ TileRange(int p0, int p1, int window, int sinks) {
    const int end = (p1 + TK) / TK;  // p1 >= -1
    const int lo = window ? max(max(p0, 0) - window + 1, 0) / TK : 0;
    ns = window ? min((min(sinks, p1 + 1) + TK - 1) / TK, end) : 0;
    skip = max(lo - ns, 0);
    n = max(end - skip, 0);
  }
  __device__ __forceinline__ int at(int j) const { return j < ns ? j : j + skip; }
};

// does the row at position pos see token t?
__device__ __forceinline__ bool at_sees(int pos, int t, int window, int sinks) {
  return t <= pos && (window == 0 || t > pos - window || t < sinks);
}
// do all rows at positions p0 .. p1 see all tokens of [t0, t1]?
__device__ __forceinline__ bool at_all_see(int p0, int p1, int t0, int t1, int window, int sinks) {
  return t1 <= p0 && (window == 0 || t0 > p1 - window || t1 < sinks);
}

}  // namespace qg
