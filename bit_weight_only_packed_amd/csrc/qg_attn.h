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
//
// Weights meet the values on the matrix cores as fp16 or bf16, one rounding each: in 32
// bits that product would run at a sixteenth of the rate, and in two parts at half of it, to
// take a whole output from 2.6e-4 off (fp16; bf16 2.3e-3) to the 2.0e-4 (1.7e-3) of its own
// rounding.  fp16 would lose those below 2^-14 of the largest bit by bit and those below
// 2^-25 whole: behind one token that takes nearly all the weight (a sink with a value of
// 0) that can be all of the output.  So in fp16 every weight, in o and in l alike, is larger
// by a fixed power of two, which the division by l takes away again: the largest reach
// 2^AT_FP16_TOP.
#pragma once
#include "qg_kv.h"

namespace qg {

constexpr float AT_FP16_TOP = 15.0f;

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

// s_waitcnt vmcnt(n), the other counters left alone
__host__ __device__ constexpr int at_wait_vm(int n) { return (n & 15) | 0x0F70 | (n >> 4) << 14; }

// maximum over the lanes that differ in bit 5 (32), or in bits 4 and 5 (16)
__device__ __forceinline__ float at_max32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float at_max16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return at_max32(fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])));
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
// do not, its values are looked at.  One that is not finite is taken out (0) and
// noted, a bit for +inf or NaN and a bit for -inf or NaN; after the products each
// row that does see the token gets the infinity added, or both.
template <bool BF> __device__ __forceinline__ uint32_t at_exp_mask() { return BF ? 0x7F80u : 0x7C00u; }
template <bool BF> __device__ __forceinline__ bool at_odd1(uint32_t h) { return (h & at_exp_mask<BF>()) == at_exp_mask<BF>(); }
// the larger magnitude of two halves and m: not finite from at_exp_mask on
__device__ __forceinline__ uint32_t at_top(uint32_t m, uint32_t w) { return max(max(m, w & 0x7FFFu), (w >> 16) & 0x7FFFu); }
// take what is not finite out of two values; bits `at` and `at` + 1 of pos and neg note it
template <bool BF> __device__ __forceinline__ uint32_t at_take(uint32_t w, int at, uint32_t& pos, uint32_t& neg) {
  asm volatile("" : "+v"(w));  // its classification is not carried over from the check: registers are dearer here
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = (w >> (16 * i)) & 0xFFFFu;
    const uint32_t odd = at_odd1<BF>(h), nan = (h & 0x7FFFu) > at_exp_mask<BF>(), sign = h >> 15;
    pos |= (odd & (nan | (sign ^ 1u))) << (at + i);
    neg |= (odd & (nan | sign)) << (at + i);
    if (odd) w &= ~(0xFFFFu << (16 * i));
  }
  return w;
}
// what bits p and n of a noted value add to the output of a row that sees it
__device__ __forceinline__ float at_noted(uint32_t p, uint32_t n) {
  const float inf = __builtin_inff();
  return ((p & 1) ? inf : 0.0f) + ((n & 1) ? -inf : 0.0f);
}

// Partials go past the per-XCD L2 caches (agent scope), as in qg_common.h, here
// 16 bytes at a time: buffer accesses with the cache policy of an agent-scope atomic.
constexpr int AT_AGENT = 16;  // sc1
__device__ __forceinline__ __amdgpu_buffer_rsrc_t at_slots(float* p, size_t floats) {
  return __builtin_amdgcn_make_buffer_rsrc(p, 0, (int)(floats * 4), 0x00020000);
}
__device__ __forceinline__ void at_st4(__amdgpu_buffer_rsrc_t r, uint32_t at, at_f4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(kv_u4, v), r, (int)(at * 4), 0, AT_AGENT);
}
__device__ __forceinline__ void at_st2(__amdgpu_buffer_rsrc_t r, uint32_t at, float x, float y) {
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(kv_u2, at_f2{x, y}), r, (int)(at * 4), 0, AT_AGENT);
}
__device__ __forceinline__ at_f4 at_ld4(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(at_f4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(at * 4), 0, AT_AGENT));
}
__device__ __forceinline__ at_f2 at_ld2(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(at_f2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)(at * 4), 0, AT_AGENT));
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
  const float inv = L != 0.0f ? 1.0f / L : (e.pos + i < 0 ? 0.0f : __builtin_nanf(""));
  uint16_t* to = const_cast<uint16_t*>(a.out.ptr) + (int64_t)(e.row0 + i) * a.out.row +
                 (int64_t)(head * a.G + r - i * a.G) * a.out.head + c;
  uint32_t w[N / 2];
#pragma unroll
  for (int x = 0; x < N / 2; ++x) w[x] = at_pack<BF>(o[2 * x] * inv, o[2 * x + 1] * inv);
  if constexpr (N == 2) {
    *reinterpret_cast<uint32_t*>(to) = w[0];
  } else if constexpr (N == 4) {
    *reinterpret_cast<kv_u2*>(to) = kv_u2{w[0], w[1]};
  } else {
#pragma unroll
    for (int x = 0; x < N / 2; x += 4) *reinterpret_cast<kv_u4*>(to + 2 * x) = kv_u4{w[x], w[x + 1], w[x + 2], w[x + 3]};
  }
}

// Join n partials of rows f0 .. f0 + nrows - 1 of a block of (entry, head) that begins
// with row r0; slot(k) is where the k-th lies (in floats): [ld][D] fp32, then (m, l) of each row.  Every sum runs in an
// order that n fixes.
//
// A round trip to the partials costs about 2 us, so there are two: one for all (m, l),
// whose factors 2^(m_k - M) / sum go to LDS (a wave per row), and one for the outputs,
// sixteen partials at a time; where the rows are few, several threads share an item
// of four columns, each with a contiguous part of the partials.
// fac, tot, part: AT_JOIN_CAP floats of LDS each; n <= AT_JOIN_CAP.
constexpr int AT_JOIN_CAP = 2720;  // (row, partial) pairs at a time; 4 floats of 512 threads fit as well
template <bool BF, int D, int THREADS, class F>
__device__ __forceinline__ void at_join(const AttnArgs& a, __amdgpu_buffer_rsrc_t rs, const KvEntry& e, int head, int r0, int f0,
                                        int nrows, int ld, int n, float* fac, float* tot, float* part, F slot) {
  constexpr int NB = 16, NW = THREADS / 64;
  static_assert(4 * THREADS <= AT_JOIN_CAP, "part");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = min(nrows, AT_JOIN_CAP / n);
  // fac [row][partial] m, then its factor; tot [row][partial] l, then [row][0] the sum;
  // part [thread][4] outputs of threads that share an item
  for (int rb = f0; rb < f0 + nrows; rb += chunk) {
    const int rows = min(chunk, f0 + nrows - rb);
    __syncthreads();
    for (int x = tid; x < rows * n; x += THREADS) {
      const int r = x / n, k = x - r * n;
      const at_f2 ml = at_ld2(rs, slot(k) + (uint32_t)ld * D + 2 * (rb + r));
      fac[x] = ml.x;
      tot[x] = ml.y;
    }
    __syncthreads();
    for (int r = wave; r < rows; r += NW) {
      float M = -__builtin_inff(), L = 0.0f;
      for (int k = lane; k < n; k += 64) M = fmaxf(M, fac[r * n + k]);
#pragma unroll
      for (int o = 32; o; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
      M = at_safe(M);
      for (int k = lane; k < n; k += 64) {
        const float f = at_exp2(fac[r * n + k] - M);
        fac[r * n + k] = f;
        L = __builtin_fmaf(f, tot[r * n + k], L);
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) L += __shfl_xor(L, o);
      if (lane == 0) tot[r * n] = L;
    }
    __syncthreads();
    const int items = rows * (D / 4);
    int groups = 1;  // threads per item: a power of two
    while (2 * groups * items <= THREADS && groups * NB < n) groups *= 2;
    const int g = groups > 1 ? tid / items : 0;
    const int k0 = n * g / groups, k1 = n * (g + 1) / groups;
    for (int it = tid - g * items; it < items; it += THREADS) {
      const int r = it / (D / 4), c = (it % (D / 4)) * 4;
      const uint32_t at = (uint32_t)(rb + r) * D + c;
      at_f4 o = {0, 0, 0, 0};
      if (g < groups)
        for (int kb = k0; kb < k1; kb += NB) {
          at_f4 po[NB];
#pragma unroll
          for (int k = 0; k < NB; ++k)
            if (kb + k < k1) po[k] = at_ld4(rs, at + slot(kb + k));
#pragma unroll
          for (int k = 0; k < NB; ++k)
            if (kb + k < k1) {
              const float f = fac[r * n + kb + k];
#pragma unroll
              for (int x = 0; x < 4; ++x) o[x] = __builtin_fmaf(f, po[k][x], o[x]);
            }
        }
      if (groups == 1) {
        const float res[4] = {o.x, o.y, o.z, o.w};
        at_store<BF, 4>(a, e, head, r0 + rb + r, c, res, tot[r * n]);
      } else if (g < groups) {
        *reinterpret_cast<at_f4*>(part + tid * 4) = o;
      }
    }
    if (groups == 1) continue;
    __syncthreads();
    if (tid < items) {
      const int r = tid / (D / 4), c = (tid % (D / 4)) * 4;
      float o[4] = {0, 0, 0, 0};
      for (int i = 0; i < groups; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[x] += part[(i * items + tid) * 4 + x];
      at_store<BF, 4>(a, e, head, r0 + rb + r, c, o, tot[r * n]);
    }
  }
}

// The tokens that rows at positions p0 .. p1 see between them, as tiles of TK:
// the tiles of the sinks, then those of the window up to p1.  n tiles; tile j
// of them covers tokens TK * at(j) ...
template <int TK> struct TileRange {
  int ns, skip, n;
  __device__ __forceinline__ TileRange(int p0, int p1, int window, int sinks) {
    const int end = (p1 + TK) / TK;  // p1 < 0: none (0 or less)
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
// The same for many tokens base + c of one row: t is seen iff pos - t, unsigned, is
// below `span`, or c below `first`.  (Two compares a token; and the users put up
// barriers between tokens, for a mask per token and compare would take every
// scalar register, those of the main loop among them.)
struct SeenFrom {
  int d, first;
  uint32_t span;
  __device__ __forceinline__ SeenFrom(int pos, int base, int window, int sinks)
      : d(pos - base), first(min(sinks, pos + 1) - base), span(pos < 0 ? 0u : window ? (uint32_t)window : 0x80000000u) {}
  __device__ __forceinline__ bool operator()(int c) const { return (int)((uint32_t)(d - c) < span) | (int)(c < first); }
};
// do all rows at positions p0 .. p1 see all tokens of [t0, t1]?
__device__ __forceinline__ bool at_all_see(int p0, int p1, int t0, int t1, int window, int sinks) {
  return t1 <= p0 && (window == 0 || t0 > p1 - window || t1 < sinks);
}

}  // namespace qg
