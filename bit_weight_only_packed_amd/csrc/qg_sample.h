// qg_sample.h -- picking tokens from logits: temperature, top-k, top-p, min-p.
//
//   w_i = 2^(log2(e) (l_i - max) / T); of the tokens in the order (logit down, index up) the first k,
//   then the fewest with p of their mass, then those with w >= min_p; the picked token is the first by
//   index up to which the kept mass passes u * (all of it).
//
// Which token comes out hangs on comparisons of sums, so the sums are exact: a weight is
// fp64 (exp2, off by some 2^-52 of itself), rounded to a multiple of 2^-43, and weights are added as
// 64-bit integers.  Integer sums do not depend on their order, so they may meet by atomics.
//
// The order is never made whole.  A row's logits fall into SM_BUCKETS buckets by their distance
// from the largest (log2 of the weight in steps of 44 / SM_BUCKETS); counts and masses of the buckets
// say in which one the k-th token lies, and in which one p of the mass is reached; only
// that bucket's few logits are put in order.  So four launches, each over (part of the row, row):
//   k_sample_max   the parts' largest logits
//   k_sample_hist  counts and masses of the buckets (rows with top-k or top-p)
//   k_sample_cut   the last kept token (rows with top-k or top-p; one workgroup a row)
//   k_sample_pick  masses of the kept tokens by part; the last part of a row to arrive picks
#pragma once
#include "qg_attn.h"
#include "qg_step.h"

namespace qg {

constexpr int SM_BUCKETS = SAMPLE_BUCKETS;
constexpr int SM_BITS = 43;         // weights are multiples of 2^-SM_BITS: 2^20 of them stay below 2^63
constexpr int SM_LIST = 512;        // tokens put in order against each other
constexpr int SM_T = 256;           // threads of the kernels over parts
constexpr int SM_CUT = 1024;        // threads of k_sample_cut

typedef uint32_t sm_u4 __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned long long sm_u64;

// order of logits as unsigned numbers (no NaN, no -0)
__device__ __forceinline__ uint32_t sm_key(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float sm_clean(float f) {
  f += 0.0f;  // -0 is 0
  return f == f ? f : -__builtin_inff();
}
// 8 logits at `at` of which `left` are there (the others, and NaN: -inf)
template <int TY> __device__ __forceinline__ void sm_load(float (&v)[8], const void* row, int at, int left) {
  if constexpr (TY == QGS_F32) {
    const float* p = reinterpret_cast<const float*>(row) + at;
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    if (left >= 8) {
      const f4 x = *reinterpret_cast<const f4*>(p), y = *reinterpret_cast<const f4*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = x[i], v[i + 4] = y[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : -__builtin_inff();
    }
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + at;
    constexpr uint32_t none = TY == QGS_BF16 ? 0xFF80u : 0xFC00u;
    uint32_t h[8];
    if (left >= 8) {
      const sm_u4 x = *reinterpret_cast<const sm_u4*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (x[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = i < left ? p[i] : none;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (TY == QGS_BF16) v[i] = __builtin_bit_cast(float, h[i] << 16);
      else v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)h[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = sm_clean(v[i]);
}

// what a row asks for
struct SmRow {
  float heat, p, min_p;
  int k;         // 0: no limit
  bool greedy, cut;  // cut: top-k or top-p
  __device__ __forceinline__ SmRow(const SampleArgs& a, int row) {
    heat = a.temperature ? a.temperature[row] : a.temperature1;
    k = a.top_k ? a.top_k[row] : a.top_k1;
    p = a.top_p ? a.top_p[row] : a.top_p1;
    min_p = a.min_p ? a.min_p[row] : a.min_p1;
    greedy = !(heat > 0.0f);
    k = k > 0 && k < a.vocab ? k : 0;
    p = p < 1.0f ? p : 1.0f;
    min_p = min_p > 0.0f ? min_p : 0.0f;
    cut = !greedy && (k > 0 || p < 1.0f);
  }
};

// weights of a row
struct SmScale {
  float top, per_bucket;
  double rate;
  __device__ __forceinline__ SmScale(float top_, float heat) : top(top_) {
    rate = 1.4426950408889634 / (double)heat;
    per_bucket = (float)(rate * (SM_BUCKETS / 44.0));
  }
  // Monotone in l: a rounded difference, times a constant, cut off.  SM_BUCKETS: a weight of 0.
  __device__ __forceinline__ int bucket(float l) const {
    if (l == top) return 0;
    if (l == -__builtin_inff()) return SM_BUCKETS;
    const float x = (top - l) * per_bucket;
    return x < (float)SM_BUCKETS ? (int)x : SM_BUCKETS;
  }
  __device__ __forceinline__ double share(float l) const { return l == top ? 1.0 : exp2(((double)l - (double)top) * rate); }
  __device__ __forceinline__ sm_u64 fixed(double s) const { return (sm_u64)rint(s * (double)(1ull << SM_BITS)); }
  __device__ __forceinline__ sm_u64 weight(float l) const { return bucket(l) < SM_BUCKETS ? fixed(share(l)) : 0; }
};

// a row's largest logit, from its parts' (every thread calls it)
__device__ __forceinline__ float sm_top(const SampleArgs& a, int row, int* arg = nullptr) {
  float m = -__builtin_inff();
  int at = 0;
  for (int p = 0; p < a.parts; ++p) {  // the same addresses for all lanes
    const float x = a.part_max[(int64_t)row * a.parts + p];
    if (x > m) m = x, at = p;
  }
  if (arg) *arg = a.part_arg[(int64_t)row * a.parts + at];
  return m;
}
template <int TY> __device__ __forceinline__ const void* sm_row(const SampleArgs& a, int row) {
  return reinterpret_cast<const char*>(a.logits) + (int64_t)row * a.stride * (TY == QGS_F32 ? 4 : 2);
}

template <int TY> __global__ __launch_bounds__(SM_T) void k_sample_max(SampleArgs a) {
  __shared__ float lm[SM_T / 64];
  __shared__ int la[SM_T / 64];
  const int part = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  const void* x = sm_row<TY>(a, row);
  const int a0 = part * a.part_len, a1 = min(a0 + a.part_len, a.vocab);
  // what the later kernels add to
  for (int b = part * SM_T + tid; b < SM_BUCKETS; b += a.parts * SM_T) {
    a.counts[(int64_t)row * SM_BUCKETS + b] = 0;
    a.masses[(int64_t)row * SM_BUCKETS + b] = 0;
  }
  if (part == 0 && tid == 0) a.arrived[row] = 0;
  float m = -__builtin_inff();
  int arg = a0;
  for (int at = a0 + tid * 8; at < a1; at += SM_T * 8) {
    float v[8];
    sm_load<TY>(v, x, at, a1 - at);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v[i] > m) m = v[i], arg = at + i;
  }
  const auto better = [](float x, int i, float y, int j) { return y > x || (y == x && j < i); };
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float y = __shfl_xor(m, o);
    const int j = __shfl_xor(arg, o);
    if (better(m, arg, y, j)) m = y, arg = j;
  }
  if ((tid & 63) == 0) lm[tid >> 6] = m, la[tid >> 6] = arg;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < SM_T / 64; ++w)
      if (better(m, arg, lm[w], la[w])) m = lm[w], arg = la[w];
    a.part_max[(int64_t)row * a.parts + part] = m;
    a.part_arg[(int64_t)row * a.parts + part] = arg;
  }
}

template <int TY> __global__ __launch_bounds__(SM_T) void k_sample_hist(SampleArgs a) {
  __shared__ uint32_t cnt[SM_BUCKETS];
  __shared__ sm_u64 mass[SM_BUCKETS];
  const int part = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  const SmRow r(a, row);
  if (!r.cut) return;
  const SmScale sc(sm_top(a, row), r.heat);
  const bool masses = r.p < 1.0f || r.k > 0;
  for (int b = tid; b < SM_BUCKETS; b += SM_T) cnt[b] = 0, mass[b] = 0;
  __syncthreads();
  const void* x = sm_row<TY>(a, row);
  const int a0 = part * a.part_len, a1 = min(a0 + a.part_len, a.vocab);
  for (int at = a0 + tid * 8; at < a1; at += SM_T * 8) {
    float v[8];
    sm_load<TY>(v, x, at, a1 - at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int b = sc.bucket(v[i]);
      if (b >= SM_BUCKETS) continue;
      atomicAdd(&cnt[b], 1u);
      if (masses) atomicAdd(&mass[b], sc.fixed(sc.share(v[i])));
    }
  }
  __syncthreads();
  for (int b = tid; b < SM_BUCKETS; b += SM_T)
    if (cnt[b]) {
      atomicAdd(&a.counts[(int64_t)row * SM_BUCKETS + b], cnt[b]);
      if (masses) atomicAdd(&a.masses[(int64_t)row * SM_BUCKETS + b], mass[b]);
    }
}

// inclusive sums over the SM_CUT threads; lds: a T per wave
template <class T> __device__ __forceinline__ T sm_scan(T v, T* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const T y = __shfl_up(v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 63) lds[wave] = v;
  __syncthreads();
  for (int w = 0; w < waves; ++w)
    if (w < wave) v += lds[w];
  return v;
}
// the lowest thread for which it holds, or blockDim.x
__device__ __forceinline__ int sm_first(bool hit, int* lds) {
  __syncthreads();
  if (threadIdx.x == 0) *lds = blockDim.x;
  __syncthreads();
  if (hit) atomicMin(lds, (int)threadIdx.x);
  __syncthreads();
  return *lds;
}

// a token's place in the order: larger is earlier
__device__ __forceinline__ sm_u64 sm_place(uint32_t key, int index) { return (sm_u64)key << 32 | (uint32_t)~index; }

struct SmCutLds {
  uint32_t cnt[SM_BUCKETS];
  sm_u64 mass[SM_BUCKETS];
  sm_u64 list[SM_LIST], weight[SM_LIST];
  sm_u64 sums[SM_CUT / 64];
  int counts[SM_CUT / 64];
  int n, first;
  uint32_t lo, hi;
  sm_u64 last, got, taken;
};

// every token of the row: f(logit, index)
template <int TY, class F> __device__ __forceinline__ void sm_each(const SampleArgs& a, const void* x, F f) {
  for (int at = threadIdx.x * 8; at < a.vocab; at += SM_CUT * 8) {
    float v[8];
    sm_load<TY>(v, x, at, a.vocab - at);
#pragma unroll
    for (int i = 0; i < 8; ++i) f(v[i], at + i);
  }
}

// The last kept token's place among those of a bucket that lie at `limit` or before it in the
// order: the need-th of them (need > 0), or the first at which `before` and their weights reach
// `goal`.  kept: the mass of the bucket's kept tokens.
template <int TY>
__device__ sm_u64 sm_refine(const SampleArgs& a, const void* x, const SmScale& sc, int bucket, sm_u64 limit, int need,
                            sm_u64 before, double goal, SmCutLds& s, sm_u64* kept) {
  const int tid = threadIdx.x;
  uint32_t lo = 0, hi = 0xFFFFFFFFu;
  int skipped = 0;     // tokens of the bucket that lie before the range, and their mass
  sm_u64 passed = 0;
  const auto inside = [&](float l, int i) {
    const uint32_t k = sm_key(l);
    return k >= lo && k <= hi && sc.bucket(l) == bucket && sm_place(k, i) >= limit;
  };
  for (;;) {
    // how many, from where to where; the first SM_LIST of them
    __syncthreads();
    if (tid == 0) s.n = 0, s.lo = 0xFFFFFFFFu, s.hi = 0;
    __syncthreads();
    sm_each<TY>(a, x, [&](float l, int i) {
      if (!inside(l, i)) return;
      const uint32_t k = sm_key(l);
      const int at = atomicAdd(&s.n, 1);
      if (at < SM_LIST) s.list[at] = sm_place(k, i), s.weight[at] = sc.weight(l);
      atomicMin(&s.lo, k);
      atomicMax(&s.hi, k);
    });
    __syncthreads();
    const int n = s.n;
    lo = s.lo, hi = s.hi;
    if (n <= SM_LIST) {
      if (tid == 0) s.last = ~0ull, s.got = 0;
      __syncthreads();
      if (tid < n) {
        const sm_u64 mine = s.list[tid];
        int rank = 0;
        sm_u64 mass = passed;
        for (int j = 0; j < n; ++j) {
          const bool early = s.list[j] > mine;
          rank += early;
          mass += early ? s.weight[j] : 0;
        }
        const bool in = need > 0 ? skipped + rank < need : (before + mass == 0) || (double)(before + mass) < goal;
        if (in) {
          atomicMin(&s.last, mine);
          atomicMax(&s.got, mass + s.weight[tid]);
        }
      }
      __syncthreads();
      *kept = s.got;
      return s.last;
    }
    if (lo == hi) {
      // equal logits: so many of them, by index
      float l = 0.0f;
      {
        const uint32_t b = (lo >> 31) ? lo ^ 0x80000000u : ~lo;
        l = __builtin_bit_cast(float, b);
      }
      const sm_u64 w = sc.weight(l);
      int m = need > 0 ? need - skipped : n;
      if (need <= 0 && w > 0) {
        const double left = (goal - (double)(before + passed)) / (double)w;
        m = left >= n ? n : max((int)left - 1, 1);
        while (m < n && (double)(before + passed + (sm_u64)m * w) < goal) ++m;
      }
      // the index of the m-th
      int seen = 0, index = a.vocab;
      for (int at0 = 0; at0 < a.vocab; at0 += SM_CUT * 8) {
        const int at = at0 + tid * 8;
        float v[8];
        sm_load<TY>(v, x, at, a.vocab - at);
        int c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) c += at + i < a.vocab && sm_key(v[i]) == lo && sm_place(lo, at + i) >= limit;
        const int upto = seen + sm_scan(c, s.counts);
        if (tid == SM_CUT - 1) s.n = upto;
        if (upto >= m && upto - c < m) {
          int k = upto - c;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            k += at + i < a.vocab && sm_key(v[i]) == lo && sm_place(lo, at + i) >= limit;
            if (k == m) {
              s.first = at + i;
              break;
            }
          }
        }
        __syncthreads();
        seen = s.n;
        if (seen >= m) {
          index = s.first;
          break;
        }
      }
      __syncthreads();
      *kept = passed + (sm_u64)m * w;
      return sm_place(lo, index);
    }
    // cut the range into SM_BUCKETS pieces
    int shift = 0;
    while (((hi - lo) >> shift) >= SM_BUCKETS) ++shift;
    s.cnt[tid] = 0, s.mass[tid] = 0;
    __syncthreads();
    sm_each<TY>(a, x, [&](float l, int i) {
      if (!inside(l, i)) return;
      const int b = (int)((hi - sm_key(l)) >> shift);
      atomicAdd(&s.cnt[b], 1u);
      atomicAdd(&s.mass[b], sc.weight(l));
    });
    __syncthreads();
    const int c = (int)s.cnt[tid];
    const sm_u64 w = s.mass[tid];
    const int cc = skipped + sm_scan(c, s.counts);
    const sm_u64 ww = passed + sm_scan(w, s.sums);
    int b = sm_first(c > 0 && (need > 0 ? cc >= need : (double)(before + ww) >= goal), &s.first);
    if (b >= SM_BUCKETS) b = (int)((hi - lo) >> shift);  // (the goal lies past a rounding: the last)
    __syncthreads();
    if (tid == b) s.n = cc - c, s.taken = ww - w;
    __syncthreads();
    skipped = s.n, passed = s.taken;
    const uint32_t top = hi - ((uint32_t)b << shift), span = (1u << shift) - 1;
    lo = top - lo > span ? top - span : lo;
    hi = top;
  }
}

template <int TY> __global__ __launch_bounds__(SM_CUT) void k_sample_cut(SampleArgs a) {
  __shared__ SmCutLds s;
  const int row = blockIdx.x, tid = threadIdx.x;
  const SmRow r(a, row);
  sm_u64 last = 0;  // everything is kept
  if (r.cut) {
    const SmScale sc(sm_top(a, row), r.heat);
    if (sc.top > -__builtin_inff()) {
      const void* x = sm_row<TY>(a, row);
      const int c = (int)a.counts[(int64_t)row * SM_BUCKETS + tid];
      const sm_u64 w = a.masses[(int64_t)row * SM_BUCKETS + tid];
      const int cc = sm_scan(c, s.counts);
      const sm_u64 ww = sm_scan(w, s.sums);
      __syncthreads();
      if (tid == SM_CUT - 1) s.taken = ww;
      __syncthreads();
      sm_u64 all = s.taken;
      int bk = SM_BUCKETS;
      if (r.k > 0) {
        bk = sm_first(cc >= r.k, &s.first);
        if (bk < SM_BUCKETS) {  // (else the k-th token has a weight of 0: nothing of weight is cut)
          __syncthreads();
          if (tid == bk) s.n = cc - c, s.taken = ww - w;
          __syncthreads();
          const int need = r.k - s.n;
          const sm_u64 before = s.taken;
          sm_u64 kept;
          last = sm_refine<TY>(a, x, sc, bk, 0, need, before, 0.0, s, &kept);
          all = before + kept;
        }
      }
      if (r.p < 1.0f) {
        const double goal = (double)r.p * (double)all;
        const int bp = min(sm_first((double)ww >= goal && c > 0, &s.first), bk);
        if (bp < SM_BUCKETS) {
          __syncthreads();
          if (tid == bp) s.taken = ww - w;
          __syncthreads();
          const sm_u64 before = s.taken;
          sm_u64 kept;
          last = sm_refine<TY>(a, x, sc, bp, bp == bk ? last : 0, 0, before, goal, s, &kept);
        }
      }
    }
  }
  if (tid == 0) a.last[row] = last;
}

template <int TY> __global__ __launch_bounds__(SM_T) void k_sample_pick(SampleArgs a) {
  __shared__ sm_u64 sums[SM_T / 64];
  __shared__ int flag, found;
  __shared__ sm_u64 mine;
  const int part = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  const SmRow r(a, row);
  int arg;
  const float top = sm_top(a, row, &arg);
  if (r.greedy || top == -__builtin_inff()) {
    if (part == 0 && tid == 0) {
      const bool none = top == -__builtin_inff();
      a.tokens[row] = none ? -1 : arg;
      if (a.probs) a.probs[row] = none ? 0.0f : 1.0f;
    }
    return;
  }
  const SmScale sc(top, r.heat);
  const sm_u64 last = r.cut ? a.last[row] : 0;
  const uint32_t least = (uint32_t)(last >> 32);
  const double min_p = fmin((double)r.min_p, 1.0);
  const void* x = sm_row<TY>(a, row);
  // the weight of a kept token, 0 of others
  const auto weight = [&](float l, int i) -> sm_u64 {
    const uint32_t k = sm_key(l);
    if (k < least || (k == least && sm_place(k, i) < last) || sc.bucket(l) >= SM_BUCKETS) return 0;
    const double s = sc.share(l);
    return s >= min_p ? sc.fixed(s) : 0;
  };
  const auto eight = [&](int at, int end, sm_u64 (&w)[8]) {
    float v[8];
    sm_load<TY>(v, x, at, end - at);
    sm_u64 t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += w[i] = weight(v[i], at + i);
    return t;
  };
  const int a0 = part * a.part_len, a1 = min(a0 + a.part_len, a.vocab);
  sm_u64 sum = 0, w[8];
  for (int at = a0 + tid * 8; at < a1; at += SM_T * 8) sum += eight(at, a1, w);
  sum = sm_scan(sum, sums);
  if (tid == SM_T - 1) __hip_atomic_store(&a.part_sum[(int64_t)row * a.parts + part], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!at_last(a.arrived + row, a.parts, &flag)) return;
  // the part that holds the token
  sm_u64 total = 0;
  for (int p = 0; p < a.parts; ++p)
    total += __hip_atomic_load(&a.part_sum[(int64_t)row * a.parts + p], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const float u = a.u[row];
  sm_u64 goal = u > 0.0f ? (sm_u64)fmin((double)u * (double)total, 9.2e18) : 0;
  goal = goal < total ? goal : total - 1;
  sm_u64 passed = 0;
  int p = 0;
  for (; p < a.parts - 1; ++p) {
    const sm_u64 t = __hip_atomic_load(&a.part_sum[(int64_t)row * a.parts + p], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (passed + t > goal) break;
    passed += t;
  }
  const int b0 = p * a.part_len, b1 = min(b0 + a.part_len, a.vocab);
  if (tid == 0) found = -1;
  for (int at0 = b0; at0 < b1; at0 += SM_T * 8) {
    const int at = at0 + tid * 8;
    const sm_u64 t = eight(at, b1, w);
    const sm_u64 upto = passed + sm_scan(t, sums);
    if (upto > goal && upto - t <= goal) {
      sm_u64 run = upto - t;
      bool open = true;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        run += w[i];
        if (open && run > goal) {
          open = false;
          found = at + i;
          a.tokens[row] = at + i;
          if (a.probs) a.probs[row] = (float)((double)w[i] / (double)total);
        }
      }
    }
    __syncthreads();
    if (found >= 0) return;
    if (tid == SM_T - 1) mine = upto;
    __syncthreads();
    passed = mine;
  }
}

}  // namespace qg
