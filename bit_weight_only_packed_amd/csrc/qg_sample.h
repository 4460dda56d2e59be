// qg_sample.h -- picking tokens from logits: temperature, top-k, top-p, min-p.
//
//   w_i = 2^(log2(e) (l_i - max) / T); of the tokens in the order (logit down, index up) the first k,
//   then the fewest with p of their mass, then those with w >= min_p; the picked token is the first by
//   index up to which the kept mass passes u * (all of it).
//
// Which token comes out hangs on comparisons of sums, so the sums are exact: a weight is
// fp64 (a table and a series, off by 2^-49 of itself at most), rounded to a multiple of 2^-43, and weights are added as
// 64-bit integers.  Integer sums do not depend on their order, so they may meet by atomics.
//
// The order is never made whole.  A row's logits fall into SM_BUCKETS buckets by their distance
// from the largest (log2 of the weight in steps of 44 / SM_BUCKETS); counts and masses of the buckets
// say in which ones the k-th token lies and p of the mass is reached.  The tokens of these buckets, or,
// where they are few, all kept ones, come together in a list that is sorted in LDS.  Four launches, each
// over (part of the row, row), of which a row takes what it needs; the last part of a row to
// arrive does what is done once a row:
//   k_sample_max   the parts' largest logits
//   k_sample_hist  rows with top-k or top-p: the buckets' counts and masses; which of them are listed
//   k_sample_list  the same rows: the list; the last kept token, and if all kept ones are listed, the
//                  picked one.  (A list that overflows, as of thousands of equal logits: the
//                  row is gone through again by one workgroup, in as many passes as it takes.)
//   k_sample_pick  the other rows, and those with more kept tokens than a list: masses of the parts,
//                  then the part that holds the picked one
// Bound: the chain of dependent round trips (three arrivals of the parts among them) where rows are few, the
// LDS additions and fp64 weights of every token where they are many; reading the logits is a small part.  One
// row of 131,071 (top-k 50, top-p 0.95): 3.1 + 11.4 + 15.0 + 3.9 us; 128 rows of 100,003 with settings of every
// kind: 9 + 23 + 33 + 23 us.  Rows that are short go whole to a workgroup each (k_sample_row), one launch.
#pragma once
#include "qg_attn.h"
#include "qg_step.h"

namespace qg {

constexpr int SM_BUCKETS = SAMPLE_BUCKETS;
constexpr int SM_BITS = 43;         // weights are multiples of 2^-SM_BITS: 2^20 of them stay below 2^63
constexpr int SM_LIST = 512;        // tokens ranked against each other where a list has overflowed
constexpr int SM_CAP = SAMPLE_LIST; // tokens of a list
constexpr int SM_WHOLE = 512;       // kept tokens that are listed all
constexpr int SM_RANK = 512;        // words sorted by counting
constexpr int SM_T = 256;           // threads of a workgroup that has a part of a row,
constexpr int SM_ROW_T = 512;       // and of one that has all of it

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

// 2^(i / 128), which the workgroup makes once
constexpr int SM_TAB = 128;
__device__ __forceinline__ void sm_table(double* tab) {
  for (int i = threadIdx.x; i < SM_TAB; i += blockDim.x) tab[i] = exp2((double)i / SM_TAB);
  __syncthreads();
}

// weights of a row
struct SmScale {
  float top, per_bucket;
  double rate;         // log2(e) / temperature
  // Temperatures so large that logits whose difference passes fp32 have weights, or so small that
  // per_bucket does: buckets in fp64, for all of the row.
  bool wide;
  const double* tab;
  __device__ __forceinline__ SmScale(float top_, float heat, const double* tab_) : top(top_), tab(tab_) {
    rate = 1.4426950408889634 / (double)heat;
    per_bucket = (float)(rate * (SM_BUCKETS / 44.0));
    wide = !(per_bucket >= 0x1p-117f && per_bucket < __builtin_inff());
  }
  // Monotone in l: a rounded difference, times a constant, cut off.  SM_BUCKETS: a weight of 0.
  __device__ __forceinline__ int bucket(float l) const {
    if (l == top) return 0;
    float x = (top - l) * per_bucket;  // (infinite where l is -inf)
    if (__builtin_expect(wide, 0)) {
      if (l == -__builtin_inff() || top == __builtin_inff()) return SM_BUCKETS;
      x = (float)(((double)top - (double)l) * (rate * (SM_BUCKETS / 44.0)));
    }
    return x < (float)SM_BUCKETS ? (int)x : SM_BUCKETS;
  }
  // The weight of a logit in a bucket, in units of 2^-SM_BITS, before its rounding: 2^e = 2^(n / 128) 2^f
  // with |f| <= 2^-8, and 2^f by its series to f^4 (the next term is at most 2^-49.5): 15 instructions, where
  // exp2 takes some 40 (one row of 131,071 by one workgroup: 91 us against 108).
  __device__ __forceinline__ double scaled(float l) const {
    if (l == top) return (double)(1ull << SM_BITS);  // (infinities among them)
    const double e = ((double)l - (double)top) * rate, r = rint(e * SM_TAB), f = __builtin_fma(r, -1.0 / SM_TAB, e);
    constexpr double c1 = 0.6931471805599453, c2 = c1 * c1 / 2, c3 = c1 * c1 * c1 / 6, c4 = c1 * c1 * c1 * c1 / 24;
    const double p = __builtin_fma(f, __builtin_fma(f, __builtin_fma(f, __builtin_fma(f, c4, c3), c2), c1), 1.0);
    const int n = (int)r;
    return ldexp(p * tab[n & (SM_TAB - 1)], (n >> 7) + SM_BITS);
  }
  static_assert(SM_TAB == 1 << 7);
  // rounded to a whole number by the addition of 2^52, which leaves it in the low bits
  __device__ __forceinline__ static sm_u64 fixed(double w) { return __builtin_bit_cast(sm_u64, w + 0x1p52) - __builtin_bit_cast(sm_u64, 0x1p52); }
  __device__ __forceinline__ sm_u64 weight(float l) const { return bucket(l) < SM_BUCKETS ? fixed(scaled(l)) : 0; }
};
// min_p in the same units; at most that of the largest
__device__ __forceinline__ double sm_min(const SmRow& r) { return fmin((double)r.min_p, 1.0) * (double)(1ull << SM_BITS); }

// a row's largest logit and where it first stands, from its parts' (64 at most: a lane each)
__device__ __forceinline__ bool sm_better(float x, int i, float y, int j) { return y > x || (y == x && j < i); }
__device__ __forceinline__ float sm_top(const SampleArgs& a, int row, int* arg = nullptr) {
  const int lane = threadIdx.x & 63;
  float m = -__builtin_inff();
  int at = 0x7FFFFFFF;
  if (lane < a.parts) m = a.part_max[(int64_t)row * a.parts + lane], at = a.part_arg[(int64_t)row * a.parts + lane];
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float y = __shfl_xor(m, o);
    const int j = __shfl_xor(at, o);
    if (sm_better(m, at, y, j)) m = y, at = j;
  }
  if (arg) *arg = at;
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
  if (part == 0 && tid < 4) a.arrived[4 * row + tid] = 0;
  float m = -__builtin_inff();
  int arg = a0;
  for (int at = a0 + tid * 8; at < a1; at += SM_T * 8) {
    float v[8];
    sm_load<TY>(v, x, at, a1 - at);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v[i] > m) m = v[i], arg = at + i;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float y = __shfl_xor(m, o);
    const int j = __shfl_xor(arg, o);
    if (sm_better(m, arg, y, j)) m = y, arg = j;
  }
  if ((tid & 63) == 0) lm[tid >> 6] = m, la[tid >> 6] = arg;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < SM_T / 64; ++w)
      if (sm_better(m, arg, lm[w], la[w])) m = lm[w], arg = la[w];
    a.part_max[(int64_t)row * a.parts + part] = m;
    a.part_arg[(int64_t)row * a.parts + part] = arg;
  }
}

// inclusive sums over the workgroup; lds: a word per wave
template <int T, class V> __device__ __forceinline__ V sm_scan(V v, V* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const V y = __shfl_up(v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 63) lds[wave] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; ++w)
    if (w < wave) v += lds[w];
  return v;
}

// a token's place in the order: larger is earlier
__device__ __forceinline__ sm_u64 sm_place(uint32_t key, int index) { return (sm_u64)key << 32 | (uint32_t)~index; }
__device__ __forceinline__ float sm_logit(uint32_t key) {
  return __builtin_bit_cast(float, (key >> 31) ? key ^ 0x80000000u : ~key);
}

// Counts and masses of the buckets, PER consecutive ones a thread, and where they cross.
struct SmScanLds {
  sm_u64 sums[SM_ROW_T / 64], mass;
  int counts[SM_ROW_T / 64], at, count, own;
};
struct SmAt {
  int bucket;    // SM_BUCKETS: none
  int count;     // tokens in the buckets before it,
  sm_u64 mass;   // their mass,
  int own;       // and its own tokens
};
template <int T> struct SmBuckets {
  static constexpr int PER = SM_BUCKETS / T;
  int c[PER], c0;       // c0, w0: of the buckets before this thread's
  sm_u64 w[PER], w0;
  __device__ __forceinline__ void scan(SmScanLds& s) {
    int ct = 0;
    sm_u64 wt = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) ct += c[i], wt += w[i];
    c0 = sm_scan<T>(ct, s.counts) - ct;
    w0 = sm_scan<T>(wt, s.sums) - wt;
  }
  // the first bucket with tokens at whose end hit(count, mass) holds
  template <class F> __device__ __forceinline__ SmAt cross(SmScanLds& s, F hit) const {
    int mine = SM_BUCKETS, own = 0, cc = c0, cb = 0;
    sm_u64 ww = w0, wb = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (mine == SM_BUCKETS && c[i] > 0 && hit(cc + c[i], ww + w[i])) mine = PER * threadIdx.x + i, cb = cc, wb = ww, own = c[i];
      cc += c[i], ww += w[i];
    }
    __syncthreads();
    if (threadIdx.x == 0) s.at = SM_BUCKETS, s.count = 0, s.mass = 0, s.own = 0;
    __syncthreads();
    if (mine < SM_BUCKETS) atomicMin(&s.at, mine);
    __syncthreads();
    if (mine < SM_BUCKETS && mine == s.at) s.count = cb, s.mass = wb, s.own = own;
    __syncthreads();
    return SmAt{s.at, s.count, s.mass, s.own};
  }
  __device__ __forceinline__ sm_u64 all(SmScanLds& s) const {  // the whole mass
    sm_u64 t = w0;
#pragma unroll
    for (int i = 0; i < PER; ++i) t += w[i];
    __syncthreads();
    if (threadIdx.x == T - 1) s.mass = t;
    __syncthreads();
    return s.mass;
  }
};

// What a row's buckets have said.
enum { SM_PICK = 0, SM_ALL = 1, SM_SOME = 2, SM_SLOW = 3, SM_DONE = 4 };

// whether the masses are asked for: they say nothing that a list of all tokens down to the k-th would not
__device__ __forceinline__ bool sm_masses(const SmRow& r) { return r.p < 1.0f && !(r.k > 0 && r.k <= SM_WHOLE / 2); }

// What the buckets (scanned) say: which of them are listed, and what lies before them.
template <int T> __device__ __forceinline__ SmPlan sm_plan(const SmBuckets<T>& h, const SmRow& r, bool masses, SmScanLds& s) {
  SmPlan p{SM_PICK};
  p.k_bucket = SM_BUCKETS, p.hi = SM_BUCKETS - 1;
  bool bounded = false;  // whether something of weight is cut off by top-k
  if (r.k > 0) {
    const SmAt k = h.cross(s, [&](int c, sm_u64) { return c >= r.k; });
    bounded = k.bucket < SM_BUCKETS;  // (else the k-th token has a weight of 0)
    if (bounded) {
      p.k_bucket = k.bucket, p.k_count = k.count, p.k_mass = k.mass;
      p.mode = k.count + k.own <= SM_WHOLE ? SM_ALL : r.p < 1.0f ? (masses ? SM_SOME : SM_SLOW) : k.own <= SM_CAP ? SM_SOME : SM_SLOW;
      p.lo = p.hi = k.bucket, p.lo_mass = k.mass;
      if (p.mode == SM_ALL) p.lo = 0;
      if (p.mode == SM_SOME && r.p < 1.0f) {
        // p of the mass lies between p of it without the k-th token's bucket and p of it with
        const sm_u64 most = h.cross(s, [&](int c, sm_u64) { return c > k.count + k.own; }).mass;  // up to that bucket's end
        const sm_u64 upto = most > 0 ? most : h.all(s);
        const double from = (double)r.p * (double)k.mass, to = (double)r.p * (double)upto;
        const SmAt l = h.cross(s, [&](int, sm_u64 w) { return (double)w >= from; });
        const SmAt e = h.cross(s, [&](int, sm_u64 w) { return (double)w >= to; });
        p.lo = l.bucket, p.lo_mass = l.mass;
        p.hi = min(e.bucket, k.bucket);
        const int n = e.count + e.own - l.count + (p.hi < k.bucket ? k.own : 0);
        if (n > SM_CAP) p.mode = SM_SLOW;
      }
    }
  }
  if (!bounded && r.p < 1.0f) {
    if (!masses) {
      p.mode = SM_ALL;  // fewer than k tokens have any weight
      p.lo = 0;
    } else {
      const double goal = (double)r.p * (double)h.all(s);
      const SmAt e = h.cross(s, [&](int, sm_u64 w) { return (double)w >= goal; });
      p.mode = e.count + e.own <= SM_WHOLE ? SM_ALL : e.own <= SM_CAP ? SM_SOME : SM_SLOW;
      p.lo = p.mode == SM_ALL ? 0 : e.bucket, p.hi = e.bucket;
      p.lo_mass = p.mode == SM_ALL ? 0 : e.mass;
    }
  }
  p.total = masses ? h.all(s) : 0;
  return p;
}

template <int TY> __global__ __launch_bounds__(SM_T) void k_sample_hist(SampleArgs a) {
  __shared__ uint32_t cnt[SM_BUCKETS];
  __shared__ sm_u64 mass[SM_BUCKETS];
  __shared__ SmScanLds s;
  __shared__ int flag;
  const int part = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  const SmRow r(a, row);
  if (!r.cut) return;
  __shared__ double tab[SM_TAB];
  sm_table(tab);
  const SmScale sc(sm_top(a, row), r.heat, tab);
  SmPlan& plan = a.plan[row];
  if (sc.top == -__builtin_inff()) {
    if (part == 0 && tid == 0) plan = SmPlan{SM_PICK};
    return;
  }
  const bool masses = sm_masses(r);
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
      if (masses) atomicAdd(&mass[b], sc.fixed(sc.scaled(v[i])));
    }
  }
  __syncthreads();
  // Of a part that holds k tokens alone, the buckets past its own k-th have none of the row's first k.
  int upto = SM_BUCKETS - 1;
  SmBuckets<SM_T> h;
  constexpr int PER = SmBuckets<SM_T>::PER;
  if (r.k > 0 && r.k < a1 - a0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) h.c[i] = (int)cnt[PER * tid + i], h.w[i] = 0;
    h.scan(s);
    upto = min(h.cross(s, [&](int c, sm_u64) { return c >= r.k; }).bucket, upto);
  }
  uint32_t* counts = a.counts + (int64_t)row * SM_BUCKETS;
  sm_u64* sums = a.masses + (int64_t)row * SM_BUCKETS;
  for (int b = tid; b <= upto; b += SM_T)
    if (cnt[b]) {
      atomicAdd(&counts[b], cnt[b]);
      if (masses) atomicAdd(&sums[b], mass[b]);
    }
  if (!at_last(a.arrived + 4 * row, a.parts, &flag)) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    h.c[i] = (int)__hip_atomic_load(&counts[PER * tid + i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    h.w[i] = masses ? __hip_atomic_load(&sums[PER * tid + i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
  }
  h.scan(s);
  const SmPlan p = sm_plan<SM_T>(h, r, masses, s);
  if (tid == 0) plan = p;
}

// ---- a list that has overflowed: one workgroup, as many passes over the row as it takes ----

struct SmSlowLds {
  uint32_t cnt[SM_BUCKETS];
  sm_u64 mass[SM_BUCKETS];
  sm_u64 list[SM_LIST], weight[SM_LIST];
  int n, first;
  uint32_t lo, hi;
  sm_u64 last, got;
};

// every token of the row: f(logit, index)
template <int TY, int T, class F> __device__ __forceinline__ void sm_each(const SampleArgs& a, const void* x, F f) {
  for (int at = threadIdx.x * 8; at < a.vocab; at += T * 8) {
    float v[8];
    sm_load<TY>(v, x, at, a.vocab - at);
#pragma unroll
    for (int i = 0; i < 8; ++i) f(v[i], at + i);
  }
}
// counts and masses of the tokens by which(logit, index), SM_BUCKETS or more: none
template <int TY, int T, class F>
__device__ __forceinline__ void sm_count(SmBuckets<T>& h, const SampleArgs& a, const void* x, const SmScale& sc, SmSlowLds& s, SmScanLds& t, F which) {
  __syncthreads();
  for (int b = threadIdx.x; b < SM_BUCKETS; b += T) s.cnt[b] = 0, s.mass[b] = 0;
  __syncthreads();
  sm_each<TY, T>(a, x, [&](float l, int i) {
    const int b = which(l, i);
    if (b >= SM_BUCKETS) return;
    atomicAdd(&s.cnt[b], 1u);
    atomicAdd(&s.mass[b], sc.weight(l));
  });
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SmBuckets<T>::PER; ++i) h.c[i] = (int)s.cnt[SmBuckets<T>::PER * threadIdx.x + i], h.w[i] = s.mass[SmBuckets<T>::PER * threadIdx.x + i];
  h.scan(t);
}

// The last kept token's place among those of a bucket that lie at `limit` or before it in the
// order: the need-th of them (need > 0), or the first at which `before` and their weights reach
// `goal`.  kept: the mass of the bucket's kept tokens.
template <int TY, int T>
__device__ __forceinline__ sm_u64 sm_refine(const SampleArgs& a, const void* x, const SmScale& sc, int bucket, sm_u64 limit, int need,
                                            sm_u64 before, double goal, SmSlowLds& s, SmScanLds& t, sm_u64* kept) {
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
    sm_each<TY, T>(a, x, [&](float l, int i) {
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
      for (int e = tid; e < n; e += T) {
        const sm_u64 mine = s.list[e];
        int rank = 0;
        sm_u64 mass = passed;
        for (int j = 0; j < n; ++j) {
          const bool early = s.list[j] > mine;
          rank += early;
          mass += early ? s.weight[j] : 0;
        }
        const bool in = need > 0 ? skipped + rank < need : before + mass == 0 || (double)(before + mass) < goal;
        if (in) {
          atomicMin(&s.last, mine);
          atomicMax(&s.got, mass + s.weight[e]);
        }
      }
      __syncthreads();
      *kept = s.got;
      return s.last;
    }
    if (lo == hi) {
      // equal logits: so many of them, by index
      const sm_u64 w = sc.weight(sm_logit(lo));
      int m = need > 0 ? need - skipped : n;
      if (need <= 0 && w > 0) {
        const double left = (goal - (double)(before + passed)) / (double)w;
        m = left >= n ? n : max((int)left - 1, 1);
        while (m < n && (double)(before + passed + (sm_u64)m * w) < goal) ++m;
      }
      // the index of the m-th
      int seen = 0, index = a.vocab;
      for (int at0 = 0; at0 < a.vocab; at0 += T * 8) {
        const int at = at0 + tid * 8;
        float v[8];
        sm_load<TY>(v, x, at, a.vocab - at);
        int c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) c += at + i < a.vocab && sm_key(v[i]) == lo && sm_place(lo, at + i) >= limit;
        const int upto = seen + sm_scan<T>(c, t.counts);
        if (tid == T - 1) s.n = upto;
        if (upto >= m && upto - c < m) {
          int k = upto - c, found = -1;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            k += at + i < a.vocab && sm_key(v[i]) == lo && sm_place(lo, at + i) >= limit;
            if (found < 0 && k == m) found = at + i;
          }
          s.first = found;
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
    SmBuckets<T> h;
    sm_count<TY, T>(h, a, x, sc, s, t, [&](float l, int i) { return inside(l, i) ? (int)((hi - sm_key(l)) >> shift) : SM_BUCKETS; });
    SmAt b = h.cross(t, [&](int c, sm_u64 w) { return need > 0 ? skipped + c >= need : (double)(before + passed + w) >= goal; });
    if (b.bucket >= SM_BUCKETS) {  // (the goal lies past a rounding: the last)
      const int end = (int)((hi - lo) >> shift);
      b = h.cross(t, [&](int c, sm_u64) { return c == n; });
      b.bucket = end;
    }
    skipped += b.count, passed += b.mass;
    const uint32_t top = hi - ((uint32_t)b.bucket << shift), span = (1u << shift) - 1;
    lo = top - lo > span ? top - span : lo;
    hi = top;
  }
}

template <int TY, int T>
__device__ __forceinline__ sm_u64 sm_slow(const SampleArgs& a, const void* x, const SmRow& r, const SmScale& sc, SmSlowLds& s, SmScanLds& t) {
  SmBuckets<T> h;
  sm_u64 last = 0, all = 0, kept;
  int bk = SM_BUCKETS;
#pragma unroll 1
  for (int stage = 0; stage < 2; ++stage) {  // top-k, then top-p of what that leaves
    if (stage == 0 ? r.k <= 0 : r.p >= 1.0f) continue;
    sm_count<TY, T>(h, a, x, sc, s, t, [&](float l, int) { return sc.bucket(l); });
    if (bk == SM_BUCKETS) all = h.all(t);
    const double goal = (double)r.p * (double)all;
    const SmAt e = h.cross(t, [&](int c, sm_u64 w) { return stage == 0 ? c >= r.k : (double)w >= goal; });
    if (e.bucket >= SM_BUCKETS) continue;
    last = sm_refine<TY, T>(a, x, sc, e.bucket, stage == 1 && e.bucket == bk ? last : 0, stage == 0 ? r.k - e.count : 0, e.mass, goal, s, t, &kept);
    if (stage == 0) bk = e.bucket, all = e.mass + kept;
  }
  return last;
}

// ---- lists ----

// n distinct words in LDS, falling.  Up to SM_RANK of them each thread counts the words above
// its own, all reads on their way at once and the same for all lanes (64 words: 0.3 us, where the 21
// dependent steps of a sorting network take 4.6); above that the network.
template <int T> __device__ __forceinline__ void sm_sort(sm_u64* list, int n) {
  constexpr int E = SM_RANK > T ? SM_RANK / T : 1;
  __syncthreads();
  if (n <= SM_RANK) {
    sm_u64 mine[E];
    int rank[E];
#pragma unroll
    for (int e = 0; e < E; ++e) mine[e] = threadIdx.x + e * T < n ? list[threadIdx.x + e * T] : ~0ull, rank[e] = 0;
    if (n <= T) {
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank[0] += list[j] > mine[0];
    } else {
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const sm_u64 x = list[j];
#pragma unroll
        for (int e = 0; e < E; ++e) rank[e] += x > mine[e];
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (threadIdx.x + e * T < n) list[rank[e]] = mine[e];
  } else {
    int size = SM_RANK;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += T) list[i] = 0;  // (no word is 0)
    for (int k = 2; k <= size; k <<= 1)
      for (int j = k >> 1; j; j >>= 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < size / 2; i += T) {
          const int x = 2 * i - (i & (j - 1));
          const sm_u64 u = list[x], v = list[x + j];
          if ((u < v) == ((x & k) == 0)) list[x] = v, list[x + j] = u;
        }
      }
  }
  __syncthreads();
}

// the multiple of 2^-SM_BITS that u of a total is, held to [0, total)
__device__ __forceinline__ sm_u64 sm_goal(float u, sm_u64 total) {
  const sm_u64 g = u > 0.0f ? (sm_u64)fmin((double)u * (double)total, 9.2e18) : 0;
  return g < total ? g : total - 1;
}

// The n listed tokens of a row put in order, and what is kept of them.  SM_SOME: the last kept token's
// place is returned.  SM_ALL: the token is picked and written, and ~0 is returned.
template <int T>
__device__ __forceinline__ sm_u64 sm_finish(const SampleArgs& a, int row, const SmRow& r, const SmScale& sc, const SmPlan& plan,
                                            sm_u64* list, int n, SmScanLds& t) {
  const int tid = threadIdx.x;
  sm_sort<T>(list, n);
  // this thread's consecutive tokens, their weights, and the mass before them
  constexpr int MOST = SM_CAP / T;
  const int per = (n + T - 1) / T, i0 = tid * per;
  sm_u64 w[MOST], before;
  const auto masses = [&](auto weight) {
    sm_u64 sum = 0;
#pragma unroll
    for (int e = 0; e < MOST; ++e) {
      w[e] = e < per && i0 + e < n ? weight(i0 + e) : 0;
      sum += w[e];
    }
    before = sm_scan<T>(sum, t.sums) - sum;
  };
  const auto logit = [&](int i) { return sm_logit((uint32_t)(list[i] >> 32)); };
  masses([&](int i) { return sc.weight(logit(i)); });
  // the first token of the list at which hit(index, mass up to and with it) holds (n: none), and that mass
  const auto first = [&](auto hit, int none, sm_u64* upto) {
    __syncthreads();
    if (tid == 0) t.at = none;
    __syncthreads();
    sm_u64 run = before;
#pragma unroll
    for (int e = 0; e < MOST; ++e) {
      run += w[e];
      if (e < per && i0 + e < n && hit(i0 + e, run)) atomicMin(&t.at, i0 + e);
    }
    __syncthreads();
    const int at = t.at;
    run = before;
#pragma unroll
    for (int e = 0; e < MOST; ++e) {
      run += w[e];
      if (e < per && i0 + e == at) t.mass = run;
    }
    __syncthreads();
    *upto = t.mass;
    return at;
  };
  int kept = n;       // of the list
  sm_u64 total, got;  // total: the mass of what top-k leaves
  if (plan.k_bucket < SM_BUCKETS) {
    // the tokens before the k-th one's bucket that are listed
    const int skip = first([&](int i, sm_u64) { return sc.bucket(logit(i)) >= plan.k_bucket; }, n, &got);
    kept = min(skip + r.k - plan.k_count, n);
    first([&](int i, sm_u64) { return i == kept - 1; }, kept - 1, &total);
    if (plan.mode == SM_SOME) {
      sm_u64 ahead = 0;  // mass of the listed tokens before that bucket
      if (skip > 0) first([&](int i, sm_u64) { return i == skip - 1; }, skip - 1, &ahead);
      total = total - ahead + plan.k_mass;
    }
  } else if (plan.mode == SM_SOME) {
    total = plan.total;
  } else {
    first([&](int i, sm_u64) { return i == n - 1; }, n - 1, &total);
    if (plan.total > 0) total = plan.total;  // (the list ends with the bucket that p is reached in)
  }
  if (r.p < 1.0f) {
    const double goal = (double)r.p * (double)total;
    const sm_u64 base = plan.mode == SM_SOME ? plan.lo_mass : 0;
    kept = min(kept, first([&](int, sm_u64 run) { return (double)(base + run) >= goal; }, kept - 1, &got) + 1);
  }
  if (plan.mode == SM_SOME) return list[kept - 1];
  // everything that is kept is listed: min-p, then the token
  const double min_p = sm_min(r);
  kept = min(kept, first([&](int i, sm_u64) { return sc.scaled(logit(i)) < min_p; }, n, &got));
  // by rising index: ~index falls
  for (int i = tid; i < kept; i += T) list[i] = list[i] << 32 | list[i] >> 32;
  sm_sort<T>(list, kept);
  const auto logit2 = [&](int i) { return sm_logit((uint32_t)list[i]); };
  masses([&](int i) { return i < kept ? sc.weight(logit2(i)) : 0; });
  first([&](int i, sm_u64) { return i == kept - 1; }, kept - 1, &total);
  const sm_u64 goal = sm_goal(a.u[row], total);
  const int at = first([&](int i, sm_u64 run) { return run > goal; }, kept - 1, &got);
  if (tid == 0) {
    const sm_u64 e = list[at];
    a.tokens[row] = (int)~(uint32_t)(e >> 32);
    if (a.probs) a.probs[row] = (float)((double)sc.weight(sm_logit((uint32_t)e)) / (double)total);
  }
  return ~0ull;
}

template <int TY> __global__ __launch_bounds__(SM_T) void k_sample_list(SampleArgs a) {
  __shared__ union {
    sm_u64 list[SM_CAP];
    SmSlowLds slow;
  } m;
  __shared__ SmScanLds t;
  __shared__ int flag, cut;
  const int part = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  const SmRow r(a, row);
  if (!r.cut) return;
  const SmPlan plan = a.plan[row];
  if (plan.mode == SM_PICK) {
    if (part == 0 && tid == 0) a.last[row] = 0;
    return;
  }
  __shared__ double tab[SM_TAB];
  sm_table(tab);
  const SmScale sc(sm_top(a, row), r.heat, tab);
  const void* x = sm_row<TY>(a, row);
  if (plan.mode == SM_SLOW) {
    if (part > 0) return;
    const sm_u64 last = sm_slow<TY, SM_T>(a, x, r, sc, m.slow, t);
    if (tid == 0) a.last[row] = last;
    return;
  }
  sm_u64* list = a.list + (int64_t)row * SM_CAP;
  int* length = a.arrived + 4 * row + 3;
  const int a0 = part * a.part_len, a1 = min(a0 + a.part_len, a.vocab);
  if (tid == 0) cut = 0;
  __syncthreads();
  for (int at = a0 + tid * 8; at < a1; at += SM_T * 8) {
    float v[8];
    sm_load<TY>(v, x, at, a1 - at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int b = sc.bucket(v[i]);
      if (((b < plan.lo) | (b > plan.hi)) & (b != plan.k_bucket) | (b >= SM_BUCKETS)) continue;
      const int to = atomicAdd(&cut, 1);  // (the part's: the list's places are asked for once a part)
      if (to < SM_CAP) m.list[to] = sm_place(sm_key(v[i]), at + i);
    }
  }
  __syncthreads();
  const int mine = min(cut, SM_CAP);
  if (tid == 0 && mine > 0) flag = atomicAdd(length, mine);
  __syncthreads();
  for (int i = tid; i < mine; i += SM_T)
    if (flag + i < SM_CAP) __hip_atomic_store(&list[flag + i], m.list[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (!at_last(a.arrived + 4 * row + 1, a.parts, &flag)) return;
  const int n = min(__hip_atomic_load(length, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), SM_CAP);
  for (int i = tid; i < n; i += SM_T) m.list[i] = __hip_atomic_load(&list[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const sm_u64 last = sm_finish<SM_T>(a, row, r, sc, plan, m.list, n, t);
  if (tid == 0) {
    a.last[row] = last;
    if (plan.mode == SM_ALL) a.plan[row].mode = SM_DONE;
  }
}

// the weights of the tokens of a row that are kept
struct SmKept {
  const SmScale& sc;
  sm_u64 last;    // the last kept token's place
  uint32_t least;
  double min_p;
  int most;       // buckets past which no weight reaches min_p (one more, for the roundings)
  __device__ __forceinline__ SmKept(const SmRow& r, const SmScale& sc_, sm_u64 last_) : sc(sc_), last(last_) {
    least = (uint32_t)(last >> 32);
    min_p = sm_min(r);
    most = r.min_p > 0.0f ? (int)fmin(1.0 - log2((double)r.min_p) * (SM_BUCKETS / 44.0), (double)SM_BUCKETS) : SM_BUCKETS;
    most = max(most, 0);
  }
  __device__ __forceinline__ sm_u64 weight(float l, int i) const {
    const uint32_t k = sm_key(l);
    const int b = sc.bucket(l);
    if (k < least || (k == least && sm_place(k, i) < last) || b >= SM_BUCKETS || b > most) return 0;
    const double s = sc.scaled(l);
    return s >= min_p ? sc.fixed(s) : 0;
  }
  // of 8 tokens from `at` on, and their sum
  template <int TY> __device__ __forceinline__ sm_u64 eight(const void* x, int at, int end, sm_u64 (&w)[8]) const {
    float v[8];
    sm_load<TY>(v, x, at, end - at);
    sm_u64 t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += w[i] = weight(v[i], at + i);
    return t;
  }
};

template <int TY> __global__ __launch_bounds__(SM_T) void k_sample_pick(SampleArgs a) {
  __shared__ sm_u64 sums[SM_T / 64];
  __shared__ int flag, found;
  __shared__ sm_u64 mine;
  const int part = blockIdx.x, row = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const SmRow r(a, row);
  if (r.cut && a.plan[row].mode == SM_DONE) return;
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
  __shared__ double tab[SM_TAB];
  sm_table(tab);
  const SmScale sc(top, r.heat, tab);
  const sm_u64 last = r.cut ? a.last[row] : 0;
  const SmKept keep(r, sc, last);
  const void* x = sm_row<TY>(a, row);
  const auto eight = [&](int at, int end, sm_u64 (&w)[8]) { return keep.template eight<TY>(x, at, end, w); };
  const int a0 = part * a.part_len, a1 = min(a0 + a.part_len, a.vocab);
  sm_u64 sum = 0, w[8];
  for (int at = a0 + tid * 8; at < a1; at += SM_T * 8) sum += eight(at, a1, w);
  sum = sm_scan<SM_T>(sum, sums);
  if (tid == SM_T - 1) __hip_atomic_store(&a.part_sum[(int64_t)row * a.parts + part], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!at_last(a.arrived + 4 * row + 2, a.parts, &flag)) return;
  // the part that holds the token (64 at most: a lane each)
  sm_u64 passed = 0;
  if (lane < a.parts) passed = __hip_atomic_load(&a.part_sum[(int64_t)row * a.parts + lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const sm_u64 own = passed;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const sm_u64 y = __shfl_up(passed, o);
    if (lane >= o) passed += y;
  }
  const sm_u64 total = __shfl(passed, 63), goal = sm_goal(a.u[row], total);
  const int p = __builtin_ctzll(__ballot(passed > goal));
  passed = __shfl(passed - own, p);
  const int b0 = p * a.part_len, b1 = min(b0 + a.part_len, a.vocab);
  if (tid == 0) found = -1;
  for (int at0 = b0; at0 < b1; at0 += SM_T * 8) {
    const int at = at0 + tid * 8;
    const sm_u64 t = eight(at, b1, w);
    const sm_u64 upto = passed + sm_scan<SM_T>(t, sums);
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

// The whole of it for a row by one workgroup, in one launch: where rows are short the launches cost more than
// the passes, and where rows are many the parts' meetings do (sample_whole in k_sample.hip).
template <int TY> __global__ __launch_bounds__(SM_ROW_T) void k_sample_row(SampleArgs a) {
  constexpr int T = SM_ROW_T, W = T / 64;
  __shared__ union {
    sm_u64 list[SM_CAP];
    SmSlowLds slow;
    sm_u64 waves[QGS_MAX_VOCAB / 512];  // masses of 512 tokens each
  } m;
  __shared__ SmScanLds t;
  __shared__ float lm[W];
  __shared__ int la[W], cut;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const SmRow r(a, row);
  const void* x = sm_row<TY>(a, row);
  float top = -__builtin_inff();
  int arg = 0x7FFFFFFF;
  sm_each<TY, T>(a, x, [&](float l, int i) {
    if (l > top) top = l, arg = i;
  });
  const auto meet = [&](int o) {
    const float y = __shfl_xor(top, o);
    const int j = __shfl_xor(arg, o);
    if (sm_better(top, arg, y, j)) top = y, arg = j;
  };
#pragma unroll
  for (int o = 32; o; o >>= 1) meet(o);
  if (lane == 0) lm[wave] = top, la[wave] = arg;
  __syncthreads();
  top = lm[lane % W], arg = la[lane % W];
#pragma unroll
  for (int o = W / 2; o; o >>= 1) meet(o);
  if (r.greedy || top == -__builtin_inff()) {
    if (tid == 0) {
      const bool none = top == -__builtin_inff();
      a.tokens[row] = none ? -1 : arg;
      if (a.probs) a.probs[row] = none ? 0.0f : 1.0f;
    }
    return;
  }
  __shared__ double tab[SM_TAB];
  sm_table(tab);
  const SmScale sc(top, r.heat, tab);
  sm_u64 last = 0;
  if (r.cut) {
    const bool masses = sm_masses(r);
    for (int b = tid; b < SM_BUCKETS; b += T) m.slow.cnt[b] = 0, m.slow.mass[b] = 0;
    __syncthreads();
    sm_each<TY, T>(a, x, [&](float l, int) {
      const int b = sc.bucket(l);
      if (b >= SM_BUCKETS) return;
      atomicAdd(&m.slow.cnt[b], 1u);
      if (masses) atomicAdd(&m.slow.mass[b], sc.fixed(sc.scaled(l)));
    });
    __syncthreads();
    SmBuckets<T> h;
#pragma unroll
    for (int i = 0; i < h.PER; ++i) h.c[i] = (int)m.slow.cnt[h.PER * tid + i], h.w[i] = m.slow.mass[h.PER * tid + i];
    h.scan(t);
    const SmPlan plan = sm_plan<T>(h, r, masses, t);
    if (plan.mode == SM_SLOW) {
      last = sm_slow<TY, T>(a, x, r, sc, m.slow, t);
    } else if (plan.mode != SM_PICK) {
      __syncthreads();
      if (tid == 0) cut = 0;
      __syncthreads();
      sm_each<TY, T>(a, x, [&](float l, int i) {
        const int b = sc.bucket(l);
        if (((b < plan.lo) | (b > plan.hi)) & (b != plan.k_bucket) | (b >= SM_BUCKETS)) return;
        const int to = atomicAdd(&cut, 1);
        if (to < SM_CAP) m.list[to] = sm_place(sm_key(l), i);
      });
      __syncthreads();
      last = sm_finish<T>(a, row, r, sc, plan, m.list, min(cut, SM_CAP), t);
      if (plan.mode == SM_ALL) return;
    }
    __syncthreads();
  }
  // masses of the kept tokens, 512 consecutive ones a wave, then the ones that hold the token
  const SmKept keep(r, sc, last);
  const int n = (a.vocab + 511) / 512;
  sm_u64 w[8];
  for (int k = wave; k < n; k += W) {
    sm_u64 sum = keep.template eight<TY>(x, k * 512 + lane * 8, a.vocab, w);
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) m.waves[k] = sum;
  }
  __syncthreads();
  constexpr int PER = QGS_MAX_VOCAB / 512 / T;
  sm_u64 part[PER], mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    part[i] = tid * PER + i < n ? m.waves[tid * PER + i] : 0;
    mine += part[i];
  }
  sm_u64 run = sm_scan<T>(mine, t.sums);
  if (tid == T - 1) t.mass = run;
  run -= mine;
  __syncthreads();
  const sm_u64 total = t.mass, goal = sm_goal(a.u[row], total);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (run <= goal && goal < run + part[i]) t.at = tid * PER + i, t.mass = run;
    run += part[i];
  }
  __syncthreads();
  if (wave > 0) return;
  const int at = t.at * 512 + lane * 8;
  const sm_u64 own = keep.template eight<TY>(x, at, a.vocab, w);
  run = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const sm_u64 y = __shfl_up(run, o);
    if (lane >= o) run += y;
  }
  run += t.mass - own;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (run <= goal && goal < run + w[i]) {
      a.tokens[row] = at + i;
      if (a.probs) a.probs[row] = (float)((double)w[i] / (double)total);
    }
    run += w[i];
  }
}

}  // namespace qg
