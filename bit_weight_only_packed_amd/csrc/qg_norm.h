// qg_norm.h -- root-mean-square norm of rows, with the residual's addition before it
// and, if wanted, its output in 8 bits with scales.
//
//   h = round(x + r),  y = h w / sqrt(mean h^2 + eps),  codes round(y / s), s = max |y| / top
//
// Bound.  HBM where rows are many: each operand is read once and each output written
// once, and a row lives in registers between its sum and its outputs.  8,191 rows of 5,120 with the residual
// (bf16): 53 us, 336 MB at 6.3 TB/s (some of the residual from the last-level cache); 2,047 rows of 17,408 to e4m3
// with a scale for each 128: 39 us, 107 MB at 2.8 TB/s.  There a row is a block of 12 waves, of which a CU holds
// two (77 registers a thread: 6 waves a SIMD), and nothing of a block's is on its way while it sums its row
// (with four chunks a thread, 97 registers, 55 us).
// Where rows are few, the call: one round trip to memory, one sum over the workgroup, one store (one row of
// 5,120: 3.2 us).
#pragma once
#include "qg_attn.h"
#include "qg_step.h"

namespace qg {

typedef uint32_t nm_u4 __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes of 16-bit elements, where they are
typedef uint32_t nm_u2 __attribute__((ext_vector_type(2), aligned(1)));  // 8 codes

constexpr int NM_TEAMS = 256;  // threads of a workgroup of several rows

template <bool BF> __device__ __forceinline__ float nm_f32(uint32_t h) {
  if constexpr (BF) return __builtin_bit_cast(float, h << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
// 8 elements at p of which `left` are there; the others are 0
__device__ __forceinline__ kv_u4 nm_load(const uint16_t* p, int left) {
  if (left >= 8) return *reinterpret_cast<const nm_u4*>(p);
  kv_u4 w = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
  return w;
}
__device__ __forceinline__ void nm_store(uint16_t* p, kv_u4 w, int left) {
  if (left >= 8) {
    *reinterpret_cast<nm_u4*>(p) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}
template <bool BF> __device__ __forceinline__ float nm_at(kv_u4 w, int i) { return nm_f32<BF>((w[i / 2] >> (16 * (i & 1))) & 0xFFFFu); }

// sum or maximum over the workgroup, in a fixed order; lds: a float per wave
template <bool MAX> __device__ __forceinline__ float nm_all(float x, float* lds) {
  const auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int o = 32; o; o >>= 1) x = op(x, __shfl_xor(x, o));
  const int waves = blockDim.x >> 6;
  if (waves == 1) return x;
  __syncthreads();  // the last use's readers are done
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  float t = lds[0];
  for (int w = 1; w < waves; ++w) t = op(t, lds[w]);
  return t;
}

// the same over the T (a power of two) lanes of a row
template <bool MAX> __device__ __forceinline__ float nm_team(float x, int T) {
  for (int o = T >> 1; o; o >>= 1) {
    const float y = __shfl_xor(x, o);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  return x;
}

template <int CODES> constexpr float nm_top = CODES == QGS_INT8 ? 127.0f : 448.0f;

// codes of 8 values: v / s rounded to nearest even.  |v| / s is at most the type's largest but
// for the rounding of s, which the rounding of the code takes away where s has its 24 bits.  (max / top may
// have none: of 176 units of 2^-149 it is one, and |v| / s 176.  So there it is held to the largest.)
template <int CODES> __device__ __forceinline__ kv_u2 nm_codes(const float (&v)[8], float s) {
  kv_u2 w = {0, 0};
  if (!(s > 0.0f)) return w;  // zeros, or a NaN scale
  constexpr float TOP = nm_top<CODES>;
  float c[8];
  if (__builtin_expect(s < 0x1p-80f, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(v[i] / s, -TOP), TOP);
  } else {
    // The quotient as fp32 division rounds it: 1 / s in two parts gives it to one unit, and one step by the
    // remainder brings it there (Markstein's theorem; the remainder is exact for quotients of 2^-11 and more, s
    // being 2^-80 at least, and what is smaller has a code of 0 either way).  Against v r alone, which is 1.5 units
    // off: 33 us and 32 (2,047 rows of 17,408 to e4m3, from the last-level cache).
    const float r = 1.0f / s, r2 = __builtin_fmaf(-r, s, 1.0f) * r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __builtin_fmaf(v[i], r, v[i] * r2);
      c[i] = __builtin_fmaf(__builtin_fmaf(-q, s, v[i]), r, q);
    }
  }
  if constexpr (CODES == QGS_INT8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)(int)rintf(c[i]) & 0xFFu) << (8 * (i & 3));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int x = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], x, true);
    }
  }
  return w;
}

// Thread t of a row holds its chunks t, t + T, ... of 8 elements, as the 16-bit values that
// they are.  A row is a workgroup's, or, where it is short (TEAM: the heads of q and k), a.team lanes'
// of a wave: 60,000 rows of 128 elements with the residual (61 MB) 15.1 us, with a wave each 27.9.
template <bool BF, int C, int CODES, bool TEAM> __global__ __launch_bounds__(TEAM ? NM_TEAMS : 1024) void k_rms_norm(NormArgs a) {
  __shared__ float lds[16];
  const int T = TEAM ? a.team : (int)blockDim.x, tid = TEAM ? (int)threadIdx.x & (T - 1) : (int)threadIdx.x;
  const int64_t row = a.first + (TEAM ? (int64_t)blockIdx.x * (NM_TEAMS / T) + threadIdx.x / T : (int64_t)blockIdx.x);
  if (TEAM && row >= a.rows) a.n = 0;  // (its lanes go along for the sums)
  const auto place = [&](int c) { return (c * T + tid) * 8; };
  const auto sum = [&](float x) { return TEAM ? nm_team<false>(x, T) : nm_all<false>(x, lds); };
  const auto most = [&](float x) { return TEAM ? nm_team<true>(x, T) : nm_all<true>(x, lds); };
  const uint16_t* x = a.x + row * a.x_stride;
  kv_u4 h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = nm_load(x + place(c), a.n - place(c));
  if (a.residual) {
    uint16_t* res = a.residual + row * a.residual_stride;
    kv_u4 r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] = nm_load(res + place(c), a.n - place(c));
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[c][i] = at_pack<BF>(nm_at<BF>(h[c], 2 * i) + nm_at<BF>(r[c], 2 * i), nm_at<BF>(h[c], 2 * i + 1) + nm_at<BF>(r[c], 2 * i + 1));
      nm_store(res + place(c), h[c], a.n - place(c));
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(nm_at<BF>(h[c], i), nm_at<BF>(h[c], i), ss);
  ss = sum(ss);
  const float n = (float)a.n;
  const float mean = ss / n + a.eps;
  float rs = 1.0f / sqrtf(mean), rs2 = 1.0f;  // (rs2 is 1 but where one factor would lose bits)
  if (__builtin_expect(!(ss < __builtin_inff()) | (mean < 0x1p-100f), 0)) {
    // squares that overflow fp32 (bf16 values past 2^63), or lose bits that count (with an eps as small as they are): the
    // row's sum again, times 2^-2e
    int e = -60;
    bool again = true;
    if (!(ss < __builtin_inff())) {
      float top = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = fabsf(nm_at<BF>(h[c], i));
          top = fmaxf(top, v == v ? v : __builtin_inff());
        }
      top = most(top);
      again = top < __builtin_inff();  // (NaN and infinities stay as the formula has them)
      e = again ? ilogbf(top) : 0;
    }
    if (again) {
      ss = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = ldexpf(nm_at<BF>(h[c], i), -e);
          ss = __builtin_fmaf(v, v, ss);
        }
      ss = sum(ss);
      // The factor of the row as it is, in halves: h * 2^-e would have lost the small elements' bits.
      rs = ldexpf(1.0f / sqrtf(ss / n + ldexpf(a.eps, -2 * e)), -(e / 2));
      rs2 = ldexpf(1.0f, -(e - e / 2));
    }
  }
  const auto normed = [&](float (&y)[8], int c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = nm_at<BF>(h[c], i) * rs;
    if (__builtin_expect(rs2 != 1.0f, 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= rs2;
    }
    if (a.weight) {
      const kv_u4 w = nm_load(a.weight + place(c), a.n - place(c));
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= nm_at<BF>(w, i);
    }
  };
  if constexpr (CODES == QGS_SAME) {
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[8];
      normed(y, c);
      kv_u4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = at_pack<BF>(y[2 * i], y[2 * i + 1]);
      nm_store(out + place(c), w, a.n - place(c));
    }
  } else {
    constexpr float TOP = nm_top<CODES>;
    uint8_t* out = reinterpret_cast<uint8_t*>(a.out) + row * a.out_stride;
    // the largest magnitudes; a NaN counts as infinity
    const auto largest = [](const float (&v)[8], float m) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i] == v[i] ? fabsf(v[i]) : __builtin_inff());
      return m;
    };
    float all = 0.0f;
    if (a.group == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float y[8];
        normed(y, c);
        all = largest(y, all);
      }
      all = most(all);
    }
    const int per = a.group ? (a.n + a.group - 1) / a.group : 1;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = place(c);
      float y[8];
      normed(y, c);
      float m = all;
      if (a.group) {  // 4, 8 or 16 lanes share a group
        m = largest(y, 0.0f);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1)
          if (8 * o < a.group && o < T) m = fmaxf(m, __shfl_xor(m, o));
      }
      const float s = m < __builtin_inff() ? m / TOP : __builtin_nanf("");
      if (at < a.n && (a.group ? at % a.group == 0 : at == 0)) a.scales[row * per + (a.group ? at / a.group : 0)] = s;
      const kv_u2 w = nm_codes<CODES>(y, s);
      if (at + 8 <= a.n) {
        *reinterpret_cast<nm_u2*>(out + at) = w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < a.n) out[at + i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
      }
    }
  }
}

}  // namespace qg
