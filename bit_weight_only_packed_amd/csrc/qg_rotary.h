// qg_rotary.h -- rotary positions: of rows by themselves, and of a step's q and k on
// k's way into the pages of a cache.
//
//   (a, b) -> size (a cos t - b sin t, a sin t + b cos t),  t = 2 pi p turns / 2^64
//
// The phase p * turns is taken modulo 2^64, which is modulo one turn, so it is exact; its
// upper 32 bits, as a signed fraction of half a turn, go through sincospi.
//
// A thread has a unit of 16 elements, 8 pairs (two runs of 8 elements half a rotation
// apart, or one of 16), of several heads of one row: the sines and cosines, some 300
// instructions, are its own for all of them.  Bound: HBM where rows are many, the call where
// they are few.  8,191 rows of 40 heads of 128 (fp16, pairs): 34 us, 168 MB moved at 4.9 TB/s; 9 prompts of 63 to
// 3,001 rows of 40 q and 8 k and v heads: 41.5 us, 222 MB at 5.3 TB/s; one row of each of 64 slots: 4.2 us.
#pragma once
#include "qg_attn.h"
#include "qg_step.h"

namespace qg {

struct RotAngles {
  float c[8], s[8];
};

// angles of pairs 8 unit .. 8 unit + 7 at position p
__device__ __forceinline__ void rot_angles(RotAngles& a, const RotDev& r, int p, int unit) {
  typedef uint64_t u2 __attribute__((ext_vector_type(2)));
  const u2* f = reinterpret_cast<const u2*>(r.turns + 8 * unit);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u2 w = f[i];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t phase = (uint64_t)(int64_t)p * w[e] + 0x80000000u;  // the upper half rounded
      float s, c;
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
      a.c[2 * i + e] = c * r.size;
      a.s[2 * i + e] = s * r.size;
    }
  }
}

// where a unit's two runs of 8 elements begin
__device__ __forceinline__ void rot_runs(const RotDev& r, int unit, int& e0, int& e1) {
  const bool apart = !r.pairs && 16 * unit < r.dim;
  e0 = apart ? 8 * unit : 16 * unit;
  e1 = apart ? e0 + r.dim / 2 : e0 + 8;
}

template <bool BF> __device__ __forceinline__ float rot_f32(uint32_t w, int hi) {
  if constexpr (BF) return __builtin_bit_cast(float, hi ? w & 0xFFFF0000u : w << 16);
  else return (float)__builtin_bit_cast(at_h2, w)[hi];
}

// a unit's two runs, rotated
template <bool BF> __device__ __forceinline__ void rot_unit(kv_u4& x, kv_u4& y, const RotAngles& t, bool pairs) {
  if (pairs) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? reinterpret_cast<uint32_t*>(&x)[i & 3] : reinterpret_cast<uint32_t*>(&y)[i & 3];
      const float a = rot_f32<BF>(w, 0), b = rot_f32<BF>(w, 1);
      w = at_pack<BF>(a * t.c[i] - b * t.s[i], a * t.s[i] + b * t.c[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u[2], v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float a = rot_f32<BF>(x[i], e), b = rot_f32<BF>(y[i], e), c = t.c[2 * i + e], s = t.s[2 * i + e];
        u[e] = a * c - b * s;
        v[e] = a * s + b * c;
      }
      x[i] = at_pack<BF>(u[0], u[1]);
      y[i] = at_pack<BF>(v[0], v[1]);
    }
  }
}

template <bool BF> __global__ __launch_bounds__(256) void k_rotate(RotArgs a) {
  const uint32_t units = (uint32_t)a.head_dim / 16, per = units * (uint32_t)a.slots;
  const int64_t items = (int64_t)a.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
    const int row = (int)(i / per);
    const uint32_t k = (uint32_t)(i - (int64_t)row * per);
    const int slot = (int)(k / units), unit = (int)(k - slot * units);
    const bool turned = 16 * unit < a.r.dim;
    RotAngles t;
    if (turned) rot_angles(t, a.r, a.positions[row], unit);
    int e0, e1;
    rot_runs(a.r, unit, e0, e1);
    for (int h = slot; h < a.heads; h += a.slots) {
      const uint16_t* from = a.x + row * a.x_row + h * a.x_head;
      uint16_t* to = a.out + row * a.out_row + h * a.out_head;
      kv_u4 x = *reinterpret_cast<const kv_u4*>(from + e0), y = *reinterpret_cast<const kv_u4*>(from + e1);
      if (turned) rot_unit<BF>(x, y, t, a.r.pairs);
      *reinterpret_cast<kv_u4*>(to + e0) = x;
      *reinterpret_cast<kv_u4*>(to + e1) = y;
    }
  }
}

// A step's rows on their way: q rotated into q_out, k rotated and v as it is into their
// pages.  Heads are counted through q, k and v.  A row at a position before 0 (an idle
// slot's) is written to no page, and its q_out is 0.  Nothing is written to pages while a
// refused extend stands, as in k_kv_append.
template <int D, bool BF>
__global__ __launch_bounds__(256) void k_kv_append_rotary(RotAppend a) {
  constexpr int U = D / 16;
  const bool refused = (*a.refused & *a.info) != 0;
  const KvEntry e = kv_entry(a.c, a.b, blockIdx.y);
  const uint32_t per = (uint32_t)U * a.slots, items = (uint32_t)e.rows * per;  // below 2^31 (checked on the host)
  const int KH = a.c.kv_heads, heads = a.q_heads + 2 * KH;
  const int32_t* table = a.c.tables + (int64_t)e.slot * a.c.max_pages;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < items; i += gridDim.x * 256) {
    const int row = (int)(i / per);
    const uint32_t k = i - (uint32_t)row * per;
    const int slot = (int)(k / U), unit = (int)(k % U);
    const int pos = e.pos + row;
    int id = -1;
    if (pos >= 0 && !refused) id = table[pos >> a.c.page_shift];
    const bool paged = (unsigned)id < (unsigned)a.c.pages, turned = 16 * unit < a.r.dim;
    uint16_t* const page = const_cast<uint16_t*>(a.c.pool) + (paged ? id : 0) * a.c.page_stride +
                           (int64_t)(pos & ((1 << a.c.page_shift) - 1)) * D;
    RotAngles t;
    if (turned) rot_angles(t, a.r, pos, unit);
    int e0, e1;
    rot_runs(a.r, unit, e0, e1);
    const int64_t at = e.row0 + row;
    for (int h = slot; h < heads; h += a.slots) {
      const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + KH;
      if (!is_q && !paged) continue;
      const int hk = h - a.q_heads - (is_v ? KH : 0);
      const uint16_t* from = is_q ? a.q.ptr + at * a.q.row + h * a.q.head
                             : is_v ? a.v.ptr + at * a.v.row + hk * a.v.head
                                    : a.k.ptr + at * a.k.row + hk * a.k.head;
      uint16_t* to = is_q ? const_cast<uint16_t*>(a.out.ptr) + at * a.out.row + h * a.out.head
                          : page + (is_v ? a.c.v_off : 0) + (((int64_t)hk << a.c.page_shift) * D);
      kv_u4 x = *reinterpret_cast<const kv_u4*>(from + e0), y = *reinterpret_cast<const kv_u4*>(from + e1);
      if (turned && !is_v) rot_unit<BF>(x, y, t, a.r.pairs);
      if (pos < 0) x = y = kv_u4{0, 0, 0, 0};
      *reinterpret_cast<kv_u4*>(to + e0) = x;
      *reinterpret_cast<kv_u4*>(to + e1) = y;
    }
  }
}

}  // namespace qg
