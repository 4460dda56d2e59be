// qg_attn_rows.h -- attention of many rows over a paged cache: prompts, chunks of
// prompts behind a history, and verify batches too wide for the few-row kernel.
//
// Bound.  4 D flops per visible (row, q head, token) on the matrix cores.
//
// A block is 32 rows per wave of one (entry, kv head): row r is new token r / G, q
// head r % G of the group, so the q heads that share a kv head share its tokens,
// and a block spans few positions (little is computed past the diagonal).  Tokens
// come in tiles of KT = 8192 / D, keys and values 16 KiB each, straight from memory
// into one of two LDS buffers (no registers); the next tile is on its way while
// this one is computed, and one barrier per tile orders both.
//
//   scores   S^T = K Q^T on 32x32x16 (A: keys from LDS, B: q from registers).  A
//            lane holds 16 tokens of one row per 32, as token 8 (i / 4) + 4 h + i % 4
//            (h = lane / 32).
//   products O^T = V^T P^T: the B operand of step kk is the lane's own weights
//            8 kk .. 8 kk + 7, packed where they are: tokens 4 h .. 4 h + 3 and
//            8 + 4 h .. of 16.  The A operand, four tokens of one column at a time,
//            comes from the transposing LDS read.
// 16-byte chunks are placed by an exclusive-or with the row, so that the rows of a
// read fall on distinct banks.
//
// The running maximum is raised, and what has been summed rescaled, only where a
// row's new maximum is more than 2^8 above it in the exponent: weights stay below
// 2^8, far inside fp16, and the rescaling of the accumulators almost never runs.
#pragma once
#include "qg_attn.h"

namespace qg {

constexpr int RW_MIN_TILES = 4;     // tiles of a split at least
constexpr float RW_SLACK = 8.0f;    // exponent that a weight may reach

template <int D> struct RowsShape {
  static constexpr int NW = rows_waves(D);  // waves of a workgroup
  static constexpr int BM = rows_block(D);  // rows of a block
  static constexpr int KT = 8192 / D;       // tokens of a tile
  static constexpr int KC = D / 8;          // 16-byte chunks of a token's key or value
  static constexpr int NT = KT / 32;        // 32-token groups
  static constexpr int ND = D / 32;         // 32-column groups
  static constexpr int LD = 16 / NW;        // 1 KiB copies per wave of a tile's keys (or values)
  static constexpr int RW = KT / NW;        // tokens that a wave copies (they lie in one page)
  static constexpr int bytes = 16384;       // a tile's keys (or values)
};

// what a token's chunk index is exclusive-or'ed with.  Keys: 16 lanes read one chunk
// of 16 tokens.  Values: 16 lanes read 32 bytes of 4 tokens, beside those of the next
// 16 columns, so tokens 0..3 go to distinct 64-byte slots.
template <int D> __device__ __forceinline__ int rw_key_swz(int t) { return t & (D == 64 ? 7 : 15); }
template <int D> __device__ __forceinline__ int rw_val_swz(int t) {
  return D == 64 ? ((t >> 1) & 1) << 2 | ((t >> 2) & 3) : (t & 3) << 2 | ((t >> 2) & 3);
}

typedef short rw_s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) rw_s4* rw_lds4;

// four tokens of one column per lane (16 lanes: 4 tokens x 16 columns)
__device__ __forceinline__ kv_u2 rw_read_tr(const char* p) {
  return __builtin_bit_cast(kv_u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((rw_lds4)(p)));
}

// this wave's part of a tile's copies: `base` the page's first key of the head
template <int D>
__device__ __forceinline__ void rw_copy(const uint16_t* base, int64_t v_off, int slot, char* keys, char* vals, int wave, int lane) {
  using S = RowsShape<D>;
#pragma unroll
  for (int i = 0; i < S::LD; ++i) {
    const int x = i * 64 + lane, t = x / S::KC, c = x % S::KC;  // token of the wave's, chunk's place
    const int tt = wave * S::RW + t;                            // token of the tile
    const uint16_t* k = base + (slot + t) * D + (c ^ rw_key_swz<D>(tt)) * 8;
    const uint16_t* v = base + v_off + (slot + t) * D + (c ^ rw_val_swz<D>(tt)) * 8;
    const int to = (wave * S::LD + i) * 1024;
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)k,
                                     (__attribute__((address_space(3))) void*)(keys + to), 16, 0, 0);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)v,
                                     (__attribute__((address_space(3))) void*)(vals + to), 16, 0, 0);
  }
}

__device__ __forceinline__ void rw_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
constexpr int RW_WAIT_VM = 0x0F70;  // s_waitcnt vmcnt(0), the other counters left alone

// a wave's 32 rows
template <int D> struct RowsState {
  using S = RowsShape<D>;
  kv_u4 Q[D / 16];
  at_f16 O[S::ND];
  float m, l;   // m: in units of q . k
  int pos;      // this lane's row's position
};

// one tile of tokens tok .. tok + KT - 1 for a wave whose rows stand at pw0 .. pw1.
// noted: the tile's values that were not finite and have been taken out, or NULL.
template <int D, bool BF>
__device__ __forceinline__ void rw_tile(RowsState<D>& r, const AttnArgs& a, const char* keys, const char* vals, int tok, int pw0,
                                        int pw1, const uint8_t* noted, int lane) {
  using S = RowsShape<D>;
  const int h = lane >> 5, col = lane & 31;
  constexpr int RB = D * 2;  // bytes of a token
  // Byte of this lane's part of the reads below, but for what is constant per
  // read: an exclusive-or for the chunk, an immediate for the token.  Computed
  // anew for each tile (one instruction per read), for the registers are needed.
  int kb = col * RB + ((h ^ rw_key_swz<D>(col)) << 4);
  // the transposing read's lane: token i / 4 of four, columns 4 (i % 4) .. (i = lane % 16)
  const int i16 = lane & 15, t4 = 4 * h + (i16 >> 2);
  int vb = t4 * RB + (((((lane >> 4) & 1) * 2 + ((i16 >> 1) & 1)) ^ rw_val_swz<D>(t4)) << 4) + (i16 & 1) * 8;
  asm volatile("" : "+v"(kb), "+v"(vb));
  const auto val = [&](int x, int k, int b) {  // 32-column group x, 16-token step k, tokens 8 b + t4
    return rw_read_tr(vals + (vb ^ (x << 6) ^ (b << 5)) + (16 * k + 8 * b) * RB);
  };
  at_f16 s[S::NT];
#pragma unroll
  for (int g = 0; g < S::NT; ++g) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[g][i] = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const kv_u4 K = *reinterpret_cast<const kv_u4*>(keys + (kb ^ (c << 5)) + g * 32 * RB);
      s[g] = at_mfma32<BF>(K, r.Q[c], s[g]);
    }
  }
  const bool masked = !at_all_see(pw0, pw1, tok, tok + S::KT - 1, a.window, a.sinks);
  if (masked) {
#pragma unroll
    for (int g = 0; g < S::NT; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!at_sees(r.pos, tok + g * 32 + 8 * (i >> 2) + 4 * h + (i & 3), a.window, a.sinks)) s[g][i] = -__builtin_inff();
  }
  float mx = s[0][0];
#pragma unroll
  for (int g = 0; g < S::NT; ++g)
#pragma unroll
    for (int i = g == 0 ? 1 : 0; i < 16; ++i) mx = fmaxf(mx, s[g][i]);
  mx = at_max32(mx);
  if (__any((mx - r.m) * a.scale_log2 > RW_SLACK || (mx > r.m && r.m == -__builtin_inff()))) {
    const float mn = fmaxf(r.m, mx);
    const float f = at_exp2((r.m - at_safe(mn)) * a.scale_log2);
    r.m = mn;
    r.l *= f;
#pragma unroll
    for (int x = 0; x < S::ND; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) r.O[x][i] *= f;
  }
  const float ms = at_safe(r.m) * a.scale_log2;
  kv_u4 P[2 * S::NT];
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int g = 0; g < S::NT; ++g)
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float x = at_exp2(__builtin_fmaf(s[g][i], a.scale_log2, -ms));
      const float y = at_exp2(__builtin_fmaf(s[g][i + 1], a.scale_log2, -ms));
      sum[0] += x;
      sum[1] += y;
      P[2 * g + i / 8][(i & 7) / 2] = at_pack<BF>(x, y);
    }
  r.l += sum[0] + sum[1];

#pragma unroll
  for (int x = 0; x < S::ND; ++x)
#pragma unroll
    for (int k = 0; k < 2 * S::NT; ++k) {
      const kv_u2 v0 = val(x, k, 0), v1 = val(x, k, 1);
      r.O[x] = at_mfma32<BF>(kv_u4{v0.x, v0.y, v1.x, v1.y}, P[k], r.O[x]);
    }
  if (noted) {
    // rare: [token][16-byte chunk] bytes of noted +inf or NaN, then of -inf or NaN
#pragma unroll 1
    for (int t = 0; t < S::KT; ++t) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(noted + t * S::KC);
      if (!at_sees(r.pos, tok + t, a.window, a.sinks)) continue;
#pragma unroll
      for (int x = 0; x < S::ND; ++x) {
        const uint32_t p = w[x], n = w[x + S::bytes / 64];
        if ((p | n) == 0) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 8 * (i >> 2) + 4 * h + (i & 3);
          r.O[x][i] += at_noted(p >> c, n >> c);
        }
      }
    }
  }
}

template <int D, bool BF>
__global__ __launch_bounds__(64 * RowsShape<D>::NW) __attribute__((amdgpu_waves_per_eu(RowsShape<D>::NW / 4)))
void k_attn_rows(AttnArgs a) {
  using S = RowsShape<D>;
  // arrays of their own, so that a read of one buffer is known not to wait for the
  // copies that are under way into the other
  __shared__ __align__(1024) char K0[S::bytes], V0[S::bytes], K1[S::bytes], V1[S::bytes];
  __shared__ __align__(16) uint8_t notes[S::bytes / 8];
  __shared__ int odd_at, flag;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, col = lane & 31;

  // the blocks of the call, longest first: the last block of every (entry, kv
  // head), then the one before, ...; kv heads fastest, so that with 8 of them (or
  // a multiple) a head's blocks meet its tokens in one XCD's L2
  int id = blockIdx.x;
  const int z = id % a.splits;
  id /= a.splits;
  const int head = id % a.c.kv_heads, j = (id / a.c.kv_heads) % a.b.n, back = id / (a.c.kv_heads * a.b.n);
  const KvEntry e = kv_entry(a.c, a.b, j);
  const int total = e.rows * a.G;
  const int rb = (total + S::BM - 1) / S::BM - 1 - back;
  if (rb < 0) return;
  const int r0 = rb * S::BM, nrows = min(total - r0, S::BM);
  const int pe = e.len - e.rows;
  const int p0 = pe + r0 / a.G, p1 = pe + (r0 + nrows - 1) / a.G;
  const TileRange<S::KT> tr(p0, p1, a.window, a.sinks);
  const int parts = max(min(a.splits, tr.n / RW_MIN_TILES), 1);
  if (z >= parts) return;
  const int t0 = (int)((int64_t)tr.n * z / parts), t1 = (int)((int64_t)tr.n * (z + 1) / parts);
  const int32_t* table = a.c.tables + (int64_t)e.slot * a.c.max_pages;

  // this wave's rows
  RowsState<D> r;
  const int rw = r0 + wave * 32 + col;
  const bool live = rw < total;
  const int ri = live ? rw / a.G : 0;
  r.pos = live ? pe + ri : -1;
  const int pw0 = pe + (r0 + wave * 32) / a.G, pw1 = min(pe + (r0 + wave * 32 + 31) / a.G, p1);
  {
    const uint16_t* qp = a.q.ptr + (int64_t)(e.row0 + ri) * a.q.row +
                         (int64_t)(head * a.G + (live ? rw - ri * a.G : 0)) * a.q.head + h * 8;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      r.Q[c] = *reinterpret_cast<const kv_u4*>(qp + 16 * c);
      if (!live) r.Q[c] = kv_u4{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int x = 0; x < S::ND; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) r.O[x][i] = 0.0f;
  r.m = -__builtin_inff(), r.l = 0.0f;

  if (tid == 0) odd_at = 0;
  // page of this wave's tokens of tile t, and the copy of its part
  const auto page_of = [&](int t) {
    return kv_page(a.c, kv_table(table, min(tr.at(min(t, t1 - 1)) * S::KT + wave * S::RW, p1) >> a.c.page_shift));
  };
  const auto copy = [&](int t, int page, char* keys, char* vals) {
    const int slot = (tr.at(t) * S::KT + wave * S::RW) & ((1 << a.c.page_shift) - 1);
    rw_copy<D>(a.c.pool + page * a.c.page_stride + ((int64_t)head << a.c.page_shift) * D, a.c.v_off, slot, keys, vals, wave, lane);
  };
  int page = 0;
  if (t0 < t1) {
    copy(t0, page_of(t0), K0, V0);
    page = page_of(t0 + 1);
  }
  const auto step = [&](int t, char* keys, char* vals, char* keys2, char* vals2) {
    const int tok = tr.at(t) * S::KT;
    __builtin_amdgcn_s_waitcnt(RW_WAIT_VM);  // this wave's copies have landed
    rw_barrier();                            // everyone's have, and the other buffer is free
    if (t + 1 < t1) {
      copy(t + 1, page, keys2, vals2);
      page = page_of(t + 2);
    }
    const uint8_t* noted = nullptr;
    if (!at_all_see(p0, p1, tok, tok + S::KT - 1, a.window, a.sinks)) {
      // values of tokens that no row of the block sees become 0, whatever their
      // memory held; is one that some rows see and others may not not finite?
      bool nf = false;
#pragma unroll
      for (int i = 0; i < S::LD; ++i) {
        const int k = tok + wave * S::RW + (i * 64 + lane) / S::KC;
        kv_u4* p = reinterpret_cast<kv_u4*>(vals + (wave * S::LD + i) * 1024 + lane * 16);
        const bool seen = k <= p1 && (a.window == 0 || k > max(p0, 0) - a.window || k < a.sinks);
        if (seen) {
          const kv_u4 v = *p;
          nf = nf | at_odd<BF>(v.x) | at_odd<BF>(v.y) | at_odd<BF>(v.z) | at_odd<BF>(v.w);
        } else {
          *p = kv_u4{0, 0, 0, 0};
        }
      }
      if (__any(nf) && lane == 0) odd_at = t + 1;
      rw_barrier();
      if (odd_at == t + 1) {
#pragma unroll 1
        for (int i = 0; i < S::LD; ++i) {
          const int x = i * 64 + lane, tt = wave * S::RW + x / S::KC, c = (x % S::KC) ^ rw_val_swz<D>(tt);
          kv_u4* p = reinterpret_cast<kv_u4*>(vals + (wave * S::LD + i) * 1024 + lane * 16);
          kv_u4 v = *p;
          uint32_t bp = 0, bn = 0;
#pragma unroll
          for (int y = 0; y < 4; ++y) v[y] = at_take<BF>(v[y], 2 * y, bp, bn);
          *p = v;
          notes[tt * S::KC + c] = (uint8_t)bp;
          notes[S::bytes / 16 + tt * S::KC + c] = (uint8_t)bn;
        }
        rw_barrier();
        noted = notes;
      }
    }
    // a wave none of whose rows sees the tile passes it by
    if (pw0 <= pw1 && tok <= pw1 && (a.window == 0 || tok + S::KT - 1 > pw0 - a.window || tok < a.sinks))
      rw_tile<D, BF>(r, a, keys, vals, tok, pw0, pw1, noted, lane);
  };
  for (int t = t0; t < t1; t += 2) {
    step(t, K0, V0, K1, V1);
    if (t + 1 < t1) step(t + 1, K1, V1, K0, V0);
  }

  r.l += __shfl_xor(r.l, 32);
  if (parts == 1) {
    if (live) {
#pragma unroll
      for (int x = 0; x < S::ND; ++x)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float o[4] = {r.O[x][i], r.O[x][i + 1], r.O[x][i + 2], r.O[x][i + 3]};
          at_store<BF, 4>(a, e, head, rw, x * 32 + 2 * i + 4 * h, o, r.l);
        }
    }
    return;
  }
  // several workgroups share the block: the last to arrive joins their partials in order
  const auto rs = at_slots(a.partial, a.partial_floats);
  const uint32_t slot = blockIdx.x * (uint32_t)rows_slot(D), row = wave * 32 + col;
  if (live) {
#pragma unroll
    for (int x = 0; x < S::ND; ++x)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        at_st4(rs, slot + row * D + x * 32 + 2 * i + 4 * h, at_f4{r.O[x][i], r.O[x][i + 1], r.O[x][i + 2], r.O[x][i + 3]});
    if (h == 0) at_st2(rs, slot + S::BM * D + 2 * row, r.m * a.scale_log2, r.l);
  }
  if (!at_last(a.counters + blockIdx.x / a.splits, parts, &flag)) return;
  at_join<BF, D, 64 * S::NW>(a, rs, e, head, r0, nrows, S::BM, parts, reinterpret_cast<float*>(K0),
                 [&](int k) { return (blockIdx.x - z + k) * (uint32_t)rows_slot(D); });
}

}  // namespace qg
