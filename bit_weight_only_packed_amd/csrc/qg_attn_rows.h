// qg_attn_rows.h -- attention of many rows over a paged cache: prompts, chunks of
// prompts behind a history, and verify batches too wide for the few-row kernel.
//
// Bound.  4 D flops per visible (row, q head, token) on the matrix cores.
//
// A block is 128 rows of one (entry, kv head): row r is new token r / G, q head
// r % G of the group, so the q heads that share a kv head share its tokens, and a
// block spans few positions (little is computed past the diagonal).  Four waves
// of 32 rows.  Tokens come in tiles of KT = 8192 / D, keys and values 16 KiB each,
// through LDS in two buffers: the next tile's loads are issued before this one is
// computed and stored after.
//
//   scores   S^T = K Q^T on 32x32x16 (A: keys from LDS, B: q from registers).  A
//            lane holds 16 tokens of one row per 32, as token 8 (i / 4) + 4 h + i % 4
//            (h = lane / 32).
//   products O^T = V^T P^T: the B operand of step kk is the lane's own weights
//            8 kk .. 8 kk + 7, packed where they are.  Values are turned over on
//            the way into LDS (byte permutes, [column][token]), their tokens in the
//            order that a lane holds its weights in, so an A operand is one
//            16-byte read.
// 16-byte chunks are placed by an exclusive-or with the row, so that the rows of a
// read fall on distinct banks.
#pragma once
#include "qg_attn.h"

namespace qg {

constexpr int RW_NW = 4;  // waves of a workgroup
constexpr int RW_MIN_TILES = 4;  // tiles of a split at least

template <int D> struct RowsShape {
  static constexpr int KT = 8192 / D;       // tokens of a tile
  static constexpr int KC = D / 8;          // 16-byte chunks of a key
  static constexpr int VC = KT / 8;         // 16-byte chunks of a column of values
  static constexpr int NT = KT / 32;        // 32-token groups
  static constexpr int ND = D / 32;         // 32-column groups
  static constexpr size_t half = 16384;     // bytes of a tile's keys (or values)
  static constexpr size_t lds = 4 * half + 64;
};

// byte of chunk c of key t
template <int D> __device__ __forceinline__ int rw_key(int t, int c) {
  constexpr int M = RowsShape<D>::KC < 16 ? RowsShape<D>::KC - 1 : 15;
  return (t * RowsShape<D>::KC + (c ^ (t & M))) * 16;
}
// byte of chunk c (8 tokens) of column d
template <int D> __device__ __forceinline__ int rw_val(int d, int c) {
  constexpr int VC = RowsShape<D>::VC;
  constexpr int SH = VC == 16 ? 0 : (VC == 8 ? 1 : 2);  // columns that share 256 bytes, as a power of two
  return (d * VC + (c ^ (((d >> SH) ^ (d >> 4)) & (VC - 1)))) * 16;
}

template <int D> struct RowsStage {
  kv_u4 k[4], v[4];
};

// this thread's part of a tile: keys 4 x 16 bytes; values 4 tokens x 8 columns
template <int D>
__device__ __forceinline__ void rw_load(RowsStage<D>& s, const KvDev& c, const int32_t* table, int tok, int last, int head) {
  constexpr int KC = RowsShape<D>::KC;
  const int mask = (1 << c.page_shift) - 1, tid = threadIdx.x;
  const int64_t hoff = ((int64_t)head << c.page_shift) * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = i * 256 + tid, t = min(tok + x / KC, last);
    const uint16_t* p = c.pool + kv_page(c, table[t >> c.page_shift]) * c.page_stride + hoff;
    s.k[i] = *reinterpret_cast<const kv_u4*>(p + (t & mask) * D + (x % KC) * 8);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = min(tok + (tid / KC) * 4 + i, last);
    const uint16_t* p = c.pool + kv_page(c, table[t >> c.page_shift]) * c.page_stride + hoff + c.v_off;
    s.v[i] = *reinterpret_cast<const kv_u4*>(p + (t & mask) * D + (tid % KC) * 8);
  }
}

// into LDS.  masked: values of tokens that no row of the block sees become 0;
// returns whether one that remains is not finite
template <int D, bool BF>
__device__ __forceinline__ bool rw_put(RowsStage<D>& s, char* keys, char* vals, bool masked, int tok, int p0, int p1,
                                       int window, int sinks) {
  constexpr int KC = RowsShape<D>::KC;
  const int tid = threadIdx.x;
  bool odd = false;
  if (masked) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = tok + (tid / KC) * 4 + i;
      const bool seen = t <= p1 && (window == 0 || t > max(p0, 0) - window || t < sinks);
      if (!seen) s.v[i] = kv_u4{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 4; ++x) odd |= at_odd<BF>(s.v[i][x]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = i * 256 + tid;
    *reinterpret_cast<kv_u4*>(keys + rw_key<D>(x / KC, x % KC)) = s.k[i];
  }
  const int g4 = tid / KC;                                       // group of 4 tokens
  const int at = (g4 & ~3) | ((g4 & 1) << 1) | ((g4 >> 1) & 1);  // its place: the middle bits exchanged
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const uint32_t a = s.v[0][x >> 1], b = s.v[1][x >> 1], c = s.v[2][x >> 1], d = s.v[3][x >> 1];
    const kv_u2 w = (x & 1) ? kv_u2{at_halves<1>(a, b), at_halves<1>(c, d)} : kv_u2{at_halves<0>(a, b), at_halves<0>(c, d)};
    *reinterpret_cast<kv_u2*>(vals + rw_val<D>((tid % KC) * 8 + x, at >> 1) + (at & 1) * 8) = w;
  }
  return odd;
}

template <int D, bool BF>
__global__ __launch_bounds__(64 * RW_NW) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
void k_attn_rows(AttnArgs a) {
  using S = RowsShape<D>;
  extern __shared__ __align__(16) char smem[];
  int* flag = reinterpret_cast<int*>(smem + 4 * S::half);
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
  const int rb = (total + ROWS_BM - 1) / ROWS_BM - 1 - back;
  if (rb < 0) return;
  const int r0 = rb * ROWS_BM, nrows = min(total - r0, ROWS_BM);
  const int pe = e.len - e.rows;
  const int p0 = pe + r0 / a.G, p1 = pe + (r0 + nrows - 1) / a.G;
  const TileRange<S::KT> tr(p0, p1, a.window, a.sinks);
  const int parts = max(min(a.splits, tr.n / RW_MIN_TILES), 1);
  if (z >= parts) return;
  const int t0 = (int)((int64_t)tr.n * z / parts), t1 = (int)((int64_t)tr.n * (z + 1) / parts);
  const int32_t* table = a.c.tables + (int64_t)e.slot * a.c.max_pages;

  // this wave's rows
  const int rw = r0 + wave * 32 + col;
  const bool live = rw < total;
  const int ri = live ? rw / a.G : 0;
  const int pos = live ? pe + ri : -1;
  const int pw0 = pe + (r0 + wave * 32) / a.G, pw1 = min(pe + (r0 + wave * 32 + 31) / a.G, p1);
  kv_u4 Q[D / 16];
  {
    const uint16_t* qp = a.q.ptr + (int64_t)(e.row0 + ri) * a.q.row +
                         (int64_t)(head * a.G + (live ? rw - ri * a.G : 0)) * a.q.head + h * 8;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      Q[c] = *reinterpret_cast<const kv_u4*>(qp + 16 * c);
      if (!live) Q[c] = kv_u4{0, 0, 0, 0};
    }
  }
  at_f16 O[S::ND];
#pragma unroll
  for (int x = 0; x < S::ND; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) O[x][i] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;

  RowsStage<D> st;
  bool odd = false;
  int buf = 0;
  if (t0 < t1) {
    const int tok = tr.at(t0) * S::KT;
    const bool masked = !at_all_see(p0, p1, tok, tok + S::KT - 1, a.window, a.sinks);
    rw_load<D>(st, a.c, table, tok, p1, head);
    odd = rw_put<D, BF>(st, smem, smem + S::half, masked, tok, p0, p1, a.window, a.sinks);
    odd = __syncthreads_or(odd);
  }
  for (int t = t0; t < t1; ++t) {
    const int tok = tr.at(t) * S::KT;
    const bool more = t + 1 < t1;
    const int tok2 = more ? tr.at(t + 1) * S::KT : tok;
    if (more) rw_load<D>(st, a.c, table, tok2, p1, head);

    // a wave none of whose rows sees the tile passes it by
    if (pw0 <= pw1 && tok <= pw1 && (a.window == 0 || tok + S::KT - 1 > pw0 - a.window || tok < a.sinks)) {
      const char* keys = smem + buf * 2 * S::half;
      const char* vals = keys + S::half;
      at_f16 s[S::NT];
#pragma unroll
      for (int g = 0; g < S::NT; ++g) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[g][i] = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const kv_u4 K = *reinterpret_cast<const kv_u4*>(keys + rw_key<D>(g * 32 + col, 2 * c + h));
          s[g] = at_mfma32<BF>(K, Q[c], s[g]);
        }
      }
      const bool masked = !at_all_see(pw0, pw1, tok, tok + S::KT - 1, a.window, a.sinks);
      float mx = -__builtin_inff();
#pragma unroll
      for (int g = 0; g < S::NT; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[g][i] *= a.scale_log2;
          if (masked && !at_sees(pos, tok + g * 32 + 8 * (i >> 2) + 4 * h + (i & 3), a.window, a.sinks))
            s[g][i] = -__builtin_inff();
          mx = fmaxf(mx, s[g][i]);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      if (__any(mx > m)) {
        const float mn = fmaxf(m, mx);
        const float f = at_exp2(m - at_safe(mn));
        m = mn;
        l *= f;
#pragma unroll
        for (int x = 0; x < S::ND; ++x)
#pragma unroll
          for (int i = 0; i < 16; ++i) O[x][i] *= f;
      }
      const float ms = at_safe(m);
      kv_u4 P[2 * S::NT];
#pragma unroll
      for (int g = 0; g < S::NT; ++g)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float x = at_exp2(s[g][i] - ms), y = at_exp2(s[g][i + 1] - ms);
          l += x + y;
          P[2 * g + i / 8][(i & 7) / 2] = at_pack<BF>(x, y);
        }
      if (!(masked && odd)) {
#pragma unroll
        for (int x = 0; x < S::ND; ++x)
#pragma unroll
          for (int k = 0; k < 2 * S::NT; ++k) {
            const kv_u4 V = *reinterpret_cast<const kv_u4*>(vals + rw_val<D>(x * 32 + col, 2 * k + h));
            O[x] = at_mfma32<BF>(V, P[k], O[x]);
          }
      } else {
#pragma unroll 1
        for (int k = 0; k < 2 * S::NT; ++k) {
          kv_u4 I, Pk = P[0];
#pragma unroll
          for (int y = 1; y < 2 * S::NT; ++y)
            if (y == k) Pk = P[y];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // weights 2 i and 2 i + 1 of step k
            const int key = tok + k * 16 + 8 * (i >> 1) + 4 * h + (i & 1) * 2;
            I[i] = (at_sees(pos, key, a.window, a.sinks) ? at_one<BF>() : 0u) |
                   (at_sees(pos, key + 1, a.window, a.sinks) ? at_one<BF>() << 16 : 0u);
          }
#pragma unroll
          for (int x = 0; x < S::ND; ++x) {
            const kv_u4 V = *reinterpret_cast<const kv_u4*>(vals + rw_val<D>(x * 32 + col, 2 * k + h));
            kv_u4 F, Ip, In;
#pragma unroll
            for (int i = 0; i < 4; ++i) F[i] = at_fin<BF>(V[i]), Ip[i] = at_ind<BF>(V[i], false), In[i] = at_ind<BF>(V[i], true);
            at_f16 zero;
#pragma unroll
            for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
            O[x] = at_mfma32<BF>(F, Pk, O[x]);
            const at_f16 np = at_mfma32<BF>(Ip, I, zero), nn = at_mfma32<BF>(In, I, zero);
#pragma unroll
            for (int i = 0; i < 16; ++i) O[x][i] += at_add_odd(np[i], nn[i]);
          }
        }
      }
    }

    buf ^= 1;
    const bool masked2 = more && !at_all_see(p0, p1, tok2, tok2 + S::KT - 1, a.window, a.sinks);
    bool odd2 = false;
    if (more) {
      char* keys = smem + buf * 2 * S::half;
      odd2 = rw_put<D, BF>(st, keys, keys + S::half, masked2, tok2, p0, p1, a.window, a.sinks);
    }
    if (masked2) odd = __syncthreads_or(odd2);
    else __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (parts == 1) {
    if (live) {
#pragma unroll
      for (int x = 0; x < S::ND; ++x)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float o[4] = {O[x][i], O[x][i + 1], O[x][i + 2], O[x][i + 3]};
          at_store<BF, 4>(a, e, head, rw, x * 32 + 2 * i + 4 * h, o, l);
        }
    }
    return;
  }
  // several workgroups share the block: the last to arrive joins their partials in order
  float* slot = a.partial + (size_t)blockIdx.x * rows_slot(D);
  const int r = wave * 32 + col;
  if (live) {
#pragma unroll
    for (int x = 0; x < S::ND; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) at_st(slot + (size_t)r * D + x * 32 + 8 * (i >> 2) + 4 * h + (i & 3), O[x][i]);
    if (h == 0) {
      at_st(slot + (size_t)ROWS_BM * D + 2 * r, m);
      at_st(slot + (size_t)ROWS_BM * D + 2 * r + 1, l);
    }
  }
  if (!at_last(a.counters + blockIdx.x / a.splits, parts, flag)) return;
  at_join<BF, D>(a, e, head, r0, nrows, ROWS_BM, parts,
                 [&](int k) { return a.partial + (size_t)(blockIdx.x - z + k) * rows_slot(D); });
}

}  // namespace qg
