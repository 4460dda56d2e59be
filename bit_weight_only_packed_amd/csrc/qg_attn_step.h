// qg_attn_step.h -- attention of few rows over a paged cache: one new token per
// sequence, or the rows of a verify batch.
//
// Bound.  Every cached token's key and value are read once per kv head,
// 4 D bytes, for 4 D G R flops (G q heads per kv head, R new rows: 5 to 160 at
// the shapes met) -- HBM, with matrix-core work to spare.  So the G * R rows that
// share a kv head are packed into tiles of 16 (MT of them, up to 64 rows) and
// all served by one read of the tokens, and the kernel is built to keep reads in
// flight.
//
// A wave takes tiles of 32 tokens.  Keys and values go from memory straight to
// registers, 16 bytes a lane, with no pass through LDS:
//   scores   S^T = K Q^T on 16x16x32: the A operand is a lane's 8 elements of one
//            key, which is how keys lie in the page.  Row r of sub-tile t stands
//            for token 8 (r / 4) + 4 t + r % 4, so that a lane's 2 x 4 scores are
//            those of tokens 8 q .. 8 q + 7 (q = lane / 16) of one row (lane % 16).
//   products O^T = V^T P^T: the B operand wants a lane's 8 tokens of one row --
//            the lane's own weights, packed where they are.  The A operand wants
//            8 tokens of one column: the lane loads 8 tokens x D / 16 columns and
//            pairs them up with one byte permute per two elements.
// The next tile's keys are loaded as soon as the scores have used this one's, the
// next values as soon as the products have: one buffer each, always in use.
//
// Split.  The (entry, kv head, tile) triples of the call form one list; each
// workgroup takes an equal contiguous run of it, whatever the sequences'
// lengths, its four waves every fourth tile of a run's part.  A (entry, kv head)
// that one workgroup covers is finished there; one that several cover is joined
// by the last of them to arrive, from partials in a fixed order.
#pragma once
#include "qg_attn.h"

namespace qg {

constexpr int ST_TK = 32;  // tokens of a tile
constexpr int ST_NW = 4;   // waves of a workgroup

template <int D> struct StepShape {
  static constexpr int VE = D / 16;              // columns of a lane
  static constexpr int VB = D == 64 ? 8 : 16;    // bytes of a lane's value load
  static constexpr int VL = VE * 2 / VB;         // value loads per token
  static constexpr int LD = D + 4;               // padded row of the cross-wave buffer (floats)
  static constexpr int NB = VL * 16;             // bytes of noted values per token (one per value load)
  static constexpr size_t notes = (size_t)ST_NW * 2 * ST_TK * NB;
  static constexpr size_t lds = (size_t)ST_NW * 16 * LD * 4 + ST_NW * 16 * 8 + notes + 16;
};

template <int D, bool BF, int MT> struct StepTile {
  using S = StepShape<D>;
  kv_u4 k[2][D / 32];
  uint32_t v[8][S::VE / 2];
};

// first bytes of the pages of a tile's two halves of 16 tokens
struct StepPages {
  const uint16_t* p[2];
};
__device__ __forceinline__ StepPages step_pages(const KvDev& c, const int32_t* table, int tok, int last, int head, int D) {
  StepPages r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = min((tok + 16 * i) >> c.page_shift, last >> c.page_shift);
    r.p[i] = c.pool + kv_page(c, table[at]) * c.page_stride + (((int64_t)head << c.page_shift)) * D;
  }
  return r;
}

template <int D, bool BF, int MT>
__device__ __forceinline__ void step_load_k(StepTile<D, BF, MT>& t, const KvDev& c, const StepPages& pg, int tok, int lane) {
  const int mask = (1 << c.page_shift) - 1, r = lane & 15;
  const int blk = r >> 2;  // the row's 8-token block
  const uint16_t* base = (blk & 2) ? pg.p[1] : pg.p[0];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int slot = (tok + 8 * blk + 4 * u + (r & 3)) & mask;
    const uint16_t* a = base + slot * D + (lane >> 4) * 8;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) t.k[u][i] = *reinterpret_cast<const kv_u4*>(a + 32 * i);
  }
}

template <int D, bool BF, int MT>
__device__ __forceinline__ void step_load_v(StepTile<D, BF, MT>& t, const KvDev& c, const StepPages& pg, int tok, int lane) {
  using S = StepShape<D>;
  const int mask = (1 << c.page_shift) - 1, q = lane >> 4, col = lane & 15;
  const uint16_t* base = ((q & 2) ? pg.p[1] : pg.p[0]) + c.v_off + col * (S::VB / 2);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint16_t* a = base + ((tok + 8 * q + j) & mask) * D;
#pragma unroll
    for (int e = 0; e < S::VL; ++e) {
      if constexpr (S::VB == 16) {
        const kv_u4 x = *reinterpret_cast<const kv_u4*>(a + 128 * e);
        t.v[j][4 * e] = x.x, t.v[j][4 * e + 1] = x.y, t.v[j][4 * e + 2] = x.z, t.v[j][4 * e + 3] = x.w;
      } else {
        const kv_u2 x = *reinterpret_cast<const kv_u2*>(a);
        t.v[j][0] = x.x, t.v[j][1] = x.y;
      }
    }
  }
}

// the lane's 8 tokens of its column x: the A operand of product tile x
template <int VE> __device__ __forceinline__ kv_u4 step_column(const uint32_t (&v)[8][VE / 2], int x) {
  kv_u4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = v[2 * i][x >> 1], b = v[2 * i + 1][x >> 1];
    r[i] = (x & 1) ? at_halves<1>(a, b) : at_halves<0>(a, b);
  }
  return r;
}

// column of product tile x, row i of it: D-index of O^T element (tile x, register i) of lane quarter q
template <int D> __device__ __forceinline__ int step_col(int q, int i, int x) {
  using S = StepShape<D>;
  return (x / (S::VB / 2)) * 128 + (q * 4 + i) * (S::VB / 2) + x % (S::VB / 2);
}

template <int D, bool BF, int MT>
__global__ __launch_bounds__(64 * ST_NW) __attribute__((amdgpu_waves_per_eu(step_per_cu(MT, D))))
void k_attn_step(AttnArgs a) {
  using S = StepShape<D>;
  extern __shared__ __align__(16) char smem[];
  float* buf = reinterpret_cast<float*>(smem);                                    // [wave][16][LD]
  float* ml = buf + ST_NW * 16 * S::LD;                                           // [wave][16][2]
  uint8_t* notes = reinterpret_cast<uint8_t*>(ml + ST_NW * 16 * 2);               // [wave][2][32][NB]
  int* flag = reinterpret_cast<int*>(notes + S::notes);
  int* pre = flag + 4;                                                            // [n + 1]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, col = lane & 15;
  const int n = a.b.n, heads = a.c.kv_heads;
  notes += (size_t)wave * 2 * ST_TK * S::NB;
  const auto rs = at_slots(a.partial, a.partial_floats);

  // prefix sums of the entries' tiles (at least one for an entry with rows, which
  // has outputs to write even where it sees nothing)
  {
    int carry = 0;
    int* sums = flag;  // the four waves' sums
    for (int j0 = 0; j0 < n; j0 += 64 * ST_NW) {
      const int j = j0 + tid;
      int t = 0;
      if (j < n) {
        const KvEntry e = kv_entry(a.c, a.b, j);
        if (e.rows > 0) t = max(TileRange<ST_TK>(e.len - e.rows, e.len - 1, a.window, a.sinks).n, 1);
      }
      int x = t;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
      }
      if (lane == 63) sums[wave] = x;
      __syncthreads();
      int before = carry;
#pragma unroll
      for (int w = 0; w < ST_NW; ++w) {
        before += w < wave ? sums[w] : 0;
        carry += sums[w];
      }
      if (j < n) pre[j + 1] = before + x;
      __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
  }
  const int64_t units = (int64_t)pre[n] * heads;
  const int64_t per = max((units + a.workers - 1) / a.workers, (int64_t)ST_NW);
  int64_t u = blockIdx.x * per;
  const int64_t u1 = min(u + per, units);

  int j = 0;  // the entry that holds unit u
  if (u < u1)
    for (;; j += 64) {
      const uint64_t past = __ballot(j + lane < n && (int64_t)pre[min(j + lane, n - 1) + 1] * heads > u);
      if (past) {
        j += __builtin_ctzll(past);
        break;
      }
    }
  for (bool first = true; u < u1; first = false) {
    // entry, kv head and tiles of the run's next part
    while ((int64_t)pre[j + 1] * heads <= u) ++j;
    j = __builtin_amdgcn_readfirstlane(j);
    const int nt = __builtin_amdgcn_readfirstlane(pre[j + 1] - pre[j]);
    const int64_t seg0 = (int64_t)pre[j] * heads;
    const int head = __builtin_amdgcn_readfirstlane((int)((u - seg0) / nt));
    const int64_t useg = seg0 + (int64_t)head * nt;  // first unit of (entry, head)
    const int t0 = __builtin_amdgcn_readfirstlane((int)(u - useg));
    const int t1 = __builtin_amdgcn_readfirstlane((int)min((int64_t)nt, u1 - useg));
    u = useg + t1;
    const KvEntry e = kv_entry(a.c, a.b, j);
    const int p0 = e.len - e.rows, p1 = e.len - 1, nrows = e.rows * a.G;
    const TileRange<ST_TK> tr(p0, p1, a.window, a.sinks);
    const int32_t* table = a.c.tables + (int64_t)e.slot * a.c.max_pages;

    // the rows of this kv head: row r is new token r / G, q head head * G + r % G
    kv_u4 Q[MT][D / 32];
    int pos[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = mt * 16 + col;
      const bool live = r < nrows;
      const int i = live ? r / a.G : 0;
      pos[mt] = live ? p0 + i : -1;
      const uint16_t* qp = a.q.ptr + (int64_t)(e.row0 + i) * a.q.row + (int64_t)(head * a.G + (live ? r - i * a.G : 0)) * a.q.head + q * 8;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        Q[mt][c] = *reinterpret_cast<const kv_u4*>(qp + 32 * c);
        if (!live) Q[mt][c] = kv_u4{0, 0, 0, 0};
      }
    }
    at_f4 O[MT][S::VE];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt] = -__builtin_inff(), l[mt] = 0.0f;
#pragma unroll
      for (int x = 0; x < S::VE; ++x) O[mt][x] = at_f4{0, 0, 0, 0};
    }

    StepTile<D, BF, MT> t;
    int tl = t0 + wave;
    StepPages pg;
    const bool any = tr.n > 0;  // else the one tile of an entry that sees nothing
    if (any && tl < t1) {
      const int tok = tr.at(tl) * ST_TK;
      pg = step_pages(a.c, table, tok, p1, head, D);
      step_load_k(t, a.c, pg, tok, lane);
      step_load_v(t, a.c, pg, tok, lane);
    }
    for (; any && tl < t1; tl += ST_NW) {
      const int tok = tr.at(tl) * ST_TK;
      const bool more = tl + ST_NW < t1;
      const int tok2 = more ? tr.at(tl + ST_NW) * ST_TK : tok;
      pg = step_pages(a.c, table, tok2, p1, head, D);

      at_f4 s[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[mt][h] = at_f4{0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < D / 32; ++c) s[mt][h] = at_mfma16<BF>(t.k[h][c], Q[mt][c], s[mt][h]);
        }
      if (more) step_load_k(t, a.c, pg, tok2, lane);

      const bool masked = !at_all_see(p0, p1, tok, tok + ST_TK - 1, a.window, a.sinks);
      kv_u4 P[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = s[mt][i >> 2][i & 3] * a.scale_log2;
        if (masked) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!at_sees(pos[mt], tok + 8 * q + i, a.window, a.sinks)) x[i] = -__builtin_inff();
        }
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__any(mx > m[mt])) {
          const float mn = fmaxf(m[mt], mx);
          const float f = at_exp2(m[mt] - at_safe(mn));
          m[mt] = mn;
          l[mt] *= f;
#pragma unroll
          for (int c = 0; c < S::VE; ++c) O[mt][c] *= f;
        }
        const float ms = at_safe(m[mt]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = at_exp2(x[i] - ms);
          l[mt] += x[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) P[mt][i] = at_pack<BF>(x[2 * i], x[2 * i + 1]);
      }

      bool odd = false;
      if (masked) {
        // tokens that no row sees count for nothing, whatever their memory holds;
        // what only some rows see needs care where it is not finite
        bool nf = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = tok + 8 * q + i;
          const bool seen = key <= p1 && (a.window == 0 || key > max(p0, 0) - a.window || key < a.sinks);
#pragma unroll
          for (int c = 0; c < S::VE / 2; ++c) {
            t.v[i][c] = seen ? t.v[i][c] : 0;
            nf |= at_odd<BF>(t.v[i][c]);
          }
        }
        odd = __any(nf);
        if (odd) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int x = 0; x < S::VL; ++x) {
              uint32_t bp = 0, bn = 0;
#pragma unroll
              for (int c = 0; c < S::VB / 4; ++c)
                t.v[i][x * S::VB / 4 + c] = at_take<BF>(t.v[i][x * S::VB / 4 + c], 2 * c, bp, bn);
              notes[(8 * q + i) * S::NB + x * 16 + col] = (uint8_t)bp;
              notes[(ST_TK + 8 * q + i) * S::NB + x * 16 + col] = (uint8_t)bn;
              __builtin_amdgcn_sched_barrier(0);
            }
        }
      }
#pragma unroll
      for (int c = 0; c < S::VE; ++c) {
        const kv_u4 A = step_column<S::VE>(t.v, c);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) O[mt][c] = at_mfma16<BF>(A, P[mt], O[mt][c]);
      }
      if (odd) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
        for (int k = 0; k < ST_TK; ++k)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (!at_sees(pos[mt], tok + k, a.window, a.sinks)) continue;
#pragma unroll
            for (int x = 0; x < S::VL; ++x) {
              // the notes of this lane's 4 groups of columns
              const uint32_t p = *reinterpret_cast<const uint32_t*>(notes + k * S::NB + x * 16 + 4 * q);
              const uint32_t n = *reinterpret_cast<const uint32_t*>(notes + (ST_TK + k) * S::NB + x * 16 + 4 * q);
              if ((p | n) == 0) continue;
#pragma unroll
              for (int c = 0; c < S::VB / 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) O[mt][x * (S::VB / 2) + c][i] += at_noted(p >> (8 * i + c), n >> (8 * i + c));
            }
          }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      if (more) step_load_v(t, a.c, pg, tok2, lane);
    }

    // the waves' results, joined in wave order; thread (row, c) has D / 16 columns
    const bool whole = t0 == 0 && t1 == nt;
    const uint32_t slot = (2 * blockIdx.x + (first ? 0 : 1)) * (uint32_t)step_slot(MT, D);
    const int row = tid >> 4, c0 = (tid & 15) * S::VE;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= nrows) break;
      float lt = l[mt];
      lt += __shfl_xor(lt, 16);
      lt += __shfl_xor(lt, 32);
      __syncthreads();  // the buffer's last readers are done
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < S::VE; x += 4) {
          const at_f4 w = {O[mt][x][i], O[mt][x + 1][i], O[mt][x + 2][i], O[mt][x + 3][i]};
          *reinterpret_cast<at_f4*>(buf + (wave * 16 + col) * S::LD + step_col<D>(q, i, x)) = w;
        }
      if (q == 0) {
        ml[(wave * 16 + col) * 2] = m[mt];
        ml[(wave * 16 + col) * 2 + 1] = lt;
      }
      __syncthreads();
      const int r = mt * 16 + row;
      if (r < nrows) {
        float M = -__builtin_inff(), L = 0.0f, o[S::VE];
#pragma unroll
        for (int w = 0; w < ST_NW; ++w) M = fmaxf(M, ml[(w * 16 + row) * 2]);
#pragma unroll
        for (int x = 0; x < S::VE; ++x) o[x] = 0.0f;
#pragma unroll
        for (int w = 0; w < ST_NW; ++w) {
          const float f = at_exp2(ml[(w * 16 + row) * 2] - at_safe(M));
          L += f * ml[(w * 16 + row) * 2 + 1];
#pragma unroll
          for (int x = 0; x < S::VE; ++x) o[x] = __builtin_fmaf(f, buf[(w * 16 + row) * S::LD + c0 + x], o[x]);
        }
        if (whole) {
          at_store<BF, S::VE>(a, e, head, r, c0, o, L);
        } else {
#pragma unroll
          for (int x = 0; x < S::VE; x += 4) at_st4(rs, slot + r * D + c0 + x, at_f4{o[x], o[x + 1], o[x + 2], o[x + 3]});
          if (c0 == 0) at_st2(rs, slot + MT * 16 * D + 2 * r, M, L);
        }
      }
    }
    if (whole) continue;

    // several workgroups share (entry, head): the last to arrive joins them, in
    // list order.  The first of them has it as the last part of its run, the
    // others as the first part of theirs.
    const int64_t w0 = useg / per, w1 = (useg + nt - 1) / per;
    if (!at_last(a.counters + j * heads + head, (int)(w1 - w0) + 1, flag)) continue;
    const int before = w0 * per == useg ? 0 : 1;  // w0's slot: its first part or its last
    at_join<BF, D>(a, rs, e, head, 0, nrows, MT * 16, (int)(w1 - w0) + 1,
                   [&](int k) { return (uint32_t)(2 * (w0 + k) + (k == 0 ? before : 0)) * (uint32_t)step_slot(MT, D); });
  }
}

}  // namespace qg
