// qg_attn_step.h -- attention of few rows over a paged cache: one new token per
// sequence, or the rows of a verify batch.
//
// Bound.  Every cached token's key and value are read once per kv head,
// 4 D bytes, for 4 D G R flops (G q heads per kv head, R new rows: up to 32 of
// them together) -- HBM, with matrix-core work to spare.  So the G * R rows that
// share a kv head are packed into tiles of 16 (MT of them, one or two) and
// all served by one read of the tokens, and the kernel is built to keep reads in
// flight.
//
// A wave takes tiles of 32 tokens, each load instruction whole rows side by side
// (keys loaded 16 bytes of 16 rows at a time, as the scores want them, cost 20 %
// of the bandwidth):
//   scores   S^T = K Q^T on 16x16x32: the A operand is a lane's 8 elements of one
//            key.  Keys go straight to the wave's own LDS and come back as operands.
//            A lane's 2 x 4 scores are those of tokens 4 q .. and 16 + 4 q .. (q =
//            lane / 16) of one row (lane % 16).
//   products O^T = V^T P^T: the B operand wants a lane's 8 tokens of one row --
//            the lane's own weights, packed where they are.  The A operand wants
//            8 tokens of one column: the lane loads 8 tokens x D / 16 columns into
//            registers and pairs them up with one byte permute per two elements.
// The next tile's keys are copied as soon as the scores have used this one's, the
// next values loaded as soon as the products have: one buffer each, always in use.
//
// Split.  The (entry, kv head, tile) triples of the call form one list, each (entry,
// kv head) lengthened by ST_COST places for what it costs to begin and end it; each
// workgroup takes an equal contiguous run, whatever the sequences' lengths, its
// waves every NW-th tile of a run's part.  An (entry, kv head) that one workgroup
// covers is finished there; one that several cover is joined by the last of them
// to arrive, from partials in a fixed order.
//
// Measured, 40 q and 8 kv heads of 128, fp16, where the card's large read reaches 5.7
// TB/s: one row of 131,071 tokens 103 us (537 MB, 5.2 TB/s); of 48 sequences of 3 to
// 24,577 tokens each (bf16) 108 us (578 MB, 5.3 TB/s); one row of 1,025 tokens 11 to 13
// us, a chain of some eight memory round trips (entry, table, keys, join).  16 q and 2 kv
// heads of 256, 32 sequences, window 4,096: 50 us (204 MB, 4.1 TB/s; 256 vector and 74
// accumulation registers, one wave a SIMD).
// The scalar registers run out: 51 (heads of 64), 56 (128) and 68 (256) values are kept in
// lanes of vector registers, and some are moved there and back every tile.
#pragma once
#include "qg_attn.h"

namespace qg {

constexpr int ST_TK = 32;  // tokens of a tile
// Tiles that beginning and ending an (entry, kv head) is worth: without it a workgroup
// whose run holds many short sequences ends last (48 sequences of 3 to 24,577 tokens, 8
// kv heads of 128, an (entry, kv head) counted as its tiles alone: 384 us; at 16: 109).
constexpr int ST_COST = 16;
// added to a weight's exponent, at most 0, for the matrix cores' sake
template <bool BF> constexpr float ST_BIAS = BF ? 0.0f : AT_FP16_TOP;

template <int D, int MT = 1> struct StepShape {
  static constexpr int NW = step_waves(D);       // waves of a workgroup
  static constexpr int VE = D / 16;              // columns of a lane
  static constexpr int VB = D == 64 ? 8 : 16;    // bytes of a lane's value load
  static constexpr int VL = VE * 2 / VB;         // value loads per token
  static constexpr int LD = D + 4;               // padded row of the cross-wave buffer (floats)
  static constexpr int NB = VL * 16;             // bytes of noted values per token (one per value load)
  static constexpr size_t notes = (size_t)NW * 2 * ST_TK * NB;
  static constexpr size_t lds = (size_t)NW * 16 * LD * 4 + NW * 16 * 8 + notes + 64;
  static_assert(NW * 16 * LD >= 3 * AT_JOIN_CAP && LD * 4 * 16 >= ST_TK * D * 2, "what shares the buffer");
};

// the call's list in LDS: an entry's slot, position, first row and rows, and its places
// in the list before it (n + 1 of these)
constexpr size_t step_list_bytes(int n) { return (size_t)n * 16 + ((size_t)n + 1) * 4; }

template <int D> struct StepTile {
  using S = StepShape<D>;
  uint32_t v[8][S::VE / 2];
};

// what a token's chunk index is exclusive-or'ed with in LDS, so that the 16 tokens of a
// score read fall on distinct banks
template <int D> __device__ __forceinline__ int step_swz(int t) { return D == 64 ? (t >> 1) & 7 : t & 15; }

// pages of a tile's two halves of 16 tokens, and the first bytes of a head's keys in them
struct StepIds {
  int id[2];
};
struct StepPages {
  __amdgpu_buffer_rsrc_t k[2], v[2];
};
__device__ __forceinline__ StepIds step_ids(const KvDev& c, const int32_t* table, int tok, int last) {
  StepIds r;
#pragma unroll
  for (int i = 0; i < 2; ++i) r.id[i] = kv_table(table, min((tok + 16 * i) >> c.page_shift, last >> c.page_shift));
  return r;
}
// a tile that is none (live false) loads from an empty range: zeros, no memory access.
// So every tile issues the same loads and the waits for them are exact.
__device__ __forceinline__ StepPages step_pages(const KvDev& c, const StepIds& ids, int tok, int head, int D, bool live) {
  StepPages r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int slot = (tok + 16 * i) & ((1 << c.page_shift) - 1);
    const uint16_t* p = c.pool + kv_page(c, ids.id[i]) * c.page_stride + (((int64_t)head << c.page_shift) + slot) * D;
    const int bytes = live ? 16 * D * 2 : 0;
    r.k[i] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, bytes, 0x00020000);
    r.v[i] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p) + c.v_off, 0, bytes, 0x00020000);
  }
  return r;
}

// a tile's keys into the wave's part of LDS, whole rows side by side
template <int D> __device__ __forceinline__ void step_copy_k(char* to, const StepPages& pg, int lane) {
  constexpr int KC = D / 8;   // 16-byte chunks of a key
  constexpr int IN = D / 32;  // copies of 1 KiB per half
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < IN; ++i) {
      const int t = (i * 64 + lane) / KC;
      const int at = t * D * 2 + (((i * 64 + lane) % KC) ^ step_swz<D>(t)) * 16;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(pg.k[h], (__attribute__((address_space(3))) void*)(to + (h * IN + i) * 1024), 16,
                                               at, 0, 0, 0);
    }
}

// a tile's values: register j of a lane is token 16 (j / 4) + 4 q + j % 4 (q = lane / 16)
template <int D> __device__ __forceinline__ void step_load_v(StepTile<D>& t, const StepPages& pg, int lane) {
  using S = StepShape<D>;
  const int at = (lane >> 4) * 4 * D * 2 + (lane & 15) * S::VB;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < S::VL; ++e) {
      const int o = (j & 3) * D * 2 + 256 * e;
      if constexpr (S::VB == 16) {
        const kv_u4 x = __builtin_amdgcn_raw_buffer_load_b128(pg.v[j >> 2], at + o, 0, 0);
        t.v[j][4 * e] = x.x, t.v[j][4 * e + 1] = x.y, t.v[j][4 * e + 2] = x.z, t.v[j][4 * e + 3] = x.w;
      } else {
        const kv_u2 x = __builtin_amdgcn_raw_buffer_load_b64(pg.v[j >> 2], at + o, 0, 0);
        t.v[j][0] = x.x, t.v[j][1] = x.y;
      }
    }
}

// token of a tile that a lane quarter's register (weight, value) j stands for
__device__ __forceinline__ int step_tok(int q, int j) { return 16 * (j >> 2) + 4 * q + (j & 3); }

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
__global__ __launch_bounds__(64 * step_waves(D)) __attribute__((amdgpu_waves_per_eu(step_waves(D) / 4)))
void k_attn_step(AttnArgs a) {
  using S = StepShape<D, MT>;
  constexpr int NW = S::NW;
  extern __shared__ __align__(16) char smem[];
  float* buf = reinterpret_cast<float*>(smem);                                    // [wave][16][LD]
  float* ml = buf + NW * 16 * S::LD;                                              // [wave][16][2]
  uint8_t* notes = reinterpret_cast<uint8_t*>(ml + NW * 16 * 2);                  // [wave][2][32][NB]
  int* flag = reinterpret_cast<int*>(notes + S::notes);                           // [16]
  KvEntry* list = reinterpret_cast<KvEntry*>(flag + 16);                          // [n]
  int* pre = reinterpret_cast<int*>(list + a.b.n);                                // [n + 1]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, col = lane & 15;
  const int n = a.b.n, heads = a.c.kv_heads;
  notes += (size_t)wave * 2 * ST_TK * S::NB;
  // this wave's tile of keys lies where the results are joined once the tiles are
  // done; kb: this lane's part of its reads, but for the column step and the sub-tile
  char* const keys = smem + wave * (ST_TK * D * 2);
  const int kb = col * D * 2 + ((q ^ step_swz<D>(col)) << 4);
  const auto rs = at_slots(a.partial, a.partial_floats);

  // the list: prefix sums of the entries' places per kv head (an entry with rows has
  // outputs to write even where it sees nothing: one tile at least)
  {
    int carry = 0;
    for (int j0 = 0; j0 < n; j0 += 64 * NW) {
      const int j = j0 + tid;
      int t = 0;
      if (j < n) {
        const KvEntry e = kv_entry(a.c, a.b, j);
        list[j] = e;
        if (e.rows > 0) t = ST_COST + max(TileRange<ST_TK>(e.pos, e.pos + e.rows - 1, a.window, a.sinks).n, 1);
      }
      int x = t;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
      }
      if (lane == 63) flag[wave] = x;
      __syncthreads();
      int before = carry;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        before += w < wave ? flag[w] : 0;
        carry += flag[w];
      }
      if (j < n) pre[j + 1] = before + x;
      if (j0 == 0 && tid == 0) pre[0] = 0;
      __syncthreads();
    }
  }
  // (the host has made sure that the places of all heads stay below 2^30)
  const int places = __builtin_amdgcn_readfirstlane(pre[n]) * heads;
  const int per = max((places + a.workers - 1) / a.workers, a.min_run);
  int u = min((int)blockIdx.x, places / per + 1) * per;
  const int u1 = min(u + per, places);

  int j = 0;  // the entry that holds place u
  if (u < u1)
    for (;; j += 64) {
      const uint64_t past = __ballot(j + lane < n && pre[min(j + lane, n - 1) + 1] * heads > u);
      if (past) {
        j += __builtin_ctzll(past);
        break;
      }
    }
  while (u < u1) {
    // entry, kv head and tiles of the run's next part
    while (pre[j + 1] * heads <= u) ++j;
    j = __builtin_amdgcn_readfirstlane(j);
    const int before = __builtin_amdgcn_readfirstlane(pre[j]);
    const int len = __builtin_amdgcn_readfirstlane(pre[j + 1]) - before, nt = len - ST_COST;
    const int seg = before * heads, head = (u - seg) / len;
    const int tile0 = seg + head * len + ST_COST;  // place of (entry, head)'s first tile
    const int t0 = max(u - tile0, 0), t1 = min(nt, u1 - tile0);
    u = tile0 + nt;
    if (t0 >= t1) continue;  // the run ends before its first tile
    KvEntry e = list[j];
    e.slot = __builtin_amdgcn_readfirstlane(e.slot), e.pos = __builtin_amdgcn_readfirstlane(e.pos);
    e.row0 = __builtin_amdgcn_readfirstlane(e.row0), e.rows = __builtin_amdgcn_readfirstlane(e.rows);
    const int p0 = e.pos, p1 = p0 + e.rows - 1, nrows = e.rows * a.G;
    const TileRange<ST_TK> tr(p0, p1, a.window, a.sinks);
    const int32_t* table = a.c.tables + (int64_t)e.slot * a.c.max_pages;

    // the rows of this kv head: row r is new token r / G, q head head * G + r % G
    kv_u4 Q[MT][D / 32];
    int pos[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = mt * 16 + col;
      const bool live = r < nrows;
      const int ri = live ? r / a.G : 0;
      pos[mt] = live ? p0 + ri : -1;
      const uint16_t* qp = a.q.ptr + (int64_t)(e.row0 + ri) * a.q.row +
                           (int64_t)(head * a.G + (live ? r - ri * a.G : 0)) * a.q.head + q * 8;
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

    StepTile<D> t;
    __syncthreads();  // the last part's use of LDS is over
    int tl = t0 + wave;
    StepPages pg;
    StepIds ids;  // of the tile after the one whose keys and values are on their way
    const bool any = tr.n > 0;  // else the one tile of an entry that sees nothing
    const auto token = [&](int i) { return tr.at(min(i, t1 - 1)) * ST_TK; };
    if (any && tl < t1) {
      ids = step_ids(a.c, table, token(tl), p1);
      pg = step_pages(a.c, ids, token(tl), head, D, true);
      step_copy_k<D>(keys, pg, lane);
      __builtin_amdgcn_sched_barrier(0);  // the order that the wait below counts on
      step_load_v(t, pg, lane);
      ids = step_ids(a.c, table, token(tl + NW), p1);
    }
    if (any && tl < t1) for (;; tl += NW) {
      const int tok = token(tl), tok2 = token(tl + NW);
      const bool more = tl + NW < t1;
      pg = step_pages(a.c, ids, tok2, head, D, more);
      // the keys have landed when only the value loads, issued after them, are left
      __builtin_amdgcn_s_waitcnt(at_wait_vm(8 * S::VL));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      at_f4 s[MT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        kv_u4 K[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) K[c] = *reinterpret_cast<const kv_u4*>(keys + (kb ^ (c << 6)) + 16 * h * D * 2);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          s[mt][h] = at_f4{0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < D / 32; ++c) s[mt][h] = at_mfma16<BF>(K[c], Q[mt][c], s[mt][h]);
        }
      }
      // the reads have returned before the next tile's copy may overwrite what they read
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      __builtin_amdgcn_sched_barrier(0);
      step_copy_k<D>(keys, pg, lane);
      __builtin_amdgcn_sched_barrier(0);
      ids = step_ids(a.c, table, token(tl + 2 * NW), p1);

      const bool masked = !at_all_see(p0, p1, tok, tok + ST_TK - 1, a.window, a.sinks);
      kv_u4 P[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = s[mt][i >> 2][i & 3] * a.scale_log2;
        if (masked) {
          const SeenFrom seen(pos[mt], tok + 4 * q, a.window, a.sinks);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = seen(step_tok(0, i)) ? x[i] : -__builtin_inff();
            if (i & 1) __builtin_amdgcn_sched_barrier(0);
          }
        }
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i]);
        mx = at_max16(mx);
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
          x[i] = at_exp2((x[i] - ms) + ST_BIAS<BF>);
          l[mt] += x[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) P[mt][i] = at_pack<BF>(x[2 * i], x[2 * i + 1]);
      }

      bool odd = false;
      if (masked) {
        // tokens that no row sees count for nothing, whatever their memory holds;
        // what only some rows see needs care where it is not finite
        uint32_t top = 0;
        const int far = a.window ? max(p0, 0) - a.window + 1 : 0;  // the first row's oldest token
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = tok + step_tok(q, i);
          const bool seen = (int)(key <= p1) & ((int)(key >= far) | (int)(key < a.sinks));
#pragma unroll
          for (int c = 0; c < S::VE / 2; ++c) {
            t.v[i][c] = seen ? t.v[i][c] : 0;
            top = at_top(top, t.v[i][c]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        odd = __any(top >= at_exp_mask<BF>());
        if (__builtin_expect(odd, 0)) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int x = 0; x < S::VL; ++x) {
              uint32_t bp = 0, bn = 0;
#pragma unroll
              for (int c = 0; c < S::VB / 4; ++c)
                t.v[i][x * S::VB / 4 + c] = at_take<BF>(t.v[i][x * S::VB / 4 + c], 2 * c, bp, bn);
              notes[step_tok(q, i) * S::NB + x * 16 + col] = (uint8_t)bp;
              notes[(ST_TK + step_tok(q, i)) * S::NB + x * 16 + col] = (uint8_t)bn;
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
      if (__builtin_expect(odd, 0)) {
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
      step_load_v(t, pg, lane);
      if (!more) break;
    }

    // the waves' results, joined in wave order; 16 rows over all threads
    const bool whole = t0 == 0 && t1 == nt;
    // a workgroup has at most one part that begins past its first tile (its run's
    // first) and one that begins there and does not end (its last)
    const uint32_t slot = (2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * (uint32_t)step_slot(MT, D);
    constexpr int CW = 16 * D / (64 * NW);  // columns of a thread below
    const int row = tid / (D / CW), c0 = (tid % (D / CW)) * CW;
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
        float M = -__builtin_inff(), L = 0.0f, o[CW];
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[(w * 16 + row) * 2]);
#pragma unroll
        for (int x = 0; x < CW; ++x) o[x] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = at_exp2(ml[(w * 16 + row) * 2] - at_safe(M));
          L += f * ml[(w * 16 + row) * 2 + 1];
#pragma unroll
          for (int x = 0; x < CW; ++x) o[x] = __builtin_fmaf(f, buf[(w * 16 + row) * S::LD + c0 + x], o[x]);
        }
        if (whole) {
          at_store<BF, CW>(a, e, head, r, c0, o, L);
        } else {
#pragma unroll
          for (int x = 0; x < CW; x += 4) {
            if constexpr (CW >= 4) at_st4(rs, slot + r * D + c0 + x, at_f4{o[x], o[x + 1], o[x + 2], o[x + 3]});
            else at_st2(rs, slot + r * D + c0, o[0], o[1]);
          }
          if (c0 == 0) at_st2(rs, slot + MT * 16 * D + 2 * r, M, L);
        }
      }
    }
    if (whole) continue;

    // several workgroups share (entry, head): the last to arrive joins them, in list order
    const int w0 = tile0 / per, parts = (tile0 + nt - 1) / per - w0 + 1;
    if (!at_last(a.counters + j * heads + head, parts, flag)) continue;
    at_join<BF, D, 64 * NW>(a, rs, e, head, 0, 0, nrows, MT * 16, parts, buf, buf + AT_JOIN_CAP, buf + 2 * AT_JOIN_CAP, [&](int k) {
      return (uint32_t)(2 * (w0 + k) + (k == 0 ? 1 : 0)) * (uint32_t)step_slot(MT, D);
    });
    __syncthreads();  // the join's use of the buffer is over
  }
}

}  // namespace qg
