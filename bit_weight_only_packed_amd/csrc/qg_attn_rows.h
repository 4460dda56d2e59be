// qg_attn_rows.h -- attention of many rows over a paged cache: prompts, chunks of
// prompts behind a history, and verify batches too wide for the few-row kernel.
//
// Bound.  4 D flops per visible (row, q head, token) on the matrix cores, and one
// exponential per 4 D flops beside them.  8,191 prompt tokens, 40 q and 8 kv heads of
// 128 (687 GFLOP): 707 to 731 us by card, 940 to 972 TFLOP/s, where the card's best fp16
// matrix product reaches 1,154; the last 4,096 rows of 16,411 tokens through a window of
// 2,048 with 8 sinks (bf16, 172 GFLOP): 217 to 220 us, 782 to 793 TFLOP/s (1,280 blocks of one
// length on 512 places: 2.5 rounds in the time of 3; 7 % is computed past the window's edges).
//
// A block is 32 rows per wave of one (entry, kv head): row r is new token r / G, q
// head r % G of the group, so the q heads that share a kv head share its tokens,
// and a block spans few positions (little is computed past the diagonal).  Tokens
// come in tiles of KT, keys and values straight from memory into LDS (no registers),
// the next tiles on their way while one is computed.
//
// Four waves make a block; two blocks share a CU (three with heads of 64) and each runs
// at its own pace: one's exponentials fall beside the other's products.  Against one
// block of eight waves per CU, four of them half a step behind the other four (8,191
// tokens: 702 against 691 us): half the rows per block waste less on short prompts, 47
// against 33 us at 1,024 tokens.  Three blocks against two with heads of 64: 16 prompts of
// 1 to 1,901 tokens 52 against 60 us, 8,192 tokens 176 against 183.  Two against one, which
// would have had registers to spare, with heads of 256: 8,192 tokens 661 against 898 us
// (with two, q and the sums leave some 60 of 256 registers, and what spills is q).
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
// row's new maximum is more than RW_SLACK above it in the exponent, so the rescaling of
// the accumulators almost never runs.  In fp16 that is 2^4 (8,191 tokens: 731 us, 734 at 2^8) and
// weights are carried 2^11 times larger: up to 2^15, and only those below 2^-36 of the row's
// largest are lost.
#pragma once
#include "qg_attn.h"

namespace qg {

// Tiles of a part at least, of a block that several workgroups share: a part costs its
// rows' partials, 4 D bytes each to write and to read, and its turn of the pipeline's
// start.  The first where CUs would else have no workgroup (splits1 parts give each one),
// the second for what a second workgroup of a CU brings over one (2 prompts of 1,500 rows
// of 3,000 tokens, 8 q heads of 128 and one kv head: 67 us unshared, 76 at 23 tiles a part).
constexpr int RW_MIN_TILES = 8, RW_LONG_TILES = 32;
constexpr int RW_REST_TILES = 3;     // (of an entry's own tokens behind shared ones, which are few)
// parts of a block with so many shared tokens
constexpr int RW_PREFIX_PART = 128, RW_PREFIX_LONG = 1024;
__device__ __forceinline__ int rw_prefix_parts(int tokens, int splits, int splits1) {
  return max(min(splits, max(min(tokens / RW_PREFIX_PART, splits1), tokens / RW_PREFIX_LONG)), 1);
}
__host__ __device__ constexpr int rw_parts(int tiles, int splits1, int least = RW_MIN_TILES) {
  const int few = tiles / least < splits1 ? tiles / least : splits1;
  return few > tiles / RW_LONG_TILES ? few : tiles / RW_LONG_TILES;
}
// operands read from LDS ahead of the product that takes them: 4 where there are
// registers for them (8,191 tokens, heads of 128: 691 us at 4, 689 at 2, 728 at 1), 1 where
// there are none (8,192 tokens, 16 q and 4 kv heads of 256: 661 us at 1, 685 at 2, 742 at
// 3); and the scheduler's names of the two instructions
template <int D> constexpr int RW_DEEP = D == 256 ? 1 : 4;
constexpr int RW_MFMA = 0x8, RW_DS_READ = 0x100;

template <int D> struct RowsShape {
  static constexpr int NW = ROWS_WAVES;     // waves of a workgroup
  static constexpr int BM = ROWS_BLOCK;     // rows of a block
  static constexpr int KT = D == 256 ? 32 : 64;  // tokens of a tile
  static constexpr int KC = D / 8;          // 16-byte chunks of a token's key or value
  static constexpr int NT = KT / 32;        // 32-token groups
  static constexpr int ND = D / 32;         // 32-column groups
  static constexpr int bytes = KT * D * 2;  // a tile's keys (or values)
  static constexpr int LD = bytes / 1024 / NW;  // 1 KiB copies per wave of them
  static constexpr int RW = KT / NW;        // tokens that a wave copies (they lie in one page)
  static constexpr int NB = 2;              // tiles of keys, and of values, in LDS
  static_assert(RW <= 16, "a wave's tokens of a tile lie in one page");
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

// 64 lanes copy 16 bytes each, from `from` (the same for the wave) + ofs, side by side to `to`
__device__ __forceinline__ void rw_copy(const char* from, int ofs, char* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + (uint32_t)ofs),
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Workgroup barrier that waits for this wave's LDS accesses but not for its copies on
// their way into LDS (a fence would: to it they are LDS writes like any other).
__device__ __forceinline__ void rw_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// a wave's 32 rows
template <int D> struct RowsState {
  using S = RowsShape<D>;
  kv_u4 Q[D / 16];
  at_f16 O[S::ND];
  float m, l;   // m: in units of q . k
  int pos;      // this lane's row's position
  bool large;   // (the same for the wave) some row's c m is 2^20 or more
};

// its scores with a tile, and their weights
template <int D> using RowsScores = at_f16[RowsShape<D>::NT];
template <int D> using RowsWeights = kv_u4[2 * RowsShape<D>::NT];

// byte of this lane's part of the key reads, and of the value reads, but for what is
// constant per read: an exclusive-or for the chunk, an immediate for the token
template <int D> __device__ __forceinline__ int rw_key_byte(int lane) {
  const int h = lane >> 5, col = lane & 31;
  return col * D * 2 + ((h ^ rw_key_swz<D>(col)) << 4);
}
template <int D> __device__ __forceinline__ int rw_val_byte(int lane) {
  // the transposing read's lane: token i / 4 of four, columns 4 (i % 4) .. (i = lane % 16)
  const int i = lane & 15, t = 4 * (lane >> 5) + (i >> 2);
  return t * D * 2 + (((((lane >> 4) & 1) * 2 + ((i >> 1) & 1)) ^ rw_val_swz<D>(t)) << 4) + (i & 1) * 8;
}

// scores of the wave's rows with a tile of keys
template <int D, bool BF>
__device__ __forceinline__ void rw_scores(RowsScores<D>& s, const RowsState<D>& r, const char* keys, int lane) {
  using S = RowsShape<D>;
  int kb = rw_key_byte<D>(lane);
  asm volatile("" : "+v"(kb));  // one instruction per read, not a register each: they are needed
  constexpr int N = S::NT * (D / 16), DEEP = RW_DEEP<D>;
  const auto key = [&](int i) {  // column step i / NT, 32-token group i % NT
    return *reinterpret_cast<const kv_u4*>(keys + (kb ^ ((i / S::NT) << 5)) + (i % S::NT) * 32 * D * 2);
  };
  kv_u4 K[N];
#pragma unroll
  for (int i = 0; i < DEEP; ++i) K[i] = key(i);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + DEEP < N) K[i + DEEP] = key(i + DEEP);
    at_f16& x = s[i % S::NT];
    x = at_mfma32<BF>(K[i], r.Q[i / S::NT], i < S::NT ? at_f16{} : x);
  }
  __builtin_amdgcn_sched_group_barrier(RW_DS_READ, DEEP, 0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(RW_MFMA, 1, 0);
    if (i + DEEP < N) __builtin_amdgcn_sched_group_barrier(RW_DS_READ, 1, 0);
  }
}

// scores of tile tok .. tok + KT - 1 to weights; masked: some row does not see all of it
template <int D, bool BF>
__device__ __forceinline__ void rw_softmax(RowsWeights<D>& P, RowsScores<D>& s, RowsState<D>& r,
                                           const AttnArgs& a, int tok, bool masked, int lane) {
  using S = RowsShape<D>;
  const int h = lane >> 5;
  if (masked) {
    const SeenFrom seen(r.pos, tok + 4 * h, a.window, a.sinks);
#pragma unroll
    for (int g = 0; g < S::NT; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[g][i] = seen(g * 32 + 8 * (i >> 2) + (i & 3)) ? s[g][i] : -__builtin_inff();
        if (i & 1) __builtin_amdgcn_sched_barrier(0);
      }
  }
  float mx = s[0][0];
#pragma unroll
  for (int g = 0; g < S::NT; ++g)
#pragma unroll
    for (int i = g == 0 ? 1 : 0; i < 16; ++i) mx = fmaxf(mx, s[g][i]);
  mx = at_max32(mx);
  // (r.m = -inf, nothing seen yet: the difference is inf, or NaN where mx is -inf too)
  if (__builtin_expect(__any((mx - r.m) * a.scale_log2 > RW_SLACK<BF>), 0)) {
    const float mn = fmaxf(r.m, mx);
    const float f = at_exp2((r.m - at_safe(mn)) * a.scale_log2);
    r.m = mn;
    r.large = __any(fabsf(at_safe(mn) * a.scale_log2) >= 0x1p20f);
    r.l *= f;
#pragma unroll
    for (int x = 0; x < S::ND; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) r.O[x][i] *= f;
  }
  float ms = at_safe(r.m) * a.scale_log2 - RW_BIAS<BF>;
  // c s - ms, rounded once, is off by the rounding of ms: by 2^-5 at most below 2^20.  Scores so
  // large that it could overflow the weights are subtracted first (taken everywhere that
  // costs 8,191 tokens 709 against 694 us).
  if (__builtin_expect(r.large, 0)) {
#pragma unroll
    for (int g = 0; g < S::NT; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[g][i] -= at_safe(r.m);
    ms = -RW_BIAS<BF>;
  }
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
  // here, and not among the products that follow the barrier
#pragma unroll
  for (int k = 0; k < 2 * S::NT; ++k) asm volatile("" : "+v"(P[k]));
}

// products of the weights of tile tok with its values
// noted: the tile's values that were not finite and have been taken out, or NULL
template <int D, bool BF>
__device__ __forceinline__ void rw_products(RowsState<D>& r, const RowsWeights<D>& P, const AttnArgs& a,
                                            const char* vals, int tok, const uint8_t* noted, int lane) {
  using S = RowsShape<D>;
  int vb = rw_val_byte<D>(lane);
  asm volatile("" : "+v"(vb));
  const auto val = [&](int x, int k, int b) {  // 32-column group x, 16-token step k, tokens 8 b ..
    return rw_read_tr(vals + (vb ^ (x << 6) ^ (b << 5)) + (16 * k + 8 * b) * D * 2);
  };
  constexpr int N = S::ND * 2 * S::NT, DEEP = RW_DEEP<D>;
  const auto op = [&](int i) {  // 16-token step i / ND, column group i % ND
    const kv_u2 v0 = val(i % S::ND, i / S::ND, 0), v1 = val(i % S::ND, i / S::ND, 1);
    return kv_u4{v0.x, v0.y, v1.x, v1.y};
  };
  kv_u4 V[N];
#pragma unroll
  for (int i = 0; i < DEEP; ++i) V[i] = op(i);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + DEEP < N) V[i + DEEP] = op(i + DEEP);
    r.O[i % S::ND] = at_mfma32<BF>(V[i], P[i / S::ND], r.O[i % S::ND]);
  }
  __builtin_amdgcn_sched_group_barrier(RW_DS_READ, 2 * DEEP, 0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(RW_MFMA, 1, 0);
    if (i + DEEP < N) __builtin_amdgcn_sched_group_barrier(RW_DS_READ, 2, 0);
  }
  if (__builtin_expect(noted != nullptr, 0)) {
    // [token][16-byte chunk] bytes of noted +inf or NaN, then of -inf or NaN
    const int h = lane >> 5;
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

// A block of the call.  Longest first: the last block of every (entry, kv head), then
// the one before, ...; kv heads fastest, so that with 8 of them (or a multiple) a
// head's blocks meet its tokens in one XCD's L2.
enum { RW_WHOLE = 0, RW_PREFIX = 1, RW_REST = 2 };  // all tokens; a group's shared ones; an entry's others
template <int D, int MODE = RW_WHOLE> struct RowsBlock {
  using S = RowsShape<D>;
  int head, rb, total, r0, nrows, pe, p0, p1, parts;  // rb < 0: none; parts that share its tiles
  int cut = 0;  // tiles of the list that are others' to compute
  KvEntry e;
  ShareEntry shared;
  TileRange<S::KT> tr;
  __device__ __forceinline__ RowsBlock(const AttnArgs& a, int id) : tr(-1, -1, 0, 0) {
    head = id % a.c.kv_heads;
    const int back = id / (a.c.kv_heads * a.b.n), j = (id / a.c.kv_heads) % a.b.n;
    e = kv_entry(a.c, a.b, j);
    total = e.rows * a.G;
    rb = (total + S::BM - 1) / S::BM - 1 - back;
    if (rb < 0) return;
    r0 = rb * S::BM, nrows = min(total - r0, S::BM);
    pe = e.pos;
    p0 = pe + r0 / a.G, p1 = pe + (r0 + nrows - 1) / a.G;
    tr = TileRange<S::KT>(p0, p1, a.window, a.sinks);
    if constexpr (MODE == RW_REST) {
      shared = a.share[j];
      cut = tr.before(shared.tokens / S::KT);
    }
    // (an entry that shares nothing has the parts, and the bits, of a call without sharing)
    parts = max(min(a.splits, rw_parts(tr.n - cut, a.splits1, MODE == RW_REST && shared.tokens > 0 ? RW_REST_TILES : RW_MIN_TILES)), 1);
  }
};
// a block of a group's rows with its shared tokens
template <int D> struct RowsBlock<D, RW_PREFIX> {
  using S = RowsShape<D>;
  int head, rb, total, r0, nrows, pe, p0, p1, parts;
  static constexpr int cut = 0;
  KvEntry e;
  TileRange<S::KT> tr;
  __device__ __forceinline__ RowsBlock(const AttnArgs& a, int id) : tr(-1, -1, 0, 0) {
    head = id % a.c.kv_heads;
    const ShareBlock s = a.share_blocks[id / a.c.kv_heads];
    rb = s.tokens > 0 ? 0 : -1;
    if (rb < 0) return;
    r0 = s.r0, total = s.total, nrows = min(total - r0, S::BM);
    pe = 0, p0 = s.p0, p1 = s.p1;
    e = KvEntry{s.slot, 0, s.row0, total / a.G};
    tr = TileRange<S::KT>(p0, p1, a.window, a.sinks);
    tr.n = tr.before(s.tokens / S::KT);
    parts = rw_prefix_parts(tr.n * S::KT, a.splits, a.splits1);
  }
};

// The prefix kernel's part and block.  Row blocks of one head and part read the same tokens: they
// are numbered eight apart, so that they meet in one XCD's L2 whatever the number of heads
// (the last few (head, part) pairs, where that is no multiple of eight, are not).
__device__ __forceinline__ void rw_prefix_place(const AttnArgs& a, unsigned blocks, int& z, int& id) {
  const int heads = a.c.kv_heads, nb = (int)blocks / heads, units = heads * a.splits, whole = units / 8 * 8;
  const int x = blockIdx.x;
  int u, b;
  if (x < whole * nb) {
    u = x / (8 * nb) * 8 + x % 8;
    b = x % (8 * nb) / 8;
  } else {
    const int y = x - whole * nb;
    u = whole + y / nb;
    b = y % nb;
  }
  z = u / heads;
  id = b * heads + u % heads;
}

template <int D, bool BF, int MODE = RW_WHOLE>
__global__ __launch_bounds__(64 * ROWS_WAVES) __attribute__((amdgpu_waves_per_eu(D == 64 ? 3 : 2)))
void k_attn_rows(AttnArgs a) {
  using S = RowsShape<D>;
  __shared__ __align__(1024) char keys[S::NB * S::bytes];
  __shared__ __align__(1024) char vals[S::NB * S::bytes];
  __shared__ __align__(16) uint8_t notes[S::bytes / 8];
  __shared__ int odd_at;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, col = lane & 31;

  // parts slowest: the workgroups past a block's parts come last, and the CUs between
  // those that work do not wait for them (the last 16 rows of 16,384 tokens: 29 us against
  // 36 with parts fastest)
  const unsigned blocks = gridDim.x / (unsigned)a.splits;
  int z = blockIdx.x / blocks, id = a.first + (int)(blockIdx.x - z * blocks);
  if constexpr (MODE == RW_PREFIX) rw_prefix_place(a, blocks, z, id);
  const RowsBlock<D, MODE> blk(a, id);
  if (blk.rb < 0 || z >= blk.parts) return;
  const KvEntry& e = blk.e;
  const TileRange<S::KT>& tr = blk.tr;
  const int head = blk.head, total = blk.total, r0 = blk.r0, pe = blk.pe, p0 = blk.p0, p1 = blk.p1, parts = blk.parts;
  const int tiles = tr.n - blk.cut;
  const int t0 = blk.cut + (int)((int64_t)tiles * z / parts), t1 = blk.cut + (int)((int64_t)tiles * (z + 1) / parts);
  const int32_t* table = a.c.tables + (int64_t)e.slot * a.c.max_pages;

  // this wave's rows
  RowsState<D> r;
  const int rw = r0 + wave * 32 + col;
  const bool live = rw < total, alive = r0 + wave * 32 < total;
  const int ri = live ? rw / a.G : 0;
  int pw0, pw1;  // first and last position of the wave's rows
  bool counts = live;
  if constexpr (MODE == RW_PREFIX) {
    // Rows of many entries.  What comes of those that see nothing, or that max_rows leaves out (-1), is not
    // looked at: a position that masks nothing costs least, and a q of 0 raises no maximum, which would
    // change the roundings of the wave's other rows.
    const int p = live ? a.share_pos[e.row0 + ri] : -1;
    counts = p >= 0;
    r.pos = live ? ((unsigned)p < (unsigned)p1 ? p : p1) : -1;
    pw0 = live ? r.pos : 0x7FFFFFFF, pw1 = r.pos;
#pragma unroll
    for (int o = 16; o; o >>= 1) pw0 = min(pw0, __shfl_xor(pw0, o)), pw1 = max(pw1, __shfl_xor(pw1, o));
    pw0 = __builtin_amdgcn_readfirstlane(pw0), pw1 = __builtin_amdgcn_readfirstlane(pw1);
  } else {
    r.pos = live ? pe + ri : -1;
    pw0 = pe + (r0 + wave * 32) / a.G, pw1 = min(pe + (r0 + wave * 32 + 31) / a.G, p1);
  }
  {
    const uint16_t* qp = a.q.ptr + (int64_t)(e.row0 + ri) * a.q.row +
                         (int64_t)(head * a.G + (live ? rw - ri * a.G : 0)) * a.q.head + h * 8;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      r.Q[c] = *reinterpret_cast<const kv_u4*>(qp + 16 * c);
      if (!counts) r.Q[c] = kv_u4{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int x = 0; x < S::ND; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) r.O[x][i] = 0.0f;
  r.m = -__builtin_inff(), r.l = 0.0f, r.large = false;

  if (tid == 0) odd_at = 0;
  const int nt = t1 - t0;
  const auto token = [&](int t) { return tr.at(t0 + t) * S::KT; };
  // Tiles [clear0, clear1) are seen whole by every row of the block, [wclear0, wclear1)
  // by every row of the wave (of a window's tiles those past the sinks).
  const auto clear = [&](int a0, int a1, int& from, int& to) {
    // tok + KT - 1 <= a0, and tok > a1 - window
    to = min((a0 + 1) / S::KT - (t0 + tr.skip), nt);
    from = a.window ? max((max(a1 - a.window, -1) + S::KT) / S::KT, tr.ns + tr.skip) - (t0 + tr.skip) : 0;
    from = max(from, 0);
    if (a0 < 0) to = 0;
  };
  int clear0, clear1, wclear0, wclear1;
  clear(p0, p1, clear0, clear1);
  clear(pw0, max(pw0, pw1), wclear0, wclear1);
  // values of tile t, once they have landed: those of tokens that no row of the block
  // sees become 0, whatever their memory held; the notes if one that some rows see and
  // others may not is not finite
  const auto mend = [&](int t, char* v) -> const uint8_t* {
    if (t >= clear0 && t < clear1) return nullptr;
    const int tok = token(t);
    uint32_t top = 0;
    const int far = a.window ? max(p0, 0) - a.window + 1 : 0;  // the first row's oldest token
#pragma unroll
    for (int i = 0; i < S::LD; ++i) {
      const int k = tok + wave * S::RW + (i * 64 + lane) / S::KC;
      kv_u4* p = reinterpret_cast<kv_u4*>(v + (wave * S::LD + i) * 1024 + lane * 16);
      if (k <= p1 && ((int)(k >= far) | (int)(k < a.sinks))) {
        const kv_u4 w = *p;
        top = at_top(at_top(at_top(at_top(top, w.x), w.y), w.z), w.w);
      } else {
        *p = kv_u4{0, 0, 0, 0};
      }
    }
    if (__any(top >= at_exp_mask<BF>()) && lane == 0) odd_at = t + 1;
    rw_barrier();
    if (odd_at != t + 1) return nullptr;
#pragma unroll 1
    for (int i = 0; i < S::LD; ++i) {
      const int x = i * 64 + lane, tt = wave * S::RW + x / S::KC, c = (x % S::KC) ^ rw_val_swz<D>(tt);
      kv_u4* p = reinterpret_cast<kv_u4*>(v + (wave * S::LD + i) * 1024 + lane * 16);
      kv_u4 w = *p;
      uint32_t bp = 0, bn = 0;
#pragma unroll
      for (int y = 0; y < 4; ++y) w[y] = at_take<BF>(w[y], 2 * y, bp, bn);
      *p = w;
      notes[tt * S::KC + c] = (uint8_t)bp;
      notes[S::bytes / 16 + tt * S::KC + c] = (uint8_t)bn;
    }
    rw_barrier();
    return notes;
  };

  // The tiles, one barrier each.
  //   bound(t):  keys t and values t - 1 are there, and every wave is done with step t - 1
  //              products t - 1, scores t
  //              send t: the copies of keys t + 1 and values t, into the buffers that
  //              tile t - 1 has left
  //              softmax t
  at_f16 s[S::NT];
  kv_u4 P[2 * S::NT];
  const uint8_t* noted = nullptr;
  const auto key_buf = [&](int t) { return keys + (t & (S::NB - 1)) * S::bytes; };
  const auto val_buf = [&](int t) { return vals + (t & (S::NB - 1)) * S::bytes; };
  // The copies.  What a send needs is made while the one before is on its way: the
  // table entry of this wave's tokens of the next tile is loaded then and looked at
  // only when it is used, and the values' address is the keys' of a send before.
  const int mask = (1 << a.c.page_shift) - 1;
  const char* const pool0 = reinterpret_cast<const char*>(a.c.pool) + (((int64_t)head << a.c.page_shift)) * D * 2;
  const int64_t page_bytes = a.c.page_stride * 2, v_bytes = a.c.v_off * 2;
  const int lane0 = wave * S::RW;
  int at_tok = 0, at_id = 0;        // this wave's first token of the tile to be sent next, its page's id
  const char* before = pool0;    // where the keys sent last came from
  int kofs[S::LD], vofs[S::LD];  // this lane's byte of each copy
#pragma unroll
  for (int i = 0; i < S::LD; ++i) {
    const int x = i * 64 + lane, k = x / S::KC, c = x % S::KC;  // token of the wave's, chunk's place
    kofs[i] = k * D * 2 + (c ^ rw_key_swz<D>(lane0 + k)) * 16;
    vofs[i] = k * D * 2 + (c ^ rw_val_swz<D>(lane0 + k)) * 16;
  }
  const auto look = [&](int t) {
    at_tok = token(min(t, nt - 1)) + lane0;
    at_id = kv_table(table, min(at_tok, p1) >> a.c.page_shift);
  };
  const auto send = [&](int t) {
    const int to = (t + 1) & (S::NB - 1), to1 = t & (S::NB - 1);
    const char* const from = pool0 + kv_page(a.c, at_id) * page_bytes + (at_tok & mask) * (D * 2);
    if (t + 1 < nt)
#pragma unroll
      for (int i = 0; i < S::LD; ++i) rw_copy(from, kofs[i], keys + to * S::bytes + (wave * S::LD + i) * 1024);
    if (t >= 0)
#pragma unroll
      for (int i = 0; i < S::LD; ++i) rw_copy(before + v_bytes, vofs[i], vals + to1 * S::bytes + (wave * S::LD + i) * 1024);
    before = from;
    look(t + 2);
  };
  const auto bound = [&](int t) {
    __builtin_amdgcn_s_waitcnt(at_wait_vm(0));  // this wave's copies of keys t and values t - 1 have landed
    rw_barrier();  // everyone's have, and the buffers of the tile before are free
    noted = t > 0 ? mend(t - 1, val_buf(t - 1)) : nullptr;
  };
  if (nt > 0) {
    look(0);
    send(-1);
    bound(0);
    // (a wave without rows only copies and keeps step)
    if (alive) rw_scores<D, BF>(s, r, key_buf(0), lane);
    for (int t = 0; t < nt; ++t) {
      send(t);
      if (alive) rw_softmax<D, BF>(P, s, r, a, token(t), t < wclear0 || t >= wclear1, lane);
      bound(t + 1);
      if (!alive) continue;
      __builtin_amdgcn_s_setprio(1);  // a product is one issue in eight: let it have it
      rw_products<D, BF>(r, P, a, val_buf(t), token(t), noted, lane);
      if (t + 1 < nt) rw_scores<D, BF>(s, r, key_buf(t + 1), lane);
      __builtin_amdgcn_s_setprio(0);
    }
  }

  r.l += __shfl_xor(r.l, 32);
  if (MODE != RW_PREFIX && parts == 1) {
    if (live) {
      if constexpr (MODE == RW_REST) if (blk.shared.tokens > 0) {
        const AtPrefix<D> p(a, blk.shared, head, 0.0f);
        const at_f2 ml = p.ml(rw);
        const float m = r.m * a.scale_log2, M = at_safe(fmaxf(m, ml.x));
        const float f = at_exp2(m - M), g = at_exp2(ml.x - M);
        r.l = f * r.l + g * ml.y;
#pragma unroll
        for (int x = 0; x < S::ND; ++x)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const at_f4 v = p.o(rw, x * 32 + 2 * i + 4 * h);
#pragma unroll
            for (int k = 0; k < 4; ++k) r.O[x][i + k] = f * r.O[x][i + k] + g * v[k];
          }
      }
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
  // several workgroups share the block: k_attn_rows_join puts their partials together
  const auto rs = at_slots(a.partial, a.partial_floats);
  const uint32_t slot = (MODE == RW_PREFIX ? z * blocks + (unsigned)id : blockIdx.x) * (uint32_t)rows_slot(D), row = wave * 32 + col;
  if (live) {
#pragma unroll
    for (int x = 0; x < S::ND; ++x)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        at_st4(rs, slot + row * D + x * 32 + 2 * i + 4 * h, at_f4{r.O[x][i], r.O[x][i + 1], r.O[x][i + 2], r.O[x][i + 3]});
    if (h == 0) at_st2(rs, slot + S::BM * D + 2 * row, r.m * a.scale_log2, r.l);
  }
}

// The blocks that several workgroups have shared, eight rows to a workgroup: a launch
// of its own, for one workgroup per block (the last to arrive) would have to read all
// of a block's partials alone.  The last 16 rows of 16,384 tokens, 40 q and 8 kv heads of
// 128: 40 us against 97 in the same parts; a prompt of 1,024 tokens: 33 against 94.
constexpr int RJ_ROWS = 8, RJ_THREADS = 256;
template <int D, bool BF, int MODE = RW_WHOLE> __global__ __launch_bounds__(RJ_THREADS) void k_attn_rows_join(AttnArgs a) {
  using S = RowsShape<D>;
  __shared__ __align__(16) float lds[3 * AT_JOIN_CAP];
  constexpr int PER = S::BM / RJ_ROWS;
  const unsigned id = blockIdx.x / PER, blocks = gridDim.x / PER;
  const RowsBlock<D, MODE> b(a, id);
  const int f0 = (blockIdx.x % PER) * RJ_ROWS;
  if (b.rb < 0 || b.parts == 1 || f0 >= b.nrows) return;
  const auto slot = [&](int k) { return (k * blocks + id) * (uint32_t)rows_slot(D); };
  const int n = min(b.nrows - f0, RJ_ROWS);
  if constexpr (MODE == RW_REST)
    at_join<BF, D, RJ_THREADS>(a, at_slots(a.partial, a.partial_floats), b.e, b.head, b.r0, f0, n, S::BM, b.parts, lds,
                               lds + AT_JOIN_CAP, lds + 2 * AT_JOIN_CAP, slot, AtPrefix<D>(a, b.shared, b.head, 0.0f));
  else
    at_join<BF, D, RJ_THREADS>(a, at_slots(a.partial, a.partial_floats), b.e, b.head, b.r0, f0, n, S::BM, b.parts, lds,
                               lds + AT_JOIN_CAP, lds + 2 * AT_JOIN_CAP, slot);
}

}  // namespace qg
