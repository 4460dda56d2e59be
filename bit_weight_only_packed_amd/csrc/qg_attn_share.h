// qg_attn_share.h -- attention of entries that name the same first pages: their shared
// tokens are computed once for all rows of a group, then each entry's own.
//
// Forked answers to one prompt, or requests behind one system prompt, hold the same pages
// (qgkv_fork): n of them read one by one cost n times the bytes.  Here the rows of all entries of
// a group are one batch of rows for the many-row kernel, which reads the shared tokens once
// per ROWS_BLOCK of them; the entries' other tokens go the usual way, and a row's two
// results join like any partials.
//
//   k_share_plan        how many tokens each group shares: the leading table entries
//                       that all its entries have alike, up to the first row's position, in whole
//                       tiles.  From the tables as they are, so nothing has to be told or kept.
//   k_attn_rows         (RW_PREFIX) the shared tokens, in parts
//   k_share_join        a block's parts into one result
//   k_attn_step, _rows  (SH, RW_REST) the other tokens, joined with that result
//
// Measured: one row each of 64 answers to 32,768 tokens, 9 to 1,500 tokens of their own, bf16, 40 q and 8 kv heads
// of 128: 115 us (208 MB that it cannot do without, 43 GFLOP), as qgkv_attend 1,260.  The plan 9.4 us (some eight
// dependent round trips), the shared tokens 71 (320 rows in three blocks of 128: 51 GFLOP computed, 720 TFLOP/s, what
// the many-row kernel reaches on long windows; read from HBM once), their join 9, the rest 32 (76 MB; two or three
// entries' beginnings and ends in each workgroup).
#pragma once
#include "qg_attn_rows.h"

namespace qg {

constexpr int SP_T = 256;  // threads of the plan

__device__ __forceinline__ void sp_st(int* p, int v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ int sp_ld(int* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// One workgroup per entry compares its table with that of its group's first entry that sees
// anything; the last to arrive makes the groups' plans.
__global__ __launch_bounds__(SP_T) void k_share_plan(ShareArgs a) {
  __shared__ int group, lead, same, flag;
  __shared__ KvEntry entry[KV_MAX_SEQS];
  __shared__ int g_tokens[KV_MAX_SEQS], g_live[KV_MAX_SEQS], g_lo[KV_MAX_SEQS], g_hi[KV_MAX_SEQS], g_p0[KV_MAX_SEQS],
      g_p1[KV_MAX_SEQS], g_slot[KV_MAX_SEQS], g_base[KV_MAX_SEQS];
  const int j = blockIdx.x, tid = threadIdx.x, n = a.b.n;
  const auto first = [&](int g) { return a.groups ? min(max(a.groups[g], 0), n) : g * n; };
  const auto sees = [](const KvEntry& e) { return e.rows > 0 && e.pos + e.rows > 0; };
  if (tid == 0) group = a.ngroups, lead = n;
  for (int k = tid; k < n; k += SP_T) entry[k] = kv_entry(a.c, a.b, k);
  __syncthreads();
  for (int g = tid; g < a.ngroups; g += SP_T)
    if (first(g) <= j && j < first(g + 1)) atomicMin(&group, g);
  __syncthreads();
  const bool grouped = group < a.ngroups;
  if (grouped)
    for (int k = first(group) + tid; k < first(group + 1); k += SP_T)
      if (sees(entry[k])) {
        atomicMin(&lead, k);
        break;
      }
  const KvEntry e = entry[j];
  // (-1: left out by max_rows; every row between a group's first and last has its position from this call)
  const int all = kv_all_rows(a.b, e, j);
  for (int i = tid; i < all; i += SP_T) a.pos[e.row0 + i] = i < e.rows ? e.pos + i : -1;
  __syncthreads();
  // -1: no constraint on the others (an entry that sees nothing)
  int tokens = -1;
  if (grouped && sees(e)) {
    const KvEntry l = entry[lead];
    const int pages = min(e.pos + 1, l.pos + 1) >> a.c.page_shift;  // whole pages before both's first rows
    if (tid == 0) same = max(pages, 0);
    __syncthreads();
    const int32_t *x = a.c.tables + (int64_t)e.slot * a.c.max_pages, *y = a.c.tables + (int64_t)l.slot * a.c.max_pages;
    if (e.slot != l.slot) {
      int bad = pages;
      for (int i = tid; i < pages && bad == pages; i += 4 * SP_T) {
        bool d[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) d[k] = i + k * SP_T < pages && x[i + k * SP_T] != y[i + k * SP_T];
#pragma unroll
        for (int k = 3; k >= 0; --k) bad = d[k] ? i + k * SP_T : bad;
      }
      if (bad < pages) atomicMin(&same, bad);
      __syncthreads();
    }
    tokens = same << a.c.page_shift;
  }
  if (tid == 0) {
    sp_st(&a.want[j].x, tokens);
    sp_st(&a.want[j].y, grouped ? group : -1);
  }
  if (!at_last(a.counter, n, &flag)) return;

  for (int g = tid; g < a.ngroups; g += SP_T)
    g_tokens[g] = 0x7FFFFFFF, g_live[g] = 0, g_lo[g] = 0x7FFFFFFF, g_hi[g] = 0, g_p0[g] = 0x7FFFFFFF, g_p1[g] = -1, g_slot[g] = n;
  __syncthreads();
  constexpr int PER = KV_MAX_SEQS / SP_T;
  int wt[PER], wg[PER];  // what entries tid, tid + SP_T, ... want
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int k = tid + i * SP_T;
    wt[i] = -1, wg[i] = -1;
    if (k < n) wt[i] = sp_ld(&a.want[k].x), wg[i] = sp_ld(&a.want[k].y);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int k = tid + i * SP_T, t = wt[i], g = wg[i];
    if (g < 0) continue;
    const KvEntry f = entry[k];
    if (f.rows == 0) continue;
    atomicMin(&g_lo[g], f.row0);
    atomicMax(&g_hi[g], f.row0 + f.rows);
    if (t < 0) continue;
    atomicMin(&g_tokens[g], t);
    atomicAdd(&g_live[g], 1);
    atomicMin(&g_p0[g], f.pos);
    atomicMax(&g_p1[g], f.pos + f.rows - 1);
    atomicMin(&g_slot[g], k);
  }
  __syncthreads();
  // blocks of the groups, one after another (few groups: one thread); none where all that sharing
  // would save is less than it costs
  if (tid == 0) {
    int64_t saved = 0;  // tokens less to read, in eighths
    for (int g = 0; g < a.ngroups; ++g) {
      int t = g_live[g] > 1 ? g_tokens[g] / SHARE_TILE * SHARE_TILE : 0;
      if (t < SHARE_MIN) t = 0;
      g_tokens[g] = t;
      if (t == 0) continue;
      const int64_t read = a.window ? min((int64_t)t, (int64_t)a.window + a.sinks) : t;
      const int64_t waves = ((int64_t)(g_hi[g] - g_lo[g]) * a.G + 31) / 32;
      saved += read * (8 * (g_live[g] + a.extra) - a.cost * waves);
    }
    const bool pays = saved >= 8 * a.least;
    int base = 0;
    for (int g = 0; g < a.ngroups; ++g) {
      const int t = pays ? g_tokens[g] : 0;
      const int64_t blocks = t ? ((int64_t)(g_hi[g] - g_lo[g]) * a.G + ROWS_BLOCK - 1) / ROWS_BLOCK : 0;
      const bool fits = blocks <= a.blocks - base;  // (not so where groups overlap, which no allowed call's do)
      g_tokens[g] = fits ? t : 0;
      g_base[g] = base;
      base += fits ? (int)blocks : 0;
    }
    same = base;
  }
  __syncthreads();
  for (int b = tid; b < a.blocks; b += SP_T) {
    ShareBlock s{};
    if (b < same) {
      int g = 0;
      while (g + 1 < a.ngroups && g_base[g + 1] <= b) ++g;  // (groups without blocks begin where the next does)
      while (g_tokens[g] == 0) --g;
      s = ShareBlock{g_tokens[g], entry[g_slot[g]].slot, g_lo[g], (b - g_base[g]) * ROWS_BLOCK,
                     (g_hi[g] - g_lo[g]) * a.G, g_p0[g], g_p1[g]};
    }
    a.share_blocks[b] = s;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int k = tid + i * SP_T, g = wg[i];
    if (k >= n) break;
    ShareEntry s{};
    if (g >= 0 && wt[i] >= 0 && g_tokens[g] > 0)
      s = ShareEntry{g_tokens[g], g_base[g] * ROWS_BLOCK + (entry[k].row0 - g_lo[g]) * a.G};
    a.share[k] = s;
  }
}

// A block's parts, joined in part order into the first one's slot; RJ_ROWS rows a workgroup.
template <int D> __global__ __launch_bounds__(RJ_THREADS) void k_share_join(AttnArgs a) {
  using S = RowsShape<D>;
  constexpr int PER = S::BM / RJ_ROWS, MOST = 512;  // (parts of a block: the slots of the workspace at most)
  __shared__ float fac[RJ_ROWS][MOST];
  const unsigned id = blockIdx.x / PER, blocks = gridDim.x / PER;
  const RowsBlock<D, RW_PREFIX> b(a, id);
  const int f0 = (blockIdx.x % PER) * RJ_ROWS, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (b.rb < 0 || b.parts == 1 || f0 >= b.nrows) return;
  const int n = b.parts, rows = min(b.nrows - f0, RJ_ROWS);
  const auto rs = at_slots(a.prefix, a.prefix_floats);
  const auto slot = [&](int k) { return (k * blocks + id) * (uint32_t)rows_slot(D); };
  float Ms[RJ_ROWS * 64 / RJ_THREADS], Ls[RJ_ROWS * 64 / RJ_THREADS];
#pragma unroll
  for (int i = 0; i < RJ_ROWS * 64 / RJ_THREADS; ++i) {  // a wave per row
    const int r = wave + i * (RJ_THREADS / 64);
    float M = -__builtin_inff(), L = 0.0f;
    if (r < rows) {
      for (int k = lane; k < n; k += 64) M = fmaxf(M, at_ld2(rs, slot(k) + S::BM * D + 2 * (f0 + r)).x);
#pragma unroll
      for (int o = 32; o; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
      for (int k = lane; k < n; k += 64) {
        const at_f2 ml = at_ld2(rs, slot(k) + S::BM * D + 2 * (f0 + r));
        const float f = at_exp2(ml.x - at_safe(M));
        fac[r][k] = f;
        L = __builtin_fmaf(f, ml.y, L);
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) L += __shfl_xor(L, o);
    }
    Ms[i] = M, Ls[i] = L;
  }
  __syncthreads();
  for (int it = tid; it < rows * (D / 4); it += RJ_THREADS) {
    const int r = it / (D / 4), c = (it % (D / 4)) * 4;
    const uint32_t at = (uint32_t)(f0 + r) * D + c;
    at_f4 o = {0, 0, 0, 0};
    constexpr int NB = 16;
    for (int kb = 0; kb < n; kb += NB) {
      at_f4 po[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (kb + k < n) po[k] = at_ld4(rs, at + slot(kb + k));
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (kb + k < n) {
          const float f = fac[r][kb + k];
#pragma unroll
          for (int x = 0; x < 4; ++x) o[x] = __builtin_fmaf(f, po[k][x], o[x]);
        }
    }
    at_st4(rs, at + slot(0), o);
  }
#pragma unroll
  for (int i = 0; i < RJ_ROWS * 64 / RJ_THREADS; ++i) {
    const int r = wave + i * (RJ_THREADS / 64);
    if (r < rows && lane == 0) at_st2(rs, slot(0) + S::BM * D + 2 * (f0 + r), Ms[i], Ls[i]);
  }
}

}  // namespace qg
