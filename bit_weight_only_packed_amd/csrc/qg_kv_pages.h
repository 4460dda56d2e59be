// qg_kv_pages.h -- what is done to the pages of a key-value cache: forking,
// cutting and freeing sequences, making room for new tokens (with the copy of
// shared tails), moving the live pages together, and writing new tokens.
//
// The decisions (which pages are free, who takes which, what moves) are integer
// work on small arrays: one workgroup makes them, so they need no order between
// workgroups and come out the same every time.  What has weight is the copying
// of pages, layers * 2 * kv_heads * page_size * head_dim elements each,
// contiguous: a launch of its own that reads its list from the workspace and
// covers the chip.  Its bound is HBM, 2 bytes moved per byte copied.
#pragma once
#include "qg_kv.h"

namespace qg {

constexpr int KV_PLAN = 1024;  // threads of the deciding workgroup

// exclusive prefix sum over the workgroup's KV_PLAN threads; *total gets the sum
__device__ __forceinline__ int plan_scan(int v, int* lds, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of a scan before this one have been read
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < KV_PLAN / 64; ++w) {
    const int t = lds[w];
    before += w < wave ? t : 0;
    all += t;
  }
  *total = all;
  return before + x - v;
}

// refs[4 i .. 4 i + 3] (past the end: -1, neither free nor live)
__device__ __forceinline__ int4 plan_refs(const KvPool& p, int i) {
  if (4 * i + 3 < p.pages) return reinterpret_cast<const int4*>(p.refs)[i];
  int4 r = make_int4(-1, -1, -1, -1);
  if (4 * i < p.pages) r.x = p.refs[4 * i];
  if (4 * i + 1 < p.pages) r.y = p.refs[4 * i + 1];
  if (4 * i + 2 < p.pages) r.z = p.refs[4 * i + 2];
  return r;
}

__device__ __forceinline__ int kv_used(int len, int shift) { return (int)(((int64_t)len + (1 << shift) - 1) >> shift); }

// tokens of a slot: never more than its table holds
__device__ __forceinline__ int kv_len(const KvPool& p, int s) {
  return (int)min<int64_t>(max(p.lens[s], 0), (int64_t)p.max_pages << p.page_shift);
}

// One workgroup per pair.  A pair decides for itself: it looks at the call's
// other pairs, and the slots it reads or writes are no other accepted pair's to
// write (an earlier pair's dst refuses it, and so does a source that any pair
// has as dst).
__global__ __launch_bounds__(256) void k_kv_fork(KvPool p, const int32_t* src, const int32_t* dst, int n) {
  const int i = blockIdx.x, s = src[i], d = dst[i];
  bool bad = (unsigned)s >= (unsigned)p.max_seqs || (unsigned)d >= (unsigned)p.max_seqs;
  for (int k = threadIdx.x; k < n; k += 256) bad |= dst[k] == s || (k < i && dst[k] == d);
  bool refused = __syncthreads_or(bad);
  if (!refused) refused = p.lens[d] != 0;
  if (__syncthreads_or(refused)) {
    if (threadIdx.x == 0) atomicOr(p.info, 4);
    return;
  }
  const int len = kv_len(p, s), used = kv_used(len, p.page_shift);
  const int32_t* from = p.tables + (int64_t)s * p.max_pages;
  int32_t* to = p.tables + (int64_t)d * p.max_pages;
  for (int k = threadIdx.x; k < used; k += 256) {
    const int id = from[k];
    to[k] = id;
    if ((unsigned)id < (unsigned)p.pages) atomicAdd(p.refs + id, 1);
  }
  if (threadIdx.x == 0) p.lens[d] = len;  // every thread has seen lens[d] == 0 (the barrier above)
}

// One workgroup per entry; the pages of different slots meet in refs only, by
// integer atomics (any order, one result).
__global__ __launch_bounds__(256) void k_kv_trim(KvPool p, const int32_t* seqs, const int32_t* keep) {
  const int i = blockIdx.x, s = seqs[i];
  bool bad = (unsigned)s >= (unsigned)p.max_seqs;
  for (int k = threadIdx.x; k < i; k += 256) bad |= seqs[k] == s;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(p.info, 4);
    return;
  }
  const int len = kv_len(p, s), left = min(keep ? max(keep[i], 0) : 0, len);
  const int u0 = kv_used(left, p.page_shift), u1 = kv_used(len, p.page_shift);
  int32_t* t = p.tables + (int64_t)s * p.max_pages;
  for (int k = u0 + threadIdx.x; k < u1; k += 256) {
    const int id = t[k];
    if ((unsigned)id < (unsigned)p.pages) atomicSub(p.refs + id, 1);
    t[k] = -1;
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) p.lens[s] = left;
}

// Room for new tokens: thread s decides for slot s.
__global__ __launch_bounds__(KV_PLAN) void k_kv_extend(KvPool p, const int32_t* n_new) {
  __shared__ int sums[KV_PLAN / 64];
  __shared__ __align__(16) int tails[KV_PLAN];  // shared tail page that the slot would write to, or -1
  __shared__ int begin[KV_PLAN];  // pages taken by the slots before
  __shared__ int first[KV_PLAN];  // table entry of the slot's first new page; bit 30: a copy of its tail comes before
  const int s = threadIdx.x, P = 1 << p.page_shift;
  const bool slot = s < p.max_seqs;
  const int len = slot ? kv_len(p, s) : 0, add = slot ? max(n_new[s], 0) : 0;
  const int64_t grown = (int64_t)len + add;
  const bool too_long = grown > ((int64_t)p.max_pages << p.page_shift);
  const int used = kv_used(len, p.page_shift);
  // more than the pool holds is short anyway (and 1024 of these stay below 2^31)
  const int wanted = too_long ? 0 : kv_used((int)grown, p.page_shift) - used;  // at most 2^26
  const int need = min(wanted, p.pages + 1);
  int32_t* table = p.tables + (int64_t)(slot ? s : 0) * p.max_pages;
  int tail = -1, holders = 0;
  if (add > 0 && (len & (P - 1)) != 0 && !too_long) {
    tail = table[used - 1];
    holders = (unsigned)tail < (unsigned)p.pages ? p.refs[tail] : 0;
    if (holders <= 1) tail = -1;
  }
  tails[s] = tail;
  __syncthreads();
  bool copy = false;
  if (tail >= 0) {
    int growing = 0;
    bool lowest = true;
#pragma unroll 4
    for (int k = 0; k < p.max_seqs; k += 4) {  // (slots past max_seqs have -1)
      const int4 t = *reinterpret_cast<const int4*>(tails + k);
      growing += (t.x == tail) + (t.y == tail) + (t.z == tail) + (t.w == tail);
      lowest = lowest & !((t.x == tail) & (k < s)) & !((t.y == tail) & (k + 1 < s)) & !((t.z == tail) & (k + 2 < s)) &
               !((t.w == tail) & (k + 3 < s));
    }
    copy = !(growing == holders && lowest);
  }
  int total, copies;
  const int b0 = plan_scan(need + copy, sums, &total);
  const int c0 = plan_scan(copy, sums, &copies);
  begin[s] = b0;
  first[s] = used | (copy ? 1 << 30 : 0);
  if (__syncthreads_or(too_long)) {
    if (s == 0) {
      p.head[0] = 0;
      p.head[2] = 2;
      atomicOr(p.info, 2);
    }
    return;
  }
  // the lowest `total` free ids, ascending, into the list `place`
  int found = 0;
  for (int i0 = 0; 4 * (int64_t)i0 < p.pages && found < total; i0 += KV_PLAN) {
    const int4 r = plan_refs(p, i0 + s);
    const int f = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int chunk;
    int k = found + plan_scan(f, sums, &chunk);
    const int id = 4 * (i0 + s);
    if (r.x == 0) { if (k < total) p.place[k] = id; ++k; }
    if (r.y == 0) { if (k < total) p.place[k] = id + 1; ++k; }
    if (r.z == 0) { if (k < total) p.place[k] = id + 2; ++k; }
    if (r.w == 0) { if (k < total) p.place[k] = id + 3; ++k; }
    found += chunk;
  }
  __syncthreads();
  if (found < total) {
    int lo, hi;  // of the pages wanted, all slots together
    plan_scan((wanted & 0xFFFF) + copy, sums, &lo);
    plan_scan(wanted >> 16, sums, &hi);
    if (s == 0) {
      p.head[0] = 0;
      p.head[2] = 1;
      p.info[1] = (int)min<int64_t>(((int64_t)hi << 16) + lo - found, INT32_MAX);
      atomicOr(p.info, 1);
    }
    return;
  }
  if (slot) {
    if (copy) {
      p.from[c0] = tail;
      p.to[c0] = p.place[b0];
      atomicSub(p.refs + tail, 1);
    }
    p.lens[s] = (int)grown;
  }
  if (s == 0) {
    p.head[0] = copies;
    p.head[2] = 0;
  }
  // page k of the list belongs to the last slot whose run starts at or before it
  // (a slot that takes none starts where the next one does, so the last is the taker)
  for (int k = s; k < total; k += KV_PLAN) {
    int lo = 0, hi = p.max_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (begin[mid] <= k) lo = mid;
      else hi = mid - 1;
    }
    const int id = p.place[k], at = k - begin[lo], c = first[lo] >> 30, u = first[lo] & ((1 << 30) - 1);
    p.refs[id] = 1;
    p.tables[(int64_t)lo * p.max_pages + u + at - c] = id;  // the copy takes entry u - 1, the tail's
  }
}

// Which pages move: m live pages; the live ids >= m, in order, take the free ids < m, in order.
__global__ __launch_bounds__(KV_PLAN) void k_kv_compact(KvPool p) {
  __shared__ int sums[KV_PLAN / 64];
  const int t = threadIdx.x;
  int mine = 0;
  for (int i = t; 4 * (int64_t)i < p.pages; i += KV_PLAN) {
    const int4 r = plan_refs(p, i);
    mine += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  int m;
  plan_scan(mine, sums, &m);
  int nf = 0, nt = 0;
  for (int i0 = 0; 4 * (int64_t)i0 < p.pages; i0 += KV_PLAN) {
    const int4 r4 = plan_refs(p, i0 + t);
    const int id = 4 * (i0 + t);
    const int r[4] = {r4.x, r4.y, r4.z, r4.w};
    int f = 0, g = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f += r[e] > 0 && id + e >= m;
      g += r[e] == 0 && id + e < m;
    }
    int cf, cg;
    int kf = nf + plan_scan(f, sums, &cf);
    int kg = nt + plan_scan(g, sums, &cg);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (r[e] > 0 && id + e >= m) p.from[kf++] = id + e;
      if (r[e] == 0 && id + e < m) p.to[kg++] = id + e;
    }
    nf += cf;
    nt += cg;
  }
  __syncthreads();
  // as many live ids lie past m as free ones before it (negative counts, which no
  // operation here leaves, are neither: the shorter list decides)
  const int moves = min(nf, nt);
  for (int k = t; k < moves; k += KV_PLAN) {
    const int a = p.from[k], b = p.to[k];
    p.place[a] = b;
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  for (int k = moves + t; k < nf; k += KV_PLAN) p.place[p.from[k]] = p.from[k];
  if (t == 0) {
    p.head[0] = moves;
    p.head[1] = m;
    p.info[2] = m;
    p.info[3] = moves;
  }
}

// Copy the listed pages (RENAME: and put the moved pages' new ids into the
// tables).  A piece is 16 KiB of a page: 4 x 16 bytes per thread, all loads
// before the stores.  350 pages of 1 MiB moved together, plan included: 159 us, 734 MB
// read and written at 4.6 TB/s, where the card's large copy moves 4.9.
constexpr int KV_PIECE = 16384;
template <bool RENAME>
__global__ __launch_bounds__(256) void k_kv_copy(KvPool p) {
  const int n = p.head[0];
  if constexpr (RENAME) {
    const int m = p.head[1];
    const int64_t all = (int64_t)p.max_seqs * p.max_pages;
    if (n > 0)
      for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int id = p.tables[i];
        if (id >= m && id < p.pages) p.tables[i] = p.place[id];
      }
  }
  const int64_t pieces = (p.page_bytes + KV_PIECE - 1) / KV_PIECE, all = pieces * n;
  char* pool = reinterpret_cast<char*>(p.pool);
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    const int i = (int)(w / pieces);
    const int64_t at = (w - i * pieces) * KV_PIECE;
    const char* a = pool + p.from[i] * p.page_bytes + at;
    char* b = pool + p.to[i] * p.page_bytes + at;
    const int64_t left = p.page_bytes - at;
    kv_u4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int o = (e * 256 + (int)threadIdx.x) * 16;
      if (o < left) x[e] = *reinterpret_cast<const kv_u4*>(a + o);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int o = (e * 256 + (int)threadIdx.x) * 16;
      if (o < left) *reinterpret_cast<kv_u4*>(b + o) = x[e];
    }
  }
}

// New tokens into their pages: a group of D / 8 lanes moves one (row, head) of k
// or of v, 16 bytes a lane.  blockIdx.y is the entry.  16,383 tokens of 8 heads of 128:
// 32 us (134 MB read and written, 4.2 TB/s); one token of each of 64 slots: 3.5 us, the
// launch and three dependent loads (length, table, key).
// Nothing is written while a refused extend stands: the lengths have not grown, so the
// rows would take the places of tokens that the slots, or others through shared pages,
// hold.
template <int D>
__global__ __launch_bounds__(256) void k_kv_append(KvDev c, KvBatchDev b, KvRows k, KvRows v, const int32_t* refused,
                                                   const int32_t* info) {
  if (*refused & *info) return;
  const KvEntry e = kv_entry(c, b, blockIdx.y);
  const int per = 2 * c.kv_heads;  // (k or v, head) pairs of a row
  const uint32_t items = (uint32_t)e.rows * per;  // below 2^31 (checked on the host)
  const int lane = threadIdx.x % (D / 8);
  const int32_t* table = c.tables + (int64_t)e.slot * c.max_pages;
  for (uint32_t i = blockIdx.x * (256 / (D / 8)) + threadIdx.x / (D / 8); i < items;
       i += gridDim.x * (256 / (D / 8))) {
    const int row = (int)(i / per), w = (int)(i - (uint32_t)row * per);
    const int pos = e.pos + row;
    if (pos < 0) continue;
    const int id = table[pos >> c.page_shift];
    if ((unsigned)id >= (unsigned)c.pages) continue;
    const int head = w >> 1;
    const KvRows& x = (w & 1) ? v : k;
    const int slot = pos & ((1 << c.page_shift) - 1);
    uint16_t* to = const_cast<uint16_t*>(c.pool) + id * c.page_stride + ((w & 1) ? c.v_off : 0) +
                   (((int64_t)head << c.page_shift) + slot) * D + lane * 8;
    *reinterpret_cast<kv_u4*>(to) =
        *reinterpret_cast<const kv_u4*>(x.ptr + (int64_t)(e.row0 + row) * x.row + head * x.head + lane * 8);
  }
}

}  // namespace qg
