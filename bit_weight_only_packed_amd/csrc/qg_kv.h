// qg_kv.h -- the paged key-value cache as its kernels see it: the device view of
// a cache, the rows of a call, and the launchers (host code: qgkv.hip).  The
// kernels: qg_kv_pages.h (page operations, append), qg_attn_step.h (attention of
// few rows), qg_attn_rows.h (attention of many rows).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qg {

constexpr int KV_MAX_SEQS = 1024;

// one layer of a cache
struct KvDev {
  const uint16_t* pool;  // this layer's keys of page 0
  const int32_t* tables;
  const int32_t* lens;
  int64_t page_stride;   // elements from a page to the next
  int64_t v_off;         // elements from a page's keys to its values
  int pages, max_pages, max_seqs, page_shift, kv_heads;
  int cap;               // max_pages * page_size
};

struct KvRows {
  const uint16_t* ptr;
  int64_t row, head;     // strides in elements
};

struct KvBatchDev {
  const int32_t* seqs;       // or NULL
  const int32_t* row_start;  // or NULL
  int n, rows, max_rows;     // entries, rows in all, rows of an entry at most
};

// entry j of a call: slot, position of its first row, first row, rows.  Everything that
// comes from device memory is cut to what the cache and the call's operands hold.  Rows
// past max_rows are left out, but count for the position: the others stand where they
// would without the cut.
struct KvEntry {
  int slot, pos, row0, rows;
};
__device__ __forceinline__ KvEntry kv_entry(const KvDev& c, const KvBatchDev& b, int j) {
  KvEntry e;
  int s = b.seqs ? b.seqs[j] : j;
  const bool ok = (unsigned)s < (unsigned)c.max_seqs;
  e.slot = ok ? s : 0;
  const int l = c.lens[e.slot], len = ok ? min(max(l, 0), c.cap) : 0;
  int rows = b.max_rows;
  if (b.row_start) {
    e.row0 = min(max(b.row_start[j], 0), b.rows);
    rows = min(max(b.row_start[j + 1], e.row0), b.rows) - e.row0;
  } else {
    e.row0 = j * b.max_rows;
  }
  e.pos = len - rows;
  e.rows = min(rows, b.max_rows);
  return e;
}

// An entry of a page table, at an address that is the same for the whole wave, by a
// scalar load: it neither takes a place among the vector loads in flight, which are
// waited for in order, nor a vector register.  (No kernel that reads tables this way
// writes them.)
__device__ __forceinline__ int kv_table(const int32_t* table, int i) {
  return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)(table + i);
}

// page that a table names, or page 0 where it names none of the pool
__device__ __forceinline__ int kv_page(const KvDev& c, int id) { return (unsigned)id < (unsigned)c.pages ? id : 0; }

// 16 bytes = 8 elements
typedef uint32_t kv_u4 __attribute__((ext_vector_type(4)));
typedef uint32_t kv_u2 __attribute__((ext_vector_type(2)));

// ---- page operations ---------------------------------------------------------
struct KvPool {
  uint16_t* pool;
  int32_t *tables, *lens, *refs, *info;
  int64_t page_bytes;
  int pages, max_seqs, max_pages, page_shift;
  // workspace: [0] copies to make, [1] first id that moves (compact), [2] the bit of info
  // that the last extend was refused with (0: it was granted), then the lists of source
  // and destination pages and the moved pages' new ids
  int32_t* head;
  int32_t *from, *to, *place;
};

hipError_t launch_kv_fork(const KvPool& p, const int32_t* src, const int32_t* dst, int n, hipStream_t st);
hipError_t launch_kv_trim(const KvPool& p, const int32_t* seqs, const int32_t* keep, int n, hipStream_t st);
hipError_t launch_kv_extend(const KvPool& p, const int32_t* n_new, int cus, hipStream_t st);
hipError_t launch_kv_compact(const KvPool& p, int cus, hipStream_t st);
// refused, info: KvPool's head + 2 and info
hipError_t launch_kv_append(const KvDev& c, const KvBatchDev& b, const KvRows& k, const KvRows& v, const int32_t* refused,
                            const int32_t* info, int D, hipStream_t st);

// ---- attention ---------------------------------------------------------------
struct AttnArgs {
  KvDev c;
  KvBatchDev b;
  KvRows q, out;
  int G;               // q heads per kv head
  float scale_log2;    // scale * log2(e)
  int window, sinks;   // window 0: none
  float* partial;      // partials of work that several workgroups share (o, max, sum of a row)
  size_t partial_floats;
  int* counters;       // few rows: arrivals at a shared (entry, kv head), zero between launches
  int workers;         // few rows: workgroups that share the tiles,
  int min_run;         // and places of their list that each takes at least
  int splits, splits1; // many rows: workgroups that may share a block's tiles, however many it has; and if few
  int first;           // many rows: the launch's first block (0 where blocks are shared)
};

// Rows of one kv head that the few-row kernel takes, (new rows) * (q heads per kv head).
// us of the few-row and of the many-row kernel, fp16, 8 kv heads of 128 (2 of 256):
//   rows          one slot of 8,192   8 of 2,048     16 of 8,192
//   25            25.9 / 24.7         27.7 / 31.6    107.7 / 116.5
//   32            26.7 / 25.3         28.1 / 32.3    108.5 / 120.5
//   45            33.7 / 27.1         34.5 / 33.5    117.4 / 121.2
//   64            54.4 / 27.7         47.1 / 35.5    128.2 / 126.2
//   16, heads 256 28.0 / 32.1         27.7 / 35.0    66.4 / 95.0
//   32, heads 256 50.3 / 33.4         44.4 / 36.9    87.2 / 97.7
__host__ __device__ constexpr int step_max_rows(int D) { return D == 256 ? 16 : 32; }
// waves of a workgroup, one workgroup per CU: two waves per SIMD where the registers allow
__host__ __device__ constexpr int step_waves(int D) { return D == 256 ? 4 : 8; }
// Places of the list that a workgroup takes at least.  One request of 1,025 tokens, 40
// q and 8 kv heads of 128: 13.4 us at 8, 13.1 at 12, 13.8 at 16, 16.0 at 24, 21.1 at 48
// (fewer, longer runs save joins and cost round trips); from a few thousand tokens on
// the runs are longer by themselves.
constexpr int STEP_MIN_RUN = 12;
// fp32 words of one partial of MT row tiles: o, then (max, sum) of each row
__host__ __device__ constexpr size_t step_slot(int MT, int D) { return (size_t)MT * 16 * (D + 2); }
hipError_t launch_attn_step(const AttnArgs& a, int D, bool bf16, int MT, hipStream_t st);

// the many-row kernel: waves of a workgroup, rows of a block (32 a wave), fp32 words of
// its partial
constexpr int ROWS_WAVES = 4, ROWS_BLOCK = 32 * ROWS_WAVES;
__host__ __device__ constexpr size_t rows_slot(int D) { return (size_t)ROWS_BLOCK * (D + 2); }
// parts of a block that sees every token of a slot that holds cap
int rows_parts(int D, int cap, int splits1);
hipError_t launch_attn_rows(const AttnArgs& a, int D, bool bf16, unsigned blocks, hipStream_t st);
hipError_t attn_step_allow_lds();

}  // namespace qg
