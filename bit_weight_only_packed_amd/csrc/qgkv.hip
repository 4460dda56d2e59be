// qgkv.hip -- host side of the C ABI declared in include/qgkv.h: descriptor and
// argument checks, the handle's workspace, and the choice between the few-row and
// the many-row attention kernel.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <new>

#include "../../include/qgkv.h"
#include "qg_error.h"
#include "qg_kv.h"
#include "qg_launch.h"

using namespace qg;

struct qg_kv {
  qg_kv_desc d{};
  int device = 0, cus = 0, shift = 0, elem = 2;
  bool debug_sync = false;
  KvPool pool{};
  float* partial = nullptr;   // attention partials
  size_t partial_floats = 0;
  int* counters = nullptr;    // arrivals, zero between launches
  int32_t* lists = nullptr;   // head | from | to | place of the page operations
  int ncounters = 0;
};

namespace {

constexpr int kMaxPages = 1 << 20;
// (block, part) pairs of a many-row call whose blocks are shared: two workgroups for each
// of 256 CUs where the parts are long, one where they are short
constexpr int kRowsSlots = 512;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

void free_kv(qg_kv* h) {
  if (!h) return;
  if (h->partial) hipFree(h->partial);
  if (h->counters) hipFree(h->counters);
  if (h->lists) hipFree(h->lists);
  delete h;
}

qg_status done(const qg_kv* h, hipError_t e, hipStream_t st) {
  if (e != hipSuccess) return fail(QG_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
  if (h->debug_sync) {
    e = hipStreamSynchronize(st);
    if (e != hipSuccess) return fail(QG_ERR_DEVICE, "kernel failed: %s", hipGetErrorString(e));
  }
  return QG_OK;
}

// the handle, and that its device is the current one
qg_status check_handle(const qg_kv* h) {
  clear_error();
  if (!h) return fail(QG_ERR_INVALID_ARG, "cache handle is NULL");
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return fail(QG_ERR_DEVICE, "no current HIP device");
  if (dev != h->device) return fail(QG_ERR_INVALID_ARG, "current device %d is not the cache's %d", dev, h->device);
  return QG_OK;
}

qg_status check_list(const qg_kv* h, const void* p, int n, const char* name) {
  if (n < 1 || n > h->d.max_seqs) return fail(QG_ERR_INVALID_ARG, "n = %d is not in [1, max_seqs = %d]", n, h->d.max_seqs);
  if (!p || !aligned4(p)) return fail(QG_ERR_INVALID_ARG, "%s must be a 4-byte aligned device pointer", name);
  return QG_OK;
}

qg_status batch_of(const qg_kv* h, int layer, const qg_kv_batch* b, KvDev* c, KvBatchDev* out) {
  if (layer < 0 || layer >= h->d.layers) return fail(QG_ERR_INVALID_ARG, "layer = %d is not in [0, %d)", layer, h->d.layers);
  if (!b) return fail(QG_ERR_INVALID_ARG, "batch is NULL");
  if (b->n < (b->rows ? 1 : 0) || b->n > h->d.max_seqs)
    return fail(QG_ERR_INVALID_ARG, "n = %d is not in [1, max_seqs = %d]", b->n, h->d.max_seqs);
  if (b->rows < 0) return fail(QG_ERR_INVALID_ARG, "rows = %d is negative", b->rows);
  if (!aligned4(b->seqs) || !aligned4(b->row_start))
    return fail(QG_ERR_INVALID_ARG, "seqs and row_start must be 4-byte aligned");
  out->rows = b->rows;
  if (b->rows == 0) return QG_OK;  // nothing to do, and no more to check
  if (b->row_start) {
    if (b->max_rows < 1 || b->max_rows > b->rows)
      return fail(QG_ERR_INVALID_ARG, "max_rows = %d is not in [1, rows = %d]", b->max_rows, b->rows);
  } else if (b->rows % b->n) {
    return fail(QG_ERR_INVALID_ARG, "rows = %d is not a multiple of n = %d (pass row_start)", b->rows, b->n);
  }
  const qg_kv_desc& d = h->d;
  const int64_t half = (int64_t)d.kv_heads * d.page_size * d.head_dim;
  c->pool = static_cast<const uint16_t*>(d.pool) + 2 * half * layer;
  c->tables = d.tables;
  c->lens = d.lens;
  c->page_stride = 2 * half * d.layers;
  c->v_off = half;
  c->pages = d.pages;
  c->max_pages = d.max_pages;
  c->max_seqs = d.max_seqs;
  c->page_shift = h->shift;
  c->kv_heads = d.kv_heads;
  c->cap = d.max_pages * d.page_size;
  out->seqs = b->seqs;
  out->row_start = b->row_start;
  out->n = b->n;
  out->max_rows = b->row_start ? b->max_rows : b->rows / b->n;
  return QG_OK;
}

// an operand of so many rows and heads (the stride of one alone is never used, and may be anything)
qg_status rows_of(const qg_kv_rows* r, const char* name, int64_t rows, int64_t heads, KvRows* out) {
  if (!r || !r->ptr) return fail(QG_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(r->ptr)) return fail(QG_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  const int64_t row = rows > 1 ? r->row_stride : 0, head = heads > 1 ? r->head_stride : 0;
  if (row % 8 || head % 8 || row < 0 || head < 0)
    return fail(QG_ERR_INVALID_ARG, "%s: strides %lld, %lld are not multiples of 8 elements", name,
                (long long)r->row_stride, (long long)r->head_stride);
  *out = KvRows{static_cast<const uint16_t*>(r->ptr), row, head};
  return QG_OK;
}

// Whether two of the D-element runs that begin at r * row + h * head (r < rows, h < heads)
// and at those places + ofs share elements; with ofs 0 two runs of the same kind.
bool runs_meet(int64_t row, int64_t head, int64_t rows, int64_t heads, int64_t D, int64_t ofs) {
  if (ofs == 0 && rows > 1 && row < D) return true;
  for (int64_t dh = 1 - heads; dh < heads; ++dh) {
    if (ofs == 0 && dh == 0) continue;
    const int64_t to = ofs + dh * head;  // less the dr rows that come nearest to it
    const int64_t dr = row > 0 ? std::clamp(to / row, 1 - rows, rows - 1) : 0;
    for (int64_t x = std::max(dr - 1, 1 - rows); x <= std::min(dr + 1, rows - 1); ++x)
      if (std::abs(to - x * row) < D) return true;
  }
  return false;
}

// out [rows][heads][D] against itself and against q of the same shape.  What is plainly apart
// is not looked into: rows that hold their heads, operands in different memory or in columns of
// one tensor's rows.  (Operands of different strides that share memory are left to the caller.)
qg_status check_overlap(const KvRows& q, const KvRows& out, int64_t rows, int64_t heads, int64_t D) {
  const int64_t ow = (heads - 1) * out.head + D, qw = (heads - 1) * q.head + D;  // a row's extent
  const bool nested = (heads == 1 || out.head >= D) && (rows == 1 || out.row >= ow);
  if (!nested && runs_meet(out.row, out.head, rows, heads, D, 0))
    return fail(QG_ERR_INVALID_ARG, "out: strides %lld, %lld: rows or heads overlap", (long long)out.row, (long long)out.head);
  const int64_t ofs = (int64_t)((intptr_t)out.ptr - (intptr_t)q.ptr) / 2;
  if (ofs >= (rows - 1) * q.row + qw || -ofs >= (rows - 1) * out.row + ow) return QG_OK;
  if (rows > 1 && q.row == out.row && q.row > 0) {
    const int64_t at = (ofs % q.row + q.row) % q.row;
    if (at >= qw && at + ow <= q.row) return QG_OK;
  }
  if (ofs == 0 || ((rows == 1 || q.row == out.row) && (heads == 1 || q.head == out.head) &&
                   runs_meet(q.row, q.head, rows, heads, D, ofs)))
    return fail(QG_ERR_INVALID_ARG, "out overlaps q");
  return QG_OK;
}

}  // namespace

extern "C" {

qg_status qgkv_create(qg_kv_handle* out, const qg_kv_desc* d, void* stream) {
  clear_error();
  if (!out) return fail(QG_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!d) return fail(QG_ERR_INVALID_ARG, "desc is NULL");
  if (d->pages < 1 || d->pages > kMaxPages) return fail(QG_ERR_INVALID_ARG, "pages = %d is not in [1, %d]", d->pages, kMaxPages);
  if (d->layers < 1) return fail(QG_ERR_INVALID_ARG, "layers = %d is not positive", d->layers);
  if (d->kv_heads < 1 || d->kv_heads > 1024) return fail(QG_ERR_INVALID_ARG, "kv_heads = %d is not in [1, 1024]", d->kv_heads);
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return fail(QG_ERR_UNSUPPORTED, "head_dim = %d is not 64, 128 or 256", d->head_dim);
  int shift = 0;
  while ((1 << shift) < d->page_size && shift < 30) ++shift;
  if (d->page_size < QG_KV_MIN_PAGE || d->page_size > QG_KV_MAX_PAGE || (1 << shift) != d->page_size)
    return fail(QG_ERR_INVALID_ARG, "page_size = %d is not a power of two in [%d, %d]", d->page_size, QG_KV_MIN_PAGE,
                QG_KV_MAX_PAGE);
  if (d->max_seqs < 1 || d->max_seqs > QG_KV_MAX_SEQS)
    return fail(QG_ERR_INVALID_ARG, "max_seqs = %d is not in [1, %d]", d->max_seqs, QG_KV_MAX_SEQS);
  if (d->max_pages < 1 || (int64_t)d->max_pages * d->page_size > (1 << 30))
    return fail(QG_ERR_INVALID_ARG, "max_pages = %d: a slot holds 1 page to 2^30 tokens", d->max_pages);
  if (d->dtype != QG_KV_F16 && d->dtype != QG_KV_BF16) return fail(QG_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
  if (!d->pool || !d->tables || !d->lens || !d->refs || !d->info)
    return fail(QG_ERR_INVALID_ARG, "pool, tables, lens, refs and info must be device pointers");
  if (!aligned16(d->pool) || !aligned16(d->refs)) return fail(QG_ERR_INVALID_ARG, "pool and refs must be 16-byte aligned");
  if (!aligned4(d->tables) || !aligned4(d->lens) || !aligned4(d->info))
    return fail(QG_ERR_INVALID_ARG, "tables, lens and info must be 4-byte aligned");
  int dev = 0;
  qg_status s = check_device(&dev);
  if (s != QG_OK) return s;
  qg_kv* h = new (std::nothrow) qg_kv();
  if (!h) return fail(QG_ERR_OOM, "host allocation failed");
  h->d = *d;
  h->device = dev;
  h->shift = shift;
  h->debug_sync = getenv("QG_DEBUG_SYNC") != nullptr;
  if (hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || h->cus < 1) {
    free_kv(h);
    return fail(QG_ERR_DEVICE, "cannot query the compute-unit count");
  }
  const size_t step = (size_t)2 * h->cus * step_slot(step_max_rows(d->head_dim) / 16, d->head_dim);
  const size_t rows = (size_t)kRowsSlots * rows_slot(d->head_dim);
  const size_t entries = (size_t)std::max(d->pages, d->max_seqs);
  h->ncounters = (d->max_seqs * d->kv_heads + 3) / 4 * 4;
  hipStream_t st = (hipStream_t)stream;
  h->partial_floats = std::max(step, rows);
  if (hipMalloc(&h->partial, h->partial_floats * sizeof(float)) != hipSuccess ||
      hipMalloc(&h->counters, (size_t)h->ncounters * sizeof(int)) != hipSuccess ||
      hipMalloc(&h->lists, (4 + 3 * entries) * sizeof(int32_t)) != hipSuccess) {
    (void)hipGetLastError();
    s = fail(QG_ERR_OOM, "workspace allocation failed");
  }
  if (s == QG_OK && attn_step_allow_lds() != hipSuccess)
    s = fail(QG_ERR_DEVICE, "cannot raise the LDS limit of the kernels");
  if (s == QG_OK && (launch_fill_zero(h->counters, (int64_t)h->ncounters * sizeof(int), st) != hipSuccess ||
                     launch_fill_zero(h->lists, 4 * sizeof(int32_t), st) != hipSuccess))
    s = fail(QG_ERR_DEVICE, "workspace initialisation failed");
  if (hipStreamSynchronize(st) != hipSuccess && s == QG_OK) s = fail(QG_ERR_DEVICE, "stream synchronisation failed");
  if (s != QG_OK) {
    free_kv(h);
    return s;
  }
  KvPool& p = h->pool;
  p.pool = static_cast<uint16_t*>(d->pool);
  p.tables = d->tables;
  p.lens = d->lens;
  p.refs = d->refs;
  p.info = d->info;
  p.page_bytes = (int64_t)4 * d->layers * d->kv_heads * d->page_size * d->head_dim;
  p.pages = d->pages;
  p.max_seqs = d->max_seqs;
  p.max_pages = d->max_pages;
  p.page_shift = shift;
  p.head = h->lists;
  p.from = h->lists + 4;
  p.to = p.from + entries;
  p.place = p.to + entries;
  *out = h;
  return QG_OK;
}

qg_status qgkv_destroy(qg_kv_handle h) {
  clear_error();
  free_kv(h);
  return QG_OK;
}

qg_status qgkv_extend(qg_kv_handle h, const int32_t* n_new, void* stream) {
  qg_status s = check_handle(h);
  if (s != QG_OK) return s;
  if (!n_new || !aligned4(n_new)) return fail(QG_ERR_INVALID_ARG, "n_new must be a 4-byte aligned device pointer");
  hipStream_t st = (hipStream_t)stream;
  return done(h, launch_kv_extend(h->pool, n_new, h->cus, st), st);
}

qg_status qgkv_fork(qg_kv_handle h, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  qg_status s = check_handle(h);
  if (s == QG_OK) s = check_list(h, src, n, "src");
  if (s == QG_OK) s = check_list(h, dst, n, "dst");
  if (s != QG_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  return done(h, launch_kv_fork(h->pool, src, dst, n, st), st);
}

qg_status qgkv_trim(qg_kv_handle h, const int32_t* seqs, const int32_t* keep, int32_t n, void* stream) {
  qg_status s = check_handle(h);
  if (s == QG_OK) s = check_list(h, seqs, n, "seqs");
  if (s != QG_OK) return s;
  if (!aligned4(keep)) return fail(QG_ERR_INVALID_ARG, "keep must be 4-byte aligned");
  hipStream_t st = (hipStream_t)stream;
  return done(h, launch_kv_trim(h->pool, seqs, keep, n, st), st);
}

qg_status qgkv_compact(qg_kv_handle h, void* stream) {
  qg_status s = check_handle(h);
  if (s != QG_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  return done(h, launch_kv_compact(h->pool, h->cus, st), st);
}

qg_status qgkv_append(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* k, const qg_kv_rows* v,
                      void* stream) {
  qg_status s = check_handle(h);
  KvDev c;
  KvBatchDev bd;
  KvRows kr, vr;
  if (s == QG_OK) s = batch_of(h, layer, b, &c, &bd);
  if (s == QG_OK && bd.rows == 0) return QG_OK;
  if (s == QG_OK) s = rows_of(k, "k", bd.rows, c.kv_heads, &kr);
  if (s == QG_OK) s = rows_of(v, "v", bd.rows, c.kv_heads, &vr);
  if (s != QG_OK) return s;
  if ((int64_t)bd.max_rows * 2 * c.kv_heads >= (int64_t)1 << 31)
    return fail(QG_ERR_UNSUPPORTED, "%d rows of %d heads in one call", bd.max_rows, c.kv_heads);
  hipStream_t st = (hipStream_t)stream;
  return done(h, launch_kv_append(c, bd, kr, vr, h->pool.head + 2, h->pool.info, h->d.head_dim, st), st);
}

qg_status qgkv_attend(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* q, const qg_kv_rows* out,
                      int32_t q_heads, float scale, int32_t window, int32_t sinks, void* stream) {
  qg_status s = check_handle(h);
  AttnArgs a{};
  if (s == QG_OK) s = batch_of(h, layer, b, &a.c, &a.b);
  if (s == QG_OK && a.b.rows == 0) return QG_OK;
  if (s == QG_OK) s = rows_of(q, "q", a.b.rows, q_heads, &a.q);
  if (s == QG_OK) s = rows_of(out, "out", a.b.rows, q_heads, &a.out);
  if (s != QG_OK) return s;
  if (q_heads < 1 || q_heads % a.c.kv_heads)
    return fail(QG_ERR_INVALID_ARG, "q_heads = %d is not a positive multiple of kv_heads = %d", q_heads, a.c.kv_heads);
  if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(QG_ERR_INVALID_ARG, "scale = %g is not positive and finite", scale);
  if (window < 0 || sinks < 0) return fail(QG_ERR_INVALID_ARG, "window = %d, sinks = %d: negative", window, sinks);
  a.G = q_heads / a.c.kv_heads;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!std::isfinite(a.scale_log2)) return fail(QG_ERR_INVALID_ARG, "scale = %g is too large", scale);
  s = check_overlap(a.q, a.out, a.b.rows, q_heads, h->d.head_dim);
  if (s != QG_OK) return s;
  a.window = window;
  a.sinks = sinks;
  a.partial = h->partial;
  a.partial_floats = h->partial_floats;
  a.counters = h->counters;
  const int D = h->d.head_dim;
  const bool bf16 = h->d.dtype == QG_KV_BF16;
  const int64_t rows = (int64_t)a.b.max_rows * a.G;  // rows of a kv head
  if (rows >= (int64_t)1 << 30) return fail(QG_ERR_UNSUPPORTED, "%d rows of %d heads in one call", a.b.max_rows, a.G);
  hipStream_t st = (hipStream_t)stream;
  if (rows <= step_max_rows(D)) {
    const int MT = (int)(rows + 15) / 16;
    // places of the few-row kernel's list
    if ((int64_t)(a.c.cap / 32 + 32) * a.b.n * a.c.kv_heads >= (int64_t)1 << 30)
      return fail(QG_ERR_UNSUPPORTED, "%d entries of up to %d tokens and %d kv heads in one call", a.b.n, a.c.cap, a.c.kv_heads);
    a.workers = h->cus;
    a.min_run = STEP_MIN_RUN;
    return done(h, launch_attn_step(a, D, bf16, MT, st), st);
  }
  // A call of few blocks is split over the tokens until it covers the chip: once for parts
  // of few tiles, twice for parts of many (the last 512 rows of 65,536 tokens, 40 q and 8
  // kv heads of 128: 741 us with two, 1,507 with one; the last 16 of each of 4 slots of
  // 8,192: 53 and 47).  A cache whose slots hold too little for parts saves the join.
  const int64_t blocks = (rows + ROWS_BLOCK - 1) / ROWS_BLOCK * a.b.n * a.c.kv_heads;
  a.splits1 = (int)std::max<int64_t>(1, kRowsSlots / 2 / blocks);
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(kRowsSlots / blocks, rows_parts(D, a.c.cap, a.splits1)));
  if (blocks * a.splits >= (int64_t)1 << 31) return fail(QG_ERR_UNSUPPORTED, "%lld blocks in one call", (long long)blocks);
  return done(h, launch_attn_rows(a, D, bf16, (unsigned)blocks, st), st);
}

}  // extern "C"
