// qgkv.hip -- host side of the C ABI declared in include/qgkv.h: descriptor and
// argument checks, the handle's workspace, and the choice between the few-row and
// the many-row attention kernel.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <new>

#include "../../include/qgkv.h"
#include "qg_check.h"
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
  // attention of shared tokens: its blocks' results and plan
  float* prefix = nullptr;
  size_t prefix_floats = 0;
  int* plan = nullptr;
  ShareArgs share{};
};

namespace {

constexpr int kMaxPages = 1 << 20;
// (block, part) pairs of a many-row call whose blocks are shared: two workgroups for each
// of 256 CUs where the parts are long, one where they are short
constexpr int kRowsSlots = 512;

// arrival counter | blocks | what each entry wants | entries | rows' positions
size_t plan_bytes(int max_seqs) {
  return 16 + kRowsSlots * sizeof(ShareBlock) + (size_t)max_seqs * (sizeof(int2) + sizeof(ShareEntry)) + SHARE_ROWS * sizeof(int);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

void free_kv(qg_kv* h) {
  if (!h) return;
  if (h->partial) hipFree(h->partial);
  if (h->counters) hipFree(h->counters);
  if (h->lists) hipFree(h->lists);
  if (h->prefix) hipFree(h->prefix);
  if (h->plan) hipFree(h->plan);
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
  *out = KvRows{static_cast<const uint16_t*>(r->ptr), rows > 1 ? r->row_stride : 0, heads > 1 ? r->head_stride : 0};
  return check_strides(name, out->row, out->head);
}

// the checked arguments of an attention call
qg_status attn_of(qg_kv* h, int layer, const qg_kv_batch* b, const qg_kv_rows* q, const qg_kv_rows* out, int q_heads, float scale,
                  int window, int sinks, AttnArgs* to) {
  qg_status s = check_handle(h);
  AttnArgs& a = *to;
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
  s = check_overlap(a.q, a.out, a.b.rows, q_heads, h->d.head_dim, "out overlaps q");
  if (s != QG_OK) return s;
  a.window = window;
  a.sinks = sinks;
  a.partial = h->partial;
  a.partial_floats = h->partial_floats;
  a.counters = h->counters;
  return QG_OK;
}

// shared: the entries' first tokens have been attended to
qg_status attend(qg_kv* h, AttnArgs& a, bool shared, hipStream_t st) {
  const int D = h->d.head_dim;
  const bool bf16 = h->d.dtype == QG_KV_BF16;
  const int64_t rows = (int64_t)a.b.max_rows * a.G;  // rows of a kv head
  if (rows >= (int64_t)1 << 30) return fail(QG_ERR_UNSUPPORTED, "%d rows of %d heads in one call", a.b.max_rows, a.G);
  if (rows <= step_max_rows(D)) {
    const int MT = (int)(rows + 15) / 16;
    // places of the few-row kernel's list
    if ((int64_t)(a.c.cap / 32 + 32) * a.b.n * a.c.kv_heads >= (int64_t)1 << 30)
      return fail(QG_ERR_UNSUPPORTED, "%d entries of up to %d tokens and %d kv heads in one call", a.b.n, a.c.cap, a.c.kv_heads);
    a.workers = h->cus;
    a.min_run = STEP_MIN_RUN;
    return done(h, launch_attn_step(a, D, bf16, MT, shared, st), st);
  }
  // A call of few blocks is split over the tokens until it covers the chip: once for parts
  // of few tiles, twice for parts of many (the last 512 rows of 65,536 tokens, 40 q and 8
  // kv heads of 128: 741 us with two, 1,507 with one; the last 16 of each of 4 slots of
  // 8,192: 53 and 47).  A cache whose slots hold too little for parts saves the join.
  const int64_t blocks = (rows + ROWS_BLOCK - 1) / ROWS_BLOCK * a.b.n * a.c.kv_heads;
  a.splits1 = (int)std::max<int64_t>(1, kRowsSlots / 2 / blocks);
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(kRowsSlots / blocks, rows_parts(D, a.c.cap, a.splits1, shared)));
  if (blocks * a.splits >= (int64_t)1 << 31) return fail(QG_ERR_UNSUPPORTED, "%lld blocks in one call", (long long)blocks);
  return done(h, launch_attn_rows(a, D, bf16, (unsigned)blocks, shared, st), st);
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
      hipMalloc(&h->lists, (4 + 3 * entries) * sizeof(int32_t)) != hipSuccess ||
      hipMalloc(&h->prefix, rows * sizeof(float)) != hipSuccess || hipMalloc(&h->plan, plan_bytes(d->max_seqs)) != hipSuccess) {
    (void)hipGetLastError();
    s = fail(QG_ERR_OOM, "workspace allocation failed");
  }
  if (s == QG_OK && attn_step_allow_lds() != hipSuccess)
    s = fail(QG_ERR_DEVICE, "cannot raise the LDS limit of the kernels");
  if (s == QG_OK && (launch_fill_zero(h->counters, (int64_t)h->ncounters * sizeof(int), st) != hipSuccess ||
                     launch_fill_zero(h->lists, 4 * sizeof(int32_t), st) != hipSuccess ||
                     launch_fill_zero(h->plan, 16, st) != hipSuccess))
    s = fail(QG_ERR_DEVICE, "workspace initialisation failed");
  if (hipStreamSynchronize(st) != hipSuccess && s == QG_OK) s = fail(QG_ERR_DEVICE, "stream synchronisation failed");
  if (s != QG_OK) {
    free_kv(h);
    return s;
  }
  h->prefix_floats = rows;
  char* at = reinterpret_cast<char*>(h->plan);
  h->share.counter = reinterpret_cast<int*>(at);
  h->share.share_blocks = reinterpret_cast<ShareBlock*>(at += 16);
  h->share.want = reinterpret_cast<int2*>(at += kRowsSlots * sizeof(ShareBlock));
  h->share.share = reinterpret_cast<ShareEntry*>(at += d->max_seqs * sizeof(int2));
  h->share.pos = reinterpret_cast<int*>(at += d->max_seqs * sizeof(ShareEntry));
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

qg_status qgkv_append_rotary(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* k, const qg_kv_rows* v,
                             const qg_kv_rows* q, const qg_kv_rows* q_out, int32_t q_heads, const qgs_rotary* rotary,
                             void* stream) {
  qg_status s = check_handle(h);
  RotAppend a{};
  if (s == QG_OK) s = batch_of(h, layer, b, &a.c, &a.b);
  if (s == QG_OK) s = rotary_of(rotary, h->d.head_dim, &a.r);
  if (s == QG_OK && q_heads < 0) s = fail(QG_ERR_INVALID_ARG, "q_heads = %d is negative", q_heads);
  if (s == QG_OK && a.b.rows == 0) return QG_OK;
  const int D = h ? h->d.head_dim : 0;
  const int64_t rows = a.b.rows, kvh = a.c.kv_heads;
  if (s == QG_OK) s = rows_of(k, "k", rows, kvh, &a.k);
  if (s == QG_OK) s = rows_of(v, "v", rows, kvh, &a.v);
  if (s == QG_OK && q_heads > 0) {
    s = rows_of(q, "q", rows, q_heads, &a.q);
    if (s == QG_OK) s = rows_of(q_out, "q_out", rows, q_heads, &a.out);
    if (s == QG_OK) {
      // in place, or apart; and never over k or v, which other workgroups read
      if (a.q.ptr == a.out.ptr && a.q.row == a.out.row && a.q.head == a.out.head)
        s = check_nested(a.out, rows, q_heads, D);
      else
        s = check_overlap(a.q, a.out, rows, q_heads, D, "q_out overlaps q");
    }
    if (s == QG_OK && (!apart(a.out, q_heads, a.k, kvh, rows, D) || !apart(a.out, q_heads, a.v, kvh, rows, D)))
      s = fail(QG_ERR_INVALID_ARG, "q_out overlaps k or v");
  }
  if (s != QG_OK) return s;
  a.q_heads = q_heads;
  if ((int64_t)a.b.max_rows * (D / 16) * (q_heads + 2 * kvh) >= (int64_t)1 << 31)
    return fail(QG_ERR_UNSUPPORTED, "%d rows of %d heads in one call", a.b.max_rows, q_heads + 2 * (int)kvh);
  a.refused = h->pool.head + 2;
  a.info = h->pool.info;
  hipStream_t st = (hipStream_t)stream;
  return done(h, launch_kv_append_rotary(a, D, h->d.dtype == QG_KV_BF16, h->cus, st), st);
}

qg_status qgkv_attend(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* q, const qg_kv_rows* out,
                      int32_t q_heads, float scale, int32_t window, int32_t sinks, void* stream) {
  AttnArgs a{};
  qg_status s = attn_of(h, layer, b, q, out, q_heads, scale, window, sinks, &a);
  if (s != QG_OK || a.b.rows == 0) return s;
  return attend(h, a, false, (hipStream_t)stream);
}

qg_status qgkv_attend_shared(qg_kv_handle h, int32_t layer, const qg_kv_batch* b, const qg_kv_rows* q, const qg_kv_rows* out,
                             int32_t q_heads, float scale, int32_t window, int32_t sinks, const int32_t* groups,
                             int32_t n_groups, int64_t least, void* stream) {
  AttnArgs a{};
  qg_status s = attn_of(h, layer, b, q, out, q_heads, scale, window, sinks, &a);
  if (s != QG_OK || a.b.rows == 0) return s;
  if (!aligned4(groups)) return fail(QG_ERR_INVALID_ARG, "groups must be 4-byte aligned");
  if (groups && (n_groups < 1 || n_groups > a.b.n)) return fail(QG_ERR_INVALID_ARG, "n_groups = %d is not in [1, n = %d]", n_groups, a.b.n);
  if (!groups) n_groups = 1;
  hipStream_t st = (hipStream_t)stream;
  // a group of k blocks holds more than 128 (k - 1) rows of a kv head
  const int64_t blocks = (int64_t)a.b.rows * a.G / ROWS_BLOCK + n_groups, grid = blocks * a.c.kv_heads;
  // without two entries in a group there is nothing to share; and calls of more rows than the
  // workspace has slots for are made of blocks that read the tokens many times either way
  const int64_t token = (int64_t)4 * a.c.kv_heads * h->d.head_dim;  // bytes of a token
  ShareRule rule{0, 0, 0};
  if (least < 0) {
    rule = share_rule(h->d.head_dim, (int64_t)a.b.max_rows * a.G <= step_max_rows(h->d.head_dim));
    least = (int64_t)rule.mib << 20;
  }
  const int64_t seen = window ? std::min<int64_t>(a.c.cap, (int64_t)window + sinks) : a.c.cap;  // tokens of an entry at most
  // what an entry can bring at most, in eighths: it has a row at least, and without row_start all of its rows
  const int64_t each = std::max<int64_t>(0, 8 - (int64_t)rule.cost * (b->row_start ? 1 : a.b.max_rows) * a.G / 32);
  if (n_groups == a.b.n || a.b.rows > SHARE_ROWS || grid > kRowsSlots ||
      seen * (a.b.n * each + 8 * (int64_t)n_groups * rule.extra) < 8 * (least / token))
    return attend(h, a, false, st);
  ShareArgs p = h->share;
  p.least = least / token;
  p.extra = rule.extra;
  p.cost = rule.cost;
  p.window = window;
  p.sinks = sinks;
  p.c = a.c;
  p.b = a.b;
  p.groups = groups;
  p.ngroups = n_groups;
  p.G = a.G;
  p.blocks = (int)blocks;
  hipError_t e = launch_share_plan(p, st);
  if (e != hipSuccess) return done(h, e, st);
  a.share = p.share;
  a.share_blocks = p.share_blocks;
  a.share_pos = p.pos;
  a.prefix = h->prefix;
  a.prefix_floats = h->prefix_floats;
  AttnArgs x = a;
  x.partial = h->prefix;
  x.partial_floats = h->prefix_floats;
  // (one workgroup a CU with heads of 256: what the partials of more cost is more than they bring, 17 answers of 2 to 5 rows
  // to prompts of 8,192 and 4,096: 79 us against 83)
  x.splits = (int)std::max<int64_t>(1, kRowsSlots / (h->d.head_dim == 256 ? 2 : 1) / grid);
  x.splits1 = (int)std::max<int64_t>(1, kRowsSlots / 2 / grid);
  e = launch_attn_prefix(x, h->d.head_dim, h->d.dtype == QG_KV_BF16, (unsigned)grid, st);
  if (e != hipSuccess) return done(h, e, st);
  return attend(h, a, true, st);
}

}  // extern "C"
