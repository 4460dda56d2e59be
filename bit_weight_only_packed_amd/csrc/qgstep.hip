// qgstep.hip -- host side of the C ABI declared in include/qgstep.h: argument checks and
// the layout of the sampling workspace.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>

#include "qg_check.h"
#include "qg_error.h"
#include "qg_kv.h"
#include "qg_step.h"

using namespace qg;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

qg_status launched(hipError_t e, hipStream_t st) {
  if (e != hipSuccess) return fail(QG_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
  static const bool sync = getenv("QG_DEBUG_SYNC") != nullptr;
  if (sync && (e = hipStreamSynchronize(st)) != hipSuccess) return fail(QG_ERR_DEVICE, "kernel failed: %s", hipGetErrorString(e));
  return QG_OK;
}

// rows of `width` bytes at every `stride` bytes
struct Span {
  const void* p;
  int64_t stride, width, rows;
  int64_t extent() const { return (rows - 1) * (rows > 1 ? stride : 0) + width; }
};
// whether they are plainly apart: in different memory, or in other columns of the same rows
bool apart(const Span& a, const Span& b) {
  const int64_t ofs = (int64_t)((intptr_t)b.p - (intptr_t)a.p);
  if (ofs >= a.extent() || -ofs >= b.extent()) return true;
  if (a.rows == 1 || b.rows == 1 || a.stride != b.stride || a.stride <= 0) return false;
  const int64_t at = (ofs % a.stride + a.stride) % a.stride;
  return at >= a.width && at + b.width <= a.stride;
}

}  // namespace

namespace qg {

qg_status rotary_of(const qgs_rotary* r, int head_dim, RotDev* out) {
  if (!r) return fail(QG_ERR_INVALID_ARG, "rotary is NULL");
  if (!r->turns || !aligned(r->turns, 16)) return fail(QG_ERR_INVALID_ARG, "turns must be a 16-byte aligned device pointer");
  if (r->dim < 16 || r->dim % 16 || r->dim > head_dim)
    return fail(QG_ERR_INVALID_ARG, "rotary dim = %d is not a multiple of 16 up to head_dim = %d", r->dim, head_dim);
  if (r->layout != QGS_HALVES && r->layout != QGS_PAIRS) return fail(QG_ERR_INVALID_ARG, "unknown layout %d", r->layout);
  if (!std::isfinite(r->size)) return fail(QG_ERR_INVALID_ARG, "size = %g is not finite", r->size);
  *out = RotDev{r->turns, r->dim, r->layout == QGS_PAIRS, r->size};
  return QG_OK;
}

qg_status known_device(int* dev, int* cus) {
  static std::atomic<int> known[64];  // compute units of a gfx950
  int d = -1;
  if (hipGetDevice(&d) != hipSuccess) return fail(QG_ERR_UNSUPPORTED, "no HIP device available");
  int n = d < 64 ? known[d].load(std::memory_order_relaxed) : 0;
  if (!n) {
    const qg_status s = check_device(&d);
    if (s != QG_OK) return s;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, d) != hipSuccess || n < 1)
      return fail(QG_ERR_DEVICE, "cannot query the compute-unit count");
    if (d < 64) known[d].store(n, std::memory_order_relaxed);
  }
  *dev = d;
  *cus = n;
  return QG_OK;
}

}  // namespace qg

extern "C" {

qg_status qgs_rms_norm(const qgs_norm* d, void* stream) {
  clear_error();
  if (!d) return fail(QG_ERR_INVALID_ARG, "desc is NULL");
  if (d->rows < 0) return fail(QG_ERR_INVALID_ARG, "rows = %d is negative", d->rows);
  if (d->n < 1 || d->n > QGS_MAX_NORM) return fail(QG_ERR_INVALID_ARG, "n = %d is not in [1, %d]", d->n, QGS_MAX_NORM);
  if (d->dtype != QGS_F16 && d->dtype != QGS_BF16) return fail(QG_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
  if (d->codes < QGS_SAME || d->codes > QGS_E4M3) return fail(QG_ERR_INVALID_ARG, "unknown codes %d", d->codes);
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return fail(QG_ERR_INVALID_ARG, "eps = %g is not positive and finite", d->eps);
  if (d->codes == QGS_SAME ? d->group != 0 : d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128)
    return fail(QG_ERR_INVALID_ARG, "group = %d is not 0%s", d->group, d->codes == QGS_SAME ? "" : ", 32, 64 or 128");
  if (d->rows == 0) return QG_OK;
  if (!d->x || !d->out) return fail(QG_ERR_INVALID_ARG, "x and out must be device pointers");
  if (!aligned(d->x, 2) || !aligned(d->residual, 2) || !aligned(d->weight, 2) || (d->codes == QGS_SAME && !aligned(d->out, 2)))
    return fail(QG_ERR_INVALID_ARG, "x, residual, weight and out must be aligned to their types");
  if (d->codes != QGS_SAME && (!d->scales || !aligned(d->scales, 4)))
    return fail(QG_ERR_INVALID_ARG, "scales must be a 4-byte aligned device pointer");
  if (d->rows > 1) {
    if (d->x_stride < 0) return fail(QG_ERR_INVALID_ARG, "x_stride = %lld is negative", (long long)d->x_stride);
    if (d->out_stride < d->n) return fail(QG_ERR_INVALID_ARG, "out_stride = %lld: rows of %d overlap", (long long)d->out_stride, d->n);
    if (d->residual && d->residual_stride < d->n)
      return fail(QG_ERR_INVALID_ARG, "residual_stride = %lld: rows of %d overlap", (long long)d->residual_stride, d->n);
  }
  const int64_t el = d->codes == QGS_SAME ? 2 : 1, w = 2 * (int64_t)d->n;
  const Span x{d->x, 2 * d->x_stride, w, d->rows}, out{d->out, el * d->out_stride, el * d->n, d->rows};
  const Span res{d->residual, 2 * d->residual_stride, w, d->rows}, wt{d->weight, 0, w, 1};
  const int per = d->group ? (d->n + d->group - 1) / d->group : 1;
  const Span sc{d->scales, 4 * (int64_t)per, 4 * (int64_t)per, d->rows};
  const bool in_place = d->codes == QGS_SAME && d->out == d->x && (d->rows == 1 || d->out_stride == d->x_stride);
  if (!in_place && !apart(x, out)) return fail(QG_ERR_INVALID_ARG, "out overlaps x");
  if (d->residual && (!apart(x, res) || !apart(res, out))) return fail(QG_ERR_INVALID_ARG, "residual overlaps x or out");
  if (d->weight && (!apart(wt, out) || (d->residual && !apart(wt, res)))) return fail(QG_ERR_INVALID_ARG, "weight overlaps out or residual");
  if (d->codes != QGS_SAME && (!apart(sc, x) || !apart(sc, out) || (d->residual && !apart(sc, res)) || (d->weight && !apart(sc, wt))))
    return fail(QG_ERR_INVALID_ARG, "scales overlap another operand");
  int dev = 0, cus = 0;
  qg_status s = known_device(&dev, &cus);
  if (s != QG_OK) return s;
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(d->x);
  a.residual = static_cast<uint16_t*>(d->residual);
  a.weight = static_cast<const uint16_t*>(d->weight);
  a.out = d->out;
  a.scales = d->scales;
  a.x_stride = d->x_stride, a.residual_stride = d->residual_stride, a.out_stride = d->out_stride;
  a.rows = d->rows, a.n = d->n, a.group = d->group;
  a.eps = d->eps;
  hipStream_t st = (hipStream_t)stream;
  return launched(launch_rms_norm(a, d->dtype == QGS_BF16, d->codes, st), st);
}

qg_status qgs_rotate(const qgs_rows* d, const qgs_rotary* rotary, void* stream) {
  clear_error();
  if (!d) return fail(QG_ERR_INVALID_ARG, "desc is NULL");
  if (d->rows < 0) return fail(QG_ERR_INVALID_ARG, "rows = %d is negative", d->rows);
  if (d->heads < 1) return fail(QG_ERR_INVALID_ARG, "heads = %d is not positive", d->heads);
  if (d->head_dim < 16 || d->head_dim > 1024 || d->head_dim % 16)
    return fail(QG_ERR_INVALID_ARG, "head_dim = %d is not a multiple of 16 up to 1024", d->head_dim);
  if (d->dtype != QGS_F16 && d->dtype != QGS_BF16) return fail(QG_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
  RotArgs a{};
  qg_status s = rotary_of(rotary, d->head_dim, &a.r);
  if (s != QG_OK || d->rows == 0) return s;
  if (!d->x || !d->out || !aligned(d->x, 16) || !aligned(d->out, 16))
    return fail(QG_ERR_INVALID_ARG, "x and out must be 16-byte aligned device pointers");
  if (!d->positions || !aligned(d->positions, 4)) return fail(QG_ERR_INVALID_ARG, "positions must be a 4-byte aligned device pointer");
  a.x = static_cast<const uint16_t*>(d->x);
  a.out = static_cast<uint16_t*>(d->out);
  a.positions = d->positions;
  a.rows = d->rows, a.heads = d->heads, a.head_dim = d->head_dim;
  a.x_row = d->rows > 1 ? d->x_row : 0, a.out_row = d->rows > 1 ? d->out_row : 0;
  a.x_head = d->heads > 1 ? d->x_head : 0, a.out_head = d->heads > 1 ? d->out_head : 0;
  s = check_strides("x", a.x_row, a.x_head);
  if (s == QG_OK) s = check_strides("out", a.out_row, a.out_head);
  if (s != QG_OK) return s;
  const KvRows x{a.x, a.x_row, a.x_head}, out{a.out, a.out_row, a.out_head};
  if (!(a.x == a.out && a.x_row == a.out_row && a.x_head == a.out_head)) {
    s = check_overlap(x, out, d->rows, d->heads, d->head_dim, "out overlaps x");
  } else {
    s = check_nested(out, d->rows, d->heads, d->head_dim);
  }
  if (s != QG_OK) return s;
  int dev = 0, cus = 0;
  s = known_device(&dev, &cus);
  if (s != QG_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  return launched(launch_rotate(a, d->dtype == QGS_BF16, cus, st), st);
}

}  // extern "C"

namespace {

// the workspace's arrays, one after another on 16-byte boundaries
size_t lay_out(SampleArgs* a, int rows, int vocab, char* at) {
  if (sample_whole(rows, vocab)) return 16;  // (none, but a pointer is asked for all the same)
  sample_parts(rows, vocab, &a->parts, &a->part_len);
  const size_t r = (size_t)std::min(rows, SAMPLE_ROWS);  // rows of a launch
  size_t used = 0;
  const auto take = [&](auto*& p, size_t n) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(at + used);
    used += (n * sizeof(*p) + 15) / 16 * 16;
  };
  take(a->masses, r * SAMPLE_BUCKETS);
  take(a->counts, r * SAMPLE_BUCKETS);
  take(a->part_sum, r * a->parts);
  take(a->part_max, r * a->parts);
  take(a->part_arg, r * a->parts);
  take(a->list, r * SAMPLE_LIST);
  take(a->plan, r);
  take(a->last, r);
  take(a->arrived, 4 * r);
  return used;
}

qg_status check_sample_size(int rows, int vocab) {
  if (rows < 0) return fail(QG_ERR_INVALID_ARG, "rows = %d is negative", rows);
  if (vocab < 1 || vocab > QGS_MAX_VOCAB) return fail(QG_ERR_INVALID_ARG, "vocab = %d is not in [1, %d]", vocab, QGS_MAX_VOCAB);
  return QG_OK;
}

}  // namespace

extern "C" {

qg_status qgs_sample_workspace(int32_t rows, int32_t vocab, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(QG_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  qg_status s = check_sample_size(rows, vocab);
  if (s != QG_OK) return s;
  SampleArgs a{};
  if (rows > 0) *bytes = lay_out(&a, rows, vocab, nullptr);
  return QG_OK;
}

qg_status qgs_sample(const qgs_sampling* d, void* workspace, size_t bytes, void* stream) {
  clear_error();
  if (!d) return fail(QG_ERR_INVALID_ARG, "desc is NULL");
  qg_status s = check_sample_size(d->rows, d->vocab);
  if (s != QG_OK) return s;
  if (d->dtype != QGS_F16 && d->dtype != QGS_BF16 && d->dtype != QGS_F32) return fail(QG_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
  if (d->rows == 0) return QG_OK;
  if (!d->logits || !d->u || !d->tokens) return fail(QG_ERR_INVALID_ARG, "logits, u and tokens must be device pointers");
  if (!aligned(d->logits, d->dtype == QGS_F32 ? 4 : 2)) return fail(QG_ERR_INVALID_ARG, "logits must be aligned to their type");
  if (d->rows > 1 && d->stride < 0) return fail(QG_ERR_INVALID_ARG, "stride = %lld is negative", (long long)d->stride);
  for (const void* p : {(const void*)d->u, (const void*)d->temperature, (const void*)d->top_k, (const void*)d->top_p,
                        (const void*)d->min_p, (const void*)d->tokens, (const void*)d->probs})
    if (!aligned(p, 4)) return fail(QG_ERR_INVALID_ARG, "u, temperature, top_k, top_p, min_p, tokens and probs must be 4-byte aligned");
  SampleArgs a{};
  const size_t need = lay_out(&a, d->rows, d->vocab, static_cast<char*>(workspace));
  if (!workspace || !aligned(workspace, 16)) return fail(QG_ERR_INVALID_ARG, "workspace must be a 16-byte aligned device pointer");
  if (bytes < need) return fail(QG_ERR_INVALID_ARG, "workspace of %zu bytes: %zu are needed", bytes, need);
  int dev = 0, cus = 0;
  s = known_device(&dev, &cus);
  if (s != QG_OK) return s;
  a.logits = d->logits;
  a.stride = d->rows > 1 ? d->stride : 0;
  a.rows = d->rows, a.vocab = d->vocab;
  a.u = d->u, a.temperature = d->temperature, a.top_k = d->top_k, a.top_p = d->top_p, a.min_p = d->min_p;
  a.temperature1 = d->temperature1, a.top_k1 = d->top_k1, a.top_p1 = d->top_p1, a.min_p1 = d->min_p1;
  a.tokens = d->tokens, a.probs = d->probs;
  const bool heat = d->temperature || d->temperature1 > 0.0f;
  a.cuts = heat && (d->top_k || d->top_p || (d->top_k1 > 0 && d->top_k1 < d->vocab) || d->top_p1 < 1.0f);
  a.whole = sample_whole(d->rows, d->vocab);
  hipStream_t st = (hipStream_t)stream;
  return launched(launch_sample(a, d->dtype, st), st);
}

}  // extern "C"
