// k_sample.hip -- launchers of the sampling kernels (qg_sample.h).
#include <algorithm>

#include "qg_sample.h"

namespace qg {

namespace {

template <int TY> hipError_t go(const SampleArgs& a, hipStream_t st) {
  for (int64_t at = 0; at < a.rows; at += SAMPLE_ROWS) {  // (at may pass 2^31 at the end)
    const unsigned rows = (unsigned)std::min<int64_t>(a.rows - at, SAMPLE_ROWS);
    SampleArgs b = a;
    b.logits = reinterpret_cast<const char*>(a.logits) + at * a.stride * (TY == QGS_F32 ? 4 : 2);
    b.u += at, b.tokens += at;
    if (b.probs) b.probs += at;
    if (b.temperature) b.temperature += at;
    if (b.top_k) b.top_k += at;
    if (b.top_p) b.top_p += at;
    if (b.min_p) b.min_p += at;
    if (a.whole) {
      k_sample_row<TY><<<rows, SM_ROW_T, 0, st>>>(b);
      continue;
    }
    const dim3 grid((unsigned)a.parts, rows);
    k_sample_max<TY><<<grid, SM_T, 0, st>>>(b);
    if (a.cuts) {
      k_sample_hist<TY><<<grid, SM_T, 0, st>>>(b);
      k_sample_list<TY><<<grid, SM_T, 0, st>>>(b);
    }
    k_sample_pick<TY><<<grid, SM_T, 0, st>>>(b);
  }
  return hipGetLastError();
}

}  // namespace

// Parts of some 2,048 tokens, one load of a thread (33 parts of 2,000 or fewer for a row of 66,000), or more where there
// would be more than 64 of a row or some 4,096 in all.
// us with 1,024 / 2,048 / 4,096 / 8,192 parts: 128 rows of 100,003 98 / 91 / 86 / 90, of 131,071 without limits
// 69 / 61 / 59 / 67, 250 rows of 131,000 with top-k and top-p 147 / 138 / 149 / 177.
void sample_parts(int rows, int vocab, int* parts, int* len) {
  int p = (vocab + 2047) / 2048;
  const int most = rows >= 4096 ? 1 : 4096 / rows;
  p = p < most ? p : most;
  p = p < 64 ? p : 64;
  *len = ((vocab + p - 1) / p + 7) / 8 * 8;
  *parts = (vocab + *len - 1) / *len;
}

// Whether a workgroup takes a whole row.  us by parts / by rows, top-k 200 and top-p of all rows in bf16,
// no limits in fp32, and settings of every kind in fp16:
//   1 row     1,000    29 / 18, 21 / 13, 27 / 16     16,001  30 / 24, 20 / 18, 29 / 23     32,003  30 / 33, 20 / 28, 29 / 31
//   32 rows   16,001   49 / 39, 20 / 18, 59 / 41     32,003  51 / 58, 20 / 29, 56 / 55
//   128 rows  32,003   68 / 57, 28 / 29, 67 / 57     65,537  104 / 90, 48 / 53, 90 / 100
//   256 rows  65,537   132 / 92, 68 / 57, 106 / 103  131,071 156 / 167, 107 / 106, 138 / 199
bool sample_whole(int rows, int vocab) { return vocab <= 16384 || (vocab <= 65536 && vocab <= 256 * (int64_t)rows); }

hipError_t launch_sample(const SampleArgs& a, int type, hipStream_t st) {
  if (type == QGS_F16) return go<QGS_F16>(a, st);
  if (type == QGS_BF16) return go<QGS_BF16>(a, st);
  return go<QGS_F32>(a, st);
}

}  // namespace qg
