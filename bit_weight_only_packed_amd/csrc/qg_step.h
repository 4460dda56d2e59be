// qg_step.h -- what the host and the kernels of qgstep.h share: arguments and launchers.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qgstep.h"

namespace qg {

struct NormArgs {
  const uint16_t* x;
  uint16_t* residual;
  const uint16_t* weight;
  void* out;
  float* scales;
  int64_t x_stride, residual_stride, out_stride;
  int rows, n, group;
  int first;  // the launch's first row
  int team;   // lanes of a row, a power of two, where a wave has several
  float eps;
};
hipError_t launch_rms_norm(const NormArgs& a, bool bf16, int codes, hipStream_t st);

struct RotDev {
  const uint64_t* turns;
  int dim, pairs;  // pairs: 2 j and 2 j + 1, else j and j + dim / 2
  float size;
};
struct RotArgs {
  RotDev r;
  const uint16_t* x;
  uint16_t* out;
  const int32_t* positions;
  int64_t x_row, x_head, out_row, out_head;
  int rows, heads, head_dim;
  int slots;  // threads that share a row's heads
};
hipError_t launch_rotate(const RotArgs& a, bool bf16, int cus, hipStream_t st);

// What the buckets of a row's logits have said (qg_sample.h).
struct SmPlan {
  int mode;
  int lo, hi;                 // buckets to list, and
  int k_bucket;               // the one that holds the k-th token (SAMPLE_BUCKETS: no such)
  int k_count;                // tokens in the buckets before that
  unsigned long long k_mass;  // their mass,
  unsigned long long lo_mass; // the mass of the buckets before lo,
  unsigned long long total;   // and of all (0 where it is not known)
};
struct SampleArgs {
  const void* logits;
  int64_t stride;
  int rows, vocab;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  float temperature1, top_p1, min_p1;
  int top_k1;
  int32_t* tokens;
  float* probs;
  int parts, part_len;  // of a row
  bool cuts;            // some row may have top-k or top-p
  bool whole;           // a workgroup takes a whole row
  // workspace, of SAMPLE_ROWS rows at most
  float* part_max;      // [row][part]
  int* part_arg;        // [row][part]
  unsigned long long *part_sum, *masses, *last, *list;  // [row][part], [row][bucket], [row], [row][SAMPLE_LIST]
  uint32_t* counts;     // [row][bucket]
  int* arrived;         // [row][4]: of the parts in three kernels, and the list's length
  SmPlan* plan;         // [row]
};
constexpr int SAMPLE_BUCKETS = 1024;
constexpr int SAMPLE_LIST = 2048;
constexpr int SAMPLE_ROWS = 4096;  // rows of a launch: what the workspace holds
void sample_parts(int rows, int vocab, int* parts, int* len);
bool sample_whole(int rows, int vocab);
hipError_t launch_sample(const SampleArgs& a, int type, hipStream_t st);

// what qgs_rotate and qgkv_append_rotary check of a qgs_rotary
qg_status rotary_of(const qgs_rotary* r, int head_dim, RotDev* out);

}  // namespace qg
