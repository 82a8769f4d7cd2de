// kda_layer_internal.h -- what the kernels of the layer operators (the public
// include/kda_layer.h) and the host code that launches them share.
#pragma once

#include "kda_internal.h"

namespace kda {

// Records a failed HIP call for kda_last_hip_error() and returns KDA_ERR_HIP
// (defined with the thread's error text in kda_api.hip).
int record_hip_failure(hipError_t e, const char* step);
// Compute units of the current device (cached; no synchronisation).
hipError_t device_cus(int* cus);

constexpr int kGdrChunk = 64;  // tokens per chunk of the chunked form

// One call of the delta rule with one decay per head.  Strides in elements.
struct GdrParams {
  const uint16_t *q, *k, *v, *a, *beta;
  const float *A_log, *dt_bias;
  const void* s0;  // null: zeros
  void* sT;
  uint16_t* out;
  const int32_t* cu;   // prefill: [N + 1]
  const int32_t* idx;  // step: [N] slots of s0 == sT, null in the prefill
  int64_t slots;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, a_t, a_h, b_t, b_h, o_t, o_h;
  float scale;
  int T, Hk, Hv, N;
  int state_bf16;
  char* ws;  // prefill: see gdr_layout
  // segment-parallel schedule: its table (see SegParams), the summaries it
  // writes, the states it starts from
  const int32_t* seg;
  float* summ;
  const float* starts;
};

// Chunk slots: sequence n's j-th chunk has slot cu[n] / 64 + n + j.  The next
// sequence's first slot is never below this one's last plus one, since
// floor((c + l) / 64) + 1 >= floor(c / 64) + ceil(l / 64); T / 64 + N slots
// cover every batch of N sequences and T tokens.
struct GdrLayout {
  int64_t slots;
  size_t head, tri, coef;             // byte offsets of the parts
  size_t table, first, count, summ, starts, total;
};
GdrLayout gdr_layout(int64_t T, int Hk, int Hv, int64_t N);

// Chunked prefill: two launches, five where sequences are cut into segments.
hipError_t launch_gdr_chunked(const GdrParams& p, int cus, hipStream_t stream);
// Token after token, for the single-token step and sequences of few tokens.
hipError_t launch_gdr_serial(const GdrParams& p, hipStream_t stream);

struct NormParams {
  const uint16_t* x;
  uint16_t* res;  // null: no residual
  const uint16_t* w;
  void* out;
  float* scale;
  int64_t x_row, r_row, o_row;
  int64_t rows;
  float eps;
  int dim, fp8, group;
};
hipError_t launch_norm(const NormParams& p, hipStream_t stream);

struct W4Params {
  const uint16_t* x;
  const uint8_t* w;
  const uint16_t *scales, *zeros;
  uint16_t* y;
  int64_t x_row, y_row;
  int M, K, N, group;
};
hipError_t launch_w4(const W4Params& p, int cus, hipStream_t stream);

}  // namespace kda
