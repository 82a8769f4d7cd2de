// kda_gdr.h -- device helpers of the delta rule with one decay per head,
// shared by its chunked and its serial kernels.
#pragma once

#include "kda_layer_internal.h"
#include "kda_mfma.h"

namespace kda {

// log a = -exp(A_log) softplus(x), x = a + dt_bias, not below -120: e^-120 is 0
// in fp32, and a sum of 64 stays finite.  Above A_log = 88, where its exponential
// passes fp32, the excess c goes to x: exp(A_log) e^x = e^88 e^(x + c), softplus
// is e^x below -20, and from there on the product is beyond 120 either way.  A
// NaN stays one.
static __device__ __forceinline__ float gdr_log_decay(float a, float A_log, float dt_bias) {
  const float c = fmaxf(A_log - 88.f, 0.f), x = a + dt_bias + c;
  const float l = -expf(A_log - c) * (fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))));
  return l < -120.f ? -120.f : l;
}

static __device__ __forceinline__ float gdr_sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// Token range of sequence n, clamped to the batch (cu is read on the device
// only and is not to be trusted).
static __device__ __forceinline__ void gdr_range(const GdrParams& p, int n, int& t0, int& t1) {
  t0 = min(max(p.cu[n], 0), p.T);
  t1 = min(max(p.cu[n + 1], t0), p.T);
}

}  // namespace kda
