// Host half of the layer operators (include/kda_layer.h) under AddressSanitizer
// and UndefinedBehaviorSanitizer: the argument checks and the workspace query,
// called with every kind of bad argument and with the extremes of each integer.
// Every call here is rejected (or has nothing to do) before any HIP call, so the
// fake device pointers are never dereferenced and no GPU is needed.  Exits 0
// when every status is the documented one.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kda_layer.h"

static int failures = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    fprintf(stderr, "%s: status %d, expected %d\n", what, got, want);
    ++failures;
  }
}
#define FAKE ((void*)(uintptr_t)0x1000)
#define FAKEF ((const float*)(uintptr_t)0x1000)
#define FAKEI ((const int32_t*)(uintptr_t)0x1000)

static kda_state_dtype_t state_dtype(int v) {
  kda_state_dtype_t e;
  memcpy(&e, &v, sizeof e);
  return e;
}
static kda_out_dtype_t out_dtype(int v) {
  kda_out_dtype_t e;
  memcpy(&e, &v, sizeof e);
  return e;
}

static int prefill(int64_t T, int32_t hk, int32_t hv, int32_t n, int sdt, size_t ws, float scale,
                   const kda_gdr_strides_t* s) {
  return kda_gdr_prefill_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKEF, FAKEF, scale, NULL, FAKEI, FAKE, FAKE,
                             FAKE, NULL, T, hk, hv, n, state_dtype(sdt), ws, s);
}
static int decode(int64_t slots, int32_t n, int32_t hk, int32_t hv, int sdt, const kda_gdr_strides_t* s) {
  return kda_gdr_decode_step(FAKE, FAKE, FAKE, FAKE, FAKE, FAKEF, FAKEF, 0.1f, FAKE, slots, FAKEI, FAKE,
                             NULL, n, hk, hv, state_dtype(sdt), s);
}
static int norm(int64_t rows, int32_t dim, int64_t xr, int64_t rr, int64_t orow, int odt, int32_t group,
                float eps, float* scale) {
  return kda_add_rms_norm(FAKE, FAKE, FAKE, eps, FAKE, scale, NULL, rows, dim, xr, rr, orow, out_dtype(odt),
                          group);
}
static int w4(int32_t m, int32_t k, int32_t n, int32_t g, int64_t xr, int64_t yr) {
  return kda_w4_proj(FAKE, FAKE, FAKE, NULL, FAKE, NULL, m, k, n, g, xr, yr);
}

int main(void) {
  const int32_t ints[] = {INT32_MIN, -1, 0, 3, 65537, INT32_MAX};
  const int64_t longs[] = {INT64_MIN, -1, (int64_t)1 << 31, (int64_t)1 << 62, INT64_MAX};
  const size_t all = SIZE_MAX;

  // the workspace query: 0 for what the call refuses, monotone otherwise
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < 6; ++j)
      for (int k = 0; k < 6; ++k) {
        if (ints[i] == 3 && ints[j] == 3 && ints[k] == 3) continue;
        for (int l = 0; l < 5; ++l)
          expect(kda_gdr_get_workspace_size(longs[l], ints[i], ints[j], ints[k]) == 0, 1, "workspace size");
        if (ints[i] == 3 && ints[j] == 3) continue;
        expect(prefill(100, ints[i], ints[j], ints[k], 0, all, 0.1f, NULL), KDA_ERR_INVALID_ARG, "prefill heads");
        if (ints[k] != 0)
          expect(decode(9, ints[k], ints[i], ints[j], 0, NULL), KDA_ERR_INVALID_ARG, "decode heads");
      }
  size_t prev = 0;
  for (int64_t t = 0; t < 1 << 20; t = 2 * t + 1) {
    const size_t w = kda_gdr_get_workspace_size(t, 2, 4, 3);
    expect(w >= prev && w > 0, 1, "workspace size monotone");
    expect(prefill(t, 2, 4, 3, 0, w - 1, 0.1f, NULL), KDA_ERR_WORKSPACE_TOO_SMALL, "short workspace");
    prev = w;
  }
  for (int l = 0; l < 5; ++l) {
    expect(prefill(longs[l], 2, 4, 2, 0, all, 0.1f, NULL), KDA_ERR_INVALID_ARG, "prefill tokens");
    expect(norm(longs[l], 64, 64, 64, 64, 0, 0, 1e-6f, NULL), KDA_ERR_INVALID_ARG, "norm rows");
    expect(norm(4, 64, longs[l], 64, 64, 0, 0, 1e-6f, NULL), KDA_ERR_INVALID_ARG, "norm x stride");
    expect(norm(4, 64, 64, longs[l], 64, 0, 0, 1e-6f, NULL), KDA_ERR_INVALID_ARG, "norm residual stride");
    expect(norm(4, 64, 64, 64, longs[l], 0, 0, 1e-6f, NULL), KDA_ERR_INVALID_ARG, "norm out stride");
    expect(w4(3, 256, 40, 64, longs[l], 40), KDA_ERR_INVALID_ARG, "w4 x stride");
    expect(w4(3, 256, 40, 64, 256, longs[l]), KDA_ERR_INVALID_ARG, "w4 y stride");
    for (int f = 0; f < 12; ++f) {
      kda_gdr_strides_t s = {256, 128, 256, 128, 512, 128, 4, 1, 4, 1, 512, 128};
      memcpy((char*)&s + 8 * f, &longs[l], 8);
      expect(prefill(100, 2, 4, 2, 0, all, 0.1f, &s), KDA_ERR_INVALID_ARG, "prefill strides");
      expect(decode(9, 3, 2, 4, 0, &s), KDA_ERR_INVALID_ARG, "decode strides");
    }
  }
  expect(decode(INT64_MIN, 3, 2, 4, 0, NULL), KDA_ERR_INVALID_ARG, "decode slots");
  expect(decode(0, 3, 2, 4, 0, NULL), KDA_ERR_INVALID_ARG, "decode of no slots");
  expect(decode(9, 0, 2, 4, 0, NULL), KDA_OK, "decode of nothing");

  /* an int outside the enumerators, as a C caller may pass it */
  const int enums[] = {INT32_MIN, -1, 2, 77, INT32_MAX};
  for (int i = 0; i < 5; ++i) {
    expect(prefill(100, 2, 4, 2, enums[i], all, 0.1f, NULL), KDA_ERR_INVALID_ARG, "prefill state dtype");
    expect(decode(9, 3, 2, 4, enums[i], NULL), KDA_ERR_INVALID_ARG, "decode state dtype");
    expect(norm(4, 64, 64, 64, 64, enums[i], 0, 1e-6f, NULL), KDA_ERR_INVALID_ARG, "norm out dtype");
  }
  const float floats[] = {NAN, INFINITY, -INFINITY};
  for (int i = 0; i < 3; ++i) {
    expect(prefill(100, 2, 4, 2, 0, all, floats[i], NULL), KDA_ERR_INVALID_ARG, "prefill scale");
    expect(norm(4, 64, 64, 64, 64, 0, 0, floats[i], NULL), KDA_ERR_INVALID_ARG, "norm eps");
  }
  for (int i = 0; i < 6; ++i) {
    if (ints[i] != 3) {
      expect(norm(4, ints[i], INT32_MAX, INT32_MAX, INT32_MAX, 0, 0, 1e-6f, NULL), KDA_ERR_INVALID_ARG, "norm dim");
      if (ints[i] != 0) {
        expect(norm(4, 64, 64, 64, 64, 1, ints[i], 1e-6f, (float*)FAKE), KDA_ERR_INVALID_ARG, "norm group");
        expect(w4(ints[i], 256, 40, 64, 256, 40), KDA_ERR_INVALID_ARG, "w4 tokens");
      }
    }
    expect(w4(3, ints[i], 40, 64, 1 << 24, 40), KDA_ERR_INVALID_ARG, "w4 k");
    expect(w4(3, 256, 40, ints[i], 256, 40), KDA_ERR_INVALID_ARG, "w4 group");
    if (ints[i] <= 0 || ints[i] == INT32_MAX)
      expect(w4(3, 256, ints[i], 64, 256, INT32_MAX), KDA_ERR_INVALID_ARG, "w4 n");
  }
  expect(norm(0, 64, 0, 0, 0, 0, 0, 1e-6f, NULL), KDA_OK, "norm of nothing");
  expect(w4(0, 256, 40, 64, 0, 0), KDA_OK, "w4 of nothing");
  printf("%d failures\n", failures);
  return failures != 0;
}
