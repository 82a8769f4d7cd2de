// Host half of the operators on microscaled 4-bit numbers (include/kda_mx4.h)
// under AddressSanitizer and UndefinedBehaviorSanitizer: the argument checks and
// the workspace query, called with every kind of bad argument and with the
// extremes of each integer.  Every call here is rejected (or has nothing to do)
// before any HIP call, so the fake device pointers are never dereferenced and no
// GPU is needed.  Exits 0 when every status is the documented one.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kda_mx4.h"

static int failures = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    fprintf(stderr, "%s: status %d, expected %d\n", what, got, want);
    ++failures;
  }
}
#define FAKE ((void*)(uintptr_t)0x1000)

static kda_route_t route(int v) {
  kda_route_t e;
  memcpy(&e, &v, sizeof e);
  return e;
}
static int quant(int64_t rows, int32_t k, int64_t row) { return kda_mx4_quant(FAKE, FAKE, FAKE, NULL, rows, k, row); }
static int dequant(int64_t rows, int32_t k, int64_t row) {
  return kda_mx4_dequant(FAKE, FAKE, FAKE, NULL, rows, k, row);
}
static int proj(void* xs, int64_t m, int32_t k, int32_t n, int64_t xr, int64_t yr) {
  return kda_mx4_proj(FAKE, xs, FAKE, FAKE, FAKE, NULL, m, k, n, xr, yr);
}
static int moe(int32_t m, int32_t k, int32_t inter, int32_t e, int32_t s, int32_t top, int64_t xr, int64_t yr,
               int scoring, float scale, size_t bytes) {
  return kda_mx4_moe(FAKE, FAKE, NULL, FAKE, FAKE, FAKE, FAKE, NULL, FAKE, (int32_t*)FAKE, (float*)FAKE, FAKE, NULL,
                     m, k, inter, e, s, top, xr, yr, route(scoring), 1, scale, bytes);
}

int main(void) {
  const int32_t ints[] = {INT32_MIN, -1, 0, 7, 65567, INT32_MAX};
  const int64_t longs[] = {INT64_MIN, -1, (int64_t)1 << 31, (int64_t)1 << 62, INT64_MAX};
  const size_t all = SIZE_MAX;
  for (int i = 0; i < 6; ++i) {
    expect(quant(4, ints[i], INT32_MAX), KDA_ERR_INVALID_ARG, "quant k");
    expect(dequant(4, ints[i], INT32_MAX), KDA_ERR_INVALID_ARG, "dequant k");
    expect(proj(NULL, 3, ints[i], 40, 1 << 24, 40), KDA_ERR_INVALID_ARG, "proj k");
    expect(proj(FAKE, 3, ints[i], 40, 0, 40), KDA_ERR_INVALID_ARG, "proj k of codes");
    if (ints[i] <= 0 || ints[i] == INT32_MAX)
      expect(proj(NULL, 3, 64, ints[i], 64, INT32_MAX), KDA_ERR_INVALID_ARG, "proj n");
    if (ints[i] != 7 && ints[i] != 0) expect(moe(ints[i], 64, 64, 8, 1, 2, 64, 64, 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe tokens");
    expect(moe(3, ints[i], 64, 8, 1, 2, 1 << 24, 1 << 24, 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe k");
    expect(moe(3, 64, ints[i], 8, 1, 2, 64, 64, 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe inter");
    if (ints[i] != 7) expect(moe(3, 64, 64, ints[i], 1, 2, 64, 64, 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe experts");
    if (ints[i] != 7 && ints[i] != 0)
      expect(moe(3, 64, 64, 8, ints[i], 2, 64, 64, 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe shared");
    if (ints[i] != 7) expect(moe(3, 64, 64, 8, 1, ints[i], 64, 64, 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe top");
    for (int j = 0; j < 6; ++j)
      for (int l = 0; l < 6; ++l) {
        expect(kda_mx4_moe_workspace_size(3, ints[i], ints[j], 8, 1, ints[l]) == 0, 1, "workspace size");
        if (ints[i] != 7 && ints[i] != 0)
          expect(kda_mx4_moe_workspace_size(ints[i], 64, 64, ints[j], ints[l], 2) == 0, 1, "workspace size");
      }
  }
  for (int l = 0; l < 5; ++l) {
    expect(quant(longs[l], 64, 64), KDA_ERR_INVALID_ARG, "quant rows");
    expect(quant(4, 64, longs[l]), KDA_ERR_INVALID_ARG, "quant stride");
    expect(dequant(longs[l], 64, 64), KDA_ERR_INVALID_ARG, "dequant rows");
    expect(dequant(4, 64, longs[l]), KDA_ERR_INVALID_ARG, "dequant stride");
    expect(proj(NULL, longs[l], 64, 40, 64, 40), KDA_ERR_INVALID_ARG, "proj tokens");
    expect(proj(FAKE, longs[l], 64, 40, 64, 40), KDA_ERR_INVALID_ARG, "proj tokens of codes");
    expect(proj(NULL, 3, 64, 40, longs[l], 40), KDA_ERR_INVALID_ARG, "proj x stride");
    expect(proj(NULL, 3, 64, 40, 64, longs[l]), KDA_ERR_INVALID_ARG, "proj y stride");
    expect(proj(FAKE, 3, 64, 40, longs[l], longs[l]), KDA_ERR_INVALID_ARG, "proj y stride of codes");
    expect(moe(3, 64, 64, 8, 1, 2, longs[l], 64, 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe x stride");
    expect(moe(3, 64, 64, 8, 1, 2, 64, longs[l], 0, 1.f, all), KDA_ERR_INVALID_ARG, "moe out stride");
  }
  expect(quant((int64_t)INT32_MAX, 1 << 20, 1 << 20), KDA_ERR_INVALID_ARG, "quant of more than a grid");
  /* the largest of everything, and the workspace's size for it */
  const size_t most = kda_mx4_moe_workspace_size(64, 1 << 16, 1 << 16, 1024, 16, 32);
  expect(most > 0, 1, "largest workspace");
  expect(moe(64, 1 << 16, 1 << 16, 1024, 16, 32, 1 << 16, 1 << 16, 0, 1.f, most - 1), KDA_ERR_WORKSPACE_TOO_SMALL,
         "short workspace");
  size_t prev = 0;
  for (int m = 0; m <= 64; ++m) {
    const size_t w = kda_mx4_moe_workspace_size(m, 7168, 512, 256, 1, 8);
    expect(w >= prev && w > 0, 1, "workspace size monotone");
    if (m) expect(moe(m, 7168, 512, 256, 1, 8, 7168, 7168, 0, 1.f, w - 1), KDA_ERR_WORKSPACE_TOO_SMALL, "short workspace");
    prev = w;
  }
  const int enums[] = {INT32_MIN, -1, 2, 77, INT32_MAX};
  for (int i = 0; i < 5; ++i)
    expect(moe(3, 64, 64, 8, 1, 2, 64, 64, enums[i], 1.f, all), KDA_ERR_INVALID_ARG, "moe scoring");
  const float floats[] = {NAN, INFINITY, -INFINITY};
  for (int i = 0; i < 3; ++i)
    expect(moe(3, 64, 64, 8, 1, 2, 64, 64, 0, floats[i], all), KDA_ERR_INVALID_ARG, "moe scale");
  expect(quant(0, 64, 0), KDA_OK, "quant of nothing");
  expect(dequant(0, 64, 0), KDA_OK, "dequant of nothing");
  expect(proj(NULL, 0, 64, 40, 0, 0), KDA_OK, "proj of nothing");
  expect(proj(FAKE, 0, 64, 40, 0, 0), KDA_OK, "proj of nothing");
  expect(moe(0, 64, 64, 8, 1, 2, 0, 0, 0, 1.f, all), KDA_OK, "moe of nothing");
  printf("%d failures\n", failures);
  return failures != 0;
}
