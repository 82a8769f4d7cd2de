// kda_mx4_api.hip -- the C ABI of include/kda_mx4.h: argument checks, workspace
// sizing and the launches.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "kda_mx4.h"
#include "kda_mx4_internal.h"

namespace {

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// The integer a C caller passed for an enum parameter (any value may come).
template <typename E>
int enum_value(const E& e) {
  static_assert(sizeof(E) == sizeof(int), "enum parameters are int-sized");
  int v;
  std::memcpy(&v, &e, sizeof v);
  return v;
}

kda_status_t failed(hipError_t e, const char* step) {
  return static_cast<kda_status_t>(kda::record_hip_failure(e, step));
}

bool blocks_ok(int32_t k, int32_t most) { return k > 0 && k <= most && k % kda::kMxBlock == 0; }
// Rows of bf16 in 16-byte pieces.
bool rows_ok(int64_t rows, int64_t row, int32_t k, int64_t most) {
  return rows <= 1 || (row >= k && row <= most && row % 8 == 0);
}

kda_status_t rows_checks(const void* x, const void* codes, const void* scales, int64_t rows, int32_t k,
                         int64_t x_row) {
  if (rows < 0 || rows >= (int64_t(1) << 31) || !blocks_ok(k, 1 << 20)) return KDA_ERR_INVALID_ARG;
  if (!rows_ok(rows, x_row, k, int64_t(1) << 30)) return KDA_ERR_INVALID_ARG;
  // a grid holds fewer than 2^32 threads
  if (rows * (k / 8) >= (int64_t(1) << 33)) return KDA_ERR_INVALID_ARG;
  if (misaligned(x, 16) || misaligned(codes, 4)) return KDA_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !codes || !scales)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

bool moe_sizes_ok(int32_t m, int32_t k, int32_t inter, int32_t experts, int32_t shared, int32_t top) {
  return m >= 0 && m <= 64 && blocks_ok(k, 1 << 16) && blocks_ok(inter, 1 << 16) && experts >= 1 &&
         experts <= 1024 && shared >= 0 && shared <= 16 && top >= 1 && top <= 32 && top <= experts;
}

}  // namespace

extern "C" {

kda_status_t kda_mx4_quant(const void* x, void* codes, void* scales, void* stream, int64_t num_rows,
                           int32_t k, int64_t x_row) {
  if (kda_status_t rc = rows_checks(x, codes, scales, num_rows, k, x_row); rc != KDA_OK) return rc;
  if (num_rows == 0) return KDA_OK;
  const kda::Mx4Rows p{const_cast<uint16_t*>(static_cast<const uint16_t*>(x)), static_cast<uint8_t*>(codes),
                       static_cast<uint8_t*>(scales), num_rows, x_row, k};
  if (hipError_t e = kda::launch_mx4_quant(p, static_cast<hipStream_t>(stream)); e != hipSuccess)
    return failed(e, "4-bit quantisation launch");
  return KDA_OK;
}

kda_status_t kda_mx4_dequant(const void* codes, const void* scales, void* out, void* stream,
                             int64_t num_rows, int32_t k, int64_t out_row) {
  if (kda_status_t rc = rows_checks(out, codes, scales, num_rows, k, out_row); rc != KDA_OK) return rc;
  if (num_rows == 0) return KDA_OK;
  const kda::Mx4Rows p{static_cast<uint16_t*>(out), const_cast<uint8_t*>(static_cast<const uint8_t*>(codes)),
                       const_cast<uint8_t*>(static_cast<const uint8_t*>(scales)), num_rows, out_row, k};
  if (hipError_t e = kda::launch_mx4_dequant(p, static_cast<hipStream_t>(stream)); e != hipSuccess)
    return failed(e, "4-bit dequantisation launch");
  return KDA_OK;
}

kda_status_t kda_mx4_proj(const void* x, const void* x_scales, const void* w, const void* w_scales,
                          void* y, void* stream, int64_t num_tokens, int32_t k, int32_t n,
                          int64_t x_row, int64_t y_row) {
  if (num_tokens < 0 || num_tokens >= (int64_t(1) << 31)) return KDA_ERR_INVALID_ARG;
  if (!blocks_ok(k, 1 << 20) || n <= 0 || n > (1 << 24)) return KDA_ERR_INVALID_ARG;
  if (!w || !w_scales || misaligned(w, 16) || misaligned(x, 16) || misaligned(y, 2)) return KDA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!x || !y)) return KDA_ERR_INVALID_ARG;
  if (!x_scales && (num_tokens > 64 || !rows_ok(num_tokens, x_row, k, 1 << 24))) return KDA_ERR_INVALID_ARG;
  if (num_tokens > 1 && (y_row < n || y_row > (int64_t(1) << 30))) return KDA_ERR_INVALID_ARG;
  // a grid holds fewer than 2^32 threads: 512 for a tile
  if (((num_tokens + 255) / 256) * ((n + 255) / 256) >= (int64_t(1) << 23)) return KDA_ERR_INVALID_ARG;
  if (num_tokens == 0) return KDA_OK;
  kda::Mx4Params p{};
  p.x = x;
  p.xs = static_cast<const uint8_t*>(x_scales);
  p.w = static_cast<const uint8_t*>(w);
  p.ws = static_cast<const uint8_t*>(w_scales);
  p.y = static_cast<uint16_t*>(y);
  p.M = num_tokens;
  p.x_row = x_row;
  p.y_row = y_row;
  p.K = k;
  p.N = n;
  int cus = 0;
  if (hipError_t e = kda::device_cus(&cus); e != hipSuccess) return failed(e, "device query");
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool tile = p.xs && kda::mx4_in_tiles(p, cus);
  if (hipError_t e = tile ? kda::launch_mx4_tile(p, cus, st) : kda::launch_mx4_few(p, cus, st); e != hipSuccess)
    return failed(e, "4-bit product launch");
  return KDA_OK;
}

size_t kda_mx4_moe_workspace_size(int32_t max_tokens, int32_t k, int32_t inter, int32_t experts,
                                  int32_t shared, int32_t top_k) {
  if (!moe_sizes_ok(max_tokens, k, inter, experts, shared, top_k)) return 0;
  return kda::moe_layout(max_tokens, k, inter, experts, shared, top_k).total;
}

kda_status_t kda_mx4_moe(const void* x, const void* router, const float* router_bias,
                         const void* w_up, const void* w_up_scales, const void* w_down,
                         const void* w_down_scales, const int32_t* state_indices, void* out,
                         int32_t* expert_ids, float* expert_gates, void* workspace, void* stream,
                         int32_t num_tokens, int32_t k, int32_t inter, int32_t experts,
                         int32_t shared, int32_t top_k, int64_t x_row, int64_t out_row,
                         kda_route_t scoring, int32_t renormalise, float route_scale,
                         size_t workspace_bytes) {
  const int route = enum_value(scoring);
  if (!moe_sizes_ok(num_tokens, k, inter, experts, shared, top_k)) return KDA_ERR_INVALID_ARG;
  if (route != KDA_ROUTE_SIGMOID && route != KDA_ROUTE_SOFTMAX) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(route_scale)) return KDA_ERR_INVALID_ARG;
  if (!router || !w_up || !w_up_scales || !w_down || !w_down_scales) return KDA_ERR_INVALID_ARG;
  for (const void* q : {x, router, w_up, w_down, static_cast<const void*>(out)})
    if (misaligned(q, 16)) return KDA_ERR_INVALID_ARG;
  if (misaligned(router_bias, 4) || misaligned(state_indices, 4) || misaligned(expert_ids, 4) ||
      misaligned(expert_gates, 4))
    return KDA_ERR_INVALID_ARG;
  if (!rows_ok(num_tokens, x_row, k, 1 << 24) || !rows_ok(num_tokens, out_row, k, 1 << 24))
    return KDA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!x || !out || !expert_ids || !expert_gates)) return KDA_ERR_INVALID_ARG;
  const kda::MoeLayout lay = kda::moe_layout(num_tokens, k, inter, experts, shared, top_k);
  if (workspace_bytes < lay.total) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || misaligned(workspace, 256)) return KDA_ERR_INVALID_ARG;
  if (num_tokens == 0) return KDA_OK;
  char* ws = static_cast<char*>(workspace);
  kda::MoeParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.router = static_cast<const uint16_t*>(router);
  p.bias = router_bias;
  p.w_up = static_cast<const uint8_t*>(w_up);
  p.s_up = static_cast<const uint8_t*>(w_up_scales);
  p.w_down = static_cast<const uint8_t*>(w_down);
  p.s_down = static_cast<const uint8_t*>(w_down_scales);
  p.idx = state_indices;
  p.out = static_cast<uint16_t*>(out);
  p.ids = expert_ids;
  p.gates = expert_gates;
  p.x_row = x_row;
  p.out_row = out_row;
  p.M = num_tokens, p.K = k, p.I = inter, p.E = experts, p.S = shared, p.top = top_k;
  p.softmax = route == KDA_ROUTE_SOFTMAX;
  p.renorm = renormalise != 0;
  p.route_scale = route_scale;
  p.slices = lay.slices, p.slice_blocks = lay.slice_blocks;
  p.head = reinterpret_cast<int32_t*>(ws + lay.head);
  p.logits = reinterpret_cast<double*>(ws + lay.logits);
  p.done = reinterpret_cast<int32_t*>(ws + lay.done);
  p.slot = reinterpret_cast<kda::MoeSlot*>(ws + lay.slot);
  p.pair_gate = reinterpret_cast<float*>(ws + lay.pair_gate);
  p.h = reinterpret_cast<uint16_t*>(ws + lay.h);
  p.sums = reinterpret_cast<float*>(ws + lay.sums);
  int cus = 0;
  if (hipError_t e = kda::device_cus(&cus); e != hipSuccess) return failed(e, "device query");
  if (hipError_t e = kda::launch_moe(p, cus, static_cast<hipStream_t>(stream)); e != hipSuccess)
    return failed(e, "mixture-of-experts launch");
  return KDA_OK;
}

}  // extern "C"
