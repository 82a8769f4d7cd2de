// kda_layer_api.hip -- the C ABI of include/kda_layer.h: argument checks,
// workspace sizing and the launches.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "kda_layer.h"
#include "kda_layer_internal.h"

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

bool heads_ok(int32_t hk, int32_t hv) { return hk > 0 && hv > 0 && hv % hk == 0 && hv <= 65536; }
// a grid holds fewer than 2^32 threads: 4 workgroups of 256 per (sequence, head), and one per (chunk, head)
bool pairs_ok(int64_t n, int32_t hv) { return n * hv < (int64_t(1) << 21); }
bool chunks_ok(int64_t t, int64_t n, int32_t hv) {
  return (t / kda::kGdrChunk + n) * hv < (int64_t(1) << 24);
}

// What both forms of the delta rule check of their tensors.  rows: tokens.
kda_status_t gdr_checks(const void* q, const void* k, const void* v, const void* a, const void* beta,
                        const float* A_log, const float* dt_bias, float scale, const void* out,
                        int64_t rows, int32_t hk, int32_t hv, int sdt, const kda_gdr_strides_t& s) {
  if (!heads_ok(hk, hv)) return KDA_ERR_INVALID_ARG;
  if (sdt != KDA_STATE_FP32 && sdt != KDA_STATE_BF16) return KDA_ERR_INVALID_ARG;
  if (!A_log || !dt_bias || !std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if (rows > 0 && (!q || !k || !v || !a || !beta || !out)) return KDA_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, out})
    if (misaligned(p, 16)) return KDA_ERR_INVALID_ARG;
  if (misaligned(a, 2) || misaligned(beta, 2) || misaligned(A_log, 4) || misaligned(dt_bias, 4))
    return KDA_ERR_INVALID_ARG;
  // token strides: 32-bit byte offsets over the 64 rows of a chunk
  constexpr int64_t kMaxHead = int64_t(1) << 30, kMaxToken = int64_t(1) << 24;
  for (int64_t x : {s.q_token, s.k_token, s.v_token, s.out_token})
    if (x < 0 || x % 8 || x > kMaxToken) return KDA_ERR_INVALID_ARG;
  for (int64_t x : {s.q_head, s.k_head, s.v_head, s.out_head})
    if (x < 0 || x % 8 || x > kMaxHead) return KDA_ERR_INVALID_ARG;
  for (int64_t x : {s.a_token, s.a_head, s.beta_token, s.beta_head})
    if (x < 0 || x > kMaxHead) return KDA_ERR_INVALID_ARG;
  if ((rows > 1 && s.out_token == 0) || (hv > 1 && s.out_head == 0)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_gdr_strides_t dense(int32_t hk, int32_t hv) {
  const int64_t rk = int64_t(hk) * KDA_HEAD_DIM, rv = int64_t(hv) * KDA_HEAD_DIM;
  return kda_gdr_strides_t{rk, KDA_HEAD_DIM, rk, KDA_HEAD_DIM, rv, KDA_HEAD_DIM,
                           hv, 1,            hv, 1,            rv, KDA_HEAD_DIM};
}

kda::GdrParams gdr_params(const void* q, const void* k, const void* v, const void* a, const void* beta,
                          const float* A_log, const float* dt_bias, float scale, void* out, int32_t hk,
                          int32_t hv, int sdt, const kda_gdr_strides_t& s) {
  kda::GdrParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.a = static_cast<const uint16_t*>(a);
  p.beta = static_cast<const uint16_t*>(beta);
  p.A_log = A_log;
  p.dt_bias = dt_bias;
  p.scale = scale;
  p.out = static_cast<uint16_t*>(out);
  p.Hk = hk;
  p.Hv = hv;
  p.state_bf16 = sdt == KDA_STATE_BF16;
  p.q_t = s.q_token, p.q_h = s.q_head, p.k_t = s.k_token, p.k_h = s.k_head;
  p.v_t = s.v_token, p.v_h = s.v_head, p.a_t = s.a_token, p.a_h = s.a_head;
  p.b_t = s.beta_token, p.b_h = s.beta_head, p.o_t = s.out_token, p.o_h = s.out_head;
  return p;
}

}  // namespace

extern "C" {

size_t kda_gdr_get_workspace_size(int64_t max_tokens, int32_t key_heads, int32_t value_heads,
                                  int32_t max_seqs) {
  if (max_tokens < 0 || max_tokens >= (int64_t(1) << 31) || max_seqs <= 0 ||
      !heads_ok(key_heads, value_heads) || !pairs_ok(max_seqs, value_heads) ||
      !chunks_ok(max_tokens, max_seqs, value_heads))
    return 0;
  return kda::gdr_layout(max_tokens, key_heads, value_heads, max_seqs).total;
}

kda_status_t kda_gdr_prefill_fwd(const void* q, const void* k, const void* v, const void* a,
                                 const void* beta_logits, const float* A_log, const float* dt_bias,
                                 float scale, const void* initial_state, const int32_t* cu_seqlens,
                                 void* out, void* final_state, void* workspace, void* stream,
                                 int64_t num_tokens, int32_t key_heads, int32_t value_heads,
                                 int32_t num_seqs, kda_state_dtype_t state_dtype,
                                 size_t workspace_bytes, const kda_gdr_strides_t* strides) {
  const int sdt = enum_value(state_dtype);
  const kda_gdr_strides_t s = strides ? *strides : dense(key_heads, value_heads);
  if (num_tokens < 0 || num_tokens >= (int64_t(1) << 31) || num_seqs <= 0) return KDA_ERR_INVALID_ARG;
  if (kda_status_t rc = gdr_checks(q, k, v, a, beta_logits, A_log, dt_bias, scale, out, num_tokens,
                                   key_heads, value_heads, sdt, s);
      rc != KDA_OK)
    return rc;
  if (!pairs_ok(num_seqs, value_heads) || !chunks_ok(num_tokens, num_seqs, value_heads) || !cu_seqlens ||
      !final_state)
    return KDA_ERR_INVALID_ARG;
  if (misaligned(initial_state, 16) || misaligned(final_state, 16) || misaligned(cu_seqlens, 4))
    return KDA_ERR_INVALID_ARG;
  const kda::GdrLayout lay = kda::gdr_layout(num_tokens, key_heads, value_heads, num_seqs);
  if (workspace_bytes < lay.total) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (lay.total && (!workspace || misaligned(workspace, 256))) return KDA_ERR_INVALID_ARG;

  kda::GdrParams p = gdr_params(q, k, v, a, beta_logits, A_log, dt_bias, scale, out, key_heads,
                                value_heads, sdt, s);
  p.s0 = initial_state;
  p.sT = final_state;
  p.cu = cu_seqlens;
  p.T = int(num_tokens);
  p.N = num_seqs;
  p.ws = static_cast<char*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  // a few tokens per sequence: token after token, as kda_chunk_prefill_fwd does
  if (num_tokens <= int64_t(kda::kDecodeTokensPerSeq) * num_seqs) {
    if (hipError_t e = kda::launch_gdr_serial(p, st); e != hipSuccess)
      return failed(e, "serial delta rule launch");
    return KDA_OK;
  }
  int cus = 0;
  if (hipError_t e = kda::device_cus(&cus); e != hipSuccess) return failed(e, "device query");
  if (hipError_t e = kda::launch_gdr_chunked(p, cus, st); e != hipSuccess)
    return failed(e, "chunked delta rule launch");
  return KDA_OK;
}

kda_status_t kda_gdr_decode_step(const void* q, const void* k, const void* v, const void* a,
                                 const void* beta_logits, const float* A_log, const float* dt_bias,
                                 float scale, void* state_pool, int64_t num_slots,
                                 const int32_t* state_indices, void* out, void* stream,
                                 int32_t num_seqs, int32_t key_heads, int32_t value_heads,
                                 kda_state_dtype_t state_dtype, const kda_gdr_strides_t* strides) {
  const int sdt = enum_value(state_dtype);
  const kda_gdr_strides_t s = strides ? *strides : dense(key_heads, value_heads);
  if (num_seqs < 0 || num_slots <= 0) return KDA_ERR_INVALID_ARG;
  if (kda_status_t rc = gdr_checks(q, k, v, a, beta_logits, A_log, dt_bias, scale, out, num_seqs,
                                   key_heads, value_heads, sdt, s);
      rc != KDA_OK)
    return rc;
  if (!pairs_ok(num_seqs, value_heads) || !state_pool) return KDA_ERR_INVALID_ARG;
  if (misaligned(state_pool, 16) || misaligned(state_indices, 4)) return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0) return KDA_OK;
  if (!state_indices) return KDA_ERR_INVALID_ARG;
  kda::GdrParams p = gdr_params(q, k, v, a, beta_logits, A_log, dt_bias, scale, out, key_heads,
                                value_heads, sdt, s);
  p.s0 = state_pool;
  p.sT = state_pool;
  p.idx = state_indices;
  p.slots = num_slots;
  p.T = num_seqs;
  p.N = num_seqs;
  if (hipError_t e = kda::launch_gdr_serial(p, static_cast<hipStream_t>(stream)); e != hipSuccess)
    return failed(e, "serial delta rule launch");
  return KDA_OK;
}

kda_status_t kda_add_rms_norm(const void* x, void* residual, const void* weight, float eps, void* out,
                              float* out_scale, void* stream, int64_t num_rows, int32_t dim,
                              int64_t x_row, int64_t residual_row, int64_t out_row,
                              kda_out_dtype_t out_dtype, int32_t group_size) {
  const int odt = enum_value(out_dtype);
  if (odt != KDA_OUT_BF16 && odt != KDA_OUT_E4M3) return KDA_ERR_INVALID_ARG;
  if (num_rows < 0 || num_rows >= (int64_t(1) << 31) || dim <= 0 || dim > 32768) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || !weight || misaligned(weight, 2)) return KDA_ERR_INVALID_ARG;
  if (odt == KDA_OUT_BF16 ? (out_scale || group_size != 0) : (group_size != 0 && group_size != 128))
    return KDA_ERR_INVALID_ARG;
  if (num_rows > 0 && (!x || !out || (odt == KDA_OUT_E4M3 && !out_scale))) return KDA_ERR_INVALID_ARG;
  if (misaligned(x, 2) || misaligned(residual, 2) || misaligned(out_scale, 4) ||
      (odt == KDA_OUT_BF16 && misaligned(out, 2)))
    return KDA_ERR_INVALID_ARG;
  constexpr int64_t kMaxStride = int64_t(1) << 30;
  if (num_rows > 1) {
    if (x_row < dim || out_row < dim || (residual && residual_row < dim)) return KDA_ERR_INVALID_ARG;
    if (x_row > kMaxStride || out_row > kMaxStride || (residual && residual_row > kMaxStride))
      return KDA_ERR_INVALID_ARG;
  }
  if (num_rows == 0) return KDA_OK;
  kda::NormParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.res = static_cast<uint16_t*>(residual);
  p.w = static_cast<const uint16_t*>(weight);
  p.out = out;
  p.scale = out_scale;
  p.x_row = x_row;
  p.r_row = residual_row;
  p.o_row = out_row;
  p.rows = num_rows;
  p.eps = eps;
  p.dim = dim;
  p.fp8 = odt == KDA_OUT_E4M3;
  p.group = group_size;
  if (hipError_t e = kda::launch_norm(p, static_cast<hipStream_t>(stream)); e != hipSuccess)
    return failed(e, "norm launch");
  return KDA_OK;
}

kda_status_t kda_w4_proj(const void* x, const void* w, const void* scales, const void* zeros, void* y,
                         void* stream, int32_t num_tokens, int32_t k, int32_t n, int32_t group_size,
                         int64_t x_row, int64_t y_row) {
  if (num_tokens < 0 || num_tokens > 64) return KDA_ERR_INVALID_ARG;
  if (group_size != 32 && group_size != 64 && group_size != 128) return KDA_ERR_INVALID_ARG;
  if (k <= 0 || k > (1 << 20) || k % group_size || n <= 0 || n > (1 << 24)) return KDA_ERR_INVALID_ARG;
  if (!w || !scales || misaligned(w, 16) || misaligned(scales, 2) || misaligned(zeros, 2))
    return KDA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!x || !y)) return KDA_ERR_INVALID_ARG;
  if (misaligned(x, 16) || misaligned(y, 2)) return KDA_ERR_INVALID_ARG;
  // 32-bit byte offsets for the 64 rows of x
  if (num_tokens > 1 && (x_row < k || x_row % 8 || x_row > (1 << 24) || y_row < n || y_row > (int64_t(1) << 30)))
    return KDA_ERR_INVALID_ARG;
  if (num_tokens == 0) return KDA_OK;
  kda::W4Params p{};
  p.x = static_cast<const uint16_t*>(x);
  p.w = static_cast<const uint8_t*>(w);
  p.scales = static_cast<const uint16_t*>(scales);
  p.zeros = static_cast<const uint16_t*>(zeros);
  p.y = static_cast<uint16_t*>(y);
  p.x_row = x_row;
  p.y_row = y_row;
  p.M = num_tokens;
  p.K = k;
  p.N = n;
  p.group = group_size;
  int cus = 0;
  if (hipError_t e = kda::device_cus(&cus); e != hipSuccess) return failed(e, "device query");
  if (hipError_t e = kda::launch_w4(p, cus, static_cast<hipStream_t>(stream)); e != hipSuccess)
    return failed(e, "4-bit product launch");
  return KDA_OK;
}

}  // extern "C"
