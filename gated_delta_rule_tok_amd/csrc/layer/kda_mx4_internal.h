// kda_mx4_internal.h -- what the kernels on microscaled 4-bit numbers (the public
// include/kda_mx4.h) and the host code that launches them share.
#pragma once

#include "kda_layer_internal.h"

namespace kda {

constexpr int kMxBlock = 32;  // elements that share a scale

struct Mx4Rows {  // quantisation and its inverse
  uint16_t* x;    // bf16 rows
  uint8_t *codes, *scales;
  int64_t rows, x_row;
  int k;
};
hipError_t launch_mx4_quant(const Mx4Rows& p, hipStream_t stream);
hipError_t launch_mx4_dequant(const Mx4Rows& p, hipStream_t stream);

struct Mx4Params {
  const void* x;
  const uint8_t* xs;  // null: x is bf16
  const uint8_t *w, *ws;
  uint16_t* y;
  int64_t M, x_row, y_row;
  int K, N;
};
hipError_t launch_mx4_few(const Mx4Params& p, int cus, hipStream_t stream);
// Operands of k a multiple of 128, 512 at least, and scales at 4-byte addresses.
bool mx4_tile_ok(const Mx4Params& p);
hipError_t launch_mx4_tile(const Mx4Params& p, int cus, hipStream_t stream);

// One call of the mixture-of-experts layer.  A pair is a token and an expert that
// it goes through; pairs are listed by expert, then token.  A slot is an expert
// that is hit.
struct MoeParams {
  const uint16_t *x, *router;
  const float* bias;
  const uint8_t *w_up, *s_up, *w_down, *s_down;
  const int32_t* idx;
  uint16_t* out;
  int32_t* ids;
  float* gates;
  int64_t x_row, out_row;
  int M, K, I, E, S, top;
  int softmax, renorm;
  float route_scale;
  // workspace
  int slices, slice_blocks;  // of the router's sums over k: how many, of how many 32s
  double* logits;       // [slices][M][E]
  int32_t* head;        // [0]: tokens routed so far, [1]: slots in use
  int32_t* slot_expert; // [slots]
  int32_t* slot_begin;  // [slots + 1] into pairs
  int32_t* pairs;       // [M (top + S)]: the pair's token
  float* pair_gate;     // [M (top + S)]
  uint16_t *h_hi, *h_lo;  // [M (top + S)][I]: silu(G x) * (U x) as two bf16 pieces
};
struct MoeLayout {
  int slices, slice_blocks, slots;
  size_t logits, head, slot_expert, slot_begin, pairs, pair_gate, h_hi, h_lo, total;
};
MoeLayout moe_layout(int M, int K, int I, int E, int S, int top);
hipError_t launch_moe(const MoeParams& p, int cus, hipStream_t stream);

}  // namespace kda
