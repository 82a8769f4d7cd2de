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
// Whether rows of x in the format are worth tiles through LDS.
bool mx4_in_tiles(const Mx4Params& p, int cus);
hipError_t launch_mx4_tile(const Mx4Params& p, int cus, hipStream_t stream);

// One call of the mixture-of-experts layer.  A pair is a token and an expert that
// it goes through; pairs are numbered by expert, then token.  A slot is an expert and
// up to `chunk` of its tokens.
struct MoeSlot {
  int32_t expert, begin, n, unused;  // pairs begin .. begin + n - 1
  uint32_t token[4];                 // 16 bytes: the pairs' tokens, the last repeated
};

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
  int chunk;                 // tokens per slot: 4 or 16
  int slices, slice_blocks;  // of the router's sums over k: how many, of how many 32s
  int up_log2;               // of up's workgroups
  int parts;                 // into which down's sum over slots is cut
  // workspace
  double* logits;         // [slices][M][E]
  int32_t* head;          // [0]: tokens routed so far, [1]: slots in use
  int32_t* done;          // [K / 16]: parts of down's sums that are there
  MoeSlot* slot;
  float* pair_gate;       // [M (top + S) + 16]
  uint16_t* h;            // [3][M (top + S)][I]: gate * silu(G x) * (U x) as three bf16 pieces
  float* sums;            // [parts][M][K]
};
struct MoeLayout {
  int slices, slice_blocks;
  size_t logits, head, done, slot, pair_gate, h, sums, total;
};
// Slots that a call may have, at most.
int moe_slots(int M, int E, int S, int top, int chunk);
int moe_parts(int M, int K, int I, int E, int S, int top, int chunk);
constexpr int kMoeMostParts = 8;
MoeLayout moe_layout(int M, int K, int I, int E, int S, int top);
hipError_t launch_moe(const MoeParams& p, int cus, hipStream_t stream);

}  // namespace kda
