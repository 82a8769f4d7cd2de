// kda_mx4_dev.h -- device pieces of the products with microscaled 4-bit weights.
//
// gfx950 facts they rely on (each checked on the device, for every code, every
// scale and every bf16):
//  * v_cvt_scalef32_pk_bf16_fp4: two codes of a byte to two bf16, low four bits
//    first, times the power of two of the scale operand's exponent field e:
//    2^(e - 127), for e = 0 too, NaN for 255; exact, subnormals among them.
//  * v_cvt_scalef32_pk_fp4_bf16: the inverse, to nearest even, saturating at 6.
//  * v_mfma_scale_f32_16x16x128_f8f6f4 with both operands e2m1: lane l holds the
//    32 elements of row (column) l % 16 from k = 32 (l / 16), 16 bytes, and
//    their scale byte; scales as above (0 and 0 together underflow to 0, which
//    is how blocks behind the end of k count nothing).  Accumulators as for
//    16x16x32.  One instruction is off by less than 2^-24 of the sum of its
//    products' magnitudes.
#pragma once

#include "kda_mfma.h"

namespace kda {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// A unit, STEPS steps of 128 k (4 blocks of 32), of one tile of 16 rows as loaded:
// lane l holds of row l / 4 the block 4 j + l % 4 of step j, and the 4 scales of step
// min(l % 4, STEPS - 1).  An operand wants row l % 16 and block l / 16 instead, but a
// load whose adjacent lanes are in different rows takes a cycle a lane (64 for 1 KB:
// 10 TB/s over the device at best, with the scales 4), this one a cycle for four, and
// LDS is there to exchange them.
template <int STEPS>
struct Piece {
  u32x4 w[STEPS];
  uint32_t s;
};
constexpr int kScaleLds = 256;  // bytes of LDS for the scales of a tile's unit
template <int STEPS>
constexpr int kPieceLds = STEPS * 1024 + kScaleLds;

// codes, scales: those of the tile's first row (scalars); code_row, scale_row: bytes
// from there to this lane's row; nb: blocks of a row; unit: which STEPS steps; q = l % 4.
// Scalar bases and 32-bit offsets, since a decode step's calls are as much instructions
// as bytes.  Blocks behind the row's end repeat the last one's codes with scale 0.
// TINY: rows of fewer than 4 blocks, whose scales are read byte by byte.
template <int STEPS, bool TINY>
__device__ __forceinline__ void load_piece(Piece<STEPS>& p, const uint8_t* codes, uint32_t code_row,
                                           const uint8_t* scales, uint32_t scale_row, int nb, int unit, int q) {
  static_assert(STEPS <= 4, "a lane of four for each step");
  const int b0 = unit * (4 * STEPS), rest = nb - 1 - b0;
  const uint8_t* c = codes + uint32_t(b0) * 16;
#pragma unroll
  for (int j = 0; j < STEPS; ++j)
    p.w[j] = *reinterpret_cast<const u32x4*>(c + (code_row + uint32_t(min(4 * j + q, rest)) * 16));
  const int b = b0 + 4 * min(q, STEPS - 1);
  if (TINY) {
    p.s = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (b + i < nb) p.s |= uint32_t(scales[scale_row + b + i]) << (8 * i);
  } else {
    struct __attribute__((packed, aligned(1))) B { uint32_t v; };
    p.s = reinterpret_cast<const B*>(scales + (scale_row + uint32_t(min(b, nb - 4))))->v;
  }
}
// Rows of 64 bytes in LDS: piece c of 16 bytes of row r is at piece c ^ bank_turn(r), so
// that one piece of 8 adjacent rows covers 128 bytes and of 16 rows 256, every bank once.
__device__ __forceinline__ int bank_turn(int r) { return ((r >> 1) ^ ((r >> 3) & 1)) & 3; }
// Into the LDS that the wave has for this tile: rows of 64 bytes for each step, then 16
// bytes of scales a row.
template <int STEPS, bool TINY>
__device__ __forceinline__ void stage_piece(char* lds, const Piece<STEPS>& p, int nb, int unit, int lane) {
  const int r = lane >> 2, q = lane & 3;
#pragma unroll
  for (int j = 0; j < STEPS; ++j)
    *reinterpret_cast<u32x4*>(lds + j * 1024 + r * 64 + ((q ^ bank_turn(r)) << 4)) = p.w[j];
  uint32_t s = p.s;
  if (!TINY && (unit + 1) * (4 * STEPS) > nb) {  // a row's last bytes: down to their place, zeros behind them
    const int over = unit * (4 * STEPS) + 4 * min(q, STEPS - 1) - (nb - 4);
    s = over <= 0 ? s : over < 4 ? s >> (8 * over) : 0u;
  }
  *reinterpret_cast<uint32_t*>(lds + STEPS * 1024 + r * 16 + q * 4) = s;
}
// An operand's codes and scale byte of step j.
__device__ __forceinline__ u32x4 codes_operand(const char* lds, int j, int l16, int g) {
  return *reinterpret_cast<const u32x4*>(lds + j * 1024 + l16 * 64 + ((g ^ bank_turn(l16)) << 4));
}
template <int STEPS>
__device__ __forceinline__ uint32_t scale_operand(const char* lds, int j, int l16, int g) {
  return *reinterpret_cast<const uint8_t*>(lds + STEPS * 1024 + l16 * 16 + j * 4 + g);
}
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// Eight codes of a dword as bf16.
__device__ __forceinline__ bf16x8 dequant8(uint32_t q, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ i32x8 codes8(u32x4 v) {
  return i32x8{int(v[0]), int(v[1]), int(v[2]), int(v[3]), 0, 0, 0, 0};
}

// 16 rows x 16 columns x 128 k of codes; sa, sb: the scale byte of the lane in the low bits
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(a), codes8(b), c, 4, 4, 0, int(sa), 0, int(sb));
}

// Up to 4 RQ rows of bf16 x, 128 of k at a time, into MFMA operands through RQ KB of
// LDS that the wave has for itself: a load takes whole 256-byte rows, 4 of them,
// where loads in the operands' layout would take quarters of lines of 16.  The
// 16-byte pieces of row r are stored in the order piece ^ r (bank spread).
// Operand d of block group g is piece 4 g + d, as dword d of the lane's codes is.
template <int RQ>
struct XRows {
  u32x4 v[RQ];
};
// x: a scalar; row[q]: bytes from there to row 4 q + lane / 16; K: elements of a row;
// n: rows that are wanted (what the others' columns give is not used).
template <int RQ>
__device__ __forceinline__ void load_x(XRows<RQ>& x, const uint16_t* base, const uint32_t (&row)[RQ], int k0, int K,
                                       int l16, int n = 4 * RQ) {
  k0 = min(k0, K - 8);
  const uint16_t* at = base + k0;
  const int rest = (K - 8 - k0) >> 3;
#pragma unroll
  for (int q = 0; q < RQ; ++q)
    if (RQ == 1 || 4 * q < n)
      x.v[q] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(at) + (row[q] + uint32_t(min(l16, rest)) * 16));
}
// Pieces behind the end of k (they repeat another) as zeros.  row0: row of LDS of the first.
template <int RQ>
__device__ __forceinline__ void stage_x(char* lds, XRows<RQ>& x, int k0, int K, int l16, int g, int n = 4 * RQ,
                                        int row0 = 0) {
  if (k0 + 128 > K) {
    const bool in = k0 + 8 * l16 < K;
#pragma unroll
    for (int q = 0; q < RQ; ++q)
      if (!in) x.v[q] = u32x4{};
  }
#pragma unroll
  for (int q = 0; q < RQ; ++q) {
    const int r = row0 + 4 * q + g;
    if (RQ == 1 || 4 * q < n) *reinterpret_cast<u32x4*>(lds + r * 256 + ((l16 ^ r) << 4)) = x.v[q];
  }
}
__device__ __forceinline__ bf16x8 x_operand_of(const char* lds, int r, int d, int g) {
  return *reinterpret_cast<const bf16x8*>(lds + r * 256 + (((4 * g + d) ^ r) << 4));
}
// (rows that are not staged repeat those that are: their columns are not used)
template <int RQ>
__device__ __forceinline__ bf16x8 x_operand(const char* lds, int d, int l16, int g) {
  return x_operand_of(lds, l16 & (4 * RQ - 1), d, g);
}
// Orders the wave's own LDS accesses (they complete in order) for the compiler.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace kda
