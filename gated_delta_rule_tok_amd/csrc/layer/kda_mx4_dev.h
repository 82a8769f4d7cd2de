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

struct __attribute__((packed, aligned(1))) AnyAligned16 { uint32_t v[4]; };

// STEPS steps of 128 k (4 blocks of 32) of one tile of 16 rows, as loaded: lane l
// holds row l % 16, block 4 j + l / 16 of step j, and all 4 scales of step j in s[j].
template <int STEPS>
struct Piece {
  u32x4 w[STEPS];
  uint32_t s[STEPS];
};

// codes, scales: the row's (this lane's), of nb blocks; unit: which STEPS steps.
// Blocks behind the row's end repeat the last one's codes with scale 0.  A wave's
// 16 scale bytes of a row come in one load (one byte at a time, each load fetches
// a line a row for it: more than the codes).
template <int STEPS>
__device__ __forceinline__ void load_piece(Piece<STEPS>& p, const uint8_t* codes, const uint8_t* scales,
                                           int nb, int unit, int g) {
  const int b0 = unit * (4 * STEPS);
  if (b0 + 4 * STEPS <= nb) {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) p.w[j] = *reinterpret_cast<const u32x4*>(codes + uint32_t(b0 + 4 * j + g) * 16);
    struct __attribute__((packed, aligned(1))) B { uint32_t v[STEPS]; };
    const B b = *reinterpret_cast<const B*>(scales + b0);
#pragma unroll
    for (int j = 0; j < STEPS; ++j) p.s[j] = b.v[j];
  } else {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int b = b0 + 4 * j + g, c = min(b, nb - 1);
      p.w[j] = *reinterpret_cast<const u32x4*>(codes + uint32_t(c) * 16);
      p.s[j] = b < nb ? uint32_t(scales[c]) << (8 * g) : 0u;
    }
  }
}

// The scale of lane group g's block, as the exponent field of a float.
__device__ __forceinline__ float scale_of(uint32_t s, int g) {
  return __uint_as_float(((s >> (8 * g)) & 0xffu) << 23);
}

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
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(a), codes8(b), c, 4, 4, 0, int(sa & 0xffu), 0, int(sb & 0xffu));
}

// Up to 16 rows of bf16 x, 128 of k at a time, into MFMA operands through 4 KB of
// LDS that the wave has for itself: a load takes whole 256-byte rows, 4 of them,
// where loads in the operands' layout would take quarters of lines of 16.  The
// 16-byte pieces of row r are stored in the order piece ^ r (bank spread).
// Operand d of block group g is piece 4 g + d, as dword d of the lane's codes is.
template <int RQ>
struct XRows {
  u32x4 v[RQ];
};
template <int RQ>
__device__ __forceinline__ void load_x(XRows<RQ>& x, const uint16_t* const (&row)[RQ], int k0, int K, int l16) {
#pragma unroll
  for (int q = 0; q < RQ; ++q) {
    const int k = k0 + 8 * l16;
    x.v[q] = *reinterpret_cast<const u32x4*>(row[q] + min(k, K - 8));
    if (k >= K) x.v[q] = u32x4{};
  }
}
template <int RQ>
__device__ __forceinline__ void stage_x(char* lds, const XRows<RQ>& x, int l16, int g) {
#pragma unroll
  for (int q = 0; q < RQ; ++q) {
    const int r = 4 * q + g;
    *reinterpret_cast<u32x4*>(lds + r * 256 + ((l16 ^ r) << 4)) = x.v[q];
  }
}
__device__ __forceinline__ bf16x8 x_operand(const char* lds, int d, int l16, int g) {
  return *reinterpret_cast<const bf16x8*>(lds + l16 * 256 + (((4 * g + d) ^ l16) << 4));
}
// Orders the wave's own LDS accesses (they complete in order) for the compiler.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace kda
