// kda_mx4_quant.hip -- bf16 rows to microscaled 4-bit numbers and back.
//
// Bound by the bytes: 2 + 17/32 per element either way.  A thread takes 8 adjacent
// elements, so that a wave's loads are 1 KB in one piece; the 4 threads of a block
// of 32 find its largest magnitude by two exchanges.  bf16 magnitudes order as
// their bits, and floor(log2 m) is the exponent field, so the scale is
// max(0, field - 2): subnormals, zeros and the clamp at 2^-127 come out of that.
// The conversion instruction rounds and saturates as the format wants.
//
// 16384 x 7168: 46 us with x in the caches' reach, 72 cold (297 MB, 4.1 TB/s); back 47
// (6.3 TB/s, the codes just written).  1 x 7168: 2.2 us, a launch and two round trips.
// Four pieces a thread, 4 KB a wave in flight.
#include "kda_mx4_dev.h"
#include "kda_mx4_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;  // of 8 elements per thread, kThreads apart

// Piece i of a workgroup's run -> row and piece within it.  ppr: pieces per row, a
// multiple of 4 (so that the threads of a block of 32 are in one wave, 4 aligned lanes).
struct Where {
  int64_t row0;
  uint32_t col0, ppr;
  __device__ __forceinline__ Where(const Mx4Rows& p) {
    ppr = uint32_t(p.k) / 8;
    const uint64_t at = uint64_t(blockIdx.x) * (kThreads * kPieces);
    row0 = int64_t(at / ppr);
    col0 = uint32_t(at - uint64_t(row0) * ppr);
  }
  __device__ __forceinline__ void at(uint32_t i, int64_t& row, uint32_t& col) const {
    const uint32_t c = col0 + i, r = c / ppr;
    row = row0 + r;
    col = c - r * ppr;
  }
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of two 16-bit numbers each
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}

// (by value: a bit cast of a vector's element itself takes the vector's first)
__device__ __forceinline__ bf16x2 pair_of(uint32_t v) { return __builtin_bit_cast(bf16x2, v); }

__global__ __launch_bounds__(kThreads) void quant_kernel(Mx4Rows p) {
  const Where w(p);
  u32x4 v[kPieces];
  int64_t row[kPieces];
  uint32_t col[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    w.at(threadIdx.x + i * kThreads, row[i], col[i]);
    v[i] = row[i] < p.rows ? *reinterpret_cast<const u32x4*>(p.x + row[i] * p.x_row + col[i] * 8) : u32x4{};
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const uint32_t m = 0x7fff7fffu;
    uint32_t b = max2(max2(v[i][0] & m, v[i][1] & m), max2(v[i][2] & m, v[i][3] & m));
    b = max(b & 0xffffu, b >> 16);
    b = max(b, uint32_t(__shfl_xor(int(b), 1)));
    b = max(b, uint32_t(__shfl_xor(int(b), 2)));
    const bool finite = b < 0x7f80u;
    const uint32_t e = max(int(b >> 7) - 2, 0);
    const float sc = __uint_as_float(e << 23);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair_of(v[i][0]), sc, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair_of(v[i][1]), sc, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair_of(v[i][2]), sc, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair_of(v[i][3]), sc, 3);
    if (row[i] < p.rows) {
      *reinterpret_cast<uint32_t*>(p.codes + row[i] * (p.k / 2) + col[i] * 4) = finite ? q : 0u;
      if ((threadIdx.x & 3) == 0) p.scales[row[i] * (p.k / 32) + col[i] / 4] = uint8_t(finite ? e : 255u);
    }
  }
}

__global__ __launch_bounds__(kThreads) void dequant_kernel(Mx4Rows p) {
  const Where w(p);
  uint32_t q[kPieces], s[kPieces];
  int64_t row[kPieces];
  uint32_t col[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    w.at(threadIdx.x + i * kThreads, row[i], col[i]);
    q[i] = s[i] = 0;
    if (row[i] < p.rows) {
      q[i] = *reinterpret_cast<const uint32_t*>(p.codes + row[i] * (p.k / 2) + col[i] * 4);
      s[i] = p.scales[row[i] * (p.k / 32) + col[i] / 4];
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (row[i] < p.rows)
      *reinterpret_cast<bf16x8*>(p.x + row[i] * p.x_row + col[i] * 8) = dequant8(q[i], __uint_as_float(s[i] << 23));
}

hipError_t launch(const void* f, const Mx4Rows& p, hipStream_t st) {
  Mx4Rows arg = p;
  void* args[] = {&arg};
  const uint64_t pieces = uint64_t(p.rows) * (p.k / 8), per = kThreads * kPieces;
  return hipLaunchKernel(f, dim3(uint32_t((pieces + per - 1) / per)), dim3(kThreads), args, 0, st);
}

}  // namespace

hipError_t launch_mx4_quant(const Mx4Rows& p, hipStream_t stream) {
  return launch(reinterpret_cast<const void*>(&quant_kernel), p, stream);
}
hipError_t launch_mx4_dequant(const Mx4Rows& p, hipStream_t stream) {
  return launch(reinterpret_cast<const void*>(&dequant_kernel), p, stream);
}

}  // namespace kda
