// kda_w4.hip -- products of few tokens with 4-bit weights:
//   y[m, n] = sum_k x[m, k] (w[n, k] - z[n, g]) s[n, g],  g = k / group
//
// Bound by the weights' bytes (each is used for at most 64 tokens), so the
// kernel streams w in 16-byte loads, one pass, and feeds 16x16x32 bf16 MFMAs:
// A = 16 tokens, B = 16 rows of w.  A nibble q becomes the bf16 number 128 + q
// by an OR with 0x4300 (exact: bf16 steps by 1 there), two at a time, and the
// group's sum is corrected in fp32:
//   sum (q - z) x = sum (128 + q) x - (128 + z) sum x,
// with sum x from one more MFMA against ones, shared by all rows of w.  x
// stays bf16 and every product is exact in fp32; scales are applied to the
// group's fp32 sum.
//
// A lane's 16 bytes are 32 adjacent k of one row (lane l: row l % 16, k from
// 32 (l / 16)); two swaps of lane halves and two of lane rows transpose the
// 4 x 4 dwords of four lanes so that dword j is k = 32 j + 8 (l / 16) .. + 8,
// one MFMA's operand with k ascending through the group.  The OR takes nibble
// pairs (0,4), (1,5), (2,6), (3,7) out of a dword; x's operand is put into the
// same order.
//
// The 8 waves of a workgroup take the 128-wide blocks of k in turn and add
// their sums through LDS in wave order.
#include "kda_layer_internal.h"
#include "kda_mfma.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kW4Waves = 8;

// In: lane group g = l / 16 holds dwords j = 0..3 of its own piece; out: dword
// j holds what dword g of group j held.
__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
  // halves: lanes 32.. of the first with lanes ..31 of the second
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  // rows: odd rows of 16 of the first with even rows of the second
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ bf16x8 nibbles(uint32_t q) {
  const uint32_t m = 0x000f000fu, e = 0x43004300u;
  return __builtin_bit_cast(bf16x8, u32x4{(q & m) | e, ((q >> 4) & m) | e, ((q >> 8) & m) | e,
                                          ((q >> 12) & m) | e});
}

// 8 adjacent bf16 in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ bf16x8 interleave(u32x4 x) {
  return __builtin_bit_cast(
      bf16x8, u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100), __builtin_amdgcn_perm(x[2], x[0], 0x07060302),
                    __builtin_amdgcn_perm(x[3], x[1], 0x05040100), __builtin_amdgcn_perm(x[3], x[1], 0x07060302)});
}

// MT tiles of 16 tokens, NT tiles of 16 rows of w per workgroup; G the group.
template <int MT, int NT, int G>
__global__ __launch_bounds__(64 * kW4Waves) void w4_kernel(W4Params p) {
  __shared__ f32x4 red[kW4Waves][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT);
  const int groups = p.K / G;
  const uint8_t* wrow[NT];
  const uint16_t *srow[NT], *zrow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int n = min(n0 + 16 * i + l16, p.N - 1);
    wrow[i] = p.w + size_t(n) * (p.K / 2);
    srow[i] = p.scales + size_t(n) * groups;
    zrow[i] = p.zeros ? p.zeros + size_t(n) * groups : nullptr;
  }
  const uint16_t* xrow[MT];
  bool mok[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + l16;
    mok[i] = m < p.M;
    xrow[i] = p.x + size_t(mok[i] ? m : 0) * p.x_row;
  }
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
  constexpr int kGroups = 128 / G;   // groups in a block of 128
  constexpr int kSteps = G / 32;     // MFMA steps in a group
  f32x4 acc[MT][NT] = {};
  for (int k0 = 128 * wave; k0 < p.K; k0 += 128 * kW4Waves) {
    u32x4 w[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int k = k0 + 32 * g4;  // K % 32 == 0: a piece is inside or outside
      w[i] = k < p.K ? *reinterpret_cast<const u32x4*>(wrow[i] + k / 2) : u32x4{};
    }
    float s[NT][kGroups], z[NT][kGroups];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const int g = min(k0 / G + j, groups - 1);
        s[i][j] = bf16_to_f32(srow[i][g]);
        z[i][j] = p.zeros ? bf16_to_f32(zrow[i][g]) : 8.f;
      }
    u32x4 x[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 32 * j + 8 * g4;
        x[i][j] = mok[i] && k < p.K ? *reinterpret_cast<const u32x4*>(xrow[i] + k) : u32x4{};
      }
#pragma unroll
    for (int i = 0; i < NT; ++i) w[i] = transpose4(w[i]);
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      f32x4 sx[MT] = {}, c[MT][NT] = {};
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const int d = j * kSteps + q;
        bf16x8 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n] = nibbles(w[n][d]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const bf16x8 a = interleave(x[m][d]);
          sx[m] = mfma32(a, ones, sx[m]);
#pragma unroll
          for (int n = 0; n < NT; ++n) c[m][n] = mfma32(a, b[n], c[m][n]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[m][n][r] += s[n][j] * (c[m][n][r] - (128.f + z[n][j]) * sx[m][r]);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[wave][m * NT + n][lane] = acc[m][n];
  __syncthreads();
  for (int i = wave; i < MT * NT; i += kW4Waves) {
    f32x4 y = red[0][i][lane];
#pragma unroll
    for (int u = 1; u < kW4Waves; ++u) y += red[u][i][lane];
    const int n = n0 + 16 * (i % NT) + l16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 16 * (i / NT) + 4 * g4 + r;
      if (m < p.M && n < p.N) p.y[size_t(m) * p.y_row + n] = f32_to_bf16(y[r]);
    }
  }
}

template <int MT, int NT>
hipError_t launch(const W4Params& p, hipStream_t st) {
  W4Params arg = p;
  void* args[] = {&arg};
  const void* f = p.group == 32   ? reinterpret_cast<const void*>(&w4_kernel<MT, NT, 32>)
                  : p.group == 64 ? reinterpret_cast<const void*>(&w4_kernel<MT, NT, 64>)
                                  : reinterpret_cast<const void*>(&w4_kernel<MT, NT, 128>);
  return hipLaunchKernel(f, dim3((p.N + 16 * NT - 1) / (16 * NT)), dim3(64 * kW4Waves), args, 0, st);
}

}  // namespace

hipError_t launch_w4(const W4Params& p, int cus, hipStream_t stream) {
  if (p.M <= 16) return launch<1, 1>(p, stream);
  if (p.M <= 32) return launch<2, 2>(p, stream);
  return launch<4, 2>(p, stream);
}

}  // namespace kda
