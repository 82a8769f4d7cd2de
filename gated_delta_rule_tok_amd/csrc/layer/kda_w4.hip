// kda_w4.hip -- products of few tokens with 4-bit weights:
//   y[m, n] = sum_k x[m, k] (w[n, k] - z[n, g]) s[n, g],  g = k / group
//
// Bound by the weights' bytes (each is used for at most 64 tokens), so the
// kernel streams w in 16-byte loads, one pass, and feeds 16x16x32 bf16 MFMAs:
// A = 16 tokens, B = 16 rows of w.  A nibble q becomes the bf16 number (128 + q)
// 2^-15 by an OR with the bits of 2^-8 (exact: bf16 steps by 2^-15 there), two at
// a time, and the group's sum is corrected in fp32:
//   sum (q - z) x = sum (128 + q) x - (128 + z) sum x,
// with sum x from one more MFMA against 2^-15, shared by all rows of w.  x
// stays bf16 and every product is exact in fp32; scales are applied to the
// group's fp32 sum, and 2^15 to the last one.  That power costs nothing and
// keeps 143 |x| summed over a group inside fp32 for every finite x.
//
// A lane's 16 bytes are 32 adjacent k of one row (lane l: row l % 16, k from
// 32 (l / 16)); two swaps of lane halves and two of lane rows transpose the
// 4 x 4 dwords of four lanes so that dword j is k = 32 j + 8 (l / 16) .. + 8,
// one MFMA's operand with k ascending through the group.  The OR takes nibble
// pairs (0,4), (1,5), (2,6), (3,7) out of a dword; x's operand is put into the
// same order.
//
// The waves of a workgroup share k, in runs of 128-wide blocks, and add their
// sums through LDS in wave order.  What costs most beside the weights is x,
// which every workgroup reads whole, and the scales; both go through LDS so
// that their loads take whole cache lines.  16 tokens x 7168 x 14336 in groups
// of 64 with zeros: 18.4 us (58 MB, 3.2 TB/s; a copy reaches 5.1); an earlier
// form that took 20.4 us took 14 without the loads of x and of the scales.
#include "kda_layer_internal.h"
#include "kda_mfma.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

__device__ __forceinline__ bf16x8 nibbles(uint32_t q, uint32_t e) {
  const uint32_t m = 0x000f000fu;
  return __builtin_bit_cast(bf16x8, u32x4{(q & m) | e, ((q >> 4) & m) | e, ((q >> 8) & m) | e,
                                          ((q >> 12) & m) | e});
}

// 8 adjacent bf16 in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ bf16x8 interleave(u32x4 x) {
  return __builtin_bit_cast(
      bf16x8, u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100), __builtin_amdgcn_perm(x[2], x[0], 0x07060302),
                    __builtin_amdgcn_perm(x[3], x[1], 0x05040100), __builtin_amdgcn_perm(x[3], x[1], 0x07060302)});
}

// One 128-wide block of k as loaded: a lane's pieces of w and of x.
template <int MT, int NT, int RQ>
struct Block {
  u32x4 w[NT], x[MT][RQ];
};

// MT tiles of 16 tokens (the first 4 RQ rows of each hold tokens) and NT tiles
// of 16 rows of w per workgroup, WAVES waves that share k, U blocks in flight per
// wave; G the group.
template <int MT, int RQ, int NT, int WAVES, int U, int G, bool ZERO>
__global__ __launch_bounds__(64 * WAVES) void w4_kernel(W4Params p) {
  constexpr int kGroups = 128 / G;  // groups in a block
  constexpr int kSteps = G / 32;    // MFMA steps in a group
  // groups whose scales and zeros are in LDS at a time
  constexpr int kSegGroups = MT * NT > 4 ? 128 : 256, kScalePitch = kSegGroups + 1;
  constexpr int kXBytes = WAVES * MT * 4096, kScaleBytes = 16 * NT * kScalePitch * 4;
  constexpr int kRedBytes = WAVES * MT * NT * 64 * 16;
  __shared__ __align__(16) char lds[kXBytes + kScaleBytes > kRedBytes ? kXBytes + kScaleBytes : kRedBytes];
  uint32_t* sz = reinterpret_cast<uint32_t*>(lds + kXBytes);  // [16 NT][kScalePitch]: scale | zero << 16
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
  const int groups = p.K / G, blocks = (p.K + 127) / 128;
  // rows behind the last row or token repeat it: their sums are not stored
  // (32-bit offsets from scalar bases: 32 rows of at most 2^19 bytes of w, 64 of x at most 2^24
  // elements apart)
  const uint8_t* wbase = p.w + size_t(n0) * (p.K / 2);
  uint32_t wrow[NT], xrow[MT][RQ];
  const int last = p.K % 128 ? p.K - p.K % 128 : p.K;  // where a block that is not whole begins
  const uint32_t wpiece = 16 * g4, wtail = min(16 * g4, max(p.K - 32 - last, 0) / 2);
#pragma unroll
  for (int i = 0; i < NT; ++i) wrow[i] = uint32_t(min(16 * i + l16, p.N - 1 - n0)) * uint32_t(p.K / 2);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < RQ; ++j) xrow[i][j] = uint32_t(min(m0 + 16 * i + 4 * j + g4, p.M - 1) * p.x_row);
  const uint32_t xpiece = 8 * l16, xtail = min(8 * l16, max(p.K - 8 - last, 0));
  // this wave's x, 256 bytes a row, its 16-byte pieces in the order piece ^ row (bank spread)
  char* xl = lds + wave * (MT * 4096);
  const uint32_t xread = l16 * 256;
  typedef Block<MT, NT, RQ> B;
  // Branch-free, so that the loads of U blocks stay in flight; in the last
  // block of a K that is no multiple of 128 (it is one of 32) pieces behind it
  // repeat the last one, and add() takes zeros for x there.
  const auto load = [&](B& b, int blk) {
    const int k0 = 128 * blk;
    const uint32_t piece = k0 < last ? wpiece : wtail;
    const uint8_t* wk = wbase + k0 / 2;
#pragma unroll
    for (int i = 0; i < NT; ++i) b.w[i] = *reinterpret_cast<const u32x4*>(wk + (wrow[i] + piece));
    const uint16_t* xk = p.x + k0;
    const uint32_t xp = k0 < last ? xpiece : xtail;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < RQ; ++j) b.x[i][j] = *reinterpret_cast<const u32x4*>(xk + (xrow[i][j] + xp));
  };
  // 2^-8 in both halves, in a vector register: an instruction reads one scalar
  // only, so that two literals would make (q & m) | e two instructions
  uint32_t e128 = 0x3b803b80u;
  asm("" : "+v"(e128));
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x38003800u, 0x38003800u, 0x38003800u, 0x38003800u});  // 2^-15
  f32x4 acc[MT][NT] = {};
  const auto add = [&](B& b, int blk, int seg) {
    // x through LDS into operands: a load of it takes whole lines of 4 rows, where loads
    // in the operands' layout took half lines of 16 rows, at 2.5 times the cost
    const bool in = 128 * blk + 8 * l16 < p.K;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < RQ; ++j) {
        const int r = 4 * j + g4;
        *reinterpret_cast<bf16x8*>(xl + i * 4096 + r * 256 + ((l16 ^ r) << 4)) =
            interleave(in ? b.x[i][j] : u32x4{});
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < NT; ++i) b.w[i] = transpose4(b.w[i]);
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      f32x4 sx[MT] = {}, c[MT][NT] = {};
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const int d = j * kSteps + q;
        bf16x8 a[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          a[m] = *reinterpret_cast<const bf16x8*>(xl + m * 4096 + xread + (((4 * d + g4) ^ l16) << 4));
          sx[m] = mfma32(a[m], ones, sx[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bf16x8 f = nibbles(b.w[n][d], e128);
#pragma unroll
          for (int m = 0; m < MT; ++m) c[m][n] = mfma32(a[m], f, c[m][n]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t v = sz[(16 * n + l16) * kScalePitch + blk * kGroups + j - seg];
        const float sc = bf16_lo(v), of = 128.f + bf16_hi(v);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[m][n][r] = fmaf(sc, fmaf(-of, sx[m][r], c[m][n][r]), acc[m][n][r]);
      }
    }
  };
  // Segments of kSegGroups groups, whose scales and zeros go through LDS (one per row
  // and group straight into registers took longer than the weights: 16 lines
  // per load of 2 bytes).  A wave's blocks of a segment are adjacent.  Every
  // load is unconditional (the last block is repeated behind the end), so that
  // the waits count loads, not branches.
  for (int seg = 0; seg < groups; seg += kSegGroups) {
    const int b0 = seg / kGroups, nb = min(blocks - b0, kSegGroups / kGroups);
    const int per = (nb + WAVES - 1) / WAVES, first = b0 + wave * per;
    const int cnt = max(0, min(per, b0 + nb - first));
    B buf[U];
    if (cnt) {
#pragma unroll
      for (int u = 0; u < U; ++u) load(buf[u], first + min(u, cnt - 1));
    }
    if (seg) __syncthreads();
    // groups behind the last one of its block of 128 count nothing
    const int ns = min(groups - seg, kSegGroups), nz = (ns + kGroups - 1) / kGroups * kGroups;
    for (int r = wave; r < 16 * NT; r += WAVES) {
      const size_t row = size_t(min(n0 + r, p.N - 1)) * groups + seg;
      for (int g = lane; g < nz; g += 64)
        sz[r * kScalePitch + g] =
            g < ns ? uint32_t(p.scales[row + g]) | (ZERO ? uint32_t(p.zeros[row + g]) << 16 : 0x41000000u) : 0u;
    }
    __syncthreads();
    int i = 0;
    for (; i + U < cnt; i += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        add(buf[u], first + i + u, seg);
        load(buf[u], first + min(i + u + U, cnt - 1));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u < cnt) add(buf[u], first + i + u, seg);
  }
  __syncthreads();
  f32x4(*red)[MT * NT][64] = reinterpret_cast<f32x4(*)[MT * NT][64]>(lds);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[wave][m * NT + n][lane] = acc[m][n];
  __syncthreads();
  for (int i = wave; i < MT * NT; i += WAVES) {
    f32x4 y = red[0][i][lane];
#pragma unroll
    for (int u = 1; u < WAVES; ++u) y += red[u][i][lane];
    const int n = n0 + 16 * (i % NT) + l16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = m0 + 16 * (i / NT) + 4 * g4 + r;
      if (m < p.M && n < p.N) p.y[size_t(m) * p.y_row + n] = f32_to_bf16(y[r] * 0x1p15f);
    }
  }
}

template <int MT, int RQ, int NT, int WAVES, int U, int G>
const void* kernel(bool zero) {
  return zero ? reinterpret_cast<const void*>(&w4_kernel<MT, RQ, NT, WAVES, U, G, true>)
              : reinterpret_cast<const void*>(&w4_kernel<MT, RQ, NT, WAVES, U, G, false>);
}

template <int MT, int RQ, int NT, int WAVES, int U>
hipError_t launch(const W4Params& p, hipStream_t st) {
  W4Params arg = p;
  void* args[] = {&arg};
  const bool z = p.zeros != nullptr;
  const void* f = p.group == 32   ? kernel<MT, RQ, NT, WAVES, U, 32>(z)
                  : p.group == 64 ? kernel<MT, RQ, NT, WAVES, U, 64>(z)
                                  : kernel<MT, RQ, NT, WAVES, U, 128>(z);
  const dim3 grid((p.N + 16 * NT - 1) / (16 * NT), (p.M + 16 * MT - 1) / (16 * MT));
  return hipLaunchKernel(f, grid, dim3(64 * WAVES), args, 0, st);
}

}  // namespace

// Rows of w per workgroup: 32 read x half as often as 16, 16 give twice the
// workgroups.  Measured (us, 16 / 32 rows): 16 tokens x 7168 x 1536 7.3 / 9.0,
// x 2048 x 4096 4.8 / 5.5, x 4096 x 5120 8.6 / 8.0, x 7168 x 14336 26.9 / 20.4;
// 24 x 7168 x 1536 7.6 / 9.5, 32 x 512 x 3000 6.2 / 4.4, 64 x 7168 x 1536 14.2 /
// 10.5, 64 x 2048 x 512 4.5 / 5.6: 32 where they are more than half a workgroup
// per compute unit.  With at most 4 tokens x is a quarter of that: 4 x 7168 x
// 7168 11.3 / 11.5, 2 x 7168 x 14336 17.2 / 15.8, so 32 from one and a half on.
// 64 rows lose everywhere.
//
// Tokens per workgroup: more than 16 in tiles of 16, each with workgroups of its
// own that read w again (64 x 7168 x 1536 10.5 us against 20.4 with all 64 in
// one, 24 x 7168 x 7168 17.0 against 18.5 with 32), but more than 32 with many
// rows of w in one (61 x 2048 x 7171 12.4 against 17.8, 64 x 7168 x 7168 30.6
// against 33.0).  (That form's variants for groups of 64 spill 12 and 13 of their
// 256 registers; none of the others spills.)
hipError_t launch_w4(const W4Params& p, int cus, hipStream_t stream) {
  const int64_t wide = (p.N + 31) / 32, tiles = (p.M + 15) / 16;
  if (p.M <= 4)
    return 2 * wide > 3 * cus ? launch<1, 1, 2, 8, 2>(p, stream) : launch<1, 1, 1, 8, 2>(p, stream);
  if (p.M > 32 && 2 * wide > cus) return launch<4, 4, 2, 8, 1>(p, stream);
  return 2 * wide * tiles > cus ? launch<1, 4, 2, 8, 1>(p, stream) : launch<1, 4, 1, 16, 1>(p, stream);
}

}  // namespace kda
