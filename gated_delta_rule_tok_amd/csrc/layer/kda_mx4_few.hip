// kda_mx4_few.hip -- products of few rows x with microscaled 4-bit weights:
//   y[m, n] = sum_k x[m, k] w[n, k]
//
// Bound by the weights' bytes: a workgroup streams 16 RT rows of w in one pass,
// its waves share k.  Weights are the MFMA's A operand (rows), 16 rows of x its B
// operand (columns).  A lane's 16 bytes of w are one block of 32 of one row, with
// one scale: with x in the format too that is the operand of the scaled 4-bit
// MFMA as it is; with x in bf16 the codes become bf16 (an exact conversion, the
// scale applied) and four MFMAs take the lane's four dwords in turn, x's operand
// in the same order of k.
#include "kda_mx4_dev.h"
#include "kda_mx4_internal.h"

namespace kda {
namespace {

// The waves' sums joined in wave order, and stored.
template <int RT, int WAVES>
__device__ __forceinline__ void join(const Mx4Params& p, char* lds, const f32x4 (&acc)[RT], int n0, int64_t m0,
                                     int lane, int wave) {
  f32x4(*red)[RT][64] = reinterpret_cast<f32x4(*)[RT][64]>(lds);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RT; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  for (int t = threadIdx.x; t < RT * 256; t += 64 * WAVES) {
    // consecutive threads: consecutive rows of w of one token
    const int r = t & 15, m = (t >> 4) & 15, i = t >> 8;
    const float* at = reinterpret_cast<const float*>(&red[0][i][(r >> 2) * 16 + m]) + (r & 3);
    float y = at[0];
#pragma unroll
    for (int u = 1; u < WAVES; ++u) y += at[u * RT * 256];
    const int n = n0 + 16 * i + r;
    if (m0 + m < p.M && n < p.N) p.y[(m0 + m) * p.y_row + n] = f32_to_bf16(y);
  }
}

template <int RQ, int RT, int WAVES, int STEPS>
__global__ __launch_bounds__(64 * WAVES) void few_bf16_kernel(Mx4Params p) {
  __shared__ __align__(16) char lds[WAVES * (4096 > RT * 1024 ? 4096 : RT * 1024)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * RT);
  const int64_t m0 = int64_t(blockIdx.y) * 16;
  const int nb = p.K / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const int per = (units + WAVES - 1) / WAVES, first = wave * per, cnt = max(0, min(per, units - first));
  // rows behind the last row or token repeat it: their sums are not stored
  const uint8_t *codes[RT], *scales[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const size_t n = min(n0 + 16 * i + l16, p.N - 1);
    codes[i] = p.w + n * (p.K / 2);
    scales[i] = p.ws + n * nb;
  }
  const uint16_t* row[RQ];
#pragma unroll
  for (int q = 0; q < RQ; ++q)
    row[q] = static_cast<const uint16_t*>(p.x) + min(m0 + 4 * q + g, p.M - 1) * p.x_row;
  char* xl = lds + wave * 4096;
  f32x4 acc[RT] = {};
  if (cnt) {
    Piece<STEPS> buf[2][RT];
    XRows<RQ> x;
    const auto use = [&](Piece<STEPS>(&b)[RT], int unit) {
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        stage_x<RQ>(xl, x, l16, g);
        load_x<RQ>(x, row, (unit * STEPS + j + 1) * 128, p.K, l16);
        wave_lds_fence();
        bf16x8 o[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = x_operand(xl, d, l16, g);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float sc = scale_of(b[i].s[j], g);
#pragma unroll
          for (int d = 0; d < 4; ++d) acc[i] = mfma32(dequant8(b[i].w[j][d], sc), o[d], acc[i]);
        }
        wave_lds_fence();
      }
    };
    const auto load = [&](Piece<STEPS>(&b)[RT], int unit) {
#pragma unroll
      for (int i = 0; i < RT; ++i) load_piece<STEPS>(b[i], codes[i], scales[i], nb, unit, g);
    };
    load(buf[0], first);
    load_x<RQ>(x, row, first * STEPS * 128, p.K, l16);
    int i = 0;
    for (; i + 2 <= cnt; i += 2) {
      load(buf[1], first + i + 1);
      use(buf[0], first + i);
      load(buf[0], first + min(i + 2, cnt - 1));
      use(buf[1], first + i + 1);
    }
    if (i < cnt) use(buf[0], first + i);
  }
  join<RT, WAVES>(p, lds, acc, n0, m0, lane, wave);
}

template <int RT, int WAVES, int STEPS>
__global__ __launch_bounds__(64 * WAVES) void few_mx4_kernel(Mx4Params p) {
  __shared__ __align__(16) char lds[WAVES * RT * 1024];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * RT);
  const int64_t m0 = int64_t(blockIdx.y) * 16;
  const int nb = p.K / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const int per = (units + WAVES - 1) / WAVES, first = wave * per, cnt = max(0, min(per, units - first));
  const uint8_t *codes[RT], *scales[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const size_t n = min(n0 + 16 * i + l16, p.N - 1);
    codes[i] = p.w + n * (p.K / 2);
    scales[i] = p.ws + n * nb;
  }
  const size_t m = size_t(min(m0 + l16, p.M - 1));
  const uint8_t *xc = static_cast<const uint8_t*>(p.x) + m * (p.K / 2), *xs = p.xs + m * nb;
  f32x4 acc[RT] = {};
  if (cnt) {
    Piece<STEPS> buf[2][RT], x[2];
    const auto use = [&](Piece<STEPS>(&b)[RT], Piece<STEPS>& x) {
#pragma unroll
      for (int j = 0; j < STEPS; ++j)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[i] = mfma_mx4(b[i].w[j], b[i].s[j] >> (8 * g), x.w[j], x.s[j] >> (8 * g), acc[i]);
    };
    const auto load = [&](Piece<STEPS>(&b)[RT], Piece<STEPS>& x, int unit) {
#pragma unroll
      for (int i = 0; i < RT; ++i) load_piece<STEPS>(b[i], codes[i], scales[i], nb, unit, g);
      load_piece<STEPS>(x, xc, xs, nb, unit, g);
    };
    load(buf[0], x[0], first);
    int i = 0;
    for (; i + 2 <= cnt; i += 2) {
      load(buf[1], x[1], first + i + 1);
      use(buf[0], x[0]);
      load(buf[0], x[0], first + min(i + 2, cnt - 1));
      use(buf[1], x[1]);
    }
    if (i < cnt) use(buf[0], x[0]);
  }
  join<RT, WAVES>(p, lds, acc, n0, m0, lane, wave);
}

template <int RT, int WAVES>
hipError_t launch(const void* f, const Mx4Params& p, hipStream_t st) {
  Mx4Params arg = p;
  void* args[] = {&arg};
  const dim3 grid((p.N + 16 * RT - 1) / (16 * RT), uint32_t((p.M + 15) / 16));
  return hipLaunchKernel(f, grid, dim3(64 * WAVES), args, 0, st);
}

}  // namespace

hipError_t launch_mx4_few(const Mx4Params& p, int cus, hipStream_t stream) {
  if (p.xs) return launch<2, 8>(reinterpret_cast<const void*>(&few_mx4_kernel<2, 8, 2>), p, stream);
  if (p.M <= 4) return launch<1, 8>(reinterpret_cast<const void*>(&few_bf16_kernel<1, 1, 8, 2>), p, stream);
  return launch<2, 8>(reinterpret_cast<const void*>(&few_bf16_kernel<4, 2, 8, 2>), p, stream);
}

}  // namespace kda
