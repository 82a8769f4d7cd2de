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
//
// Next to the bytes it is vector memory instructions that cost: operands as the MFMA
// wants them, adjacent lanes in different rows, take a cycle a lane, and kept the address
// unit busy for all of 16 x 7168 x 14336 (22.3 us; with whole lines through LDS 20.1, of
// cold weights 14.9 to 15.7: 57 MB, 3.7 TB/s where a copy reaches 5.0).  x is read whole
// by every workgroup, from the L2: 51 MB with 64 rows of w each.  The smallest calls are
// round trips: 1 x 7168 x 1536 4.3 us, of which a launch is about 2.
#include "kda_mx4_dev.h"
#include "kda_mx4_internal.h"

namespace kda {
namespace {

// The waves' sums joined in wave order, and stored.  acc: tiles of 16 tokens (NT) by
// tiles of 16 rows of w (RT).
template <int NT, int RT, int WAVES>
__device__ __forceinline__ void join(const Mx4Params& p, char* lds, const f32x4 (&acc)[NT][RT], int n0, int64_t m0,
                                     int lane, int wave) {
  constexpr int kTiles = NT * RT;
  f32x4(*red)[kTiles][64] = reinterpret_cast<f32x4(*)[kTiles][64]>(lds);
  __syncthreads();
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int i = 0; i < RT; ++i) red[wave][m * RT + i][lane] = acc[m][i];
  __syncthreads();
  for (int t = threadIdx.x; t < kTiles * 256; t += 64 * WAVES) {
    // consecutive threads: consecutive rows of w of one token
    const int r = t % (16 * RT), token = t / (16 * RT);
    const int tile = (token >> 4) * RT + (r >> 4);
    const float* at = reinterpret_cast<const float*>(&red[0][tile][((r & 15) >> 2) * 16 + (token & 15)]) + (r & 3);
    float y = at[0];
#pragma unroll
    for (int u = 1; u < WAVES; ++u) y += at[u * kTiles * 256];
    if (m0 + token < p.M && n0 + r < p.N) p.y[(m0 + token) * p.y_row + n0 + r] = f32_to_bf16(y);
  }
}

// Units first .. end - 1 with U of them in flight.  (Loads only where a unit exists, so
// that the compiler's waits cannot count them: loops whose waits can took as long, other
// waves fill the time, and their extra loads cost the short calls.)
template <int U, typename Unit, typename Load, typename Use>
__device__ __forceinline__ void ring(Unit (&buf)[U], int first, int end, const Load& load, const Use& use) {
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first + u < end) load(buf[u], first + u);
  for (int unit = first; unit < end; unit += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (unit + u >= end) break;
      use(buf[u], unit + u);
      if (unit + u + U < end) load(buf[u], unit + u + U);
    }
  }
}

// NT tiles of 16 tokens (the first 4 RQ rows of each hold tokens), RT tiles of 16 rows of
// w; U units of STEPS * 128 k in flight.
template <int NT, int RQ, int RT, int WAVES, int STEPS, int U, bool TINY>
__global__ __launch_bounds__(64 * WAVES, NT > 1 ? 2 : 4) void few_bf16_kernel(Mx4Params p) {
  constexpr int kX = STEPS * NT * RQ * 1024, kWave = kX + RT * kPieceLds<STEPS>;
  __shared__ __align__(16) char lds[WAVES * (kWave > NT * RT * 1024 ? kWave : NT * RT * 1024)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * RT), m0 = blockIdx.y * (16 * NT);
  const int nb = p.K / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const int first = units * wave / WAVES, end = units * (wave + 1) / WAVES;
  // rows behind the last row or token repeat it: their sums are not stored
  const uint8_t *codes = p.w + size_t(n0) * (p.K / 2), *scales = p.ws + size_t(n0) * nb;
  uint32_t code_row[RT], scale_row[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const uint32_t r = min(16 * i + (lane >> 2), p.N - 1 - n0);
    code_row[i] = r * (p.K / 2), scale_row[i] = r * nb;
  }
  const uint16_t* x0 = static_cast<const uint16_t*>(p.x) + m0 * p.x_row;
  uint32_t row[NT][RQ];
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int q = 0; q < RQ; ++q)
      row[m][q] = uint32_t(min(16 * m + 4 * q + g, int(p.M) - 1 - m0)) * uint32_t(p.x_row * 2);
  char *xl = lds + wave * kWave, *wl = xl + kX;
  f32x4 acc[NT][RT] = {};
  struct Unit {
    Piece<STEPS> w[RT];
    XRows<RQ> x[STEPS][NT];
  } buf[U];
  const auto load = [&](Unit& b, int unit) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
      load_piece<STEPS, TINY>(b.w[i], codes, code_row[i], scales, scale_row[i], nb, unit, lane & 3);
#pragma unroll
    for (int j = 0; j < STEPS; ++j)
#pragma unroll
      for (int m = 0; m < NT; ++m) load_x<RQ>(b.x[j][m], x0, row[m], (unit * STEPS + j) * 128, p.K, l16);
  };
  const auto use = [&](Unit& b, int unit) {
#pragma unroll
    for (int i = 0; i < RT; ++i) stage_piece<STEPS, TINY>(wl + i * kPieceLds<STEPS>, b.w[i], nb, unit, lane);
#pragma unroll
    for (int j = 0; j < STEPS; ++j)
#pragma unroll
      for (int m = 0; m < NT; ++m)
        stage_x<RQ>(xl + (j * NT + m) * (RQ * 1024), b.x[j][m], (unit * STEPS + j) * 128, p.K, l16, g);
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      bf16x8 w[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const char* at = wl + i * kPieceLds<STEPS>;
        const float sc = scale_of(scale_operand<STEPS>(at, j, l16, g));
        const u32x4 c = codes_operand(at, j, l16, g);
#pragma unroll
        for (int d = 0; d < 4; ++d) w[i][d] = dequant8(c[d], sc);
      }
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const bf16x8 o = x_operand<RQ>(xl + (j * NT + m) * (RQ * 1024), d, l16, g);
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[m][i] = mfma32(w[i][d], o, acc[m][i]);
        }
    }
    wave_lds_fence();
  };
  ring<U>(buf, first, end, load, use);
  join<NT, RT, WAVES>(p, lds, acc, n0, m0, lane, wave);
}

// The same with x in the format too.
template <int NT, int RT, int WAVES, int STEPS, int U, bool TINY>
__global__ __launch_bounds__(64 * WAVES, 4) void few_mx4_kernel(Mx4Params p) {
  constexpr int kWave = (NT + RT) * kPieceLds<STEPS>;
  __shared__ __align__(16) char lds[WAVES * (kWave > NT * RT * 1024 ? kWave : NT * RT * 1024)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * RT);
  const int64_t m0 = int64_t(blockIdx.y) * (16 * NT);
  const int nb = p.K / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const int first = units * wave / WAVES, end = units * (wave + 1) / WAVES;
  const uint8_t *codes = p.w + size_t(n0) * (p.K / 2), *scales = p.ws + size_t(n0) * nb;
  const uint8_t *xc = static_cast<const uint8_t*>(p.x) + size_t(m0) * (p.K / 2), *xs = p.xs + size_t(m0) * nb;
  uint32_t code_row[RT], scale_row[RT], x_row[NT], xs_row[NT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const uint32_t r = min(16 * i + (lane >> 2), p.N - 1 - n0);
    code_row[i] = r * (p.K / 2), scale_row[i] = r * nb;
  }
  const int last = int(p.M - 1 - m0 < 16 * NT ? p.M - 1 - m0 : 16 * NT - 1);
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    const uint32_t r = min(16 * m + (lane >> 2), last);
    x_row[m] = r * (p.K / 2), xs_row[m] = r * nb;
  }
  f32x4 acc[NT][RT] = {};
  struct Unit {
    Piece<STEPS> w[RT], x[NT];
  } buf[U];
  const auto load = [&](Unit& b, int unit) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
      load_piece<STEPS, TINY>(b.w[i], codes, code_row[i], scales, scale_row[i], nb, unit, lane & 3);
#pragma unroll
    for (int m = 0; m < NT; ++m) load_piece<STEPS, TINY>(b.x[m], xc, x_row[m], xs, xs_row[m], nb, unit, lane & 3);
  };
  char *wl = lds + wave * kWave, *xl = wl + RT * kPieceLds<STEPS>;
  const auto use = [&](Unit& b, int unit) {
#pragma unroll
    for (int i = 0; i < RT; ++i) stage_piece<STEPS, TINY>(wl + i * kPieceLds<STEPS>, b.w[i], nb, unit, lane);
#pragma unroll
    for (int m = 0; m < NT; ++m) stage_piece<STEPS, TINY>(xl + m * kPieceLds<STEPS>, b.x[m], nb, unit, lane);
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      u32x4 w[RT];
      uint32_t sw[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        w[i] = codes_operand(wl + i * kPieceLds<STEPS>, j, l16, g);
        sw[i] = scale_operand<STEPS>(wl + i * kPieceLds<STEPS>, j, l16, g);
      }
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const u32x4 x = codes_operand(xl + m * kPieceLds<STEPS>, j, l16, g);
        const uint32_t sx = scale_operand<STEPS>(xl + m * kPieceLds<STEPS>, j, l16, g);
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[m][i] = mfma_mx4(w[i], sw[i], x, sx, acc[m][i]);
      }
    }
    wave_lds_fence();
  };
  ring<U>(buf, first, end, load, use);
  join<NT, RT, WAVES>(p, lds, acc, n0, m0, lane, wave);
}

// Grid: tiles of w's rows by tiles of tokens.
hipError_t go(const void* f, int nt, int rt, int waves, const Mx4Params& p, hipStream_t st) {
  Mx4Params arg = p;
  void* args[] = {&arg};
  const dim3 grid((p.N + 16 * rt - 1) / (16 * rt), uint32_t((p.M + 16 * nt - 1) / (16 * nt)));
  return hipLaunchKernel(f, grid, dim3(64 * waves), args, 0, st);
}

template <int NT, int RQ, int RT, int WAVES, int STEPS, int U>
hipError_t few_bf16(const Mx4Params& p, hipStream_t st) {
  const auto at = [](auto* f) { return reinterpret_cast<const void*>(f); };
  return go(p.K < 128 ? at(&few_bf16_kernel<NT, RQ, RT, WAVES, STEPS, U, true>)
                              : at(&few_bf16_kernel<NT, RQ, RT, WAVES, STEPS, U, false>),
            NT, RT, WAVES, p, st);
}
template <int NT, int RT, int WAVES, int STEPS, int U>
hipError_t few_mx4(const Mx4Params& p, hipStream_t st) {
  const auto at = [](auto* f) { return reinterpret_cast<const void*>(f); };
  return go(p.K < 128 ? at(&few_mx4_kernel<NT, RT, WAVES, STEPS, U, true>)
                              : at(&few_mx4_kernel<NT, RT, WAVES, STEPS, U, false>),
            NT, RT, WAVES, p, st);
}

}  // namespace

// Which form, measured on 256 compute units (us):
//  * Rows of w per workgroup: 16 give the most workgroups, 32 read x half as often.
//    bf16, 16 / 32: 16 x 7168 x 1536 6.6 / 8.4, 16 x 2048 x 4096 3.8 / 4.5, 16 x 7168 x
//    7168 15.1 / 12.7; so 16 up to 384 workgroups.  64 where they still are 154 and more:
//    16 x 4096 x 10240 12.1 against 13.0, 16 x 7168 x 14336 20.2 / 22.3, but 16 x 7168 x
//    7168 18.0 / 12.7.  With x in the format 16 up to 192 workgroups of 32: 16 x 7168 x
//    1536 4.4 / 5.9, 16 x 7168 x 7168 9.5 / 9.2.
//  * At most 4 tokens: 16 waves share k where the workgroups are half the units or fewer
//    (1 x 7168 x 1536 4.3 against 4.8 with 8, 1 x 2048 x 4096 3.4 / 3.1), 32 rows where
//    those of 16 are three times the units (1 x 7168 x 14336 13.9 against 14.5).
//  * Tokens per workgroup: 16, which for more tokens reads w again, from the L2 or the
//    cache behind it; 32 and 64 hold x of a step in registers, so that fewer waves run.
//    64: 61 x 2080 x 7171 10.6 against 12.4 with 16, 64 x 7168 x 7168 24.0 / 27.9, but 48 x
//    2048 x 7168 9.1 / 8.4, 64 x 2048 x 2048 8.8 / 4.6.  32: 30 x 7168 x 14336 29.4 / 33.4,
//    but 32 x 7168 x 1536 11.9 / 8.1.  With x in the format 32 and one unit in flight for
//    all of more than 16 tokens: 64 x 7168 x 1536 7.4 against 8.2 with 32 rows in two
//    units, 17.7 with 64 x 64 (larger calls go to kda_mx4_tile.hip).
hipError_t launch_mx4_few(const Mx4Params& p, int cus, hipStream_t stream) {
  const int64_t rows16 = (p.N + 15) / 16, rows32 = (p.N + 31) / 32, rows64 = (p.N + 63) / 64;
  if (p.xs) {
    if (p.M > 16) return few_mx4<2, 2, 8, 2, 1>(p, stream);
    return 4 * rows32 > 3 * cus ? few_mx4<1, 2, 8, 2, 2>(p, stream) : few_mx4<1, 1, 8, 2, 2>(p, stream);
  }
  if (p.M <= 4) {
    if (2 * rows16 <= cus) return few_bf16<1, 1, 1, 16, 2, 2>(p, stream);
    return rows16 > 3 * cus ? few_bf16<1, 1, 2, 8, 2, 2>(p, stream) : few_bf16<1, 1, 1, 8, 2, 2>(p, stream);
  }
  if (p.M > 48 && 2 * rows32 > cus) return few_bf16<4, 4, 2, 8, 1, 1>(p, stream);
  if (p.M > 16 && rows32 > cus) return few_bf16<2, 4, 2, 8, 1, 1>(p, stream);
  const int64_t tiles = (p.M + 15) / 16;
  if (2 * rows16 * tiles <= 3 * cus) return few_bf16<1, 4, 1, 8, 1, 2>(p, stream);
  return p.M <= 16 && 5 * rows64 > 3 * cus ? few_bf16<1, 4, 4, 8, 1, 1>(p, stream)
                                           : few_bf16<1, 4, 2, 8, 1, 2>(p, stream);
}

}  // namespace kda
